"""Tables of one engine step (tq_build_tables) against a plain loop over the
sequences on the host: every output is a whole number and has to be equal.
Sizes from one sequence to 4096, lengths of zero, paged and contiguous caches,
shared prefixes, a free list that runs out, and the call's refusals."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FILL = -77  # what the buffers hold before the call


@pytest.fixture(scope="module")
def tq(cuda_device):
    from kv_cache_vector_12_b200 import tq as tqmod
    return tqmod


@pytest.fixture(scope="module")
def ctx(tq):
    return tq.Context(128, 3, 3, 0, 42)


def reference(cached, new, table, bs, capacity, free, start, groups=None, prefixes=None):
    """A loop over the sequences, then over the members of the groups."""
    table = None if table is None else table.copy()
    seq_idx, pos, cu, taken = [], [], [0], start
    for s, (c, w) in enumerate(zip(cached, new)):
        seq_idx += [s] * w
        pos += range(c, c + w)
        cu.append(cu[-1] + w)
        if table is not None:
            for j in range(-(-c // bs), -(-(c + w) // bs)):
                table[s, j] = free[taken]
                taken += 1
    for g, prefix in enumerate(prefixes or []):
        for s in range(groups[g] + 1, groups[g + 1]):
            table[s, :prefix // bs] = table[groups[g], :prefix // bs]
    if table is None:
        slots = [s * capacity + p for s, p in zip(seq_idx, pos)]
    else:
        slots = [int(table[s, p // bs]) * bs + p % bs for s, p in zip(seq_idx, pos)]
    lens = [c + w for c, w in zip(cached, new)]
    return dict(seq_idx=seq_idx, pos=pos, cu_new=cu, seq_lens=lens, slots=slots, table=table, free_end=taken)


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def buffers(n, n_tok, with_slots=True):
    b = {k: torch.full((size,), FILL, dtype=torch.int32, device="cuda")
         for k, size in (("seq_idx", n_tok), ("pos", n_tok), ("cu_new", n + 1), ("seq_lens", n), ("free_end", 1))}
    b["slots"] = torch.full((n_tok,), FILL, dtype=torch.int64, device="cuda") if with_slots else None
    return b


def start_table(cached, bs, capacity, ids):
    """A table whose cached blocks hold the first ids, and FILL elsewhere; and how many ids it holds."""
    table, used = np.full((len(cached), capacity // bs), FILL, dtype=np.int32), 0
    for s, c in enumerate(cached):
        k = -(-c // bs)
        table[s, :k] = ids[used:used + k]
        used += k
    return table, used


def run_paged(tq, ctx, cached, new, bs, capacity, groups=None, prefixes=None, spare=5, start=2, extra_rows=0, seed=0,
              with_slots=True, offset=0):
    rng = np.random.default_rng(seed)
    need = sum(-(-(c + w) // bs) for c, w in zip(cached, new))
    ids = rng.permutation(need + spare + start).astype(np.int32)
    table, used = start_table(cached, bs, capacity, ids)
    free = ids[used:]
    ref = reference(cached, new, table, bs, capacity, free, start, groups, prefixes)
    n, n_tok = len(cached), sum(new) + extra_rows
    cache = tq.PagedCache(ctx, n, 1, capacity, bs, n_blocks=len(ids), block_table=torch.from_numpy(table))
    b = buffers(n, n_tok + offset, with_slots)
    view = {k: (b[k][offset:] if b[k] is not None and k in ("seq_idx", "pos", "slots") else b[k]) for k in b}
    args = dict(free_list=dev(free), free_start=dev([start]),
                cu_group=None if groups is None else dev(groups), prefix_lens=None if groups is None else dev(prefixes))
    for _ in range(2):  # the call is a function of its inputs: a second one writes the same
        tq.build_tables(ctx, cache, dev(cached), dev(new), **view, **args)
        ctx.check_device_errors()
        assert np.array_equal(cache.block_table.cpu().numpy(), ref["table"])
        for k in ("seq_idx", "pos", "slots"):
            if b[k] is None:
                continue
            got = b[k].cpu().numpy()
            assert np.array_equal(got[offset:offset + sum(new)], np.asarray(ref[k], dtype=got.dtype)), k
            assert np.all(got[:offset] == FILL) and np.all(got[offset + sum(new):] == FILL), k
        assert b["cu_new"].tolist() == ref["cu_new"]
        assert b["seq_lens"].tolist() == ref["seq_lens"]
        assert b["free_end"].tolist() == [ref["free_end"]]


@pytest.mark.parametrize("n,max_cached,max_new,bs", [(1, 0, 1, 64), (1, 200, 5, 64), (3, 130, 130, 128),
                                                    (32, 4000, 1, 256), (7, 0, 900, 64), (513, 300, 40, 64),
                                                    (1025, 100, 1, 64), (4096, 64, 3, 64)])
def test_paged_tables(tq, ctx, n, max_cached, max_new, bs):
    rng = np.random.default_rng(n + bs)
    cached, new = rng.integers(0, max_cached + 1, n).tolist(), rng.integers(0, max_new + 1, n).tolist()
    capacity = -(-(max_cached + max_new) // bs) * bs
    run_paged(tq, ctx, cached, new, bs, capacity, seed=n)


def test_zero_lengths_block_borders_and_full_sequences(tq, ctx):
    cached = [0, 0, 63, 64, 65, 128, 191, 192, 0]
    new = [0, 64, 1, 1, 63, 0, 1, 0, 192]
    run_paged(tq, ctx, cached, new, 64, 192)
    run_paged(tq, ctx, [0, 0], [0, 0], 64, 64)  # nothing new at all


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_unaligned_outputs_rows_behind_the_last_and_no_slots(tq, ctx, offset):
    run_paged(tq, ctx, [5, 0, 100], [60, 7, 33], 64, 192, extra_rows=11, offset=offset)
    run_paged(tq, ctx, [5, 0, 100], [60, 7, 33], 64, 192, extra_rows=3, offset=offset, with_slots=False)


def test_more_tokens_than_resident_threads(tq, ctx):
    """Four rows to a thread: sequences that begin and end inside its four, blocks that do, unaligned outputs."""
    rng = np.random.default_rng(0)
    for offset in (0, 1):
        cached, new = rng.integers(0, 500, 90).tolist(), rng.integers(0, 9000, 90).tolist()
        new[3:9] = [1, 0, 2, 3, 0, 1]
        run_paged(tq, ctx, cached, new, 64, 9600, seed=offset, offset=offset)


def test_shared_prefixes(tq, ctx):
    """Groups of one to many members; a first member that gets its prefix in
    this call; a prefix of zero; sequences behind the last group."""
    cached = [200, 128, 130, 0, 256, 256, 70, 64, 64, 10]
    new = [1, 3, 100, 300, 1, 64, 0, 1, 5, 20]
    run_paged(tq, ctx, cached, new, 64, 512, groups=[0, 3, 6, 7, 9], prefixes=[128, 256, 64, 0])


def test_many_groups(tq, ctx):
    rng = np.random.default_rng(5)
    n = 700
    cuts = [0] + sorted(rng.choice(np.arange(1, n), 99, replace=False).tolist()) + [n]
    cached = (64 * rng.integers(1, 9, n) + rng.integers(0, 64, n)).tolist()
    prefixes = [min(cached[a:b]) // 64 * 64 for a, b in zip(cuts, cuts[1:])]
    run_paged(tq, ctx, cached, rng.integers(0, 70, n).tolist(), 64, 768, groups=cuts, prefixes=prefixes)


def test_contiguous_cache(tq, ctx):
    cached, new, capacity = [7, 0, 100, 64], [3, 0, 1, 128], 192
    ref = reference(cached, new, None, 1, capacity, [], 0)
    cache = tq.Cache(ctx, 4, 1, capacity)
    b = buffers(4, sum(new))
    del b["free_end"]
    tq.build_tables(ctx, cache, dev(cached), dev(new), **b)
    ctx.check_device_errors()
    for k in b:
        assert b[k].tolist() == ref[k], k


def _flagged(tq, ctx):
    with pytest.raises(tq.TQError) as ei:
        ctx.check_device_errors()
    assert ei.value.status == tq.TQ_ERR_DEVICE
    return str(ei.value)


def test_free_list_that_runs_out(tq, ctx):
    """Five blocks wanted, three there: the rest of the entries and their slots are -1."""
    cache = tq.PagedCache(ctx, 2, 1, 256, 64, n_blocks=9, block_table=torch.full((2, 4), FILL, dtype=torch.int32))
    b = buffers(2, 300)
    tq.build_tables(ctx, cache, dev([0, 0]), dev([130, 70]), **b, free_list=dev([4, 8, 6]), free_start=dev([0]))
    assert "token outside cache" in _flagged(tq, ctx)
    assert cache.block_table.tolist() == [[4, 8, 6, FILL], [-1, -1, FILL, FILL]]
    assert b["free_end"].tolist() == [3]
    slots = b["slots"].tolist()
    assert slots[128:130] == [6 * 64, 6 * 64 + 1] and slots[130:200] == [-1] * 70 and slots[200:] == [FILL] * 100
    # a block that does not exist, and a start behind the list
    tq.build_tables(ctx, cache, dev([0, 0]), dev([64, 0]), **b, free_list=dev([9]), free_start=dev([0]))
    _flagged(tq, ctx)
    assert cache.block_table[0, 0].item() == -1 and b["slots"][:64].tolist() == [-1] * 64
    tq.build_tables(ctx, cache, dev([0, 0]), dev([64, 0]), **b, free_list=dev([3]), free_start=dev([7]))
    _flagged(tq, ctx)
    assert b["free_end"].tolist() == [1]


def test_bad_lengths_and_prefixes_are_flagged(tq, ctx):
    cache = tq.PagedCache(ctx, 4, 1, 128, 64, n_blocks=20, block_table=torch.full((4, 2), FILL, dtype=torch.int32))
    b = buffers(4, 64)
    free = dict(free_list=dev(list(range(20))), free_start=dev([0]))
    big = 2 ** 31 - 1
    tq.build_tables(ctx, cache, dev([0, -1, 100, big]), dev([2, 5, 29, big]), **b, **free)
    assert "seq_len" in _flagged(tq, ctx)
    assert b["seq_lens"].tolist() == [2, 0, 0, 0] and b["cu_new"].tolist() == [0, 2, 2, 2, 2]
    assert b["seq_idx"].tolist() == [0, 0] + [FILL] * 62
    for prefix in (63, 192, -64):  # no whole blocks; more than is cached; negative
        tq.build_tables(ctx, cache, dev([64, 128, 0, 0]), dev([1, 0, 0, 0]), **b, **free, cu_group=dev([0, 2]),
                        prefix_lens=dev([prefix]))
        assert "seq_len" in _flagged(tq, ctx), prefix
        assert cache.block_table[1].tolist() == [FILL, FILL]
    # more new tokens than rows: the rows there are get written
    tq.build_tables(ctx, cache, dev([0, 0, 0, 0]), dev([40, 40, 0, 0]), **b, **free)
    assert "token outside cache" in _flagged(tq, ctx)
    assert b["seq_idx"].tolist() == [0] * 40 + [1] * 24 and b["cu_new"].tolist() == [0, 40, 80, 80, 80]


def test_refusals(tq, ctx):
    cache = tq.PagedCache(ctx, 2, 1, 128, 64)
    b = buffers(2, 8)
    cached, new = dev([0, 0]), dev([1, 1])
    free = dict(free_list=dev([0, 1]), free_start=dev([0]))

    def refused(status=tq.TQ_ERR_INVALID, cache=cache, cached=cached, new=new, **changed):
        args = {**b, **free, **changed}
        with pytest.raises(tq.TQError) as ei:
            tq.build_tables(ctx, cache, cached, new, **args)
        assert ei.value.status == status

    refused(cached=None)
    refused(cu_new=None)
    refused(free_start=None)
    refused(free_end=free["free_start"])          # in place: another CTA still reads it
    refused(seq_lens=cached)
    refused(pos=b["seq_idx"])
    refused(seq_idx=b["seq_idx"][:4], pos=b["seq_idx"][3:7], slots=None)
    refused(prefix_lens=dev([0]))                 # groups without their bounds
    refused(prefix_lens=dev([0, 0, 0]), cu_group=dev([0, 1, 2, 2]))
    refused(status=tq.TQ_ERR_UNSUPPORTED, cache=tq.PagedCache(ctx, 4097, 1, 64, 64))
    ctx.check_device_errors()


def test_step_captured_and_replayed_feeds_quantize(tq, ctx):
    """The tables of a step and the append that reads them, captured in one
    graph and replayed with new lengths: every token lands in its block."""
    n, bs, capacity, h = 3, 64, 256, 2
    cache = tq.PagedCache(ctx, n, h, capacity, bs, n_blocks=12,
                          block_table=torch.full((n, capacity // bs), -1, dtype=torch.int32))
    cached, new, n_tok = dev([0, 0, 0]), dev([70, 1, 64]), 135
    b = buffers(n, n_tok)
    free = dict(free_list=dev(np.random.default_rng(1).permutation(12)), free_start=dev([0]))
    k = torch.randn(n_tok, h, 128, device="cuda").to(torch.bfloat16)

    def step():
        tq.build_tables(ctx, cache, cached, new, **b, **free)
        tq.quantize(ctx, cache, k, k, b["seq_idx"], b["pos"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for plane in cache.planes.values():
        if plane is not None:
            plane.zero_()
    graph.replay()
    ctx.check_device_errors()
    flat = tq.Cache(ctx, 1, h, 192)
    zero = torch.zeros(n_tok, dtype=torch.int32, device="cuda")
    tq.quantize(ctx, flat, k, k, zero, torch.arange(n_tok, dtype=torch.int32, device="cuda"))
    slots = b["slots"]
    for name in ("codes_k", "codes_v", "norm_k", "norm_v"):
        got = cache.planes[name][slots // bs, :, slots % bs]
        assert torch.equal(got, flat.planes[name][0].transpose(0, 1)[:n_tok]), name


def test_the_most_tokens(tq, ctx):
    """2^31 - 1 new tokens, an index short of what 32 bits hold: every row, and none past them."""
    half = 2 ** 30
    cache = tq.Cache(ctx, 2, 1, 64)
    cache.struct.capacity = half  # (no plane is used)
    n = 2 * half - 1
    b = buffers(2, 0)
    del b["free_end"]
    b["slots"] = None
    b["seq_idx"], b["pos"] = (torch.full((n + 1,), -7, dtype=torch.int32, device="cuda")[:n] for _ in range(2))
    tq.build_tables(ctx, cache, dev([0, 0]), dev([half, half - 1]), **b)
    ctx.check_device_errors()
    assert b["cu_new"].tolist() == [0, half, n] and b["seq_lens"].tolist() == [half, half - 1]
    for s, a, e in ((0, 0, half), (1, half, n)):
        for i in range(a, e, 2 ** 27):
            j = min(i + 2 ** 27, e)
            assert (b["seq_idx"][i:j] == s).all()
            assert torch.equal(b["pos"][i:j], torch.arange(i - a, j - a, dtype=torch.int32, device="cuda"))
    for x in (b["seq_idx"], b["pos"]):
        assert x.as_strided((1,), (1,), n).item() == -7


@pytest.mark.parametrize("groups", [[0, 5, 3, 8], [4, 6, 0, 8], [0, 8, 0, 8]])
def test_groups_that_decrease_share_nothing(tq, ctx, groups):
    """Groups that overlap would copy table entries that others write: flagged, the rest of the step as without them."""
    ids = np.arange(40, dtype=np.int32)
    cached, new = [128] * 8, [1] * 8
    table, used = start_table(cached, 64, 256, ids)
    ref = reference(cached, new, table, 64, 256, ids[used:], 0)
    cache = tq.PagedCache(ctx, 8, 1, 256, 64, n_blocks=40, block_table=torch.from_numpy(table))
    b = buffers(8, 8)
    tq.build_tables(ctx, cache, dev(cached), dev(new), **b, free_list=dev(ids[used:]), free_start=dev([0]),
                    cu_group=dev(groups), prefix_lens=dev([128, 128, 128]))
    assert "seq_len" in _flagged(tq, ctx)
    assert np.array_equal(cache.block_table.cpu().numpy(), ref["table"])
    for k in ("seq_idx", "pos", "slots", "cu_new", "seq_lens"):
        assert b[k].tolist() == ref[k], k


@pytest.mark.parametrize("offset", [0, 1])
def test_contiguous_cache_with_more_tokens_than_resident_threads(tq, ctx, offset):
    """Four rows to a thread in the contiguous layout: sequences that begin and end inside its four, of odd lengths."""
    rng = np.random.default_rng(offset)
    cached, new, capacity = rng.integers(0, 500, 90), rng.integers(0, 9000, 90), 9600
    new[3:9] = [1, 0, 2, 3, 0, 1]
    n_tok = int(new.sum())
    cache = tq.Cache(ctx, 90, 1, 64)
    cache.struct.capacity = capacity  # (no plane is used)
    b = buffers(90, n_tok + offset + 5)
    del b["free_end"]
    view = {k: b[k][offset:] if k in ("seq_idx", "pos", "slots") else b[k] for k in b}
    tq.build_tables(ctx, cache, dev(cached), dev(new), **view)
    ctx.check_device_errors()
    seq = np.repeat(np.arange(90), new)
    cu = np.concatenate([[0], np.cumsum(new)])
    pos = np.arange(n_tok) - cu[seq] + cached[seq]
    for k, ref in (("seq_idx", seq), ("pos", pos), ("slots", seq * capacity + pos)):
        got = b[k].cpu().numpy()
        assert np.array_equal(got[offset:offset + n_tok], ref), k
        assert (got[:offset] == FILL).all() and (got[offset + n_tok:] == FILL).all(), k
    assert np.array_equal(b["cu_new"].cpu().numpy(), cu) and np.array_equal(b["seq_lens"].cpu().numpy(), cached + new)


def test_members_without_tokens_keep_their_entries(tq, ctx):
    """A padded batch: finished members of a group, and a group of nothing else, are no error and change nothing."""
    ids = np.random.default_rng(3).permutation(40).astype(np.int32)
    cached, new, prefix = [192, 0, 192, 0, 0, 0, 128], [1, 0, 70, 0, 0, 0, 1], 128
    groups = [0, 4, 6, 7]
    table, used = start_table(cached, 64, 320, ids)
    ref = reference(cached, new, table, 64, 320, ids[used:], 0)
    ref["table"][2, :2] = ref["table"][0, :2]  # the only member with tokens behind its first
    cache = tq.PagedCache(ctx, 7, 1, 320, 64, n_blocks=40, block_table=torch.from_numpy(table))
    b = buffers(7, sum(new))
    tq.build_tables(ctx, cache, dev(cached), dev(new), **b, free_list=dev(ids[used:]), free_start=dev([0]),
                    cu_group=dev(groups), prefix_lens=dev([prefix, 64, prefix]))
    ctx.check_device_errors()
    assert np.array_equal(cache.block_table.cpu().numpy(), ref["table"])
    for k in ("seq_idx", "pos", "slots", "cu_new", "seq_lens"):
        assert b[k].tolist() == ref[k], k
