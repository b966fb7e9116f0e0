"""The serving operators as one program uses them, step after step on one
stream: tables of the admission, exact attention over the prompts, packing them
into the blocks the tables gave out, sequences that join behind a shared prefix,
then decode steps (a captured graph, replayed) of tables, append and
shared-prefix attention.  Checked against attention in 64 bits over the bytes
that were packed, and against tq_decode_attention on the same tables."""
import math

import numpy as np
import pytest
import torch

from oracle import turboquant_oracle as o
from tests import parity_helpers as ph

pytestmark = pytest.mark.gpu

BS, CAP, H, PER, D = 64, 640, 2, 4, 128


@pytest.fixture(scope="module")
def tq(cuda_device):
    from kv_cache_vector_12_b200 import tq as tqmod
    return tqmod


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bits_k,bits_v,qjl,tails", [(3, 3, 0, 5), (4, 2, 1, 5), (3, 4, 0, 40)])
def test_admit_join_and_decode(tq, bits_k, bits_v, qjl, tails):
    """Two prompts are admitted; `tails` sequences join behind the first one's 256 tokens; five decode steps follow."""
    ctx = tq.Context(D, bits_k, bits_v, qjl, 42)
    g = torch.Generator().manual_seed(tails)
    n = tails + 2  # sequence 0 and the ones behind it share a prefix, the last is alone
    rng = np.random.default_rng(tails)
    prefix, lone = 4 * BS, 130
    grow = rng.integers(1, 90, tails).tolist()
    cache = tq.PagedCache(ctx, n, H, CAP, BS, n_blocks=n * 5 + 12, block_table=torch.full((n, CAP // BS), -1))
    free = torch.from_numpy(rng.permutation(n * 5 + 12).astype(np.int32)).cuda()
    used = [_ints(0), _ints(0)]  # free_start and free_end change places from step to step
    groups, prefixes = _ints(0, n - 1, n), _ints(prefix, 0)
    new = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, lens = new(n + 1), torch.zeros(n, dtype=torch.int32, device="cuda")

    def tables(cached, fresh, n_tok, grouped):
        b = dict(seq_idx=new(n_tok), pos=new(n_tok), slots=torch.empty(n_tok, dtype=torch.int64, device="cuda"))
        tq.build_tables(ctx, cache, cached, fresh, b["seq_idx"], b["pos"], cu, lens, slots=b["slots"], free_list=free,
                        free_start=used[0], free_end=used[1], cu_group=groups if grouped else None,
                        prefix_lens=prefixes if grouped else None)
        used.reverse()
        return b

    def heads(rows, k):
        return torch.randn(rows, k, D, generator=g).to(torch.bfloat16).cuda()

    # ---- admission: two prompts packed in one call
    first = prefix + 7
    fresh = [first] + [0] * tails + [lone]
    q, k, v = heads(sum(fresh), H * PER), heads(sum(fresh), H), heads(sum(fresh), H)
    b = tables(_ints(*[0] * n), _ints(*fresh), sum(fresh), False)
    out, lse = torch.empty(sum(fresh), H * PER, D, device="cuda"), torch.empty(sum(fresh), H * PER, device="cuda")
    tq.prompt_attention(ctx, q, k, v, cu, max(fresh), out, lse)
    tq.quantize(ctx, cache, k, v, b["seq_idx"], b["pos"])
    ctx.check_device_errors()
    for a, e in ((0, first), (first, first + lone)):
        for h in range(H * PER):
            s = (q[a:e, h].double() @ k[a:e, h // PER].double().t() / math.sqrt(D)).masked_fill(
                torch.ones(e - a, e - a, dtype=torch.bool, device="cuda").triu(1), -math.inf)
            ref = torch.softmax(s, -1) @ v[a:e, h // PER].double()
            # weights rounded to bf16 (2^-8), scores of size ~1 in fp32: see the prompt tests
            mag = torch.softmax(s, -1) @ v[a:e, h // PER].double().abs()
            assert ((out[a:e, h].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * mag + 1e-30).all()

    # ---- the tails join behind the prefix, each with its own tokens
    fresh = [0] + grow + [0]
    b = tables(_ints(*[first] + [prefix] * tails + [lone]), _ints(*fresh), sum(fresh), True)
    k, v = heads(sum(fresh), H), heads(sum(fresh), H)
    tq.quantize(ctx, cache, k, v, b["seq_idx"], b["pos"])
    ctx.check_device_errors()
    table = cache.block_table.cpu().numpy()
    assert (table[1:n - 1, :4] == table[0, :4]).all()
    own = [set(row[row >= 0].tolist()) for row in table]
    assert len(set().union(*own)) == sum(len(x) for x in own) - 4 * tails  # nothing else is shared

    # ---- decode: one captured step, replayed; lengths and the free list go on in place
    cached, ones = lens.clone(), _ints(*[1] * n)
    start, end = used[0].clone(), _ints(0)
    seq_idx, pos = new(n), new(n)
    qd, kd, vd = heads(n, H * PER), heads(n, H), heads(n, H)
    bounds = dict(max_group=n - 1, max_prefix_len=prefix, max_suffix_len=CAP - prefix)
    ws = tq.alloc_shared_workspace(ctx, cache, H * PER, 2, **bounds)
    dout, dlse = torch.empty(n, H * PER, D, device="cuda"), torch.empty(n, H * PER, device="cuda")

    def step():
        tq.build_tables(ctx, cache, cached, ones, seq_idx, pos, cu, lens, free_list=free, free_start=start,
                        free_end=end, cu_group=groups, prefix_lens=prefixes)
        tq.quantize(ctx, cache, kd, vd, seq_idx, pos)
        tq.decode_attention_shared(ctx, cache, qd, lens, groups, prefixes, bounds["max_group"],
                                   bounds["max_prefix_len"], bounds["max_suffix_len"], dout, dlse, ws)
        cached.copy_(lens)
        start.copy_(end)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for x, rows in ((qd, H * PER), (kd, H), (vd, H)):
            x.copy_(heads(n, rows))
        graph.replay()
    ctx.check_device_errors()
    want = [first + 5] + [prefix + x + 5 for x in grow] + [lone + 5]
    assert lens.tolist() == want

    ref, ref_lse = torch.empty_like(dout), torch.empty_like(dlse)
    tq.decode_attention(ctx, cache, qd, lens, CAP, ref, ref_lse, tq.alloc_workspace(ctx, n, H * PER, CAP))
    ctx.check_device_errors()
    assert ((dout - ref).abs() <= 2e-3 * ref.abs().amax(-1, keepdim=True)).all()  # 1e-3 each
    p = o.Params(D, bits_k, bits_v, bool(qjl), 42)
    planes = {name: t.cpu().numpy() for name, t in cache.planes.items() if t is not None}
    table = cache.block_table.cpu().numpy()
    for s in {0, 1, tails, n - 1}:
        x = np.arange(want[s])
        for h in range(H):
            get = lambda name: planes[name][table[s, x // BS], h, x % BS]  # noqa: E731
            extra = {}
            if qjl:
                extra = dict(s_matrix=p.s, qjl_signs=o.unpack_signs(get("qjl_bits"), D),
                             qjl_gamma=ph.f16_bits_to_f64(get("qjl_norm")))
            hh = slice(h * PER, (h + 1) * PER)
            o_ref, l_ref, scores = o.decode_attention(
                qd[s, hh].double().cpu().numpy(), p.pi, p.ck, o.unpack_codes(get("codes_k"), bits_k, D),
                ph.f16_bits_to_f64(get("norm_k")), p.cv, o.unpack_codes(get("codes_v"), bits_v, D),
                ph.f16_bits_to_f64(get("norm_v")), 1 / math.sqrt(D), **extra)
            ok, w = ph.attention_ok(dout[s, hh].cpu().numpy(), o_ref, dlse[s, hh].cpu().numpy(), l_ref,
                                    np.abs(scores).max(axis=1))
            assert ok, (s, h, w)


def test_host_tensors_and_other_types_are_refused(tq):
    """Tensors that the kernels could not read are refused before the launch, and nothing is written."""
    ctx = tq.Context(D, 3, 3, 0, 42)
    cache = tq.PagedCache(ctx, 2, H, CAP, BS)

    def refused(call, good, **changed):
        for name, t in changed.items():
            with pytest.raises(tq.TQError) as ei:
                call(**{**good, name: t})
            assert ei.value.status == tq.TQ_ERR_INVALID, name
        ctx.check_device_errors()

    new = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    step = dict(cached_lens=_ints(0, 0), new_lens=_ints(1, 1), seq_idx=new(2), pos=new(2), cu_new=new(3), seq_lens=new(2),
                free_list=_ints(4, 5), free_start=_ints(0), free_end=new(1))
    refused(lambda **kw: tq.build_tables(ctx, cache, **kw), step, cached_lens=torch.zeros(2, dtype=torch.int32),
            new_lens=_ints(1, 1).long(), pos=new(1), cu_new=new(2), seq_lens=new(4)[::2], free_end=new(0))
    assert all((step[k] == -7).all() for k in ("seq_idx", "pos", "cu_new", "seq_lens", "free_end"))
    q = torch.randn(30, H * PER, D, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    prompt = dict(q=q, k=q[:, :H], v=q[:, :H], cu_seqlens=_ints(0, 30), max_len=30, out=out)
    refused(lambda **kw: tq.prompt_attention(ctx, **kw), prompt, k=q[:29, :H], v=q[:, :1], out=out[:29],
            cu_seqlens=_ints(0, 30).cpu(), lse=torch.empty(30, H * PER, dtype=torch.float64, device="cuda"))
    refused(lambda **kw: tq.prompt_attention(ctx, **kw), prompt, out=out.half())
    ws = tq.alloc_shared_workspace(ctx, cache, H * PER, 1, 2, 64, 64)
    shared = dict(q=q[:2], seq_lens=_ints(70, 80), cu_group=_ints(0, 2), prefix_lens=_ints(64), max_group=2,
                  max_prefix_len=64, max_suffix_len=64, out=out[:2], lse=None, workspace=ws)
    refused(lambda **kw: tq.decode_attention_shared(ctx, cache, **kw), shared, q=q[:1], seq_lens=_ints(70, 80).long(),
            cu_group=_ints(0), out=out[:2].half(), workspace=ws.cpu(), prefix_lens=_ints(64).cpu())
    assert (out == 7.0).all()


def test_all_operators_at_once(tq):
    """Prompts of both forms, shared decode on tcgen05, tables and appends on five streams: tensor memory, shared memory
    and the contexts' flags are what they have in common, and every output is the one of the call alone."""
    from tests.test_gpu_shared import Batch
    g = torch.Generator().manual_seed(1)
    heads = lambda n, k, d: torch.randn(n, k, d, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    jobs = []
    for d, lens in ((64, [200, 3, 77]), (128, [900, 130]), (256, [300, 5])):
        ctx, n = tq.Context(d, 3, 3, 0, 42), sum(lens)
        q, k, v = heads(n, 8, d), heads(n, 2, d), heads(n, 2, d)
        cu, out = _ints(0, *np.cumsum(lens).tolist()), torch.empty_like(q)
        jobs.append((out, ctx, lambda st, a=(ctx, q, k, v, cu, max(lens)), o=out: tq.prompt_attention(*a, o, stream=st)))
    b = Batch(tq, [0, 40], [2000], [2000 + s for s in range(40)])
    ws = tq.alloc_shared_workspace(b.ctx, b.cache, 8, 1, 40, 2000, 60)
    out, args = torch.empty_like(b.q), (_ints(*b.lens), _ints(0, 40), _ints(2000), 40, 2000, 60)
    jobs.append((out, b.ctx, lambda st, o=out: tq.decode_attention_shared(b.ctx, b.cache, b.q, *args, o, None, ws,
                                                                          stream=st)))
    own = tq.Context(D, 3, 3, 0, 42)
    cache = tq.Cache(own, 4, H, 1024)
    rows, fresh, none = heads(3000, H, D), _ints(1000, 900, 800, 300), _ints(0, 0, 0, 0)
    seq_idx, pos = (torch.empty(3000, dtype=torch.int32, device="cuda") for _ in range(2))
    first, ends = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")

    def append(st):
        tq.build_tables(own, cache, none, fresh, seq_idx, pos, first, ends, stream=st)
        tq.quantize(own, cache, rows, rows, seq_idx, pos, stream=st)

    jobs.append((cache.planes["codes_k"], own, append))
    refs = []
    for out, _, call in jobs:
        call(None)
        torch.cuda.synchronize()
        refs.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(40):
        for (_, _, call), st in zip(jobs, streams):
            call(st)
    torch.cuda.synchronize()
    for (out, ctx, _), ref in zip(jobs, refs):
        ctx.check_device_errors()
        assert torch.equal(out, ref)
