"""Decode attention for groups that share a prefix (tq_decode_attention_shared)
against the definition in 64 bits on the same packed bytes: the group's first
sequence holds positions below the prefix, each member the ones behind it.

The bound is the library's for attention over the packed cache, 1e-3 of a
row's largest output (and of the largest score for the lse): the softmax
weights times the value norms are rounded to fp16 (2^-11) and q to 16 bits,
all else is fp32; a bf16 output adds its own half step, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

from oracle import turboquant_oracle as o
from tests import parity_helpers as ph

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq(cuda_device):
    from kv_cache_vector_12_b200 import tq as tqmod
    return tqmod


_params = {}


def params(d, bits_k, bits_v, qjl):
    key = (d, bits_k, bits_v, qjl)
    if key not in _params:
        _params[key] = o.Params(d, bits_k, bits_v, bool(qjl), 42)
    return _params[key]


class Batch:
    """A packed cache of random bytes and norms; what no call may use is NaN
    norms (all 16 bits of the norm planes set)."""

    def __init__(self, tq, groups, prefixes, lens, n_kv=2, per=4, d=128, bits_k=3, bits_v=3, qjl=0, block=0, seed=0,
                 q_dtype=torch.float32, norm=11.0):
        self.tq, self.groups, self.prefixes, self.lens = tq, groups, prefixes, lens
        self.n_kv, self.per, self.d, self.block = n_kv, per, d, block
        self.bits_k, self.bits_v, self.qjl = bits_k, bits_v, qjl
        self.ctx = tq.Context(d, bits_k, bits_v, qjl, 42)
        n = len(lens)
        rng = np.random.default_rng(seed)
        self.group_of = [next((g for g in range(len(prefixes)) if groups[g] <= s < groups[g + 1]), None)
                         for s in range(n)]
        unit = block or 64
        longest = max([1] + list(lens) + list(prefixes))
        self.cap = -(-longest // unit) * unit + unit
        # (sequence, position) -> row of the planes
        if block:
            per_seq = self.cap // block
            table, used = np.full((n, per_seq), -1, dtype=np.int32), 0
            for s in range(n):
                g = self.group_of[s]
                lead = s if g is None else groups[g]
                p = 0 if g is None else prefixes[g]
                upto = max(lens[s], p) if s == lead else lens[s]
                # a member's table holds its own blocks from the prefix's end on (whole shared blocks: anything)
                first = 0 if s == lead else p // block
                for j in range(first, -(-upto // block)):
                    table[s, j] = used
                    used += 1
            perm = rng.permutation(used + 3)
            table = np.where(table >= 0, perm[table], table).astype(np.int32)
            self.cache = tq.PagedCache(self.ctx, n, n_kv, self.cap, block, n_blocks=used + 3,
                                       block_table=torch.from_numpy(table))
            self.table = table
        else:
            self.cache = tq.Cache(self.ctx, n, n_kv, self.cap)
        self.planes = {}
        for name, t in self.cache.planes.items():
            if t is None:
                continue
            if t.dtype == torch.uint8:
                a = rng.integers(0, 256, t.shape, dtype=np.uint8)
            else:
                x = {"norm_k": norm, "norm_v": 1.0, "qjl_norm": 0.2}[name] * np.exp(0.3 * rng.standard_normal(t.shape))
                a = x.astype(np.float16).view(np.int16)
                a = self._poison(a)
            self.planes[name] = a
            t.copy_(torch.from_numpy(a))
        self.q = torch.from_numpy(rng.standard_normal((n, n_kv * per, d)).astype(np.float32)).to(q_dtype).cuda()

    def _slot(self, s, p):
        if self.block:
            return self.table[s, p // self.block], p % self.block
        return s, p

    def _poison(self, a):
        """NaN wherever no position of the definition lies."""
        used = np.zeros((a.shape[0], a.shape[2]), dtype=bool)
        for s, n in enumerate(self.lens):
            g = self.group_of[s]
            p = 0 if g is None else self.prefixes[g]
            lead = s if g is None else self.groups[g]
            for x, seq in ((np.arange(p), lead), (np.arange(p, n), s)):
                if len(x):
                    if self.block:
                        used[self.table[seq, x // self.block], x % self.block] = True
                    else:
                        used[seq, x] = True
        for g, p in enumerate(self.prefixes):  # an inactive first sequence holds the prefix too
            if self.groups[g] < self.groups[g + 1] and p:
                x, seq = np.arange(p), self.groups[g]
                if self.block:
                    used[self.table[seq, x // self.block], x % self.block] = True
                else:
                    used[seq, x] = True
        return np.where(used[:, None, :], a, np.int16(-1))

    def rows(self, name, s, h, a, b):
        x = np.arange(a, b)
        if self.block:
            return self.planes[name][self.table[s, x // self.block], h, x % self.block]
        return self.planes[name][s, h, x]

    def call(self, out_dtype=torch.float32, scale=0.0, stream=None, max_group=None, max_prefix=None, max_suffix=None,
             workspace=None, out=None, lse=None):
        tq, dev = self.tq, "cuda"
        n = len(self.lens)
        mg = max_group or max([1] + [b - a for a, b in zip(self.groups, self.groups[1:])])
        mp = max(self.prefixes) if max_prefix is None else max_prefix
        suffix = [x - (0 if g is None else self.prefixes[g]) for x, g in zip(self.lens, self.group_of) if x]
        ms = max([0] + suffix) if max_suffix is None else max_suffix
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        if workspace is None:
            workspace = tq.alloc_shared_workspace(self.ctx, self.cache, self.n_kv * self.per, len(self.prefixes), mg, mp, ms)
            workspace.fill_(0xFF)  # NaN: nothing may be read that was not written
        if out is None:
            out = torch.full(self.q.shape, 7.0, dtype=out_dtype, device=dev)
            lse = torch.full(self.q.shape[:2], 7.0, device=dev)
        tq.decode_attention_shared(self.ctx, self.cache, self.q, ints(self.lens), ints(self.groups),
                                   ints(self.prefixes), mg, mp, ms, out, lse, workspace, scale=scale, stream=stream)
        return out, lse

    def check(self, out, lse, scale=None, skip=(), large=False, heads_of=None):
        p = params(self.d, self.bits_k, self.bits_v, self.qjl)
        f16 = ph.f16_bits_to_f64
        bf16 = out.dtype == torch.bfloat16
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        for s, n in enumerate(self.lens):
            if s in skip:
                continue
            if n == 0:
                assert (got[s] == 0).all() and (got_lse[s] == -math.inf).all(), s
                continue
            g = self.group_of[s]
            lead, pre = self.groups[g], self.prefixes[g]
            for h in heads_of or range(self.n_kv):
                cat = lambda name: np.concatenate([self.rows(name, lead, h, 0, pre), self.rows(name, s, h, pre, n)])  # noqa: E731
                heads = slice(h * self.per, (h + 1) * self.per)
                extra = {}
                if self.qjl:
                    extra = dict(s_matrix=p.s, qjl_signs=o.unpack_signs(cat("qjl_bits"), self.d),
                                 qjl_gamma=f16(cat("qjl_norm")))
                ref, ref_lse, scores = o.decode_attention(
                    q[s, heads], p.pi, p.ck, o.unpack_codes(cat("codes_k"), self.bits_k, self.d), f16(cat("norm_k")),
                    p.cv, o.unpack_codes(cat("codes_v"), self.bits_v, self.d), f16(cat("norm_v")),
                    scale or 1 / math.sqrt(self.d), **extra)
                top = np.abs(ref).max(axis=1, keepdims=True)
                tol = 1e-3 * top + (2.0 ** -8 * np.abs(ref) if bf16 else 0)
                if large:
                    # q_hat is held in steps of max|q_hat| / 32767, so a coordinate is off by at most half of one
                    # and a score by E = scale n_j |half step| sum_i |c_i| <= E_max; every weight is then off by a
                    # factor within exp(+-2 E_max), and the output by (exp(2 E_max) - 1) sum_j p_j |v_j|
                    q_hat = q[s, heads] @ p.pi.T
                    keys = np.abs(np.asarray(p.ck)[o.unpack_codes(cat("codes_k"), self.bits_k, self.d)]).sum(1)
                    e_max = (np.abs(q_hat).max(1) / 65534 * (f16(cat("norm_k")) * keys).max() / math.sqrt(self.d))[:, None]
                    w = np.exp(scores - ref_lse[:, None])
                    vals = (f16(cat("norm_v"))[:, None] * np.asarray(p.cv)[o.unpack_codes(cat("codes_v"), self.bits_v, self.d)]) @ p.pi
                    tol = tol + np.expm1(2 * e_max) * (w @ np.abs(vals))
                err = np.abs(got[s, heads] - ref)
                assert (err <= tol).all(), (s, h, (err / tol).max())
                big = np.maximum(1.0, np.abs(scores).reshape(self.per, -1).max(axis=1))
                assert (np.abs(got_lse[s, heads] - ref_lse) <= 1e-3 * big).all(), (s, h)

    def run(self, large=False, **kw):
        out, lse = self.call(**kw)
        self.ctx.check_device_errors()
        self.check(out, lse, kw.get("scale"), large=large)


SETTINGS = [(2, 2, 0), (3, 3, 0), (4, 4, 0), (3, 2, 0), (2, 4, 1), (3, 3, 1), (4, 2, 1)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bits_k,bits_v,qjl", SETTINGS)
def test_settings_and_head_dimensions(tq, d, bits_k, bits_v, qjl):
    Batch(tq, [0, 3, 5], [300, 129], [301, 380, 300, 129, 200], d=d, bits_k=bits_k, bits_v=bits_v, qjl=qjl, seed=d).run()


@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 1000])
@pytest.mark.parametrize("suffix", [0, 1, 64, 130])
def test_prefix_and_suffix_lengths(tq, prefix, suffix):
    lens = [prefix + suffix, prefix + max(0, suffix - 1), prefix]
    Batch(tq, [0, 3], [prefix], lens, seed=prefix + suffix).run()


@pytest.mark.parametrize("per", [1, 2, 3, 5, 7, 8, 11, 16])
@pytest.mark.parametrize("n", [1, 2, 6, 19])
def test_group_sizes_and_query_heads(tq, per, n):
    rng = np.random.default_rng(per * n)
    lens = (200 + rng.integers(0, 90, n)).tolist()
    Batch(tq, [0, n], [200], lens, n_kv=2, per=per, seed=n).run()


@pytest.mark.parametrize("per,n", [(4, 33), (8, 16), (8, 17), (7, 37), (16, 9), (1, 130), (3, 90)])
def test_large_groups(tq, per, n):
    """More rows than one matrix tile of 128 holds, and just as many."""
    rng = np.random.default_rng(per * n)
    lens = (500 + rng.integers(0, 40, n)).tolist()
    Batch(tq, [0, n], [500], lens, n_kv=1, per=per, seed=n, q_dtype=torch.bfloat16).run()


@pytest.mark.parametrize("block", [64, 128, 256])
@pytest.mark.parametrize("qjl", [0, 1])
def test_paged_members_tables_hold_only_their_own_blocks(tq, block, qjl):
    """Unequal groups, one of them empty, one of one sequence; sequences that take no part, the first of a group too."""
    lens = [700, 612, 0, 612, 0, 335, 333, 512, 50, 0, 0]
    Batch(tq, [0, 4, 4, 7, 8, 11], [612, 100, 333, 512, 0], lens, block=block, qjl=qjl, seed=block).run()


def test_bf16_output_and_given_scale(tq):
    b = Batch(tq, [0, 5], [900], [901, 950, 900, 1030, 1000], q_dtype=torch.bfloat16)
    b.run(out_dtype=torch.bfloat16)
    b.run(out_dtype=torch.bfloat16, scale=0.5)


def test_large_norms(tq):
    """Scores of some hundreds (key norms of some hundreds, as a model without key normalisation has)."""
    Batch(tq, [0, 4], [700], [730, 701, 720, 760], norm=400.0, bits_k=4, bits_v=4, seed=1).run(large=True)
    Batch(tq, [0, 40], [700], [700 + i for i in range(40)], norm=400.0, bits_k=4, bits_v=4, seed=1).run(large=True)


@pytest.mark.parametrize("n,per", [(4, 4), (32, 4)])
def test_long_prefix_over_many_splits(tq, n, per):
    rng = np.random.default_rng(n)
    Batch(tq, [0, n], [20001], (20001 + rng.integers(0, 700, n)).tolist(), n_kv=1, per=per, seed=3).run()


@pytest.mark.parametrize("prefix", [1400, 2049])
@pytest.mark.parametrize("bits_k,bits_v", [(3, 3), (4, 2)])
def test_many_key_tiles_in_one_split(tq, prefix, bits_k, bits_v):
    """As many (group, KV head) pairs as the GPU has SMs, so that every CTA walks its prefix alone; keys whose
    scores rise along the prefix, so that a row's maximum keeps moving."""
    groups = [5 * g for g in range(11)]
    b = Batch(tq, groups, [prefix] * 10, [prefix + 3 * (s % 7) for s in range(50)], n_kv=16, per=4, bits_k=bits_k,
              bits_v=bits_v, seed=prefix)
    up = (np.linspace(1, 40, b.cap)[None, None, :] * np.ones(b.planes["norm_k"].shape)).astype(np.float16)
    b.planes["norm_k"] = b._poison(up.view(np.int16))
    b.cache.planes["norm_k"].copy_(torch.from_numpy(b.planes["norm_k"]))
    out, lse = b.call()
    b.ctx.check_device_errors()
    b.check(out, lse, skip=[s for s in range(50) if s % 9], heads_of=(0, 15))


def test_many_groups(tq):
    """More groups than a warp holds."""
    rng = np.random.default_rng(2)
    sizes = rng.integers(0, 4, 71).tolist()
    groups = [0] + np.cumsum(sizes).tolist()
    prefixes = rng.integers(0, 200, 71).tolist()
    lens = [prefixes[g] + int(rng.integers(0, 80)) for g, k in enumerate(sizes) for _ in range(k)]
    Batch(tq, groups, prefixes, lens, n_kv=1, per=2, seed=7).run()


def test_queries_of_sequences_that_take_no_part_reach_nothing(tq):
    """Length 0, and a query of NaN, infinity or zero: the others' outputs keep their bits."""
    for n in (3, 40):
        lens = [900 + (s % 9) if s % 3 else 0 for s in range(n)]
        b, outs = Batch(tq, [0, n], [900], lens, seed=4), []
        for x in (0.0, float("nan"), float("inf"), 1e4):
            b.q[::3] = x
            out, lse = b.call()
            b.ctx.check_device_errors()
            outs.append((out, lse))
        b.check(*outs[1])
        for out, lse in outs[1:]:
            assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_equals_decode_attention_over_copies(tq):
    """The same values as tq_decode_attention where every sequence holds the prefix itself."""
    n, prefix, lens = 3, 640, [700, 641, 777]
    b = Batch(tq, [0, n], [prefix], lens)
    out, lse = b.call()
    for t in b.cache.planes.values():
        if t is not None:
            t[1:, :, :prefix] = t[:1, :, :prefix]
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    ws = tq.alloc_workspace(b.ctx, n, out.shape[1], max(lens))
    tq.decode_attention(b.ctx, b.cache, b.q, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), ref,
                        ref_lse, ws)
    b.ctx.check_device_errors()
    assert ((out - ref).abs() <= 1e-3 * ref.abs().amax(-1, keepdim=True)).all()


def test_bounds_are_flagged_and_the_others_stay_right(tq):
    def flagged(b, skip, **kw):
        out, lse = b.call(**kw)
        with pytest.raises(tq.TQError) as ei:
            b.ctx.check_device_errors()
        assert ei.value.status == tq.TQ_ERR_DEVICE and "seq_len" in str(ei.value)
        for s in skip:
            assert (out[s] == 0).all() and (lse[s] == -math.inf).all()
        b.check(out, lse, skip=skip)

    flagged(Batch(tq, [0, 3], [100], [150, 99, 120]), [1])                          # shorter than the prefix
    flagged(Batch(tq, [0, 3], [100], [150, 110, 120]), [0], max_suffix=49)          # longer than the bound
    flagged(Batch(tq, [0, 2, 4], [100, 200], [150, 110, 220, 201]), [2, 3], max_prefix=199)
    flagged(Batch(tq, [0, 3, 4], [100, 50], [150, 110, 120, 60]), [0, 1, 2], max_group=2)
    flagged(Batch(tq, [0, 2], [100], [150, 110, 120]), [2])                         # outside every group
    b = Batch(tq, [0, 2], [100], [150, 110])
    b.lens = [-5, 110]
    flagged(b, [0])
    b.lens = [2 ** 31 - 1, 110]
    flagged(b, [0], max_suffix=64)


def test_captured_replayed_and_on_another_stream(tq):
    b = Batch(tq, [0, 3, 5], [300, 129], [301, 380, 300, 129, 200])
    mg, mp, ms = 3, 300, 128
    ws = tq.alloc_shared_workspace(b.ctx, b.cache, b.n_kv * b.per, 2, mg, mp, ms)
    first, first_lse = b.call(workspace=ws, max_suffix=ms)
    torch.cuda.synchronize()
    out, lse = torch.zeros_like(first), torch.zeros_like(first_lse)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, groups, prefixes = ints(b.lens), ints(b.groups), ints(b.prefixes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.decode_attention_shared(b.ctx, b.cache, b.q, lens, groups, prefixes, mg, mp, ms, out, lse, ws)
    ws.fill_(0xFF)
    graph.replay()
    b.ctx.check_device_errors()
    assert torch.equal(out, first) and torch.equal(lse, first_lse)
    lens.copy_(ints([330, 0, 310, 257, 140]))  # other lengths under the same bounds
    graph.replay()
    b.ctx.check_device_errors()
    side = torch.cuda.Stream()
    b2 = torch.zeros_like(out), torch.zeros_like(lse)
    torch.cuda.synchronize()
    tq.decode_attention_shared(b.ctx, b.cache, b.q, lens, groups, prefixes, mg, mp, ms, *b2, ws, stream=side)
    side.synchronize()
    # bit for bit: the longer lengths reach norms that were never written (NaN), which two outputs then share
    assert torch.equal(out.view(torch.int32), b2[0].view(torch.int32))
    assert torch.equal(lse.view(torch.int32), b2[1].view(torch.int32)) and not lse[1].isnan().any()


def test_refusals(tq):
    b = Batch(tq, [0, 2], [64], [80, 90])
    ok = dict(seq_lens=torch.tensor([80, 90], dtype=torch.int32, device="cuda"),
              cu_group=torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
              prefix_lens=torch.tensor([64], dtype=torch.int32, device="cuda"), max_group=2, max_prefix_len=64,
              max_suffix_len=64, out=torch.full(b.q.shape, 7.0, device="cuda"),
              lse=torch.full(b.q.shape[:2], 7.0, device="cuda"), q=b.q)
    ws = tq.alloc_shared_workspace(b.ctx, b.cache, 8, 1, 2, 64, 64)

    def refused(status=tq.TQ_ERR_INVALID, workspace=ws, cache=b.cache, **kw):
        with pytest.raises(tq.TQError) as ei:
            tq.decode_attention_shared(b.ctx, cache, workspace=workspace, **{**ok, **kw})
        assert ei.value.status == status

    refused(max_group=0)
    refused(max_group=3)
    refused(max_prefix_len=b.cap + 1)
    refused(max_prefix_len=-1)
    refused(max_suffix_len=b.cap + 1)
    refused(seq_lens=None)
    refused(cu_group=None)
    refused(scale=float("inf"))
    refused(q=b.q[:, :7])
    refused(workspace=ws[:256])
    refused(workspace=torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:])
    refused(prefix_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    refused(status=tq.TQ_ERR_UNSUPPORTED, q=torch.zeros(2, 34, 128, device="cuda"))
    assert tq.shared_workspace_bytes(b.ctx, b.cache, 8, 1, 3, 64, 64) == 0
    assert tq.shared_workspace_bytes(b.ctx, b.cache, 7, 1, 2, 64, 64) == 0
    b.ctx.check_device_errors()
    assert (ok["out"] == 7.0).all()


@pytest.mark.parametrize("d,qjl,n", [(128, 0, 6), (128, 0, 2), (64, 0, 3), (128, 1, 4)])
def test_a_finished_group_holds_nothing(tq, d, qjl, n):
    """A padded batch: no member of the group takes part, so its table rows may name no block."""
    b = Batch(tq, [0, n, n + 3], [200, 130], [0] * n + [200, 130, 190], d=d, qjl=qjl, block=64, per=4)
    b.cache.block_table[:n] = -1
    out, lse = b.call()
    b.ctx.check_device_errors()
    b.check(out, lse)


def test_one_member_groups_fill_the_batch(tq):
    """As many groups as sequences, with room for more members than any has: units are counted by sequences."""
    n = 300
    Batch(tq, list(range(n + 1)), [65 + s % 3 for s in range(n)], [70 + s % 7 for s in range(n)], n_kv=1, per=16).run(
        max_group=n)


def test_refused_overlaps_and_capacity(tq):
    b = Batch(tq, [0, 2], [64], [80, 90])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = tq.alloc_shared_workspace(b.ctx, b.cache, 8, 1, 2, 64, 64)
    ok = dict(q=b.q, seq_lens=ints([80, 90]), cu_group=ints([0, 2]), prefix_lens=ints([64]), max_group=2,
              max_prefix_len=64, max_suffix_len=64, out=torch.full(b.q.shape, 7.0, device="cuda"),
              lse=torch.full(b.q.shape[:2], 7.0, device="cuda"), workspace=ws)
    kept = b.q.clone()

    def refused(status=tq.TQ_ERR_INVALID, **kw):
        with pytest.raises(tq.TQError) as ei:
            tq.decode_attention_shared(b.ctx, b.cache, **{**ok, **kw})
        assert ei.value.status == status

    refused(out=b.q)
    refused(lse=ok["out"].view(-1)[:16].view(2, 8))
    refused(out=ws.view(torch.float32)[:b.q.numel()].view(b.q.shape))
    refused(seq_lens=ws[256:264].view(torch.int32))
    refused(lse=b.q.view(-1)[-16:].view(2, 8))
    capacity = b.cache.struct.capacity
    b.cache.struct.capacity = 2 ** 30 + 64
    refused(status=tq.TQ_ERR_UNSUPPORTED)
    assert tq.shared_workspace_bytes(b.ctx, b.cache, 8, 1, 2, 64, 64) == 0
    b.cache.struct.capacity = capacity
    b.ctx.check_device_errors()
    assert (ok["out"] == 7.0).all() and (ok["lse"] == 7.0).all() and torch.equal(b.q, kept)


@pytest.mark.parametrize("n,per", [(3, 4), (40, 4)])
def test_two_calls_at_once(tq, n, per):
    """On two streams, each with its own workspace."""
    b = Batch(tq, [0, n], [900], [901 + s % 60 for s in range(n)], per=per)
    ref, ref_lse = b.call()
    spaces = [tq.alloc_shared_workspace(b.ctx, b.cache, b.n_kv * per, 1, n, 900, 60) for _ in range(2)]
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.zeros_like(ref) for _ in range(20)]
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (b.lens, b.groups, b.prefixes)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        tq.decode_attention_shared(b.ctx, b.cache, b.q, *ints, n, 900, 60, o, None, spaces[i % 2],
                                   stream=streams[i % 2])
    torch.cuda.synchronize()
    b.ctx.check_device_errors()
    assert all(torch.equal(o, ref) for o in outs)


@pytest.mark.parametrize("per", [4, 8])
def test_groups_that_end_behind_the_batch_or_decrease_are_flagged(tq, per):
    """Groups that the prefix pass cannot cut into units (16 rows per CTA with 4 query heads per KV head, tcgen05 with
    8): their sequences are 0, whatever the workspace held, and the others right."""
    def flagged(b, skip, **kw):
        out, lse = b.call(**kw)
        with pytest.raises(tq.TQError) as ei:
            b.ctx.check_device_errors()
        assert ei.value.status == tq.TQ_ERR_DEVICE and "seq_len" in str(ei.value)
        for s in skip:
            assert (out[s] == 0).all() and (lse[s] == -math.inf).all(), s
        b.check(out, lse, skip=skip)

    flagged(Batch(tq, [0, 2, 6], [100, 200], [150, 110, 220, 201], per=per), [2, 3])
    flagged(Batch(tq, [0, 2, 2 ** 31 - 1], [100, 200], [150, 110, 220, 201], per=per), [2, 3], max_group=4)
    lens = [300 + s for s in range(8)]
    for groups in ([4, 6, 0, 8], [0, 5, 3, 8], [0, 8, 0, 8]):
        flagged(Batch(tq, groups, [300, 290, 280], lens, per=per), range(8), max_group=8)


@pytest.mark.parametrize("d,qjl,n_kv,per,sizes,prefix", [(128, 0, 8, 4, [32], 2560), (128, 0, 2, 4, [4] * 8, 3584),
                                                        (128, 1, 2, 7, [8] * 2, 3584), (64, 0, 2, 4, [5, 3], 3840),
                                                        (256, 0, 2, 2, [2, 9], 3840)])
def test_a_workspace_for_the_largest_bounds_serves_smaller_ones(tq, d, qjl, n_kv, per, sizes, prefix):
    """The fastest split of a smaller call may take more slots: it then runs with those there are."""
    groups, n = [0] + np.cumsum(sizes).tolist(), sum(sizes)
    n_q, ms = n_kv * per, 200
    b = Batch(tq, groups, [prefix] * len(sizes), [prefix + 1 + s % 60 for s in range(n)], n_kv=n_kv, d=d, qjl=qjl, per=per,
              seed=d)
    size = tq.shared_workspace_bytes(b.ctx, b.cache, n_q, len(sizes), max(sizes), prefix, ms)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for p in (prefix, prefix - 64, prefix - 128, prefix - 192, prefix - 256, prefix // 2, 100, 1):
        for suffix in (60, ms):
            b.prefixes = [p] * len(sizes)
            b.lens = [p + 1 + s % 60 for s in range(n)]
            for norms in ("norm_k", "norm_v", "qjl_norm"):  # (no NaN outside the first call's positions: p is below)
                if norms in b.planes:
                    x = b.planes[norms]
                    b.planes[norms] = np.where(x == -1, np.float16(1).view(np.int16), x)
                    b.cache.planes[norms].copy_(torch.from_numpy(b.planes[norms]))
            ws.fill_(0xFF)
            out, lse = b.call(workspace=ws, max_suffix=suffix)
            b.ctx.check_device_errors()
            b.check(out, lse, skip=[s for s in range(n) if s % 7], heads_of=(1,))
    # pairs behind the same prefix, each held by its own first sequence
    b.groups = list(range(0, n, 2)) + [n]
    b.prefixes = [100] * (len(b.groups) - 1)
    b.group_of = [s // 2 for s in range(n)]
    b.lens = [101 + s % 60 for s in range(n)]
    out, lse = b.call(workspace=ws, max_suffix=ms)
    b.ctx.check_device_errors()
    b.check(out, lse, heads_of=(1,))


def test_the_smallest_workspace(tq):
    """One slot a row for the prefixes and one behind them; without prefixes one; a byte less is refused."""
    for n, d, qjl in ((3, 128, 0), (30, 128, 0), (3, 128, 1), (3, 64, 0), (5, 256, 0)):
        for prefix in (1500, 0):
            b = Batch(tq, [0, n], [prefix], [prefix + 300 + s for s in range(n)], d=d, qjl=qjl)
            least = n * 8 * (d + 4) * 4 * (2 if prefix else 1)
            ws = torch.full((least + 1024,), 0xFF, dtype=torch.uint8, device="cuda")
            out, lse = b.call(workspace=ws[:least])
            b.ctx.check_device_errors()
            b.check(out, lse, skip=range(5, n))
            assert (ws[least:] == 0xFF).all()
            with pytest.raises(tq.TQError) as ei:
                b.call(workspace=ws[:least - 1])
            assert ei.value.status == tq.TQ_ERR_INVALID and "workspace" in str(ei.value)


@pytest.mark.parametrize("n,per,qjl", [(4, 4, 0), (40, 4, 0), (6, 7, 1)])
def test_inputs_written_just_before_the_call(tq, n, per, qjl):
    """The pass behind the prefixes does not wait for the prefix pass, and still reads what the kernels in front of the
    call wrote: queries, lengths and cached bytes that change right before every call, captured and replayed, and a
    workspace that was used, is new or is filled in between."""
    b = Batch(tq, [0, n], [700], [900 + s % 60 for s in range(n)], per=per, qjl=qjl)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    groups, prefixes, lens = ints(b.groups), ints(b.prefixes), ints(b.lens)
    ws = tq.alloc_shared_workspace(b.ctx, b.cache, b.n_kv * per, 1, n, 700, 260)
    g = torch.Generator(device="cuda").manual_seed(n)
    planes = [t for t in b.cache.planes.values() if t is not None and t.dtype == torch.uint8]
    sets = [([torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8) for t in planes],
             torch.randn(b.q.shape, generator=g, device="cuda"), lens - 13 * i) for i in range(4)]
    src = [[t.clone() for t in sets[0][0]], sets[0][1].clone(), sets[0][2].clone()]
    out, lse = torch.zeros_like(b.q), torch.zeros(b.q.shape[:2], device="cuda")

    def step():
        for t, x in zip(planes, src[0]):
            t.copy_(x)
        b.q.copy_(src[1])
        lens.copy_(src[2])
        tq.decode_attention_shared(b.ctx, b.cache, b.q, lens, groups, prefixes, n, 700, 260, out, lse, ws)

    def select(i):
        for t, x in zip([*src[0], src[1], src[2]], [*sets[i][0], sets[i][1], sets[i][2]]):
            t.copy_(x)

    refs = []
    for i in range(4):
        select(i)
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        refs.append((out.clone(), lse.clone()))
    assert not any(torch.equal(refs[0][0], r[0]) for r in refs[1:])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    got = []
    for i in range(60):
        select(i % 4)
        if i % 3 == 0:
            ws.fill_(i)
        graph.replay() if i % 2 else step()
        got.append((out.clone(), lse.clone()))
    b.ctx.check_device_errors()
    for i, (x, y) in enumerate(got):
        assert torch.equal(x, refs[i % 4][0]) and torch.equal(y, refs[i % 4][1]), i


@pytest.mark.parametrize("d,qjl,n", [(64, 0, 3), (128, 0, 3), (128, 1, 3), (256, 0, 3), (128, 0, 40)])
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("prefix", [0, 300])
def test_a_query_of_nan_or_infinity_makes_its_row_nan(tq, d, qjl, n, value, prefix):
    """One coordinate of one head's query: that row is NaN in both passes, every other row right."""
    b = Batch(tq, [0, n], [prefix], [prefix + 40 + s for s in range(n)], d=d, qjl=qjl)
    clean, clean_lse = b.call()
    b.check(clean, clean_lse, skip=range(5, n))
    b.q[1, 2, 5] = float(value)
    out, lse = b.call()
    b.ctx.check_device_errors()
    assert out[1, 2].isnan().all() and lse[1, 2].isnan()
    others = torch.ones_like(lse, dtype=torch.bool)
    others[1, 2] = False
    # (the same inputs, and a row's maximum moves with no other row's: the same bits but for tcgen05 rescales of a
    # warp's rows together, whose factor of 1 is exact and whose moved references round anew)
    err = (out - clean).abs().amax(-1) / clean.abs().amax(-1)
    assert (err[others] <= 1e-3).all()
