"""Causal attention over packed bf16 prompts (tq_prompt_attention) against the
formula in 64 bits: lengths from nothing to several key tiles, every head
dimension, 1 to 16 query heads per KV head, strided rows, both output types,
whatever lies outside the prompts, large scores, capture and refusals.

Tolerances.  With p the softmax weights of a row and p' what the kernel
multiplies V by, |p' - p| <= u p with u = 2^-8 (rounded once to bf16, half a
step of 2^-8 relative) plus a relative 2^-18 (exp2, fp32 scores), so
|o' - o| <= u sum_j p_j |v_j|; a bf16 output adds 2^-8 |o|.  Scores: d
products of bf16 values are exact in fp32 and their sum is off by at most
d 2^-24 sum |q k|, and the argument of exp2 by 2^-23 of its size, which the
scores of a test bound: TOL_S below is that bound on a score, and enters o as
2 TOL_S sum_j p_j |v_j| and lse as TOL_S."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq(cuda_device):
    from kv_cache_vector_12_b200 import tq as tqmod
    return tqmod


_ctx = {}


def context(tq, d):
    if d not in _ctx:
        _ctx[d] = tq.Context(d, 3, 3, 0, 42)
    return _ctx[d]


def rows(n, heads, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(n, heads, d, generator=g)).to(torch.bfloat16).cuda()


def check(q, k, v, out, lse, lens, starts, scale=None):
    """Every row of every prompt within the derived bounds; the worst share of the bound used."""
    n_q, n_kv, d = q.shape[1], k.shape[1], q.shape[2]
    per, scale = n_q // n_kv, scale or 1 / math.sqrt(d)
    worst = 0.0
    for n, a in zip(lens, starts):
        if n == 0:
            continue
        for h in range(n_kv):
            kk, vv = k[a:a + n, h].double(), v[a:a + n, h].double()
            later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            for g in range(h * per, (h + 1) * per):
                qq = q[a:a + n, g].double()
                s = (qq @ kk.t() * scale).masked_fill(later, -math.inf)
                top = (qq.abs() @ kk.abs().t() * scale).masked_fill(later, 0).amax(1)
                tol_s = top * (d * 2.0 ** -24) + 2.0 ** -21 * (1 + s.masked_fill(later, 0).abs().amax(1))
                ref_lse = torch.logsumexp(s, 1)
                p = torch.exp(s - ref_lse[:, None])
                ref, mag = p @ vv, p @ vv.abs()
                tol = (2.0 ** -8 + 2.0 ** -18 + 2 * tol_s)[:, None] * mag + 1e-30
                if out.dtype == torch.bfloat16:
                    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
                err = (out[a:a + n, g].double() - ref).abs()
                assert torch.isfinite(err).all(), (n, g)
                worst = max(worst, (err / tol).max().item())
                if lse is not None:
                    worst = max(worst, ((lse[a:a + n, g].double() - ref_lse).abs() / (tol_s + 2.0 ** -21 * (1 + ref_lse.abs()))).max().item())
    assert worst <= 1.0, worst
    return worst


def run(tq, lens, n_kv, per, d, seed=0, out_dtype=torch.bfloat16, fused=False, gap=0, scale=0.0, mag=1.0):
    """lens packed behind `gap` tokens of NaN and before as many; outputs outside the prompts must stay."""
    ctx = context(tq, d)
    n_tok = sum(lens) + 2 * gap
    if fused:
        qkv = rows(n_tok, n_kv * (per + 2), d, seed, mag)
        q, k, v = qkv[:, :n_kv * per], qkv[:, n_kv * per:n_kv * (per + 1)], qkv[:, n_kv * (per + 1):]
    else:
        q, k, v = (rows(n_tok, hh, d, seed + i, mag) for i, hh in enumerate((n_kv * per, n_kv, n_kv)))
    if gap:
        for x in (q, k, v):
            x[:gap] = float("nan")
            x[n_tok - gap:] = float("inf")
    starts = [gap + int(x) for x in np.cumsum([0] + lens)]
    out = torch.full((n_tok, n_kv * per, d), 7.0, dtype=out_dtype, device="cuda")
    lse = torch.full((n_tok, n_kv * per), 7.0, device="cuda")
    tq.prompt_attention(ctx, q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), max(max(lens), 0), out,
                        lse, scale=scale)
    ctx.check_device_errors()
    if gap:
        for x in (out, lse):
            assert (x[:gap] == 7.0).all() and (x[n_tok - gap:] == 7.0).all()
    return check(q, k, v, out, lse, lens, starts, scale or None)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513, 1500])
def test_one_prompt(tq, d, n):
    run(tq, [n], 2, 4, d, seed=n)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("per", [1, 2, 3, 5, 7, 8, 11, 16])
def test_query_heads_per_kv_head(tq, d, per):
    run(tq, [130, 1, 300], 2, per, d, seed=per)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_ragged_batch_between_nan_and_inf_rows(tq, d):
    """Empty prompts, one-token prompts, prompts that end inside a key tile;
    what lies outside the prompts is NaN or infinite and reaches nothing."""
    run(tq, [0, 1, 700, 0, 0, 129, 5, 384, 1, 0], 2, 4, d, seed=3, gap=200, out_dtype=torch.float32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_strided_rows_of_a_fused_projection(tq, d):
    run(tq, [200, 77], 2, 4, d, seed=4, fused=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_large_scores_move_the_reference(tq, d, out_dtype):
    """Scores of some hundreds: a row's maximum moves from tile to tile."""
    run(tq, [900], 1, 4, d, seed=5, mag=5.0, out_dtype=out_dtype)


def test_rising_scores_rescale_every_tile(tq):
    """Keys that grow with the position: the newest always wins by far more than the lazy bound."""
    for d in (64, 128, 256):
        ctx = context(tq, d)
        n = 700
        q, k, v = rows(n, 4, d, 1), rows(n, 2, d, 2), rows(n, 2, d, 3)
        up = torch.linspace(0.1, 8, n, device="cuda")[:, None, None]
        k = (torch.ones_like(k) * up).to(torch.bfloat16)
        q = (q.abs() * 2).to(torch.bfloat16)
        out = torch.empty(n, 4, d, device="cuda")
        lse = torch.empty(n, 4, device="cuda")
        tq.prompt_attention(ctx, q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, out, lse)
        ctx.check_device_errors()
        check(q, k, v, out, lse, [n], [0])


def test_given_scale_and_no_lse(tq):
    run(tq, [300], 2, 2, 128, seed=6, scale=0.3)
    ctx = context(tq, 128)
    q, k, v = rows(50, 2, 128, 1), rows(50, 1, 128, 2), rows(50, 1, 128, 3)
    out = torch.empty_like(q)
    tq.prompt_attention(ctx, q, k, v, torch.tensor([0, 50], dtype=torch.int32, device="cuda"), 50, out)
    check(q, k, v, out, None, [50], [0])


@pytest.mark.parametrize("n", [33, 40, 200])
def test_many_prompts(tq, n):
    """More sequences than a warp holds: the other order of the query blocks."""
    rng = np.random.default_rng(n)
    run(tq, rng.integers(0, 150, n).tolist(), 2, 4, 128, seed=n)


@pytest.mark.parametrize("n", [1023, 1100, 2500])
def test_more_prompts_than_a_warp_squared(tq, n):
    rng = np.random.default_rng(n)
    run(tq, (rng.integers(0, 9, n) * rng.integers(0, 2, n)).tolist() + [70], 1, 2, 64, seed=n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [767, 768, 769, 2047, 2048, 2049])
def test_either_side_of_the_form_for_short_prompts(tq, d, n):
    run(tq, [n, 300, 0, 65], 1, 4, d, seed=n)


def test_a_nan_in_a_prompt_stays_in_it_and_after_its_tile(tq):
    ctx = context(tq, 128)
    lens = [400, 300]
    q, k, v = rows(700, 4, 128, 1), rows(700, 2, 128, 2), rows(700, 2, 128, 3)
    out = torch.empty(700, 4, 128, device="cuda")
    cu = torch.tensor([0, 400, 700], dtype=torch.int32, device="cuda")
    v[300] = float("nan")
    tq.prompt_attention(ctx, q, k, v, cu, 400, out)
    assert torch.isfinite(out[:300 - 127]).all() and torch.isfinite(out[400:]).all() and out[300:400].isnan().all()


def test_same_call_twice_and_on_another_stream_and_captured(tq):
    ctx = context(tq, 128)
    lens = [513, 100]
    q, k, v = rows(613, 8, 128, 1), rows(613, 2, 128, 2), rows(613, 2, 128, 3)
    cu = torch.tensor([0, 513, 613], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(3)]
    tq.prompt_attention(ctx, q, k, v, cu, 513, outs[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tq.prompt_attention(ctx, q, k, v, cu, 513, outs[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.prompt_attention(ctx, q, k, v, cu, 513, outs[2])
    graph.replay()
    ctx.check_device_errors()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [700, 1500])
def test_same_bits_whatever_ran_before(tq, d, n):
    """With 7 query heads a tile of 128 rows has two of no query, and the last tile more: what an earlier call left
    in their place changes no bit."""
    ctx = context(tq, d)
    q, k, v = rows(n, 14, d, 1), rows(n, 2, d, 2), rows(n, 2, d, 3)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    outs = []
    for mag in (0.0, 1.0, 300.0):
        tq.prompt_attention(ctx, rows(n, 16, d, 9, mag), k, v, cu, n, torch.empty(n, 16, d, device="cuda"))
        out, lse = torch.empty(n, 14, d, device="cuda"), torch.empty(n, 14, device="cuda")
        tq.prompt_attention(ctx, q, k, v, cu, n, out, lse)
        outs.append((out, lse))
    ctx.check_device_errors()
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_bounds_out_of_range_are_flagged(tq):
    ctx = context(tq, 128)
    q, k, v = rows(100, 2, 128, 1), rows(100, 1, 128, 2), rows(100, 1, 128, 3)
    for cu in ([0, 101], [-1, 50], [0, 60], [50, 10]):   # past n_tok, negative, longer than max_len, decreasing
        out = torch.full_like(q, 7.0)
        tq.prompt_attention(ctx, q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 50, out)
        with pytest.raises(tq.TQError) as ei:
            ctx.check_device_errors()
        assert ei.value.status == tq.TQ_ERR_DEVICE and "seq_len" in str(ei.value)
        assert (out == 7.0).all()


def test_refusals_and_empty_calls(tq):
    ctx = context(tq, 128)
    q, k, v = rows(64, 4, 128, 1), rows(64, 2, 128, 2), rows(64, 2, 128, 3)
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)

    def refused(status=tq.TQ_ERR_INVALID, **kw):
        a = dict(q=q, k=k, v=v, cu_seqlens=cu, max_len=64, out=out)
        a.update(kw)
        with pytest.raises(tq.TQError) as ei:
            tq.prompt_attention(ctx, **a)
        assert ei.value.status == status

    refused(max_len=65)
    refused(max_len=-1)
    refused(scale=float("nan"))
    refused(q=rows(64, 3, 128, 1))                                            # 3 heads over 2
    refused(q=rows(64, 17, 128, 1), k=k[:, :1], v=v[:, :1], status=tq.TQ_ERR_UNSUPPORTED)
    wide = torch.empty(64 * (512 + 4) + 8, dtype=torch.bfloat16, device="cuda")
    refused(q=wide[:64 * 516].view(64, 516)[:, :512].unflatten(1, (4, 128)))  # stride no multiple of 8
    refused(q=wide[4:4 + 64 * 512].view(64, 4, 128))                          # 8-byte aligned only
    refused(k=k[:1].expand(64, 2, 128))                                       # stride 0
    ctx.check_device_errors()
    assert (out == 7.0).all()
    tq.prompt_attention(ctx, q, k, v, cu[:1], 64, out)                        # no prompt
    tq.prompt_attention(ctx, q[:0], k[:0], v[:0], torch.zeros(2, dtype=torch.int32, device="cuda"), 0, out[:0])
    tq.prompt_attention(ctx, q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"), 64, out)  # three empty ones
    ctx.check_device_errors()
    assert (out == 7.0).all()


def test_refused_layouts_and_overlaps(tq):
    """What the strides or the types cannot say, and outputs over an input."""
    ctx = context(tq, 128)
    q, k, v = rows(64, 4, 128, 1), rows(64, 2, 128, 2), rows(64, 2, 128, 3)
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((64, 4), 7.0, device="cuda")
    kept = [t.clone() for t in (q, k, v)]

    def refused(**kw):
        with pytest.raises(tq.TQError) as ei:
            tq.prompt_attention(ctx, **{**dict(q=q, k=k, v=v, cu_seqlens=cu, max_len=64, out=out, lse=lse), **kw})
        assert ei.value.status == tq.TQ_ERR_INVALID

    refused(q=q.float())
    refused(k=k.half())
    refused(v=rows(64, 4, 128, 3)[:, ::2])              # every second head
    refused(k=rows(2, 64, 128, 2).transpose(0, 1))      # heads first
    refused(q=rows(64, 4, 64, 1))                       # another head dimension
    refused(out=torch.empty(4, 64, 128, device="cuda").transpose(0, 1))
    refused(out=q)
    whole = torch.zeros(64 * 512 + 64, dtype=torch.bfloat16, device="cuda")
    refused(q=whole[:64 * 512].view(64, 4, 128), out=whole[64:].view(64, 4, 128))
    refused(lse=k.view(-1).view(torch.float32)[:256].view(64, 4))
    refused(lse=out.view(-1).view(torch.float32)[-256:].view(64, 4))
    ctx.check_device_errors()
    assert (out == 7.0).all() and (lse == 7.0).all() and all(torch.equal(a, b) for a, b in zip(kept, (q, k, v)))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_whose_scores_are_all_minus_infinity(tq, d):
    """softmax of nothing but -inf: NaN and lse = -inf as by the formula; a row
    with one finite score gets that key's value."""
    ctx, n = context(tq, d), 300
    q, k, v = rows(n, 2, d, 1), rows(n, 1, d, 2), rows(n, 1, d, 3)
    q[:, :, 0], k[:, :, 0] = 1.0, -math.inf
    k[250] = 0.0
    out, lse = torch.empty(n, 2, d, device="cuda"), torch.empty(n, 2, device="cuda")
    tq.prompt_attention(ctx, q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, out, lse)
    ctx.check_device_errors()
    assert out[:250].isnan().all() and (lse[:250] == -math.inf).all()
    # That key's weight is 2^0, which either exp2 gives within 2^-22; rounded to bf16 (steps of 2^-8 and 2^-7 around 1)
    # it is 1, the others are at most 2^-126.  The sum keeps the 2^-22, so o = v / l and lse = ln l are off by at most
    # that and fp32's roundings of 2^-24 each (reciprocal, product; log2, product): together below 2^-21.
    ref = v[250].float().expand(n - 250, 2, d)
    assert ((out[250:] - ref).abs() <= 2.0 ** -21 * ref.abs()).all() and (lse[250:].abs() <= 2.0 ** -21).all()


def test_two_calls_at_once(tq):
    """On two streams, with nothing shared but the context and the inputs."""
    ctx, lens = context(tq, 128), [700, 1, 333, 64]
    n = sum(lens)
    q, k, v = rows(n, 8, 128, 1), rows(n, 2, 128, 2), rows(n, 2, 128, 3)
    cu = torch.tensor([0, 700, 701, 1034, n], dtype=torch.int32, device="cuda")
    ref = torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")
    tq.prompt_attention(ctx, q, k, v, cu, 700, ref)
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.zeros_like(ref) for _ in range(20)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        tq.prompt_attention(ctx, q, k, v, cu, 700, o, stream=streams[i % 2])
    torch.cuda.synchronize()
    ctx.check_device_errors()
    assert all(torch.equal(o, ref) for o in outs)


@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("d,max_len", [(64, 330), (64, 2200), (128, 330), (128, 2200), (256, 330)])
def test_one_key_of_nan_or_infinity_reaches_every_later_query(tq, d, max_len, kind):
    """A score of NaN or +inf makes its row NaN, wherever in a key tile the key lies and however many steps later the
    query; the rows before it stay within their bounds.  (The bound on the lengths selects the form.)"""
    ctx, n = context(tq, d), 330
    q, k, v = rows(2200, 2, d, 1), rows(2200, 1, d, 2), rows(2200, 1, d, 3)
    q[:, :, 0] = q[:, :, 0].abs() + 1      # (+inf in a key's first coordinate is then a score of +inf)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for j in range(64, 128):
        kk = k.clone()
        kk[j] = float("nan") if kind == "nan" else kk[j]
        kk[j, :, 0] = float(kind)
        out, lse = torch.zeros(2200, 2, d, device="cuda"), torch.zeros(2200, 2, device="cuda")
        tq.prompt_attention(ctx, q, kk, v, cu, max_len, out, lse)
        assert out[j:n].isnan().all() and not torch.isfinite(lse[j:n]).any(), j
        # (the rows before the key see none of it: the formula over those alone)
        check(q, kk, v, out, lse, [j], [0])
    ctx.check_device_errors()
