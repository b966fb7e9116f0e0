"""Measured cases of the serving operators around the packed KV cache.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and, where ``own`` is true, as a user's program
calls it through ``kv_cache_vector_12_b200.tq``:

* ``tables``  the block table, the per-token slot maps and the cumulative
              lengths of one engine step, from request lengths on the GPU
              (``tq.build_tables``);
* ``prompt``  causal attention over whole bf16 prompts of different lengths,
              packed one behind the other, with grouped query heads
              (``tq.prompt_attention``);
* ``shared``  decode attention over the packed cache for a batch whose groups
              of sequences share a long prefix (``tq.decode_attention_shared``).

Sizes are those of the package's workloads (8 KV and 32 or 64 query heads, 4 KV
and 28 query heads, contexts up to 131072 tokens, 32 serving sequences) and
generic ones around them.  The lengths of a case come from the case alone, in
an order that comes from the seed; every other value comes from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PI_SEED = 42  # the seed of the rotation, as in the package's workloads


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of the 32-sequence serving batch: a new token each, latency counts
        dict(name="tables_step", op="tables", n_seqs=32, block=256, capacity=65536, max_cached=65535, max_new=1,
             groups=0, lens=1),
        # a wide decode step, requests in groups that share a prefix, small blocks
        dict(name="tables_groups", op="tables", n_seqs=1013, block=64, capacity=32768, max_cached=32000, max_new=1,
             groups=37, lens=2),
        # admission of 32 prompts of up to 65536 tokens: a slot for each of about a million tokens
        dict(name="tables_prompts", op="tables", n_seqs=32, block=256, capacity=65536, max_cached=0, max_new=65536,
             groups=0, lens=3),
        # the smallest prompt batch: three short requests on a small model
        dict(name="prompt_short", op="prompt", n_seqs=3, min_len=1, max_len=200, n_kv=2, n_q=8, d=64, fused=False,
             lens=4),
        # ordinary ragged batch, projections fused in one buffer (strided rows)
        dict(name="prompt_ragged", op="prompt", n_seqs=17, min_len=1, max_len=4001, n_kv=8, n_q=32, d=128, fused=True,
             lens=5),
        # one long prompt, 28 query heads over 4 KV heads
        dict(name="prompt_7per", op="prompt", n_seqs=1, min_len=16384, max_len=16384, n_kv=4, n_q=28, d=128,
             fused=False, lens=6),
        # the longest: one 32768-token prompt at 32 query heads
        dict(name="prompt_long", op="prompt", n_seqs=1, min_len=32768, max_len=32768, n_kv=8, n_q=32, d=128,
             fused=False, lens=7),
        # wide heads
        dict(name="prompt_d256", op="prompt", n_seqs=5, min_len=100, max_len=5000, n_kv=4, n_q=16, d=256, fused=True,
             lens=8),
        # two short requests behind one system prompt: latency counts
        dict(name="shared_small", op="shared", n_seqs=2, n_kv=2, n_q=8, d=128, bits_k=3, bits_v=3, qjl=False, block=0,
             n_groups=1, prefix=1000, max_suffix=100, lens=9),
        # the serving batch behind one long prompt, paged cache
        dict(name="shared_serving", op="shared", n_seqs=32, n_kv=8, n_q=32, d=128, bits_k=3, bits_v=3, qjl=False,
             block=256, n_groups=1, prefix=32768, max_suffix=1500, lens=10),
        # 8 query heads per KV head, the longest context, four samples of one prompt
        dict(name="shared_131k", op="shared", n_seqs=4, n_kv=8, n_q=64, d=128, bits_k=3, bits_v=3, qjl=False, block=0,
             n_groups=1, prefix=131072 - 64, max_suffix=64, lens=11),
        # several groups of unequal size, residual signs on K, 7 query heads per KV head
        dict(name="shared_groups", op="shared", n_seqs=13, n_kv=4, n_q=28, d=128, bits_k=2, bits_v=4, qjl=True,
             block=128, n_groups=4, prefix=9000, max_suffix=700, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "prompt", "prompt", "shared", "shared"])
    lens = rng.randrange(1, 1 << 30)
    if op == "tables":
        n_seqs = _log_int(rng, 1, 2000)
        block = rng.choice([64, 128, 256])
        kind = rng.choice(["step", "mixed", "prompts"])
        room = max(256, min(65536, (1 << 20) // n_seqs))  # about a million new tokens at most
        max_new = 1 if kind == "step" else _log_int(rng, 2, room)
        max_cached = 0 if kind == "prompts" else _log_int(rng, 1, 32768)
        groups = 0 if kind == "prompts" or n_seqs < 4 else rng.choice([0, rng.randint(1, n_seqs // 2)])
        capacity = -(-(max_cached + max_new) // block) * block
        return dict(op=op, n_seqs=n_seqs, block=block, capacity=capacity, max_cached=max_cached, max_new=max_new,
                    groups=groups, lens=lens)
    n_kv, per = rng.choice([(1, 1), (2, 4), (8, 4), (4, 7), (8, 8), (2, 16), (4, 3)])
    if op == "prompt":
        n_seqs = _log_int(rng, 1, 64)
        d = rng.choice([64, 128, 128, 256])
        # the quadratic work stays below that of 32768 tokens at 32 heads of 128
        top = min(20000, math.sqrt(32768.0 ** 2 * 32 * 128 / (4.0 * n_seqs * n_kv * per * d)))
        max_len = _log_int(rng, 16, top)
        return dict(op=op, n_seqs=n_seqs, min_len=1, max_len=max_len, n_kv=n_kv, n_q=n_kv * per, d=d,
                    fused=rng.random() < 0.5, lens=lens)
    n_seqs = _log_int(rng, 2, 64)
    d = rng.choice([64, 128, 128, 128, 256])
    bits_k, bits_v = rng.choice([(2, 2), (3, 3), (4, 4), (4, 2), (2, 4), (3, 4)])
    prefix = _log_int(rng, 64, min(100000, (1 << 28) // (n_seqs * n_kv * d)))
    return dict(op=op, n_seqs=n_seqs, n_kv=n_kv, n_q=n_kv * per, d=d, bits_k=bits_k, bits_v=bits_v,
                qjl=rng.random() < 0.25, block=rng.choice([0, 64, 256]), n_groups=rng.randint(1, max(1, n_seqs // 3)),
                prefix=prefix, max_suffix=_log_int(rng, 1, min(2000, max(2, prefix))), lens=lens)


# ------------------------------------------------------- lengths and groups
def _lengths(case, seed):
    """The case's request lengths in the seed's order (host lists)."""
    r = random.Random(case["lens"])
    n = case["n_seqs"]
    if case["op"] == "prompt":
        got = [r.randint(case["min_len"], case["max_len"]) for _ in range(n)]
        got[0] = case["max_len"]
    elif case["op"] == "shared":
        got = [r.randint(0, case["max_suffix"]) for _ in range(n)]
        got[0] = case["max_suffix"]
    else:
        got = [(r.randint(min(1, case["max_cached"]), case["max_cached"]), r.randint(1, case["max_new"]))
               for _ in range(n)]
        got[0] = (case["max_cached"], case["max_new"])
    random.Random(seed).shuffle(got)
    return got


def _group_bounds(case):
    """First sequence of each group, and the end: n_groups + 1 numbers."""
    n, g = case["n_seqs"], case.get("n_groups", case.get("groups", 0))
    cuts = sorted(random.Random(case["lens"] + 1).sample(range(1, n), g - 1)) if g > 1 else []
    return [0] + cuts + [n]


def _prefixes(case):
    """The shared prefix length of each group: the first has the case's, the others between half of it and all of it."""
    r = random.Random(case["lens"] + 2)
    return [case["prefix"]] + [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(case["n_groups"] - 1)]


# ------------------------------------------------ parameters of the method
def _gaussians(seed, stream, count):
    """SplitMix64 used as a counter-based generator, Box-Muller on 53-bit uniforms."""
    with np.errstate(over="ignore"):
        n = np.arange(1, 2 * ((count + 1) // 2) + 1, dtype=np.uint64) + np.uint64(stream << 32)
        z = np.uint64(seed) + n * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    u = (z >> np.uint64(11)).astype(np.float64)
    radius = np.sqrt(-2.0 * np.log((u[0::2] + 1.0) / 2.0 ** 53))
    angle = 2.0 * math.pi * u[1::2] / 2.0 ** 53
    return np.stack([radius * np.cos(angle), radius * np.sin(angle)], 1).reshape(-1)[:count]


def _rotation(d):
    """Pi: the QR factor of a seeded Gaussian matrix, R's diagonal positive, rounded once to bf16 (8 bits)."""
    qm, rm = np.linalg.qr(_gaussians(PI_SEED, 0, d * d).reshape(d, d))
    m, e = np.frexp(qm * np.sign(np.diag(rm)))
    return torch.from_numpy(np.ldexp(np.rint(m * 256.0), e - 8))


def _centroids(bits, d):
    """Lloyd-Max centroids of N(0, 1) over sqrt(d), rounded to fp16 (made once, before any pass)."""
    c = np.linspace(-2.0, 2.0, 1 << bits)
    cdf = np.vectorize(lambda t: 0.5 * math.erfc(-t / math.sqrt(2.0)))
    for _ in range(4000):
        t = np.concatenate([[-40.0], (c[1:] + c[:-1]) / 2, [40.0]])
        f = np.exp(-0.5 * t * t) / math.sqrt(2.0 * math.pi)
        c = (f[:-1] - f[1:]) / (cdf(t[1:]) - cdf(t[:-1]))
    c = (c - c[::-1]) / 2
    return torch.from_numpy((c / math.sqrt(d)).astype(np.float16).astype(np.float64))


def _pack(codes, bits):
    """Codes [..., d] to the cache's bytes: an LSB-first stream at 2 and 4 bits; at 3 bits groups of 32 in three words
    of eight nibbles, code l < 24 in nibble l % 8 of word l / 8 and bit k of code 24 + i on top of nibble i of word k."""
    if bits == 2:
        c = codes.unflatten(-1, (-1, 4))
        return c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
    if bits == 3:
        c = codes.unflatten(-1, (-1, 4, 8))
        word = torch.arange(3, dtype=torch.uint8, device=codes.device).view(3, 1)
        codes = (c[..., :3, :] | (((c[..., 3:, :] >> word) & 1) << 3)).flatten(-3)
    c = codes.unflatten(-1, (-1, 2))
    return c[..., 0] | (c[..., 1] << 4)


def _unpack(packed, bits):
    """Bytes [..., n] to codes [..., d] (the inverse of _pack)."""
    if bits == 2:
        return torch.stack([packed & 3, (packed >> 2) & 3, (packed >> 4) & 3, packed >> 6], -1).flatten(-2)
    nib = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    if bits == 4:
        return nib
    nib = nib.unflatten(-1, (-1, 3, 8))
    top = nib >> 3
    last = top[..., 0:1, :] | (top[..., 1:2, :] << 1) | (top[..., 2:3, :] << 2)
    return torch.cat([nib & 7, last], -2).flatten(-3)


# ---------------------------------------------------------------- prepare
def _int32(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _tables_inputs(case, seed, device):
    lens = _lengths(case, seed)
    n, bs = case["n_seqs"], case["block"]
    per = case["capacity"] // bs
    cached, new = [c for c, _ in lens], [w for _, w in lens]
    st = dict(case=case, n_tok=sum(new), cached=_int32(cached, device), new=_int32(new, device),
              bounds=None, prefix=None)
    if case["groups"]:
        bounds = _group_bounds({**case, "n_groups": case["groups"]})
        # a group's prefix: whole blocks that all of its members have cached
        prefix = [min(cached[a:b]) // bs * bs for a, b in zip(bounds, bounds[1:])]
        st["bounds"], st["prefix"] = _int32(bounds, device), _int32(prefix, device)
    old = [-(-c // bs) for c in cached]
    gen = torch.Generator(device=device).manual_seed(seed)
    perm = torch.randperm(sum(old) + n * (1 + -(-case["max_new"] // bs)) + 7, generator=gen, device=device,
                          dtype=torch.int32)
    table = torch.full((n, per), -1, dtype=torch.int32, device=device)
    held = torch.arange(per, device=device).view(1, -1) < torch.tensor(old, device=device).view(-1, 1)
    table[held] = perm[:sum(old)]
    st["table"], st["n_blocks"], st["free"] = table, perm.numel(), perm[sum(old):].contiguous()
    st["free_start"] = _int32([3], device)
    return st


def _prompt_inputs(case, seed, device):
    lens = _lengths(case, seed)
    n_tok, n_q, n_kv, d = sum(lens), case["n_q"], case["n_kv"], case["d"]
    gen = torch.Generator(device=device).manual_seed(seed)
    rows = torch.randn(n_tok, n_q + 2 * n_kv, d, generator=gen, device=device).to(torch.bfloat16)
    q, k, v = rows[:, :n_q], rows[:, n_q:n_q + n_kv], rows[:, n_q + n_kv:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    bounds = [0] + np.cumsum(lens).tolist()
    return dict(case=case, q=q, k=k, v=v, bounds=bounds, cu=_int32(bounds, device), max_len=max(lens))


def _codes(shape, d, bits, centroids, gen, device):
    """Codes of Gaussian rows on the unit sphere: after the rotation a row's coordinates are Gaussian again."""
    x = torch.randn(shape + (d,), generator=gen, device=device)
    x /= torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    edges = ((centroids[1:] + centroids[:-1]) / 2).float().to(device)
    return _pack(torch.bucketize(x, edges, out_int32=True).to(torch.uint8), bits)


def _shared_inputs(case, seed, device):
    suffix = _lengths(case, seed)
    bounds, prefix = _group_bounds(case), _prefixes(case)
    n, n_kv, d, bs = case["n_seqs"], case["n_kv"], case["d"], case["block"]
    group = [g for g, (a, b) in enumerate(zip(bounds, bounds[1:])) for _ in range(b - a)]
    lens = [prefix[g] + x for g, x in zip(group, suffix)]
    unit = bs or 64
    capacity = -(-max(max(lens), 1) // unit) * unit
    gen = torch.Generator(device=device).manual_seed(seed)
    st = dict(case=case, seq_lens=_int32(lens, device), max_len=max(lens), capacity=capacity,
              leader=torch.tensor([bounds[g] for g in group], device=device),
              prefix_of=torch.tensor([prefix[g] for g in group], device=device),
              bounds=_int32(bounds, device), prefix=_int32(prefix, device),
              max_group=max(b - a for a, b in zip(bounds, bounds[1:])), max_prefix=max(prefix),
              max_suffix=case["max_suffix"])
    if bs:
        # the members' tables start with their first member's blocks, then blocks of their own in any order
        per = capacity // bs
        table = [[-1] * per for _ in range(n)]
        used = 0
        for s in range(n):
            lead = bounds[group[s]]
            for j in range(-(-lens[s] // bs)):
                if s != lead and (j + 1) * bs <= prefix[group[s]]:
                    table[s][j] = table[lead][j]
                else:
                    table[s][j] = used
                    used += 1
            if s == lead:  # the first member holds the whole prefix
                for j in range(-(-lens[s] // bs), -(-prefix[group[s]] // bs)):
                    table[s][j] = used
                    used += 1
        perm = torch.randperm(max(used, 1), generator=gen, device=device, dtype=torch.int32)
        table = torch.tensor(table, device=device)
        st["table"] = torch.where(table >= 0, perm[table.clamp(min=0)], -1).to(torch.int32)
        shape = (max(used, 1), n_kv, bs)
    else:
        st["table"] = None
        shape = (n, n_kv, capacity)
    st["pi"], st["ck"], st["cv"] = _rotation(d), _centroids(case["bits_k"], d), _centroids(case["bits_v"], d)
    norm = lambda: math.sqrt(d) * torch.exp(0.1 * torch.randn(shape, generator=gen, device=device))  # noqa: E731
    st["codes_k"] = _codes(shape, d, case["bits_k"], st["ck"], gen, device)
    st["codes_v"] = _codes(shape, d, case["bits_v"], st["cv"], gen, device)
    st["norm_k"], st["norm_v"] = norm().to(torch.float16), norm().to(torch.float16)
    if case["qjl"]:
        st["s"] = torch.from_numpy(_gaussians(PI_SEED, 1, d * d).reshape(d, d)).to(torch.float32).to(torch.float64)
        st["qjl_bits"] = torch.randint(0, 256, shape + (d // 8,), generator=gen, device=device, dtype=torch.uint8)
        # the residual of a 2-, 3- or 4-bit code is about this share of the direction
        left = {2: 0.343, 3: 0.186, 4: 0.0975}[case["bits_k"]]
        st["qjl_norm"] = (left * torch.exp(0.05 * torch.randn(shape, generator=gen, device=device))).to(torch.float16)
    st["q"] = torch.randn(n, case["n_q"], d, generator=gen, device=device).to(torch.bfloat16)
    for name in ("pi", "ck", "cv", "s"):
        if name in st:
            st[name] = st[name].to(device)
            st[name + "32"] = st[name].float()
    return st


_INPUTS = {"tables": _tables_inputs, "prompt": _prompt_inputs, "shared": _shared_inputs}


def prepare(case, seed):
    st = _INPUTS[case["op"]](case, seed, "cuda")
    if own:
        from kv_cache_vector_12_b200 import tq
        st["tq"] = tq
        _hold(st, case, tq)
    return st


def _hold(st, case, tq):
    """What a user's program holds before the call: the context, the cache, the outputs and the workspace."""
    empty = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] == "tables":
        n, n_tok = case["n_seqs"], st["n_tok"]
        st["ctx"] = tq.Context(128, 3, 3, 0, PI_SEED)
        st["cache"] = tq.PagedCache(st["ctx"], n, 1, case["capacity"], case["block"], n_blocks=st["n_blocks"],
                                    block_table=st["table"].clone())
        st["seq_idx"], st["pos"], st["slots"] = empty(n_tok), empty(n_tok), empty(n_tok, dtype=torch.int64)
        st["cu_new"], st["seq_lens"], st["free_end"] = empty(n + 1), empty(n), empty(1)
    elif case["op"] == "prompt":
        st["ctx"] = tq.Context(case["d"], 3, 3, 0, PI_SEED)
        st["out"] = empty(*st["q"].shape, dtype=torch.bfloat16)
        st["lse"] = empty(*st["q"].shape[:2], dtype=torch.float32)
    else:
        st["ctx"] = ctx = tq.Context(case["d"], case["bits_k"], case["bits_v"], int(case["qjl"]), PI_SEED)
        if st["table"] is None:
            cache = tq.Cache(ctx, case["n_seqs"], case["n_kv"], st["capacity"])
        else:
            cache = tq.PagedCache(ctx, case["n_seqs"], case["n_kv"], st["capacity"], case["block"],
                                  n_blocks=st["codes_k"].shape[0], block_table=st["table"])
        for name, plane in cache.planes.items():
            if plane is not None:
                plane.copy_(st[name].view(plane.dtype))
        st["cache"] = cache
        st["workspace"] = tq.alloc_shared_workspace(ctx, cache, case["n_q"], st["prefix"].numel(), st["max_group"],
                                                    st["max_prefix"], st["max_suffix"])
        st["out"] = empty(*st["q"].shape, dtype=torch.bfloat16)
        st["lse"] = empty(*st["q"].shape[:2], dtype=torch.float32)


# -------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


def _own_tables(st):
    st["tq"].build_tables(st["ctx"], st["cache"], st["cached"], st["new"], st["seq_idx"], st["pos"], st["cu_new"],
                          st["seq_lens"], slots=st["slots"], free_list=st["free"], free_start=st["free_start"],
                          free_end=st["free_end"], cu_group=st["bounds"], prefix_lens=st["prefix"])
    return dict(table=st["cache"].block_table, seq_idx=st["seq_idx"], pos=st["pos"], slots=st["slots"],
                cu_new=st["cu_new"], seq_lens=st["seq_lens"], free_end=st["free_end"])


def _own_prompt(st):
    st["tq"].prompt_attention(st["ctx"], st["q"], st["k"], st["v"], st["cu"], st["max_len"], st["out"], st["lse"])
    return dict(out=st["out"], lse=st["lse"])


def _own_shared(st):
    st["tq"].decode_attention_shared(st["ctx"], st["cache"], st["q"], st["seq_lens"], st["bounds"], st["prefix"],
                                     st["max_group"], st["max_prefix"], st["max_suffix"], st["out"], st["lse"],
                                     st["workspace"])
    return dict(out=st["out"], lse=st["lse"])


def _plain_tables(st):
    case, cached, new, table = st["case"], st["cached"], st["new"], st["table"]
    bs, dev = case["block"], cached.device
    seq_lens = cached + new
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    cu_new = torch.cat([zero, torch.cumsum(new, 0)])
    seq = torch.repeat_interleave(torch.arange(case["n_seqs"], device=dev), new, output_size=st["n_tok"])
    pos = torch.arange(st["n_tok"], device=dev) - cu_new[seq] + cached[seq]
    # entries first .. last - 1 of a sequence's row get the next free blocks, in the order of the sequences
    first, last = (cached + bs - 1) // bs, (seq_lens + bs - 1) // bs
    start = st["free_start"] + torch.cat([zero, torch.cumsum(last - first, 0)])
    col = torch.arange(table.shape[1], device=dev).view(1, -1)
    take = (start[:-1] - first).view(-1, 1) + col
    fresh = (col >= first.view(-1, 1)) & (col < last.view(-1, 1))
    table = torch.where(fresh, st["free"][take.clamp(0, st["free"].numel() - 1)], table)
    if st["bounds"] is not None:  # a group's members begin with the blocks of its first member
        group = torch.searchsorted(st["bounds"], torch.arange(case["n_seqs"], device=dev, dtype=torch.int32),
                                   right=True) - 1
        table = torch.where(col < (st["prefix"][group] // bs).view(-1, 1), table[st["bounds"][group].long()], table)
    slots = table[seq, pos // bs].to(torch.int64) * bs + pos % bs
    return dict(table=table, seq_idx=seq.to(torch.int32), pos=pos.to(torch.int32), slots=slots,
                cu_new=cu_new.to(torch.int32), seq_lens=seq_lens, free_end=start[-1:].to(torch.int32))


def _plain_prompt(st):
    case, bounds = st["case"], st["bounds"]
    n_kv, per, d = case["n_kv"], case["n_q"] // case["n_kv"], case["d"]
    out = torch.empty(st["q"].shape, dtype=torch.bfloat16, device=st["q"].device)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=st["q"].device)
    # one sequence after the other, as many KV heads at once as 16 GB of scores allow
    for a, b in zip(bounds, bounds[1:]):
        n = b - a
        step = max(1, min(n_kv, (16 << 30) // (4 * per * n * n)))
        later = torch.ones(n, n, dtype=torch.bool, device=out.device).triu(1)
        for h in range(0, n_kv, step):
            e = min(h + step, n_kv)
            q = st["q"][a:b, h * per:e * per].float().unflatten(1, (e - h, per)).permute(1, 2, 0, 3)
            k = st["k"][a:b, h:e].float().permute(1, 2, 0).unsqueeze(1)
            v = st["v"][a:b, h:e].float().permute(1, 0, 2).unsqueeze(1)
            s = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).masked_fill_(later, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = s.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v) / total
            out[a:b, h * per:e * per] = o.permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
            lse[a:b, h * per:e * per] = (top + total.log()).squeeze(-1).permute(2, 0, 1).flatten(1, 2)
    return dict(out=out, lse=lse)


def _at(st, plane):
    """Rows of a plane by (sequence, position): a group's prefix from its first sequence, the rest from its own."""
    case, dev = st["case"], plane.device
    pos = torch.arange(st["max_len"], device=dev).view(1, -1)
    src = torch.where(pos < st["prefix_of"].view(-1, 1), st["leader"].view(-1, 1),
                      torch.arange(case["n_seqs"], device=dev).view(-1, 1))
    if st["table"] is None:
        return plane[src, :, pos]
    blk = st["table"][src, pos // case["block"]].long().clamp(min=0)
    return plane[blk, :, pos % case["block"]]


def _plain_shared(st):
    case = st["case"]
    n, n_kv, d = case["n_seqs"], case["n_kv"], case["d"]
    per = case["n_q"] // n_kv
    q_hat = torch.matmul(st["q"].float(), st["pi32"].t()).view(n, n_kv, per, d)
    kn = _at(st, st["norm_k"]).float().permute(0, 2, 1)
    keys = st["ck32"][_unpack(_at(st, st["codes_k"]), case["bits_k"]).int()]  # [n, positions, n_kv, d]
    s = torch.einsum("bhgd,blhd->bhgl", q_hat, keys)
    del keys
    if case["qjl"]:
        bits = (_at(st, st["qjl_bits"]).unsqueeze(-1) >> torch.arange(8, device=s.device, dtype=torch.uint8)) & 1
        signs = bits.flatten(-2).float().mul_(2).sub_(1)
        q_til = torch.matmul(q_hat, st["s32"].t())
        s += torch.einsum("bhgd,blhd->bhgl", q_til, signs) * (
            math.sqrt(math.pi / 2) / d * _at(st, st["qjl_norm"]).float().permute(0, 2, 1).unsqueeze(2))
        del bits, signs
    s *= kn.unsqueeze(2) / math.sqrt(d)
    past = torch.arange(st["max_len"], device=s.device).view(1, -1) >= st["seq_lens"].view(-1, 1)
    s = s.masked_fill_(past.view(n, 1, 1, -1), -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    p *= _at(st, st["norm_v"]).float().permute(0, 2, 1).unsqueeze(2)
    values = st["cv32"][_unpack(_at(st, st["codes_v"]), case["bits_v"]).int()]
    o = torch.einsum("bhgl,blhd->bhgd", p, values) / total.clamp(min=1e-37)
    out = torch.matmul(o, st["pi32"]).view(n, n_kv * per, d)
    return dict(out=out.to(torch.bfloat16), lse=(top + total.log()).view(n, n_kv * per))


_OWN = {"tables": _own_tables, "prompt": _own_prompt, "shared": _own_shared}
_PLAIN = {"tables": _plain_tables, "prompt": _plain_prompt, "shared": _plain_shared}


# ------------------------------------------------------------------- work
def work(case):
    lens = _lengths(case, 0)
    if case["op"] == "tables":
        bs, n = case["block"], case["n_seqs"]
        tokens = sum(w for _, w in lens)
        blocks = sum(-(-(c + w) // bs) - -(-c // bs) for c, w in lens)
        # lengths in; (seq_idx, pos, slot) of each token, cu and lengths out; a list entry in and a table entry out per
        # new block, one table entry in per sequence that continues in a block
        return dict(bytes=8 * n + 16 * tokens + 8 * n + 8 * blocks + 4 * n, flops=0)
    per_q = case["n_q"] * case["d"]
    if case["op"] == "prompt":
        tokens = sum(lens)
        pairs = sum(x * (x + 1) // 2 for x in lens)
        return dict(bytes=tokens * (2 * per_q + 4 * case["n_kv"] * case["d"] + 2 * per_q + 4 * case["n_q"]),
                    flops=4 * pairs * per_q)
    bounds, prefix = _group_bounds(case), _prefixes(case)
    token = case["n_kv"] * (case["d"] * (case["bits_k"] + case["bits_v"]) // 8 + 4
                            + (case["d"] // 8 + 2 if case["qjl"] else 0))
    attended = sum(p * (b - a) for p, a, b in zip(prefix, bounds, bounds[1:])) + sum(lens)
    return dict(bytes=(sum(prefix) + sum(lens)) * token + case["n_seqs"] * (4 * per_q + 4 * case["n_q"]),
                flops=4 * attended * per_q)


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The operators from their definitions, in 64 bits (whole numbers: None, the plain form is exact)."""
    if case["op"] == "tables":
        return None
    st = _INPUTS[case["op"]](case, seed, "cuda")
    return _exact_prompt(st) if case["op"] == "prompt" else _exact_shared(st)


def _exact_prompt(st):
    case, bounds = st["case"], st["bounds"]
    per, d = case["n_q"] // case["n_kv"], case["d"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device=st["q"].device)
    for a, b in zip(bounds, bounds[1:]):
        for h in range(case["n_kv"]):
            k, v = st["k"][a:b, h].double(), st["v"][a:b, h].double()
            for r in range(0, b - a, 2048):  # query rows r .. e - 1 against the keys before e
                e = min(r + 2048, b - a)
                q = st["q"][a + r:a + e, h * per:(h + 1) * per].double().transpose(0, 1).reshape(-1, d)
                s = (q @ k[:e].t() / math.sqrt(d)).view(per, e - r, e)
                seen = torch.arange(e, device=s.device).view(1, -1) <= torch.arange(r, e, device=s.device).view(-1, 1)
                s = torch.where(seen, s, -math.inf)
                lse_r = torch.logsumexp(s, -1)
                o = torch.exp(s - lse_r.unsqueeze(-1)).view(-1, e) @ v[:e]
                out[a + r:a + e, h * per:(h + 1) * per] = o.view(per, e - r, d).transpose(0, 1)
                lse[a + r:a + e, h * per:(h + 1) * per] = lse_r.t()
    return dict(out=out, lse=lse)


def _exact_codes(rows, bits, d):
    """Codes of packed rows [n, bytes], bit by bit from the layout's definition."""
    bit = (rows.unsqueeze(-1).to(torch.int16) >> torch.arange(8, device=rows.device, dtype=torch.int16)) & 1
    bit = bit.flatten(-2)  # [n, 8 bytes]: bit i of the little-endian row
    at = []
    for c in range(d):
        if bits != 3:
            at.append([c * bits + i for i in range(bits)])
        else:
            base, x = c // 32 * 96, c % 32
            at.append([base + x // 8 * 32 + 4 * (x % 8) + i for i in range(3)] if x < 24
                      else [base + 32 * i + 4 * (x - 24) + 3 for i in range(3)])
    picked = bit[:, torch.tensor(at, device=rows.device)]
    return (picked * torch.tensor([1 << i for i in range(bits)], device=rows.device, dtype=torch.int16)).sum(-1)


def _exact_shared(st):
    case = st["case"]
    n, n_kv, d = case["n_seqs"], case["n_kv"], case["d"]
    per, bs = case["n_q"] // n_kv, case["block"]
    if sum(_lengths(case, 0)) + sum(_prefixes(case)) > 1 << 20:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device=st["q"].device)
    lens, leader, prefix = st["seq_lens"].tolist(), st["leader"].tolist(), st["prefix_of"].tolist()

    def rows(name, s, h, a, b):  # positions a .. b - 1 of sequence s, KV head h
        if st["table"] is None:
            return st[name][s, h, a:b]
        pos = torch.arange(a, b, device=out.device)
        return st[name][st["table"][s, pos // bs].long(), h, pos % bs]

    def part(s, h, a, b):
        """Reconstructed (rotated) keys, values, sign rows scaled by the residual's norm."""
        key = st["ck"][_exact_codes(rows("codes_k", s, h, a, b), case["bits_k"], d).long()]
        kn = rows("norm_k", s, h, a, b).double().unsqueeze(-1)
        val = st["cv"][_exact_codes(rows("codes_v", s, h, a, b), case["bits_v"], d).long()]
        val = val * rows("norm_v", s, h, a, b).double().unsqueeze(-1)
        if not case["qjl"]:
            return key * kn, val, None
        sign = _exact_codes(rows("qjl_bits", s, h, a, b), 1, d).double() * 2 - 1
        return key * kn, val, sign * (rows("qjl_norm", s, h, a, b).double().unsqueeze(-1) * kn)

    for h in range(n_kv):
        held = {}
        for s in range(n):
            if lens[s] == 0:
                continue
            if leader[s] not in held:
                held = {leader[s]: part(leader[s], h, 0, prefix[s])}
            parts = [held[leader[s]], part(s, h, prefix[s], lens[s])]
            keys, vals = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
            q_hat = st["q"][s, h * per:(h + 1) * per].double() @ st["pi"].t()
            score = q_hat @ keys.t()
            if case["qjl"]:
                score = score + math.sqrt(math.pi / 2) / d * ((q_hat @ st["s"].t()) @ torch.cat([p[2] for p in parts]).t())
            score = score / math.sqrt(d)
            total = torch.logsumexp(score, -1)
            out[s, h * per:(h + 1) * per] = torch.exp(score - total.unsqueeze(-1)) @ vals @ st["pi"]
            lse[s, h * per:(h + 1) * per] = total
    return dict(out=out, lse=lse)
