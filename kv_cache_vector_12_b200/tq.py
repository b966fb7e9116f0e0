"""Thin Python binding of ``libtq.so`` (argument checks and marshalling only).

Every function mirrors the C entry point of the same name in ``include/tq.h``;
every step of the hot path runs in the library's CUDA kernels.  The serving
operators (build_tables, prompt_attention, decode_attention_shared) compare
their tensors' sizes, types, layouts and devices with what the call reads and
writes; the other functions hand their pointers over as they are.  PyTorch is
used here only to allocate device memory and to hand over stream handles.
Importing this module loads the library and raises ``ImportError`` if it has
not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtq.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m kv_cache_vector_12_b200.build`")
lib = ctypes.CDLL(_LIB_PATH)

TQ_OK, TQ_ERR_INVALID, TQ_ERR_CUDA, TQ_ERR_NOMEM, TQ_ERR_UNSUPPORTED, TQ_ERR_DEVICE = range(6)
TQ_BF16, TQ_F32 = 0, 1
TQ_LAW_GAUSSIAN, TQ_LAW_SPHERE = 0, 1
LAWS = {"gaussian": TQ_LAW_GAUSSIAN, "sphere": TQ_LAW_SPHERE}
_MAX_TABLE_SEQS = 4096  # of tq_build_tables
PLANES = ("codes_k", "norm_k", "qjl_bits", "qjl_norm", "codes_v", "norm_v")

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_fp = ctypes.POINTER(ctypes.c_float)


class tq_cache(ctypes.Structure):
    _fields_ = [("codes_k", _vp), ("norm_k", _vp), ("qjl_bits", _vp), ("qjl_norm", _vp),
                ("codes_v", _vp), ("norm_v", _vp), ("capacity", _i32), ("n_seqs", _i32),
                ("n_kv_heads", _i32), ("block_table", _vp), ("block_size", _i32), ("n_blocks", _i32)]


lib.tq_create.argtypes = [ctypes.POINTER(_vp), _i32, _i32, _i32, _i32, ctypes.c_uint64]
lib.tq_create.restype = ctypes.c_int
lib.tq_create_ex.argtypes = [ctypes.POINTER(_vp), _i32, _i32, _i32, _i32, ctypes.c_uint64, _i32]
lib.tq_create_ex.restype = ctypes.c_int
lib.tq_destroy.argtypes = [_vp]
lib.tq_destroy.restype = None
lib.tq_layout.argtypes = [_vp, ctypes.POINTER(ctypes.c_size_t)]
lib.tq_layout.restype = ctypes.c_int
lib.tq_get_params.argtypes = [_vp, _fp, _fp, _fp, _fp, _fp, _fp]
lib.tq_get_params.restype = ctypes.c_int
lib.tq_host_params.argtypes = [_i32, _i32, _i32, _i32, ctypes.c_uint64, _fp, _fp, _fp, _fp, _fp, _fp]
lib.tq_host_params.restype = ctypes.c_int
lib.tq_host_params_ex.argtypes = [_i32, _i32, _i32, _i32, ctypes.c_uint64, _i32, _fp, _fp, _fp, _fp, _fp, _fp]
lib.tq_host_params_ex.restype = ctypes.c_int
lib.tq_quantize.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _vp, _vp, _vp, _i32, _vp]
lib.tq_quantize.restype = ctypes.c_int
lib.tq_workspace_bytes.argtypes = [_vp, _i32, _i32, _i32]
lib.tq_workspace_bytes.restype = ctypes.c_size_t
lib.tq_decode_attention.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _i32, _i32, _vp, _i32,
                                    ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp]
lib.tq_decode_attention.restype = ctypes.c_int
lib.tq_decode_attention_noalloc.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _i32, _i32, _vp, _i32,
                                            ctypes.c_float, _vp, _vp, _vp]
lib.tq_decode_attention_noalloc.restype = ctypes.c_int
lib.tq_prefill_attention.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _i32, _i32, _vp, _vp, _i32, _i32,
                                     ctypes.c_float, _vp, _vp, _vp]
lib.tq_prefill_attention.restype = ctypes.c_int
lib.tq_weight_quantize.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _i32, _i32, _vp]
lib.tq_weight_quantize.restype = ctypes.c_int
lib.tq_weight_workspace_bytes.argtypes = [_vp, _i32, _i32]
lib.tq_weight_workspace_bytes.restype = ctypes.c_size_t
lib.tq_weight_gemm.argtypes = [_vp, ctypes.POINTER(tq_cache), _i32, _i32, _vp, _i32, _i32, _vp, _vp,
                               ctypes.c_size_t, _vp]
lib.tq_weight_gemm.restype = ctypes.c_int
lib.tq_shared_workspace_bytes.argtypes = [_vp, ctypes.POINTER(tq_cache), _i32, _i32, _i32, _i32, _i32]
lib.tq_shared_workspace_bytes.restype = ctypes.c_size_t
lib.tq_decode_attention_shared.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32,
                                           _i32, _i32, ctypes.c_float, _vp, _i32, _vp, _vp, ctypes.c_size_t, _vp]
lib.tq_decode_attention_shared.restype = ctypes.c_int
lib.tq_prompt_attention.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _i32, _i32, _i32,
                                    _vp, _i32, _i32, ctypes.c_float, _vp, _i32, _vp, _vp]
lib.tq_prompt_attention.restype = ctypes.c_int
lib.tq_build_tables.argtypes = [_vp, ctypes.POINTER(tq_cache), _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32,
                                _i32, _vp, _vp, _vp, _vp, _vp, _vp]
lib.tq_build_tables.restype = ctypes.c_int
# The arguments of a call as one array of words (a ctypes call costs 0.1 us for each argument)
_SHARED_WORDS = struct.Struct("QQQqqQQQqqqqdQqQQQQ").pack
_PROMPT_WORDS = struct.Struct("QQQQqqqqqqQqqdQqQQ").pack
_TABLES_WORDS = struct.Struct("QQQQQQqQQQQqqQQQQQQ").pack
for _call in (lib.tq_decode_attention_shared_words, lib.tq_prompt_attention_words, lib.tq_build_tables_words):
    _call.argtypes = [ctypes.c_char_p]
    _call.restype = ctypes.c_int
lib.tq_check_device_errors.argtypes = [_vp, _vp]
lib.tq_check_device_errors.restype = ctypes.c_int
lib.tq_last_error.argtypes = []
lib.tq_last_error.restype = ctypes.c_char_p


class TQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"tq status {status}: {message}")
        self.status = status


def _check(status: int) -> None:
    if status != TQ_OK:
        raise TQError(status, lib.tq_last_error().decode())


def _ptr(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the handle alone: building the Stream object costs ten times the lookup (3.2 us against 0.3)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_device = torch._C._cuda_getDevice  # torch.cuda.current_device() without its check that CUDA is set up
_current_stream = torch._C._cuda_getCurrentRawStream
_address = ctypes.addressof
_F32, _BF16, _I32, _I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64
_INT, _OUT_TYPES = (_I32,), (_BF16, _F32)


def _handle(ctx) -> int:
    return ctx.handle.value if ctx.handle else 0


def _ints(arrays, dev: int) -> list | None:
    """The addresses of contiguous int32 tensors on device `dev`; None if one is not that."""
    at = []
    for t in arrays:
        if t is None or t.dtype is not _I32 or not t.is_contiguous() or t.get_device() != dev:
            return None
        at.append(t.data_ptr())
    return at


def _refuse(call: str, dev: int, *arrays) -> None:
    """The error for the first of (name, tensor or None, element types, least number of elements) that does not fit:
    the library gets a bare pointer, so a tensor of another type, layout, device or size is refused before the call.
    (None is left to the library.)  A call tests its arrays itself, in one expression, and comes here when one fails."""
    for name, t, dtypes, n in arrays:
        if t is None or (t.dtype in dtypes and t.numel() >= n and t.is_contiguous() and t.get_device() == dev):
            continue
        raise TQError(TQ_ERR_INVALID, f"{call}: {name} must be a contiguous tensor of {dtypes} on the current CUDA device "
                                      f"with at least {n} elements, not {t.dtype} {tuple(t.shape)}, strides {t.stride()}, "
                                      f"on {t.device}")


def _fbuf(t: torch.Tensor | None):
    return None if t is None else ctypes.cast(t.data_ptr(), _fp)


def _law(law) -> int:
    return LAWS[law] if isinstance(law, str) else int(law)


def host_params(d: int, bits_k: int, bits_v: int, qjl: int, seed: int, law="gaussian") -> dict:
    """tq_host_params_ex: the parameters tq_create_ex would upload (CPU only)."""
    out = {"pi": torch.empty(d * d), "s": torch.empty(d * d) if qjl else None,
           "centroids_k": torch.empty(1 << bits_k), "thresholds_k": torch.empty((1 << bits_k) - 1),
           "centroids_v": torch.empty(1 << bits_v), "thresholds_v": torch.empty((1 << bits_v) - 1)}
    _check(lib.tq_host_params_ex(d, bits_k, bits_v, qjl, seed, _law(law), _fbuf(out["pi"]), _fbuf(out["s"]),
                                 _fbuf(out["centroids_k"]), _fbuf(out["thresholds_k"]),
                                 _fbuf(out["centroids_v"]), _fbuf(out["thresholds_v"])))
    out["pi"] = out["pi"].view(d, d)
    if qjl:
        out["s"] = out["s"].view(d, d)
    return out


class Context:
    """Owns one tq_ctx (tq_create_ex / tq_destroy); law "gaussian" (the
    default, as tq_create) or "sphere" (tq_law)."""

    def __init__(self, d: int = 128, bits_k: int = 3, bits_v: int = 3, qjl: int = 0, seed: int = 42,
                 law="gaussian"):
        h = _vp()
        _check(lib.tq_create_ex(ctypes.byref(h), d, bits_k, bits_v, int(qjl), seed, _law(law)))
        self.handle = h
        self.d, self.bits_k, self.bits_v, self.qjl, self.seed = d, bits_k, bits_v, int(qjl), seed
        self.law = law

    def close(self) -> None:
        if self.handle:
            lib.tq_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def layout(self) -> list[int]:
        arr = (ctypes.c_size_t * 6)()
        _check(lib.tq_layout(self.handle, arr))
        return list(arr)

    def params(self) -> dict:
        d = self.d
        out = {"pi": torch.empty(d * d), "s": torch.empty(d * d) if self.qjl else None,
               "centroids_k": torch.empty(1 << self.bits_k),
               "thresholds_k": torch.empty((1 << self.bits_k) - 1),
               "centroids_v": torch.empty(1 << self.bits_v),
               "thresholds_v": torch.empty((1 << self.bits_v) - 1)}
        _check(lib.tq_get_params(self.handle, _fbuf(out["pi"]), _fbuf(out["s"]),
                                 _fbuf(out["centroids_k"]), _fbuf(out["thresholds_k"]),
                                 _fbuf(out["centroids_v"]), _fbuf(out["thresholds_v"])))
        out["pi"] = out["pi"].view(d, d)
        if self.qjl:
            out["s"] = out["s"].view(d, d)
        return out

    def check_device_errors(self, stream=None) -> None:
        _check(lib.tq_check_device_errors(self.handle, _stream(stream)))


class Cache:
    """Device planes of one layer's packed cache, allocated through torch."""

    def __init__(self, ctx: Context, n_seqs: int, n_kv_heads: int, capacity: int, device="cuda"):
        sizes = ctx.layout()
        self.planes = {}
        for name, nbytes in zip(PLANES, sizes):
            if nbytes == 0:
                self.planes[name] = None
                continue
            shape = (n_seqs, n_kv_heads, capacity, nbytes) if nbytes > 2 else (n_seqs, n_kv_heads, capacity)
            dtype = torch.uint8 if nbytes > 2 else torch.int16
            self.planes[name] = torch.zeros(shape, dtype=dtype, device=device)
        self.n_seqs, self.n_kv_heads, self.capacity = n_seqs, n_kv_heads, capacity
        self.struct = tq_cache(*[_ptr(self.planes[n]) for n in PLANES], capacity, n_seqs, n_kv_heads, None, 0, 0)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.planes.values() if t is not None)


class PagedCache:
    """Device planes of one layer's packed cache in the paged layout:
    n_blocks physical blocks of block_size tokens ([n_blocks][n_kv_heads]
    [block_size][bytes] per plane) and a block table (device int32
    [n_seqs][capacity / block_size]) mapping each sequence's logical blocks
    to physical ones.  `block_table` may be given; by default sequence s owns
    physical blocks s * per_seq ... in order."""

    def __init__(self, ctx: Context, n_seqs: int, n_kv_heads: int, capacity: int, block_size: int,
                 n_blocks: int | None = None, block_table: torch.Tensor | None = None, device="cuda"):
        per_seq = capacity // block_size
        if n_blocks is None:
            n_blocks = n_seqs * per_seq
        if block_table is None:
            block_table = torch.arange(n_seqs * per_seq, dtype=torch.int32).view(n_seqs, per_seq)
        self.block_table = block_table.to(device=device, dtype=torch.int32).contiguous()
        sizes = ctx.layout()
        self.planes = {}
        for name, nbytes in zip(PLANES, sizes):
            if nbytes == 0:
                self.planes[name] = None
                continue
            shape = (n_blocks, n_kv_heads, block_size, nbytes) if nbytes > 2 else (n_blocks, n_kv_heads, block_size)
            dtype = torch.uint8 if nbytes > 2 else torch.int16
            self.planes[name] = torch.zeros(shape, dtype=dtype, device=device)
        self.n_seqs, self.n_kv_heads, self.capacity = n_seqs, n_kv_heads, capacity
        self.block_size, self.n_blocks = block_size, n_blocks
        self.struct = tq_cache(*[_ptr(self.planes[n]) for n in PLANES], capacity, n_seqs, n_kv_heads,
                               self.block_table.data_ptr(), block_size, n_blocks)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.planes.values() if t is not None)


def quantize(ctx: Context, cache: Cache, k: torch.Tensor, v: torch.Tensor, seq_idx: torch.Tensor,
             pos: torch.Tensor, stream=None) -> None:
    """tq_quantize: k, v bf16 [n_tok, n_kv_heads, d] contiguous; seq_idx, pos int32 [n_tok]."""
    n_tok = k.shape[0]
    _check(lib.tq_quantize(ctx.handle, ctypes.byref(cache.struct), _ptr(k), _ptr(v), _ptr(seq_idx),
                           _ptr(pos), n_tok, _stream(stream)))


def workspace_bytes(ctx: Context, n_seqs: int, n_q_heads: int, max_seq_len: int) -> int:
    return int(lib.tq_workspace_bytes(ctx.handle, n_seqs, n_q_heads, max_seq_len))


def decode_attention(ctx: Context, cache: Cache, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                     out: torch.Tensor, lse: torch.Tensor | None, workspace: torch.Tensor,
                     scale: float = 0.0, stream=None) -> None:
    """tq_decode_attention: q [n_seqs, n_q_heads, d] bf16 or fp32; out fp32 [n_seqs, n_q_heads, d]."""
    q_dtype = TQ_F32 if q.dtype == torch.float32 else TQ_BF16
    n_q_heads = q.shape[1]
    _check(lib.tq_decode_attention(ctx.handle, ctypes.byref(cache.struct), _ptr(q), q_dtype, n_q_heads,
                                   _ptr(seq_lens), max_seq_len, scale, _ptr(out), _ptr(lse),
                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)))


def prefill_attention(ctx: Context, cache: Cache, q: torch.Tensor, cu_q: torch.Tensor, seq_lens: torch.Tensor,
                      max_q: int, max_seq_len: int, out: torch.Tensor, lse: torch.Tensor | None = None,
                      scale: float = 0.0, stream=None) -> None:
    """tq_prefill_attention: q [total, n_q_heads, d] bf16 or fp32, the queries of
    sequence s being rows cu_q[s]:cu_q[s+1] (its last positions below
    seq_lens[s], already quantized into the cache); out fp32 [total, n_q_heads, d]."""
    q_dtype = TQ_F32 if q.dtype == torch.float32 else TQ_BF16
    _check(lib.tq_prefill_attention(ctx.handle, ctypes.byref(cache.struct), _ptr(q), q_dtype, q.shape[1],
                                    _ptr(cu_q), _ptr(seq_lens), max_q, max_seq_len, scale, _ptr(out), _ptr(lse),
                                    _stream(stream)))


def decode_attention_noalloc(ctx: Context, cache: Cache, q: torch.Tensor, seq_lens: torch.Tensor,
                             max_seq_len: int, out: torch.Tensor, lse: torch.Tensor | None,
                             scale: float = 0.0, stream=None) -> None:
    """tq_decode_attention_noalloc: decode attention without a caller workspace,
    for callers that cannot allocate device memory (the library's static
    scratch is used instead; concurrent calls on the GPU race on it)."""
    q_dtype = TQ_F32 if q.dtype == torch.float32 else TQ_BF16
    _check(lib.tq_decode_attention_noalloc(ctx.handle, ctypes.byref(cache.struct), _ptr(q), q_dtype, q.shape[1],
                                           _ptr(seq_lens), max_seq_len, scale, _ptr(out), _ptr(lse),
                                           _stream(stream)))


def shared_workspace_bytes(ctx: Context, cache: Cache, n_q_heads: int, n_groups: int, max_group: int,
                           max_prefix_len: int, max_suffix_len: int) -> int:
    return int(lib.tq_shared_workspace_bytes(ctx.handle, ctypes.byref(cache.struct), n_q_heads, n_groups, max_group,
                                             max_prefix_len, max_suffix_len))


def decode_attention_shared(ctx: Context, cache: Cache, q: torch.Tensor, seq_lens: torch.Tensor,
                            cu_group: torch.Tensor, prefix_lens: torch.Tensor, max_group: int, max_prefix_len: int,
                            max_suffix_len: int, out: torch.Tensor, lse: torch.Tensor | None,
                            workspace: torch.Tensor, scale: float = 0.0, stream=None) -> None:
    """tq_decode_attention_shared: decode attention for groups of sequences
    (cu_group int32 [n_groups + 1]) that share their first prefix_lens[g]
    (int32 [n_groups]) positions, read from the group's first sequence; q
    [n_seqs, n_q_heads, d] bf16 or fp32, out bf16 or fp32 of the same shape."""
    _, n_q, d = q.shape
    n_seqs, n_groups = cache.struct.n_seqs, prefix_lens.numel()
    rows, dev = n_seqs * n_q, _device()
    if not (_ints((seq_lens, cu_group, prefix_lens), dev) and d == ctx.d and seq_lens.numel() >= n_seqs
            and cu_group.numel() > n_groups and q.dtype in _OUT_TYPES and q.numel() >= rows * d and q.is_contiguous()
            and out.dtype in _OUT_TYPES and out.numel() >= rows * d and out.is_contiguous() and workspace.is_contiguous()
            and q.get_device() == out.get_device() == workspace.get_device() == dev
            and (lse is None or lse.dtype is _F32 and lse.numel() >= rows and lse.is_contiguous()
                 and lse.get_device() == dev)):
        if n_q <= 16 * cache.struct.n_kv_heads:  # (more are refused by the library as unsupported)
            _refuse("decode_attention_shared", dev, ("q", q, _OUT_TYPES, rows * d), ("seq_lens", seq_lens, _INT, n_seqs),
                    ("cu_group", cu_group, _INT, n_groups + 1), ("prefix_lens", prefix_lens, _INT, 0),
                    ("out", out, _OUT_TYPES, rows * d), ("lse", lse, (_F32,), rows),
                    ("workspace", workspace, (workspace.dtype,), 0))
            if d != ctx.d:
                raise TQError(TQ_ERR_INVALID, f"decode_attention_shared: q of head dimension {d}, not {ctx.d}")
    _check(lib.tq_decode_attention_shared_words(_SHARED_WORDS(
        _handle(ctx), _address(cache.struct), q.data_ptr(), TQ_F32 if q.dtype is _F32 else TQ_BF16, n_q,
        _ptr(seq_lens) or 0, _ptr(cu_group) or 0, prefix_lens.data_ptr(), n_groups, max_group, max_prefix_len,
        max_suffix_len, scale, out.data_ptr(), TQ_F32 if out.dtype is _F32 else TQ_BF16, _ptr(lse) or 0,
        workspace.data_ptr(), workspace.nbytes, _current_stream(dev) if stream is None else _stream(stream))))


def prompt_attention(ctx: Context, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     max_len: int, out: torch.Tensor, lse: torch.Tensor | None = None, scale: float = 0.0,
                     stream=None) -> None:
    """tq_prompt_attention: causal attention over prompts packed one behind the
    other, prompt s being tokens cu_seqlens[s]:cu_seqlens[s+1]; q bf16 [n_tok,
    n_q_heads, d], k and v bf16 [n_tok, n_kv_heads, d] (slices of one fused
    projection are taken by their token stride); out bf16 or fp32 [n_tok,
    n_q_heads, d], lse fp32 [n_tok, n_q_heads]."""
    (n_tok, n_q, d), (k_tok, n_kv, k_d), (v_tok, v_heads, v_d) = q.shape, k.shape, v.shape
    (q0, q1, q2), (k0, k1, k2), (v0, v1, v2) = q.stride(), k.stride(), v.stride()
    if not (q.dtype is k.dtype is v.dtype is _BF16 and q1 == k1 == v1 == d == ctx.d and q2 == k2 == v2 == 1
            and out.is_contiguous()):
        raise TQError(TQ_ERR_INVALID, "prompt_attention takes bf16 q, k, v with the heads of a token contiguous, "
                                      "and a contiguous out")
    dev = _device()
    if not (k_tok >= n_tok <= v_tok and n_kv == v_heads and k_d == v_d == d
            and q.get_device() == k.get_device() == v.get_device() == dev):
        raise TQError(TQ_ERR_INVALID, f"prompt_attention: k {tuple(k.shape)} on {k.device} and v {tuple(v.shape)} on "
                                      f"{v.device} must have the same heads and d, at least the tokens of q {tuple(q.shape)} "
                                      f"on {q.device}, and all be on the current CUDA device")
    rows = n_tok * n_q
    if not (cu_seqlens.dtype is _I32 and cu_seqlens.is_contiguous() and out.dtype in _OUT_TYPES
            and out.numel() >= rows * d and cu_seqlens.get_device() == out.get_device() == dev
            and (lse is None or lse.dtype is _F32 and lse.numel() >= rows and lse.is_contiguous()
                 and lse.get_device() == dev)):
        if n_q <= 16 * n_kv:  # (more are refused by the library as unsupported)
            _refuse("prompt_attention", dev, ("cu_seqlens", cu_seqlens, _INT, 0), ("out", out, _OUT_TYPES, rows * d),
                    ("lse", lse, (_F32,), rows))
    _check(lib.tq_prompt_attention_words(_PROMPT_WORDS(
        _handle(ctx), q.data_ptr(), k.data_ptr(), v.data_ptr(), q0, k0, v0, n_tok, n_q, n_kv, cu_seqlens.data_ptr(),
        cu_seqlens.numel() - 1, max_len, scale, out.data_ptr(), TQ_F32 if out.dtype is _F32 else TQ_BF16,
        _ptr(lse) or 0, _current_stream(dev) if stream is None else _stream(stream))))


def build_tables(ctx: Context, cache: Cache, cached_lens: torch.Tensor, new_lens: torch.Tensor, seq_idx: torch.Tensor,
                 pos: torch.Tensor, cu_new: torch.Tensor, seq_lens: torch.Tensor, slots: torch.Tensor | None = None,
                 free_list: torch.Tensor | None = None, free_start: torch.Tensor | None = None,
                 free_end: torch.Tensor | None = None, cu_group: torch.Tensor | None = None,
                 prefix_lens: torch.Tensor | None = None, stream=None) -> None:
    """tq_build_tables: seq_idx, pos (int32 [n_tok]), slots (int64 [n_tok] or
    None), cu_new (int32 [n_seqs + 1]) and seq_lens (int32 [n_seqs]) of one
    engine step from cached_lens and new_lens (int32 [n_seqs]).  A PagedCache's
    own block table gets the new blocks from free_list (int32), starting at
    free_start (int32 [1]); free_end (int32 [1]) is where the next step
    starts.  cu_group (int32 [n_groups + 1]) and prefix_lens (int32
    [n_groups]): groups of sequences that begin with the same blocks."""
    table, n_seqs, n_tok, dev = getattr(cache, "block_table", None), cache.struct.n_seqs, seq_idx.numel(), _device()
    ints, n_free, n_groups = [cached_lens, new_lens, seq_idx, pos, cu_new, seq_lens], 0, 0
    if prefix_lens is not None:
        n_groups = prefix_lens.numel()
        ints += cu_group, prefix_lens
    if table is not None:
        n_free = 0 if free_list is None else free_list.numel()
        ints += free_list, free_start, free_end
        if table.data_ptr() != cache.struct.block_table:
            raise TQError(TQ_ERR_INVALID, "build_tables: cache.block_table is not the table that the cache was made with")
    p = _ints(ints, dev)
    if not (p and cached_lens.numel() >= n_seqs <= new_lens.numel() and pos.numel() >= n_tok
            and cu_new.numel() > n_seqs <= seq_lens.numel() and (not n_groups or cu_group.numel() > n_groups)
            and (table is None or free_start.numel() and free_end.numel())
            and (slots is None or slots.dtype is _I64 and slots.numel() >= n_tok and slots.is_contiguous()
                 and slots.get_device() == dev)):
        if n_seqs <= _MAX_TABLE_SEQS:  # (more are refused by the library as unsupported)
            _refuse("build_tables", dev, ("cached_lens", cached_lens, _INT, n_seqs), ("new_lens", new_lens, _INT, n_seqs),
                    ("seq_idx", seq_idx, _INT, 0), ("pos", pos, _INT, n_tok), ("slots", slots, (_I64,), n_tok),
                    ("cu_new", cu_new, _INT, n_seqs + 1), ("seq_lens", seq_lens, _INT, n_seqs),
                    ("cu_group", cu_group if n_groups else None, _INT, n_groups + 1),
                    ("prefix_lens", prefix_lens, _INT, 0))
            if table is not None:
                _refuse("build_tables", dev, ("free_list", free_list, _INT, 0), ("free_start", free_start, _INT, 1),
                        ("free_end", free_end, _INT, 1))
        p = [0 if t is None else t.data_ptr() for t in ints]
    groups = p[6:8] if prefix_lens is not None else (0, 0)
    free = p[-3:] if table is not None else (0, 0, 0)
    _check(lib.tq_build_tables_words(_TABLES_WORDS(
        _handle(ctx), _address(cache.struct), 0 if table is None else table.data_ptr(), p[0], p[1], free[0], n_free,
        free[1], free[2], *groups, n_groups, n_tok, p[2], p[3], 0 if slots is None else slots.data_ptr(), p[4], p[5],
        _current_stream(dev) if stream is None else _stream(stream))))


class WeightCache:
    """Packed weight rows for tq_weight_quantize / tq_weight_gemm: a cache of
    one sequence whose KV heads are the n_in / d blocks of a row and whose
    positions are the n_out rows (K planes only)."""

    def __init__(self, ctx: Context, n_out: int, n_in: int, device="cuda"):
        nb = n_in // ctx.d
        cap = (n_out + 63) // 64 * 64
        sizes = ctx.layout()
        self.codes = torch.zeros((nb, cap, sizes[0]), dtype=torch.uint8, device=device)
        self.norms = torch.zeros((nb, cap), dtype=torch.int16, device=device)
        self.n_out, self.n_in, self.capacity = n_out, n_in, cap
        self.struct = tq_cache(self.codes.data_ptr(), self.norms.data_ptr(), None, None, None, None, cap, 1, nb,
                               None, 0, 0)

    def nbytes(self) -> int:
        return self.codes.numel() + 2 * self.norms.numel()


def weight_quantize(ctx: Context, wc: WeightCache, w: torch.Tensor, stream=None) -> None:
    """tq_weight_quantize: w bf16 [n_out, n_in] contiguous."""
    _check(lib.tq_weight_quantize(ctx.handle, ctypes.byref(wc.struct), _ptr(w), wc.n_out, wc.n_in, _stream(stream)))


def weight_workspace_bytes(ctx: Context, n_tok: int, n_in: int) -> int:
    return int(lib.tq_weight_workspace_bytes(ctx.handle, n_tok, n_in))


def weight_gemm(ctx: Context, wc: WeightCache, x: torch.Tensor, y: torch.Tensor, workspace: torch.Tensor,
                stream=None) -> None:
    """tq_weight_gemm: x [n_tok, n_in] bf16 or fp32; y fp32 [n_tok, n_out]."""
    x_dtype = TQ_F32 if x.dtype == torch.float32 else TQ_BF16
    _check(lib.tq_weight_gemm(ctx.handle, ctypes.byref(wc.struct), wc.n_out, wc.n_in, _ptr(x), x_dtype, x.shape[0],
                              _ptr(y), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream)))


def alloc_workspace(ctx: Context, n_seqs: int, n_q_heads: int, max_seq_len: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(ctx, n_seqs, n_q_heads, max_seq_len)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def alloc_shared_workspace(ctx: Context, cache: Cache, n_q_heads: int, n_groups: int, max_group: int,
                           max_prefix_len: int, max_suffix_len: int, device="cuda") -> torch.Tensor:
    n = shared_workspace_bytes(ctx, cache, n_q_heads, n_groups, max_group, max_prefix_len, max_suffix_len)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)
