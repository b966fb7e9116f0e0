"""CPU-only checks of the serving operators' entry points: refused before any
CUDA call without a context, and the plan's workspace is 0 for a refused call."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_12_b200 import build
    build.build()
    from kv_cache_vector_12_b200 import tq as tqmod
    return tqmod


def test_calls_without_a_context_are_refused(tq):
    lib, c = tq.lib, tq.tq_cache()
    ref = ctypes.byref(c)
    assert lib.tq_build_tables(None, ref, None, None, None, None, 0, None, None, None, None, 0, 0, None, None, None,
                               None, None, None) == tq.TQ_ERR_INVALID
    assert b"ctx" in lib.tq_last_error()
    assert lib.tq_prompt_attention(None, None, None, None, 0, 0, 0, 0, 1, 1, None, 0, 0, 0.0, None, 0, None,
                                   None) == tq.TQ_ERR_INVALID
    assert b"ctx" in lib.tq_last_error()
    assert lib.tq_decode_attention_shared(None, ref, None, 0, 1, None, None, None, 1, 1, 0, 0, 0.0, None, 0, None, None,
                                          0, None) == tq.TQ_ERR_INVALID
    assert b"ctx" in lib.tq_last_error()
    assert lib.tq_shared_workspace_bytes(None, ref, 1, 1, 1, 64, 64) == 0
    assert lib.tq_shared_workspace_bytes(None, None, 1, 1, 1, 64, 64) == 0


class _Library:
    """Takes the library's place: counts the calls that reach it, and launches nothing."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def entry(*args):
            self.calls += 1
            return 0
        return entry


class _Held:
    """What a context and a cache hold, without their device memory."""

    def __init__(self, **kw):
        self.__dict__.update(kw)


@pytest.fixture
def bound(tq, monkeypatch):
    """The binding on CPU tensors (device -1 is the current one), its calls going to a _Library."""
    lib = _Library()
    monkeypatch.setattr(tq, "lib", lib)
    monkeypatch.setattr(tq, "_device", lambda: -1, raising=False)
    monkeypatch.setattr(tq, "_stream", lambda stream: 0, raising=False)
    monkeypatch.setattr(tq, "_current_stream", lambda dev: 0, raising=False)
    return tq, lib


def _refusals(bound, call, good, bad):
    """`good` reaches the library; with any one argument of `bad` in its place the call is refused before it."""
    tq, lib = bound
    call(**good)
    assert lib.calls == 1
    for name, values in bad.items():
        for i, value in enumerate(values):
            with pytest.raises(tq.TQError) as ei:
                call(**{**good, **(value if isinstance(value, dict) else {name: value})})
            assert ei.value.status == tq.TQ_ERR_INVALID and lib.calls == 1, (name, i)
    call(**good)
    assert lib.calls == 2


def test_prompt_attention_refuses_other_sizes_types_and_devices(bound, monkeypatch):
    tq, lib = bound
    bf = dict(dtype=torch.bfloat16)
    good = dict(q=torch.zeros(40, 8, 128, **bf), k=torch.zeros(40, 2, 128, **bf), v=torch.zeros(40, 2, 128, **bf),
                cu_seqlens=torch.tensor([0, 30, 40], dtype=torch.int32), max_len=30, out=torch.zeros(40, 8, 128, **bf),
                lse=torch.zeros(40, 8))
    ctx = _Held(handle=None, d=128)

    def call(**kw):
        tq.prompt_attention(ctx, **kw)

    _refusals(bound, call, good, dict(
        k=[torch.zeros(39, 2, 128, **bf), torch.zeros(40, 4, 128, **bf), torch.zeros(40, 2, 128, **bf)[..., :64],
           torch.zeros(40, 2, 128, dtype=torch.float16)],
        v=[torch.zeros(39, 2, 128, **bf), torch.zeros(40, 1, 128, **bf), torch.zeros(40, 2, 128, **bf)[..., :64]],
        out=[torch.zeros(39, 8, 128, **bf), torch.zeros(40, 8, 128, dtype=torch.float16), torch.zeros(40, 2, 128, **bf),
             torch.zeros(128, 8, 40, **bf).transpose(0, 2)],
        lse=[torch.zeros(39, 8), torch.zeros(40, 8, dtype=torch.float64), torch.zeros(8, 40).t(), torch.zeros(40, 8, **bf)],
        cu_seqlens=[torch.tensor([0, 30, 40]), torch.tensor([0., 30., 40.]),
                    torch.zeros(6, dtype=torch.int32)[::2], torch.zeros(1, dtype=torch.int32).expand(3)]))
    tq.prompt_attention(ctx, **{**good, "lse": None, "out": torch.zeros(50, 1024), "k": torch.zeros(41, 2, 128, **bf)})
    assert lib.calls == 3
    monkeypatch.setattr(tq, "_device", lambda: 0)  # nothing of these is there
    with pytest.raises(tq.TQError):
        call(**good)
    assert lib.calls == 3


def test_build_tables_refuses_other_sizes_types_and_devices(bound, monkeypatch):
    tq, lib = bound
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    ctx, table = _Held(handle=None, d=128), i32(12).view(3, 4)
    cache = _Held(struct=tq.tq_cache(n_seqs=3, block_table=table.data_ptr()), block_table=table)
    good = dict(cached_lens=i32(3), new_lens=i32(3), seq_idx=i32(20), pos=i32(20), cu_new=i32(4), seq_lens=i32(3),
                slots=torch.zeros(20, dtype=torch.int64), free_list=i32(9), free_start=i32(1), free_end=i32(1),
                cu_group=i32(3), prefix_lens=i32(2))

    def call(**kw):
        tq.build_tables(ctx, cache, **kw)

    long = lambda n: torch.zeros(n, dtype=torch.int64)  # noqa: E731
    bad = {name: [long(t.numel()), t.float(), i32(2 * t.numel())[::2] if t.numel() > 1 else i32(0)]
           for name, t in good.items() if name != "slots"}
    for name in ("cached_lens", "new_lens", "pos", "cu_new", "seq_lens", "cu_group", "free_start", "free_end"):
        bad[name].append(i32(good[name].numel() - 1))
    bad["new_lens"].append(i32(1).expand(3))
    bad["slots"] = [i32(20), long(19), long(40)[::2]]
    _refusals(bound, call, good, bad)
    call(**{**good, "slots": None, "free_list": None, "cu_group": None, "prefix_lens": None})
    call(**{**good, "pos": i32(25), "cu_new": i32(9), "slots": long(21)})  # more room than is used
    assert lib.calls == 4
    cache.block_table = table.clone()  # not what the cache's other calls read
    with pytest.raises(tq.TQError):
        call(**good)
    cache.block_table = table
    monkeypatch.setattr(tq, "_device", lambda: 0)
    with pytest.raises(tq.TQError):
        call(**good)
    assert lib.calls == 4


def test_decode_attention_shared_refuses_other_sizes_types_and_devices(bound, monkeypatch):
    tq, lib = bound
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    ctx, cache = _Held(handle=None, d=128), _Held(struct=tq.tq_cache(n_seqs=3, n_kv_heads=2))
    good = dict(q=torch.zeros(3, 8, 128), seq_lens=i32(3), cu_group=i32(3), prefix_lens=i32(2), max_group=2,
                max_prefix_len=64, max_suffix_len=64, out=torch.zeros(3, 8, 128, dtype=torch.bfloat16),
                lse=torch.zeros(3, 8), workspace=torch.zeros(4096, dtype=torch.uint8))

    def call(**kw):
        tq.decode_attention_shared(ctx, cache, **kw)

    _refusals(bound, call, good, dict(
        q=[torch.zeros(2, 8, 128), torch.zeros(3, 8, 64), torch.zeros(3, 8, 128, dtype=torch.float16),
           torch.zeros(3, 16, 128)[:, ::2], torch.zeros(3, 8, 128, dtype=torch.float64)],
        seq_lens=[i32(2), i32(3).long(), i32(6)[::2], i32(1).expand(3)],
        cu_group=[i32(2), i32(3).long(), i32(6)[::2]],
        prefix_lens=[i32(3), i32(2).long(), i32(4)[::2]],
        out=[torch.zeros(2, 8, 128), torch.zeros(3, 8, 128, dtype=torch.float16), torch.zeros(3, 16, 128)[:, ::2]],
        lse=[torch.zeros(3, 7), torch.zeros(3, 8, dtype=torch.float64), torch.zeros(8, 3).t()],
        workspace=[torch.zeros(64, 128, dtype=torch.uint8)[:, :64]]))
    call(**{**good, "lse": None, "seq_lens": i32(9), "workspace": torch.zeros(4096)})
    assert lib.calls == 3
    monkeypatch.setattr(tq, "_device", lambda: 0)
    with pytest.raises(tq.TQError):
        call(**good)
    assert lib.calls == 3


@pytest.mark.parametrize("entry,pack,n,scale", [("tq_decode_attention_shared_words", "_SHARED_WORDS", 19, 12),
                                                ("tq_prompt_attention_words", "_PROMPT_WORDS", 18, 13),
                                                ("tq_build_tables_words", "_TABLES_WORDS", 19, None)])
def test_calls_by_words_reach_the_calls_and_refuse_integers_that_do_not_fit(tq, entry, pack, n, scale):
    call, pack = getattr(tq.lib, entry), getattr(tq, pack)
    assert call(None) == tq.TQ_ERR_INVALID
    words = [0.0 if i == scale else 0 for i in range(n)]
    assert call(pack(*words)) == tq.TQ_ERR_INVALID and b"ctx is NULL" in tq.lib.tq_last_error()
    words[11 if n == 19 else 8] = -2 ** 31
    assert call(pack(*words)) == tq.TQ_ERR_INVALID and b"ctx is NULL" in tq.lib.tq_last_error()
    for far in (2 ** 31, -2 ** 31 - 1, 2 ** 40):
        words[11 if n == 19 else 8] = far
        assert call(pack(*words)) == tq.TQ_ERR_INVALID and b"32 bits" in tq.lib.tq_last_error()
