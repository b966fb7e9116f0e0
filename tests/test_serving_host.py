"""CPU-only checks of the serving operators' entry points: refused before any
CUDA call without a context, and the plan's workspace is 0 for a refused call."""
import ctypes

import pytest


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
