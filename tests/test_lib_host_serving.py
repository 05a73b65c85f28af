"""CPU-side refusals of the calls that read a pool for serving: a null pool is an argument
error with a message, whatever the other arguments are."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def kvq():
    from mixed_precision_kv_gb300 import build
    build.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def test_null_pool(kvq):
    L = kvq.load_library()
    one = np.zeros(1, np.int32).ctypes.data
    for rc in (L.kv_attend(None, one, one, one, None, one, one, 1, 8, 1.0, one, None),
               L.kv_decode_attn_scored(None, one, one, 1, 8, 1.0, 1.0, one, 1, one, None),
               L.kv_select_lowest(None, one, 1, one, one, 1, 0, 0, one, 1, None)):
        assert rc == kvq.KV_ERR_INVALID_ARG
        assert b"null pool" in L.kv_last_error()
