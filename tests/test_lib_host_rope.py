"""CPU-side checks of the calls that rotate, read back and share prefixes: a null pool is an argument error
with a message, and the plain forms that the GPU tests use agree with one another."""
import numpy as np
import pytest

import rope_ref


@pytest.fixture(scope="module")
def kvq():
    from mixed_precision_kv_gb300 import build
    build.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def test_null_pool(kvq):
    L = kvq.load_library()
    one = np.zeros(1, np.int64).ctypes.data
    for rc in (L.kv_rotate(None, one, one, 1, 1, one, 1, 128, one, 128, None, 0, 0, None, 0, None),
               L.kv_append_rotated(None, one, one, 1, one, 128, one, 128, one, one, 1, None),
               L.kv_read_tokens(None, one, one, one, 1, 0, one, one, None),
               L.kv_attend_shared(None, one, one, one, None, one, one, one, 1, 8, 1.0, one, None)):
        assert rc == kvq.KV_ERR_INVALID_ARG
        assert b"null pool" in L.kv_last_error()


@pytest.mark.parametrize("rot,n_axes,pairs", [(128, 1, False), (64, 3, True), (16, 2, False)])
def test_plain_forms(rot, n_axes, pairs):
    rng = np.random.default_rng(rot)
    x = rope_ref.to_bf16(rng.standard_normal((50, 3, 128)) * 4)
    tab = rope_ref.table(200, rot)
    pos = rng.integers(0, 200, (n_axes, 50))
    axis = np.arange(rot // 2) % n_axes
    y = rope_ref.rotate(x, tab, pos, axis, pairs)
    exact, tol = rope_ref.rotate_exact(x, tab, pos, axis, pairs)
    assert np.all(np.abs(y - exact) <= tol)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    # as complex numbers, one frequency at a time
    for f in range(rot // 2):
        a, b = (2 * f, 2 * f + 1) if pairs else (f, f + rot // 2)
        row = tab[pos[axis[f]]].astype(np.float64)
        z = (x[..., a] + 1j * x[..., b]) * (row[:, f] + 1j * row[:, f + rot // 2])[:, None]
        assert np.allclose(z.real, exact[..., a], rtol=0, atol=1e-12) and np.allclose(z.imag, exact[..., b], rtol=0, atol=1e-12)
    # the length of a pair stays
    n0, n1 = np.linalg.norm(x[..., :rot].astype(np.float64), axis=-1), np.linalg.norm(exact[..., :rot], axis=-1)
    assert np.allclose(n0, n1, rtol=1e-6)
