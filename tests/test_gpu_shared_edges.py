"""Attention over shared prefixes (kv_attend_shared) where its decode-step form, the choice of kernels by request and
long caches meet the ends of their ranges; against the plain 64-bit form and against kv_attend."""
import numpy as np
import pytest

from attend_ref import SCALE, attend_row
from test_gpu_attend import Pool, mixed, rand
from test_gpu_shared import U, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def step_pool(kvq, n=24, own=410, seed=1, hkv=8, prefix=200, **kw):
    """Request 0 is a prefix, 1 .. n have own caches: enough tiles for the decode's scan."""
    P = Pool(kvq, hkv, [mixed(prefix, 99)] + [mixed(own, i) for i in range(n)], seed=seed, slack=200, **kw)
    assert n * hkv * ((own + 127) // 128) > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    return P


@pytest.mark.parametrize("size", [2.0 ** 122, 2.0 ** 60, 2.0 ** -60, 2.0 ** -122])
def test_decode_step_queries_far_from_one(kvq, size):
    """Rows of q up to bf16's ends with a softmax scale that brings the logits back."""
    P = step_pool(kvq)
    n = len(P.ids) - 1
    check(P, range(1, n + 1), [0] * (n // 2) + [-1] * (n - n // 2), [1] * n, 16, with_kv=False, scale=SCALE / size, q_mult=size)
    P.pool.destroy()


def test_decode_step_large_logits(kvq):
    """Rows whose logits are large but in fp32's range, while q . k is not: the greatest key's value, as in kv_attend."""
    P = step_pool(kvq, seed=2)
    n = len(P.ids) - 1
    q = (rand((n, 16, 128), P.gen).float() * 2.0 ** 124).bfloat16()
    ids = P.ids[1:]
    out = P.pool.attend_shared(q, ids, [-1] * n, [1] * n, 2.0 ** -30)
    P.pool.sync()
    for b in (0, 7, n - 1):
        C = P.content(b + 1)
        for j in range(16):
            s = C.K[j // 2] @ q[b, j].double().cpu().numpy()
            first, second = np.sort(s)[[-1, -2]]
            # the two greatest are 2^80 apart in all but rows that tie by chance, so the weight is one key's alone
            assert (first - second) * 2.0 ** -30 > 2.0 ** 20
            o = C.V[j // 2][int(np.argmax(s))]
            # its value, rounded to binary16 (2^-11) inside and to bf16 (2^-8) once
            assert np.all(np.abs(out[b, j].double().cpu().numpy() - o) <= np.abs(o) * (2.0 ** -8 + 2 * U) + 1e-30)
    P.pool.destroy()


def test_decode_step_between_captured_decodes(kvq):
    """A captured decode and the statistics of the last decode stay what they are over decode steps of larger and
    smaller batches with shared prefixes, and the steps over decodes."""
    P = step_pool(kvq, seed=3)
    pool, n = P.pool, len(P.ids) - 1
    q, out = rand((2, 16, 128), P.gen), torch.empty(2, 16, 128, device="cuda")
    steps = [(rand((m, 16, 128), P.gen), P.ids[1:m + 1], [P.ids[0]] * m) for m in (n, n - 3)]
    first = [pool.attend_shared(x, ids, pre, [1] * len(ids), SCALE) for x, ids, pre in steps]
    want = pool.decode(q, P.ids[1:3], SCALE).clone()
    stats = pool.last_decode_stats()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        pool.decode(q, P.ids[1:3], SCALE, out=out)
    for _ in range(2):
        for (x, ids, pre), y in zip(steps, first):
            assert torch.equal(pool.attend_shared(x, ids, pre, [1] * len(ids), SCALE), y)
            assert pool.last_decode_stats() == stats
            out.zero_()
            torch.cuda.synchronize()
            g.replay()
            assert torch.equal(out, want)
    assert torch.equal(pool.decode(q, P.ids[1:3], SCALE), want)
    pool.sync()
    pool.destroy()
