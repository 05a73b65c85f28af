"""kv_attend at the edges of its inputs: rows of q that are not finite or far from one, logits past
fp32, list tokens out of range; and what the kernel for many rows per unit does with evicted and
excluded slots, trees, every width, unaligned rows and other streams (units above 384 rows)."""
import numpy as np
import pytest

from attend_ref import SCALE, attend_row
from test_gpu_attend import IMPLS, MMA, ROUND, Pool, check, kvq, mixed, rand  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def range_error(kvq, pool):
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    pool.sync()   # reported once


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("n,T", [(70, 3), (6000, 3), (70, 130), (6000, 130)])
def test_rows_of_q_that_are_not_finite(kvq, impl, n, T):
    """They give rows that are not finite and KV_ERR_RANGE, and leave the other rows alone; blocks
    done whole (short caches) and in pieces (long ones), few rows per unit and many."""
    P = Pool(kvq, 1, [mixed(n, 3)], seed=T, chunk=1000)
    pool, hq = P.pool, 4
    q, k, v = (rand((T, h, 128), P.gen) for h in (hq, 1, 1))
    odd = {(0, 1): float("nan"), (1, 0): float("inf"), (1, 2): -float("inf"), (T - 1, 3): float("nan")}
    for (t, j), x in odd.items():
        q[t, j, (7 * t + j) % 128] = x
    pool.set_decode_impl(impl)
    out = pool.attend(q, P.ids, [T], SCALE, k, v)
    range_error(kvq, pool)
    got = out.double().cpu().numpy()
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    for t, j in odd:
        assert not np.isfinite(got[t, j]).any(), (t, j)
    C = P.content(0)
    for t in {0, 1, 2, T // 2, T - 1}:
        K, V = np.concatenate([C.K[0], kh[:t + 1, 0]]), np.concatenate([C.V[0], vh[:t + 1, 0]])
        for j in range(hq):
            if (t, j) not in odd:
                o, tol = attend_row(qh[t, j], K, V, SCALE, ROUND[impl])
                assert (np.abs(got[t, j] - o) <= tol).all(), (t, j)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [1, 130])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_one_infinite_element_and_keys_of_one_sign(kvq, impl, T, sign):
    """Every logit of the row is the same infinity."""
    P = Pool(kvq, 1, [mixed(0, 1)], seed=1)
    q, k, v = (rand((T, h, 128), P.gen) for h in (4, 1, 1))
    k[:, 0, 9] = 1.0
    q[0, 2, 9] = sign * float("inf")
    P.pool.set_decode_impl(impl)
    out = P.pool.attend(q, P.ids, [T], SCALE, k, v)
    range_error(kvq, P.pool)
    assert not torch.isfinite(out[0, 2].float()).any()
    out[0, 2] = 0
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [1, 130])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_past_fp32(kvq, impl, T, sign):
    """Finite rows whose logits all pass fp32's range (-128 * 2^127 and below, or above) are not finite."""
    P = Pool(kvq, 1, [mixed(0, 1)], seed=2)
    q, k, v = (torch.ones(T, h, 128, device="cuda").bfloat16() for h in (4, 1, 1))
    q[0, 1] = sign
    q[0, 0] = q[0, 2] = q[0, 3] = 0
    q[1:] = 0
    P.pool.set_decode_impl(impl)
    out = P.pool.attend(q, P.ids, [T], 2.0 ** 126, k, v)
    range_error(kvq, P.pool)
    assert not torch.isfinite(out[0, 1].float()).any()
    out[0, 1] = 1.0
    assert (out == 1.0).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [2, 130])
def test_list_tokens_out_of_range(kvq, impl, T):
    """A list token past binary16's range (or not a number) is used as 0 there and reported."""
    P = Pool(kvq, 1, [mixed(50, 1), mixed(50, 1)], seed=9)
    P.pool.fp_configure(40)
    k, v = rand((33, 1, 128), P.gen), rand((33, 1, 128), P.gen)
    bad = [(3, 7, float("nan")), (20, 100, 1e38), (32, 0, float("-inf"))]
    k0, v0 = k.clone(), v.clone()
    for t, c, x in bad:
        k[t, 0, c], v[t, 0, (c + 5) % 128] = x, x
        k0[t, 0, c], v0[t, 0, (c + 5) % 128] = 0, 0
    P.pool.fp_append(P.ids[0], k, v)
    q, kn, vn = (rand((T, h, 128), P.gen) for h in (4, 1, 1))
    P.pool.set_decode_impl(impl)
    out = P.pool.attend(q, [P.ids[0]], [T], SCALE, kn, vn)
    range_error(kvq, P.pool)
    P.pool.fp_drop(P.ids[0], 0, 33)
    P.pool.fp_append(P.ids[0], k0, v0)
    ref = P.pool.attend(q, [P.ids[0]], [T], SCALE, kn, vn)
    P.pool.sync()
    assert torch.isfinite(out.float()).all() and torch.equal(out, ref)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("size", [1e36, 1e-36])
def test_queries_near_the_ends_of_bf16(kvq, impl, size):
    P = Pool(kvq, 1, [mixed(200, 2)], seed=24)
    check(P, impl, [0], [5], 8, scale=SCALE / size, q_mult=size)
    check(P, impl, [0], [100], 8, scale=SCALE / size, q_mult=size, rows=[0, 60, 99])


@pytest.mark.parametrize("T", [3, 100])
def test_queries_at_the_ends_of_bf16(kvq, T):
    """The greatest and the least normal elements (the CUDA cores' fp32 sums do not hold the greatest).
    The scale of the greatest is below 2^-126, so fp32 holds it, and its product with log2 e, to 2^-20
    each: logits move by 2^-19 of themselves, which is within the hundredth that the tolerance of
    attend_row() adds to the 2^-11 of rounding K."""
    P = Pool(kvq, 1, [mixed(200, 2)], seed=25)
    P.pool.set_decode_impl(MMA)
    q = rand((T, 8, 128), P.gen).clamp(-3.9, 3.9)
    C = P.content(0)
    for e in (126, -118):
        qe = (q.float() * 2.0 ** e).bfloat16()
        got = P.pool.attend(qe, P.ids, [T], SCALE * 2.0 ** -e).double().cpu().numpy()
        P.pool.sync()
        qh = qe.double().cpu().numpy() * 2.0 ** -e
        for t in {0, T // 2, T - 1}:
            for j in range(8):
                o, tol = attend_row(qh[t, j], C.K[0], C.V[0], SCALE, ROUND[MMA])
                assert (np.abs(got[t, j] - o) <= tol).all(), (e, t, j)
