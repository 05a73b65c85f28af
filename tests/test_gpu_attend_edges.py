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
@pytest.mark.parametrize("n,T", [(70, 3), (6000, 3), (70, 130), (6000, 130)])
def test_logits_far_below_the_greatest(kvq, impl, n, T):
    """Cached keys whose logits all pass fp32's range downwards weigh nothing beside a new token with a
    logit of 0, whatever pieces the work is cut into; without it, the row is not finite."""
    P = Pool(kvq, 1, [[]], seed=T, chunk=1000)
    P.pool.destroy()
    pages = n // 32 + 64
    pool = kvq.KVPool(1, pages, pages, 1, pages)
    rid = pool.open()
    k = torch.full((n, 1, 128), -1.0, device="cuda").bfloat16()
    pool.append(k, rand((n, 1, 128), P.gen), np.full(n, rid, np.int32), mixed(n, 1))
    pool.set_decode_impl(impl)
    q = torch.ones(T, 4, 128, device="cuda").bfloat16()
    kn, vn = torch.zeros(T, 1, 128, device="cuda").bfloat16(), rand((T, 1, 128), P.gen)
    kn[1:] = -1.0
    out = pool.attend(q, [rid], [T], 2.0 ** 126, kn, vn)
    pool.sync()
    assert torch.equal(out, vn[:1].expand(T, 4, 128))
    kn[0] = -1.0
    out = pool.attend(q, [rid], [T], 2.0 ** 126, kn, vn)
    range_error(kvq, pool)
    assert not torch.isfinite(out.float()).any()


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


# ---- units above 384 rows on the tensor cores ------------------------------
@pytest.mark.parametrize("T", [100, 130])
def test_many_rows_evicted_and_excluded(kvq, T):
    """Evicted slots, a request with every slot evicted, slots excluded for one kv head, a list."""
    rng = np.random.default_rng(T)
    dead = [np.sort(rng.choice(1260, 160, replace=False)), np.arange(64), []]
    P = Pool(kvq, 2, [mixed(1260, 7, (2, 3, 4, 0xF4)), mixed(64, 8), mixed(90, 9)], seed=1, dead=dead)
    rows = [0, 1, 63, 64, T - 1]
    check(P, MMA, [0, 1, 2], [T, T, T], 8, rows=rows)
    ex = {0: {(1, int(p)) for p in rng.choice(1260, 400, replace=False)}, 2: {(0, p) for p in range(90)}}
    for r, s in ex.items():
        s = sorted(s)
        P.pool.evict_head([P.ids[r]] * len(s), [p for _, p in s], [h for h, _ in s])
    check(P, MMA, [0, 1, 2], [T, T, T], 8, rows=rows, head_dead=ex)
    out = check(P, MMA, [2, 1], [T, T], 8, rows=[0], head_dead=ex, with_kv=False)
    assert (out[:T, :4] == 0).all() and (out[T:] == 0).all()
    P.pool.fp_configure(200)
    fp = {}
    for r, n in ((1, 131), (2, 3)):
        k, v = rand((n, 2, 128), P.gen), rand((n, 2, 128), P.gen)
        P.pool.fp_append(P.ids[r], k, v)
        fp[r] = (k.double().cpu().numpy(), v.double().cpu().numpy())
    check(P, MMA, [0, 1, 2], [T, T, T], 8, rows=rows, head_dead=ex, fp=fp)


@pytest.mark.parametrize("choice", [(2,), (3,), (4,), (0xF4,), (2, 3, 4, 0xF4)])
def test_many_rows_every_width(kvq, choice):
    P = Pool(kvq, 2, [mixed(450, 3, choice), mixed(70, 4, choice)], seed=len(choice) + choice[0], reorder=False)
    check(P, MMA, [0, 1], [98, 110], 8, rows=[0, 33, 64, 97, 109])


@pytest.mark.parametrize("T", [49, 64])
@pytest.mark.parametrize("n", [0, 100, 5000])
def test_many_rows_tree(kvq, T, n):
    """392 to 512 rows of random masks: ancestors, later tokens, none at all, bits past the tokens."""
    P = Pool(kvq, 1, [mixed(n, 1), mixed(0, 1)], seed=T, chunk=1000)
    rng = np.random.default_rng(T + n)
    tree = rng.integers(0, 1 << 63, 2 * T, dtype=np.uint64) * np.uint64(2) + rng.integers(0, 2, 2 * T).astype(np.uint64)
    tree[0] = tree[T] = tree[T + 40] = 0
    tree[T + 1] = np.uint64(1) << np.uint64(T - 1)
    tree[-1] = np.uint64(0xFFFFFFFFFFFFFFFF)
    out = check(P, MMA, [0, 1], [T, T], 8, tree=tree, rows=[0, 1, 31, 32, 40, T - 1])
    assert (out[T] == 0).all() and (out[T + 40] == 0).all()


@pytest.mark.parametrize("n", [140, 5000])
def test_many_rows_unaligned_guards_and_out(kvq, n):
    """Inputs and outputs one element past an aligned address, blocks whole and merged from pieces;
    what lies around out stays."""
    P = Pool(kvq, 2, [mixed(n, 1)], seed=8, chunk=1000)
    hq, T = 8, 130
    base = {name: torch.randn(T * h * 128 + 1, generator=P.gen, device="cuda").bfloat16()
            for name, h in (("q", hq), ("k", 2), ("v", 2))}
    view = {name: base[name][1:].view(T, h, 128) for name, h in (("q", hq), ("k", 2), ("v", 2))}
    flat = torch.full((T * hq * 128 + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    P.pool.set_decode_impl(MMA)
    P.pool.attend(view["q"], P.ids, [T], SCALE, view["k"], view["v"], out=flat[1:1 + T * hq * 128].view(T, hq, 128))
    out = P.pool.attend(view["q"].clone(), P.ids, [T], SCALE, view["k"].clone(), view["v"].clone())
    P.pool.sync()
    assert torch.equal(flat[1:1 + T * hq * 128].view(T, hq, 128), out)
    assert flat[0] == 7.0 and (flat[1 + T * hq * 128:] == 7.0).all()
    check(P, MMA, [0], [T], hq, rows=[0, 63, 64, 127, T - 1])


def test_many_rows_values_out_of_range(kvq):
    T = 130
    P = Pool(kvq, 1, [mixed(50, 1)], seed=9)
    q, k, v = (rand((T, h, 128), P.gen) for h in (4, 1, 1))
    k[T - 1, 0, 5], v[T - 1, 0, 7], v[T - 1, 0, 8] = float("nan"), float("inf"), 1e38
    P.pool.set_decode_impl(MMA)
    out = P.pool.attend(q, P.ids, [T], SCALE, k, v)
    range_error(kvq, P.pool)
    k[T - 1, 0, 5] = v[T - 1, 0, 7] = v[T - 1, 0, 8] = 0
    ref = P.pool.attend(q, P.ids, [T], SCALE, k, v)
    P.pool.sync()
    assert torch.isfinite(out.float()).all() and torch.equal(out, ref)


def test_many_rows_other_stream_and_two_threads(kvq):
    """On another stream, repeated, and on two pools at once: what one call alone gives."""
    import threading
    pools = [Pool(kvq, 2, [mixed(900, s), mixed(333, s + 1)], seed=s) for s in (31, 33)]
    n_new = [110, 101]
    q, k, v = (rand((sum(n_new), h, 128), pools[0].gen) for h in (8, 2, 2))
    alone = [P.pool.attend(q, P.ids, n_new, SCALE, k, v) for P in pools]
    torch.cuda.synchronize()
    wrong = []

    def work(P, want):
        s = torch.cuda.Stream()
        out = torch.empty_like(want)
        for _ in range(10):
            P.pool.attend(q, P.ids, n_new, SCALE, k, v, out=out, stream=s)
        s.synchronize()
        P.pool.sync()
        if not torch.equal(out, want):
            wrong.append(P)

    t = [threading.Thread(target=work, args=x) for x in zip(pools, alone)]
    [x.start() for x in t]
    [x.join() for x in t]
    assert not wrong


def test_many_rows_of_one_long_chunk(kvq):
    """70,001 new tokens: 274 blocks of rows, 547 tiles of new keys."""
    P = Pool(kvq, 1, [mixed(1000, 1)], seed=3, chunk=500)
    check(P, MMA, [0], [70001], 1, rows=[0, 255, 256, 40000, 65535, 65536, 70000])


@pytest.mark.parametrize("impl", IMPLS)
def test_64_kv_heads(kvq, impl):
    P = Pool(kvq, 64, [mixed(90, 1), mixed(33, 2)], seed=5)
    check(P, impl, [0, 1], [2, 1], 64)
    check(P, impl, [1], [400], 64, rows=[0, 399])
