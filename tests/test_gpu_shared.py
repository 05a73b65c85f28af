"""Attention of a batch over shared cached prefixes (kv_attend_shared) against the plain 64-bit form on
the pool's exported content, with tolerances per element from the roundings the operator makes."""
import numpy as np
import pytest

from attend_ref import SCALE, attend_row
from test_gpu_attend import Pool, mixed, rand

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -11   # unit roundoff of K, V and weights inside: binary16


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def check(P, which, prefix, n_new, hq, with_kv=True, tree=None, fp=None, head_dead=None, rows=None, scale=SCALE,
          q_mult=1.0, off=0):
    """attend_shared() on requests `which` with prefixes `prefix` (indexes, -1: none) against the plain form."""
    pool, hkv = P.pool, P.hkv
    g, N = hq // hkv, sum(n_new)
    flat = (torch.randn(N * hq * 128 + off, generator=P.gen, device="cuda") * q_mult).bfloat16()
    q = flat[off:].view(N, hq, 128)
    k, v = (rand((N, hkv, 128), P.gen), rand((N, hkv, 128), P.gen)) if with_kv else (None, None)
    td = None if tree is None else torch.from_numpy(np.asarray(tree, np.uint64).view(np.int64)).cuda()
    ids = [P.ids[r] for r in which]
    pre = [-1 if p < 0 else P.ids[p] for p in prefix]
    out = pool.attend_shared(q, ids, pre, n_new, scale, k, v, tree=td)
    pool.sync()
    got, qh = out.double().cpu().numpy(), q.double().cpu().numpy()
    kh, vh = (k.double().cpu().numpy(), v.double().cpu().numpy()) if with_kv else (None, None)
    content = {r: P.content(r, head_dead=(head_dead or {}).get(r)) for r in set(which) | {p for p in prefix if p >= 0}}

    def cached(r, h):
        K, V = content[r].K[h], content[r].V[h]
        if fp and r in fp:
            K, V = np.concatenate([K, fp[r][0][:, h]]), np.concatenate([V, fp[r][1][:, h]])
        return K, V

    first, num, den = 0, 0.0, 0.0
    for r, p, T in zip(which, prefix, n_new):
        for h in range(hkv):
            K, V = cached(r, h)
            if p >= 0:
                K, V = (np.concatenate(x) for x in zip(cached(p, h), (K, V)))
            for t in range(T) if rows is None else [x for x in rows if x < T]:
                see = []
                if with_kv:
                    see = [j for j in range(T) if (j <= t if tree is None else (int(tree[first + t]) >> j) & 1)]
                Kt = np.concatenate([K, kh[[first + j for j in see], h]]) if see else K
                Vt = np.concatenate([V, vh[[first + j for j in see], h]]) if see else V
                for j in range(h * g, (h + 1) * g):
                    o, tol = attend_row(qh[first + t, j], Kt, Vt, scale, U)
                    d = np.abs(got[first + t, j] - o)
                    assert np.all(d <= tol), (r, p, t, j, d.max(), (d - tol).max())
                    num += float((d * d).sum())
                    den += float((o * o).sum())
        first += T
    assert num <= (2.0 ** -7) ** 2 * max(den, 1e-30)
    return q, k, v, td, out


@pytest.mark.parametrize("hkv,hq,pre,own,n_new,prefix", [
    (2, 8, (100,), (0, 40), (1, 1), (0, 0)),                                   # few rows
    (1, 8, (700,), (3, 65, 0, 31), (1, 1, 1, 1), (0, 0, -1, 0)),               # one request without a prefix
    (2, 10, (300, 129), (20, 33, 7, 64, 1), (2, 1, 3, 1, 2), (0, 1, 0, 1, 0)),  # apart in the batch
    (4, 4, (128, 0), (5, 6, 7), (1, 1, 1), (1, 0, 1)),                         # an empty prefix
    (2, 16, (513,), (10,) * 9, (2,) * 9, (0,) * 9)])                           # 144 rows of the prefix
@pytest.mark.parametrize("with_kv", [True, False])
def test_shared(kvq, hkv, hq, pre, own, n_new, prefix, with_kv):
    P = Pool(kvq, hkv, [mixed(n, i) for i, n in enumerate(pre + own)], seed=hq)
    check(P, range(len(pre), len(pre) + len(own)), prefix, n_new, hq, with_kv)
    P.pool.destroy()


@pytest.mark.parametrize("rows", [65, 100, 127, 128, 129, 200])
def test_rows_of_a_prefix(kvq, rows):
    """Blocks of 128 rows of a prefix, full and not: every width, list tokens, evicted slots, few keys and many."""
    rng = np.random.default_rng(rows)
    w = (2, 3, 4, 0xF4)
    P = Pool(kvq, 1, [rng.choice(w, 900).astype(np.uint8), rng.choice(w, 20).astype(np.uint8), mixed(70, 2), mixed(40, 3)],
             seed=rows, dead=[list(range(250, 420)), [], [], []], slack=128)
    P.pool.fp_configure(140)
    k, v = rand((130, 1, 128), P.gen), rand((130, 1, 128), P.gen)
    P.pool.fp_append(P.ids[0], k, v)
    fp = {0: (k.double().cpu().numpy(), v.double().cpu().numpy())}
    some = sorted({0, 1, rows // 3 - 1, rows // 3, rows // 2, rows - rows // 3 - 1})
    check(P, [2, 3], [0, 0], [rows // 3, rows - rows // 3], 1, fp=fp, rows=some)
    check(P, [2, 3], [1, 1], [rows // 3, rows - rows // 3], 1, rows=some)
    P.pool.destroy()


@pytest.mark.parametrize("g", [1, 4, 7])
def test_decode_step(kvq, g):
    """A token per request and no new keys, enough tiles for the decode's scan: ragged own caches (one empty), a request
    without a prefix, evicted slots and slots excluded for a head, a second prefix with one request."""
    rng = np.random.default_rng(g)
    lens = [260, 33] + [0] + [int(x) for x in rng.integers(300, 600, 21)]
    dead = [list(rng.choice(n, n // 8, replace=False)) if n else [] for n in lens]
    P = Pool(kvq, 8, [mixed(n, i) for i, n in enumerate(lens)], seed=g, dead=dead, slack=200)
    P.pool.evict_head([P.ids[5]] * 2 + [P.ids[0]], [7, 200, 3], [0, 7, 2])
    head_dead = {5: {(0, 7), (7, 200)}, 0: {(2, 3)}}
    which = list(range(2, 24))
    prefix = [0] * 22
    prefix[4], prefix[9] = -1, 1
    for _ in range(2):   # the second call finds the plan in place
        check(P, which, prefix, [1] * 22, 8 * g, with_kv=False, head_dead=head_dead)
    assert sum((n + 127) // 128 * 8 for n in lens[2:]) > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    P.pool.destroy()


def test_decode_step_far_below(kvq):
    """Rows of a decode step whose logits lie below the logit that the scan gives a dead slot, that are not finite, or
    whose own cache holds nothing live: as in the other kernels.  With an empty prefix, so that the weights go by the own
    caches, whose values are taken in fp32."""
    hkv, n = 8, 24
    P = Pool(kvq, hkv, [mixed(0, 0)] + [mixed(410, i) for i in range(n)], seed=3, slack=200,
             dead=[[]] + [list(range(410)) if i == 4 else [1, 40] for i in range(n)])
    pool = P.pool
    q = rand((n, hkv, 128), P.gen)
    q[1, 0] *= 3000.0            # logits of either sign beyond 1e4
    q[2] = -q[2].abs() * 4000.0
    q[3, 1, 9] = float("nan")
    q[5, 2, 8] = float("inf")
    ids, pre = P.ids[1:], [P.ids[0]] * (n // 2) + [-1] * (n // 2)
    out = pool.attend_shared(q, ids, pre, [1] * n, SCALE)
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    got = out.double().cpu().numpy()
    for b in (0, 1, 2, 4, n - 1):
        C = P.content(b + 1)
        for h in range(hkv):
            o, tol = attend_row(q[b, h].double().cpu().numpy(), C.K[h], C.V[h], SCALE, 2.0 ** -17)
            assert np.all(np.abs(got[b, h] - o) <= tol), (b, h)
    assert np.all(got[4] == 0)
    assert not np.isfinite(got[3, 1]).all() and np.isfinite(got[3, 0]).all() and np.isfinite(got[3, 2]).all()
    assert not np.isfinite(got[5, 2]).all() and np.isfinite(got[5, 3]).all()
    # keys that all point one way: every logit far below -1e4, the softmax among them unchanged by a common offset
    pool2 = kvq.KVPool(hkv, 8, 400, n, 20)
    ids = [pool2.open() for _ in range(n)]
    x = rand((n * 410, hkv, 128), P.gen)
    x[..., 32:64] = 0
    x[..., 40] = 16.0            # exact in the page: its group holds 0 and 16 alone
    v = rand((n * 410, hkv, 128), P.gen)
    pool2.append(x, v, np.repeat(ids, 410), np.full(n * 410, 4, np.uint8))
    q = rand((n, hkv, 128), P.gen)
    near = pool2.attend_shared(q * (torch.arange(128, device="cuda") != 40), ids, [-1] * n, [1] * n, SCALE)
    q[..., 40] = -16384.0        # logit -16 * 16384 / sqrt(128) = -23170, plus those of the other channels
    far = pool2.attend_shared(q, ids, [-1] * n, [1] * n, SCALE)
    pool2.sync()
    # the other channels' sum, of up to some tens, is rounded to fp32 beside 262144: 2^-6 at most each way before the
    # scale, so a logit moves by 2^-6 / 11.3 * 128 at the very most in a sum of 128 terms; bf16 rounds both results
    lim = 2 * (np.exp(2 * 128 * 2.0 ** -6 / 11.3) - 1) * float(v.float().abs().max())
    assert (near.float() - far.float()).abs().max() <= lim
    assert bool((far.float().abs().amax(-1) > 0).all())
    pool2.destroy()
    pool.destroy()


@pytest.mark.parametrize("rows_each,batch", [(25, 6), (70, 8), (40, 2)])
def test_shared_many_rows(kvq, rows_each, batch):
    """The prefix's rows go to the kernel for many rows (600 and 2,240 of them), the requests' own to either."""
    P = Pool(kvq, 2, [mixed(260, 1)] + [mixed(50 + i, i) for i in range(batch)], seed=4)
    check(P, range(1, batch + 1), [0] * batch, [rows_each + (i % 3) for i in range(batch)], 8, rows=[0, 1, 13, 24, 69])
    P.pool.destroy()


def test_shared_mixed_kernels(kvq):
    """Chunks and single tokens over one prefix, and a second prefix with few rows."""
    P = Pool(kvq, 1, [mixed(400, 1), mixed(90, 2), mixed(30, 3), mixed(200, 4), mixed(0, 5), mixed(77, 6)], seed=5)
    check(P, [2, 3, 4, 5], [0, 0, 1, -1], [1, 150, 3, 160], 4, rows=[0, 1, 2, 100, 149, 159])
    P.pool.destroy()


def test_shared_widths_lists_evictions_tree(kvq):
    """Every width, list tokens of the prefix and of a request, slots evicted for all heads and for one, trees."""
    rng = np.random.default_rng(6)
    w = (2, 3, 4, 0xF4)
    dead = [list(range(10, 45)), [0, 3], []]
    P = Pool(kvq, 2, [rng.choice(w, 190).astype(np.uint8), rng.choice(w, 40).astype(np.uint8), mixed(8, 2)], seed=6, dead=dead)
    pool = P.pool
    pool.evict_head([P.ids[0]] * 3, [50, 51, 189], [0, 1, 1])
    head_dead = {0: {(0, 50), (1, 51), (1, 189)}}
    pool.fp_configure(200)
    fp = {}
    for r, n in ((0, 150), (2, 5)):
        k, v = rand((n, 2, 128), P.gen), rand((n, 2, 128), P.gen)
        pool.fp_append(P.ids[r], k, v)
        fp[r] = (k.double().cpu().numpy(), v.double().cpu().numpy())
    tree = []
    for T in (5, 31):
        m = []
        for t in range(T):
            up = m[int(rng.integers(max(0, t - 3), t))] if t and rng.random() < 0.8 else 0
            m.append(up | 1 << t)
        tree += m
    check(P, [1, 2], [0, 0], [5, 31], 6, tree=tree, fp=fp, head_dead=head_dead)
    check(P, [2, 1], [0, -1], [1, 1], 6, with_kv=False, fp=fp, head_dead=head_dead)
    pool.destroy()


def test_nothing_to_see(kvq):
    """Rows whose prefix and own cache hold nothing live are zero; those of one part are that part's."""
    P = Pool(kvq, 1, [mixed(33, 1, (4,)), mixed(0, 2), mixed(20, 3, (4,)), mixed(5, 4)], seed=7,
             dead=[list(range(33)), [], list(range(20)), []])
    q, _, _, _, out = check(P, [1, 2, 3], [0, 0, 0], [1, 2, 1], 8, with_kv=False)
    assert bool((out[:3] == 0).all()) and not bool((out[3] == 0).all())
    check(P, [1, 2, 3], [2, -1, 0], [2, 1, 1], 8, with_kv=True)
    P.pool.destroy()


def test_prefix_as_request(kvq):
    """A request of the batch that is also another's prefix, one listed twice, and a prefix of a prefix's request."""
    P = Pool(kvq, 2, [mixed(80, 1), mixed(45, 2), mixed(9, 3)], seed=8)
    check(P, [0, 1, 1, 2], [-1, 0, 2, 1], [1, 2, 1, 3], 4)
    P.pool.destroy()


def test_large_logits_and_values(kvq):
    """Maxima far apart between the parts."""
    P = Pool(kvq, 1, [mixed(140, 1), mixed(70, 2), mixed(3, 3)], seed=9, kv_scale=30.0)
    check(P, [1, 2], [0, 0], [3, 1], 8, q_mult=20.0)
    check(P, [1, 2], [0, 0], [3, 1], 8, scale=-0.5)
    check(P, [1, 2], [0, 0], [3, 1], 8, scale=0.0)
    P.pool.destroy()


def test_unaligned_rows(kvq):
    P = Pool(kvq, 2, [mixed(140, 1), mixed(70, 2), mixed(3, 3)], seed=10)
    check(P, [1, 2], [0, 0], [3, 1], 6, off=1)
    check(P, [1, 2, 1], [0, -1, 0], [60, 100, 70], 8, off=3, rows=[0, 59, 99])
    P.pool.destroy()


def test_not_finite_rows(kvq):
    """A row of q that is not finite gives one that is not, and is reported; the others stay."""
    P = Pool(kvq, 1, [mixed(140, 1), mixed(40, 2), mixed(30, 3)], seed=11)
    pool = P.pool
    q = rand((4, 4, 128), P.gen)
    ids, pre, n = [P.ids[1], P.ids[2]], [P.ids[0]] * 2, [2, 2]
    good = pool.attend_shared(q, ids, pre, n, SCALE)
    pool.sync()
    bad = q.clone()
    bad[1, 2, 5] = float("inf")
    bad[3, 0, 0] = float("nan")
    out = pool.attend_shared(bad, ids, pre, n, SCALE)
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    fin = torch.isfinite(out).all(-1)
    assert not bool(fin[1, 2]) and not bool(fin[3, 0]) and int(fin.sum()) == 14
    # The rows of a block refresh their maxima together, and a row without one asks for it at every key tile, so the
    # others' weights 2^(x - m + 7) may be scaled by another power of two: exact in x, each weight is still rounded by
    # 2^-11 of itself.  Both results are therefore within the operator's own tolerance of the 64-bit one.
    C = [P.content(r) for r in range(3)]
    for t, r in enumerate((1, 1, 2, 2)):
        K, V = (np.concatenate([getattr(C[0], m)[0], getattr(C[r], m)[0]]) for m in "KV")
        for j in range(4):
            if bool(fin[t, j]):
                o, tol = attend_row(q[t, j].double().cpu().numpy(), K, V, SCALE, U)
                for x in (out, good):
                    assert np.all(np.abs(x[t, j].double().cpu().numpy() - o) <= tol)
    pool.sync()
    pool.destroy()


def test_order_and_streams(kvq):
    """The same rows whatever the order of the batch, and calls in a row on two streams and pools."""
    P, Q = (Pool(kvq, 2, [mixed(300, 1), mixed(64, 2), mixed(20, 3), mixed(31, 4)], seed=12) for _ in range(2))
    q = rand((6, 8, 128), P.gen)
    n = [1, 2, 3]
    a = P.pool.attend_shared(q, P.ids[1:], [P.ids[0]] * 3, n, SCALE)
    perm = torch.tensor([3, 4, 5, 0, 1, 2], device="cuda")
    b = P.pool.attend_shared(q[perm], [P.ids[3], P.ids[1], P.ids[2]], [P.ids[0]] * 3, [3, 1, 2], SCALE)
    assert (a[perm].float() - b.float()).abs().max() <= 2.0 ** -7 * a.float().abs().max()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for x, (X, s) in enumerate(zip((P, Q), streams)):
            outs[x].append(X.pool.attend_shared(q, X.ids[1:], [X.ids[0]] * 3, n, SCALE, stream=s))
    P.pool.sync()
    Q.pool.sync()
    for x in range(2):
        assert all(torch.equal(o, a) for o in outs[x])
    P.pool.destroy()
    Q.pool.destroy()


def test_as_attend_without_prefix(kvq):
    """Without prefixes the call is kv_attend, bit for bit."""
    P = Pool(kvq, 2, [mixed(500, 1), mixed(64, 2)], seed=13)
    for n in ([1, 3], [130, 2]):
        q, k, v = rand((sum(n), 8, 128), P.gen), rand((sum(n), 2, 128), P.gen), rand((sum(n), 2, 128), P.gen)
        assert torch.equal(P.pool.attend_shared(q, P.ids, [-1, -1], n, SCALE, k, v), P.pool.attend(q, P.ids, n, SCALE, k, v))
    P.pool.destroy()


def test_timeout(kvq):
    """An expired wait is reported once, and the pool goes on."""
    P = Pool(kvq, 1, [mixed(300, 1), mixed(64, 2)], seed=14)
    q = rand((1, 8, 128), P.gen)
    good = P.pool.attend_shared(q, [P.ids[1]], [P.ids[0]], [1], SCALE)
    P.pool.sync()
    P.pool.set_wait_limit(0)
    P.pool.attend_shared(q, [P.ids[1]], [P.ids[0]], [1], SCALE)
    with pytest.raises(kvq.KVError) as e:
        P.pool.sync()
    assert e.value.status == kvq.KV_ERR_DEVICE_TIMEOUT
    P.pool.set_wait_limit(-1)
    assert torch.equal(P.pool.attend_shared(q, [P.ids[1]], [P.ids[0]], [1], SCALE), good)
    P.pool.sync()
    P.pool.destroy()


def test_a_step_as_it_is_served(kvq):
    """A document cached once, samples over it: rotated appends, rotated queries, attention over the prefix and the
    own tokens, a few steps; every step against the plain form on the pool's content."""
    import rope_ref
    from test_gpu_rope import host, make_rope
    P = Pool(kvq, 2, [[], [], [], []], seed=15, slack=64)
    pool, hq, g = P.pool, 6, 3
    rope, tab = make_rope(kvq, 600, 128)
    doc, samples = P.ids[0], P.ids[1:]
    n = 200
    x = rand((n, 4, 128), P.gen)
    bits = np.random.default_rng(1).choice([2, 4], n).astype(np.uint8)
    pool.append_rotated(x[:, :2], x[:, 2:], [doc] * n, bits, rope, torch.arange(n, dtype=torch.int32, device="cuda"))
    pool.reorder([doc])
    P.widths[0] = list(bits)
    for step in range(3):
        qkv = rand((3, hq + 4, 128), P.gen)
        pos = torch.full((3,), n + step, dtype=torch.int32, device="cuda")
        pool.append_rotated(qkv[:, hq:hq + 2], qkv[:, hq + 2:], samples, [4] * 3, rope, pos)
        for r in (1, 2, 3):
            P.widths[r].append(4)
        q = pool.rotate(qkv[:, :hq], rope, pos)
        out = pool.attend_shared(q, samples, [doc] * 3, [1] * 3, SCALE)
        pool.sync()
        qh = rope_ref.rotate(host(qkv[:, :hq]), tab, pos.cpu().numpy()).astype(np.float64)
        C = [P.content(r) for r in range(4)]
        for s in range(3):
            for j in range(hq):
                K, V = (np.concatenate([getattr(C[0], m)[j // g], getattr(C[s + 1], m)[j // g]]) for m in "KV")
                o, tol = attend_row(qh[s, j], K, V, SCALE, U)
                assert np.all(np.abs(out[s, j].double().cpu().numpy() - o) <= tol)
    # reading back what the steps left
    k, _ = pool.read([samples[0]], dtype=torch.float32)
    assert k.shape == (3, 2, 128) and np.allclose(k.cpu().numpy()[:, 0], C[1].K[0].astype(np.float32))
    pool.destroy()


def test_refusals(kvq):
    P = Pool(kvq, 2, [mixed(40, 1), mixed(10, 2)], seed=16)
    pool, (a, b) = P.pool, P.ids
    q = rand((1, 4, 128), P.gen)
    for pre in ([b], [-2], [99]):
        with pytest.raises(kvq.KVError) as e:
            pool.attend_shared(q, [b], pre, [1], SCALE)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pool.attend_shared(q, [b], [a, a], [1], SCALE)
    for bad in (dict(q=q.float()), dict(n_new=[2]), dict(k=rand((1, 2, 128), P.gen)), dict(out=q.float())):
        args = dict(q=q, req_ids=[b], prefix_ids=[a], n_new=[1], softmax_scale=SCALE)
        args.update(bad)
        with pytest.raises(ValueError):
            pool.attend_shared(**args)
    with pytest.raises(kvq.KVError):
        pool.attend_shared(q, [b], [a], [1], float("nan"))
    g = torch.cuda.CUDAGraph()
    o = torch.empty_like(q)
    with torch.cuda.graph(g):
        with pytest.raises(kvq.KVError) as e:
            pool.attend_shared(q, [b], [a], [1], SCALE, out=o)
        assert e.value.status == kvq.KV_ERR_STATE
    assert pool.attend_shared(q[:0], [b], [a], [0], SCALE).shape == (0, 4, 128)
    pool.sync()
    pool.destroy()
