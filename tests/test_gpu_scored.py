"""The decode that accumulates attention weight (kv_decode_attn_scored) and the lowest-score
selection (kv_select_lowest) against plain 64-bit forms, and both with attend() as a serving
loop uses them."""
import numpy as np
import pytest

from attend_ref import SCALE
from test_gpu_attend import MMA, Pool, kvq, mixed, rand  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def weights(C, h, qrows, scale, fp=None):
    """Per live slot of a head: the summed softmax weights of its q rows, and a bound on their
    error: a logit is an fp32 sum of 128 exact products and a few scalings (136 roundings), and
    moves numerator and denominator of a weight."""
    K = C.K[h] if fp is None else np.concatenate([C.K[h], fp])
    s = scale * (qrows @ K.T)
    w = np.exp(s - s.max(1, keepdims=True)) if K.shape[0] else s
    w /= w.sum(1, keepdims=True)
    ds = 136 * 2.0 ** -24 * scale * np.max(np.abs(qrows) @ np.abs(K).T) if K.shape[0] else 0.0
    n = C.K[h].shape[0]
    return w.sum(0)[:n], w.sum(0)[:n] * (2 * ds + 2.0 ** -20)


def step(P, hq, scores, decay, head_dead=None, fp=None, which=None, scale=SCALE):
    pool, hkv, g = P.pool, P.hkv, hq // P.hkv
    which = list(range(len(P.ids))) if which is None else which
    ids = [P.ids[r] for r in which]
    q = rand((len(ids), hq, 128), P.gen)
    before = scores.double().cpu().numpy()
    out = pool.decode_scored(q, ids, scale, scores, decay=decay)
    ref_out = pool.decode(q, ids, scale)
    pool.sync()
    assert torch.equal(out, ref_out)          # the same scan and merge
    after = scores.double().cpu().numpy()
    qh = q.double().cpu().numpy()
    for b, r in enumerate(which):
        C = P.content(r, head_dead=(head_dead or {}).get(r))
        for h in range(hkv):
            w, tol = weights(C, h, qh[b, h * g:(h + 1) * g], scale, None if not fp or r not in fp else fp[r][:, h])
            want = before[b, h].copy()
            want[C.pos[h]] = want[C.pos[h]] * decay + w
            lim = np.zeros_like(want)
            lim[C.pos[h]] = tol + np.abs(want[C.pos[h]]) * 2.0 ** -22
            d = np.abs(after[b, h] - want)
            assert (d <= lim).all(), (b, h, float(d.max()))


@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 2), (1, 3), (2, 4), (1, 5), (1, 6), (1, 7), (2, 8)])
def test_scores_of_ragged_requests(kvq, hkv, g):
    P = Pool(kvq, hkv, [mixed(n, n) for n in (1, 32, 33, 300, 0, 517)], seed=g, dead=[[], [3], [], np.arange(40, 90), [], []])
    scores = torch.rand(6, hkv, 530, device="cuda")
    step(P, hkv * g, scores, 1.0)
    step(P, hkv * g, scores, 0.75)
    step(P, hkv * g, scores, 0.0)


@pytest.mark.parametrize("choice", [(3,), (0xF4,), (2, 3, 4, 0xF4)])
def test_scores_of_every_width(kvq, choice):
    P = Pool(kvq, 2, [mixed(450, 3, choice), mixed(70, 4, choice)], seed=3, reorder=False)
    scores = torch.zeros(2, 2, 450, device="cuda")
    step(P, 8, scores, 1.0)
    step(P, 16, scores, 1.0)


def test_scores_with_exclusions_lists_and_appends(kvq):
    """Excluded slots keep their score; list tokens take part in the softmax; positions follow
    tokens through repacks, reorders and drops of pages."""
    P = Pool(kvq, 2, [mixed(260, 7), mixed(64, 8, (2,)), mixed(90, 9)], seed=1, dead=[[], np.arange(32), []])
    scores = torch.rand(3, 2, 600, device="cuda")
    step(P, 8, scores, 1.0)
    ex = {0: {(1, p) for p in range(0, 200)}, 2: {(0, p) for p in range(90)}}
    for r, s in ex.items():
        s = sorted(s)
        P.pool.evict_head([P.ids[r]] * len(s), [p for _, p in s], [h for h, _ in s])
    step(P, 8, scores, 1.0, head_dead=ex)
    P.pool.fp_configure(40)
    k, v = rand((7, 2, 128), P.gen), rand((7, 2, 128), P.gen)
    P.pool.fp_append(P.ids[0], k, v)
    step(P, 16, scores, 0.5, head_dead=ex, fp={0: k.double().cpu().numpy()})
    P.pool.fp_drop(P.ids[0], 0, 7)
    for n, seed in ((1, 1), (1, 2), (40, 3), (97, 4)):
        w = mixed(n, seed)
        for r in range(3):
            P.pool.append(rand((n, 2, 128), P.gen), rand((n, 2, 128), P.gen), [P.ids[r]] * n, w)
            P.widths[r] += list(map(int, w))
        step(P, 8, scores, 1.0, head_dead=ex)
        P.pool.reorder(P.ids)
        step(P, 8, scores, 1.0, head_dead=ex)


def test_scores_same_request_twice_and_guards(kvq):
    P = Pool(kvq, 1, [mixed(200, 1)], seed=5)
    scores = torch.zeros(3, 1, 333, device="cuda")
    step(P, 4, scores, 1.0, which=[0, 0, 0])
    assert (scores[:, :, 200:] == 0).all()
    assert torch.allclose(scores.sum(2), torch.full((3, 1), 4.0, device="cuda"), atol=1e-4)


def plain_select(P, r, scores, n, protect, per_head, b, head_dead=None):
    C = P.content(r, head_dead=head_dead)
    H = P.hkv
    limit = C.n_tokens - protect
    outs = []
    for h in range(H if per_head else 1):
        if per_head:
            pos, key = C.pos[h], scores[b, h].astype(np.float32)
        else:
            pos = np.unique(np.concatenate([np.asarray(x, np.int64) for x in C.pos]))
            key = scores[b].astype(np.float64).sum(0).astype(np.float32)
        pos = np.sort(pos[pos < limit])
        order = np.argsort(key[pos] + np.float32(0), kind="stable")
        outs.append(np.sort(pos[order[:n]]))
    return outs


def check_select(P, scores, n, protect, per_head, which=None, head_dead=None):
    which = list(range(len(P.ids))) if which is None else which
    got = P.pool.select_lowest(scores, [P.ids[r] for r in which], n, protect=protect, per_head=per_head)
    P.pool.sync()
    got, sc = got.cpu().numpy(), scores.cpu().numpy()
    n = [n] * len(which) if np.ndim(n) == 0 else n
    for b, r in enumerate(which):
        want = plain_select(P, r, sc, n[b], protect, per_head, b, (head_dead or {}).get(r))
        rows = got[b] if per_head else got[b][None]
        for x, w in zip(rows, want):
            assert np.array_equal(x[:w.size], w) and (x[w.size:] == -1).all(), (b, x[:8], w[:8])
    return got


LENS = (1, 31, 33, 200, 2500, 0, 1024)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("kind", ["random", "ties", "zero", "special"])
def test_select(kvq, per_head, kind):
    P = Pool(kvq, 2, [mixed(n, n) for n in LENS], seed=1, chunk=500,
             dead=[[], [1, 2], [], np.arange(0, 200, 3), np.arange(700, 800), [], np.arange(1024)])
    x = torch.rand(len(LENS), 2, 2500, device="cuda", generator=P.gen)
    if kind == "ties":
        x = (x * 4).floor()
    elif kind == "zero":
        x = torch.where(x < 0.5, torch.zeros_like(x), -torch.zeros_like(x))
    elif kind == "special":
        x = torch.where(x < 0.1, torch.full_like(x, float("inf")), x - 0.5)
        x = torch.where(x > 0.45, torch.full_like(x, float("-inf")), x)
        if per_head:   # a sum of opposite infinities is a NaN of either kind: only single heads here
            x = torch.where((x > 0.3) & (x < 0.35), torch.full_like(x, float("nan")), x)
        else:
            x = torch.where(x.isinf(), torch.full_like(x, 1e38) * x.sign(), x)
    for n, protect in ((1, 0), (7, 0), (40, 16), ([0, 3, 40, 100, 1500, 2, 8], 30), (2500, 0), (3, 4000)):
        check_select(P, x, n, protect, per_head)
    check_select(P, x[:3].contiguous(), 5, 0, per_head, which=[4, 3, 4])


@pytest.mark.parametrize("per_head", [False, True])
def test_select_with_exclusions(kvq, per_head):
    P = Pool(kvq, 2, [mixed(300, 1), mixed(500, 2)], seed=2)
    ex = {0: {(1, p) for p in range(0, 300, 2)}, 1: {(0, p) for p in range(500)} | {(1, p) for p in range(250)}}
    for r, s in ex.items():
        s = sorted(s)
        P.pool.evict_head([P.ids[r]] * len(s), [p for _, p in s], [h for h, _ in s])
    x = torch.rand(2, 2, 512, device="cuda", generator=P.gen)
    check_select(P, x, 100, 10, per_head, head_dead=ex)
    check_select(P, x, 400, 0, per_head, head_dead=ex)


def test_serving_loop_with_drafts_scores_and_eviction(kvq):
    """Drafts are verified, the accepted ones appended, the next step decoded with scores, the
    lowest-scored tokens evicted and their pages dropped; attend() sees the cache that is left."""
    from attend_ref import attend_row
    P = Pool(kvq, 2, [mixed(700, 1, (2, 2, 4)), mixed(350, 2)], seed=3)
    pool, ids, hq = P.pool, P.ids, 8
    pool.set_decode_impl(MMA)
    scores = torch.zeros(2, 2, 1000, device="cuda")
    gone = [set(), set()]
    for it in range(4):
        q, k, v = (rand((7, h, 128), P.gen) for h in (hq, 2, 2))
        n_new = [4, 3]
        pool.attend(q, ids, n_new, SCALE, k, v)
        keep = [0, 1, 4, 5, 6]                                   # accepted drafts
        w = np.array([4, 2, 4, 4, 2], np.uint8)
        pool.append(k[keep].contiguous(), v[keep].contiguous(), [ids[0], ids[0], ids[1], ids[1], ids[1]], w)
        P.widths[0] += [4, 2]
        P.widths[1] += [4, 4, 2]
        pool.decode_scored(rand((2, hq, 128), P.gen), ids, SCALE, scores)
        pos = pool.evict_lowest(scores, ids, [40, 25], protect=32)
        for r in range(2):
            new = set(pos[r][pos[r] >= 0].tolist())
            assert len(new) == [40, 25][r] and not (new & gone[r])
            gone[r] |= new
    q, k, v = (rand((5, h, 128), P.gen) for h in (hq, 2, 2))
    out = pool.attend(q, ids, [3, 2], SCALE, k, v).double().cpu().numpy()
    ref_dec = pool.decode(q[[2, 4]].contiguous(), ids, SCALE)
    P.slots()
    pool.sync()
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    first = 0
    for r, T in ((0, 3), (1, 2)):
        C = P.content(r)
        assert not (set(C.pos[0].tolist()) & gone[r])
        for h in range(2):
            for t in range(T):
                for j in range(4 * h, 4 * h + 4):
                    o, tol = attend_row(qh[first + t, j], np.concatenate([C.K[h], kh[first:first + t + 1, h]]),
                                        np.concatenate([C.V[h], vh[first:first + t + 1, h]]), SCALE, 2.0 ** -11)
                    assert (np.abs(out[first + t, j] - o) <= tol).all()
        first += T
    # dropping the dead pages changes nothing that is read
    pool.drop_dead_pages(ids)
    out2 = pool.attend(q, ids, [3, 2], SCALE, k, v).double().cpu().numpy()
    dec2 = pool.decode(q[[2, 4]].contiguous(), ids, SCALE)
    pool.sync()
    assert np.linalg.norm(out2 - out) <= 2 * 2.0 ** -8 * np.linalg.norm(out)
    assert float((dec2 - ref_dec).norm()) <= 1e-4 * float(ref_dec.norm())
    left = pool.evict_lowest(scores, ids, 3, protect=0, per_head=True)
    assert left.shape == (2, 2, 3)


def test_refusals(kvq):
    P = Pool(kvq, 2, [mixed(40, 1)], seed=12)
    pool, r = P.pool, P.ids[0]
    q = rand((1, 8, 128), P.gen)
    sc = torch.zeros(1, 2, 64, device="cuda")
    for args, kw in [((q, [r], SCALE, sc.double()), {}), ((q, [r], SCALE, sc.cpu()), {}), ((q, [r], SCALE, sc[:, :1]), {}),
                     ((q, [r], SCALE, sc[:, :, ::2]), {}), ((q, [r, r], SCALE, sc), {}), ((q.float(), [r], SCALE, sc), {}),
                     ((q, [r], SCALE, sc), dict(out=torch.empty(1, 8, 64, device="cuda")))]:
        with pytest.raises(ValueError):
            pool.decode_scored(*args, **kw)
    for args, kw in [((q, [r + 1], SCALE, sc), {}), ((q, [r], SCALE, sc[:, :, :39].contiguous()), {}),
                     ((q, [r], float("inf"), sc), {}), ((q, [r], SCALE, sc), dict(decay=float("nan"))),
                     ((q[:, :7].contiguous(), [r], SCALE, sc), {})]:
        with pytest.raises(kvq.KVError) as e:
            pool.decode_scored(*args, **kw)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    assert (sc == 0).all()
    for args, kw in [((sc, [r], [1, 2]), {}), ((sc, [r], -1), {}), ((sc, [r, r], 1), {}),
                     ((sc, [r], 3), dict(out=torch.empty(1, 2, dtype=torch.int32, device="cuda")))]:
        with pytest.raises(ValueError):
            pool.select_lowest(*args, **kw)
    for args, kw in [((sc, [r + 1], 1), {}), ((sc, [r], 1), dict(protect=-1)), ((sc[:, :, :39].contiguous(), [r], 1), {})]:
        with pytest.raises(kvq.KVError) as e:
            pool.select_lowest(*args, **kw)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pool.evict_lowest(sc.expand(2, 2, 64).contiguous(), [r, r], 1)
    assert pool.select_lowest(sc, [r], 0).shape == (1, 0)


@pytest.mark.parametrize("rows,n", [(160, 40000), (1, 40000), (3, 110000)])
def test_select_long_and_many(kvq, rows, n):
    """One CTA per row with more pages than its warps hold at once, and clusters; a request listed
    as often as there are rows, every third token evicted in a stretch."""
    pool = kvq.KVPool(1, n // 32 + 16, n // 32 + 16, 1, n // 32 + 32)
    rid = pool.open()
    gen = torch.Generator("cuda").manual_seed(n + rows)
    w = mixed(n, 3)
    for a in range(0, n, 10000):
        pool.append(rand((10000, 1, 128), gen), rand((10000, 1, 128), gen), np.full(10000, rid, np.int32), w[a:a + 10000])
    dead = np.arange(5000, 20000, 3)
    pool.evict(np.full(dead.size, rid, np.int32), dead)
    x = torch.rand(rows, 1, n + 5, device="cuda", generator=gen)
    x = torch.where(x < 0.3, torch.zeros_like(x), x)   # many ties
    got = pool.select_lowest(x, [rid] * rows, 17000, protect=100).cpu().numpy()
    pool.sync()
    live = np.setdiff1d(np.arange(n - 100), dead)
    for b, key in enumerate(x[:, 0].cpu().numpy()):
        assert np.array_equal(got[b], np.sort(live[np.argsort(key[live], kind="stable")[:17000]])), b
