"""Attention of new tokens over the cache (kv_attend) against a plain 64-bit form on the pool's
exported content, with tolerances per element from the roundings the operator makes."""
import numpy as np
import pytest

from attend_ref import SCALE, Content, attend_row

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIMT, MMA = 1, 2
# unit roundoff of K, V and weights inside: binary16 on the tensor cores, fp32 sums on the CUDA cores
ROUND = {SIMT: 2.0 ** -17, MMA: 2.0 ** -11}


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def rand(shape, gen, mult=None):
    x = torch.randn(*shape, generator=gen, device="cuda")
    return (x if mult is None else x * mult).bfloat16()


class Pool:
    """A pool with requests of given widths per token; knows every slot's token position."""

    def __init__(self, kvq, hkv, widths, seed=0, dead=(), reorder=True, chunk=97, mult=None, slack=64, kv_scale=1.0):
        self.kvq = kvq
        gen = torch.Generator("cuda").manual_seed(seed)
        self.gen = gen
        total = sum(len(w) for w in widths)
        pages = total // 32 + 8 * len(widths) + slack
        self.pool = kvq.KVPool(hkv, pages, pages, len(widths), max([len(w) for w in widths] + [1]) // 32 + 16,
                               n_int3_pages=pages, n_fp4_pages=pages)
        self.pool.first_fp4 = 3 * pages
        self.ids = [self.pool.open() for _ in widths]
        self.hkv = hkv
        self.widths = [list(map(int, w)) for w in widths]
        for r, w in enumerate(self.widths):
            w = np.asarray(w, np.uint8)
            for t in range(0, w.size, chunk):
                n = min(chunk, w.size - t)
                k, v = rand((n, hkv, 128), gen, mult), rand((n, hkv, 128), gen)
                if kv_scale != 1.0:
                    k, v = (k.float() * kv_scale).bfloat16(), (v.float() * kv_scale).bfloat16()
                self.pool.append(k, v, np.full(n, self.ids[r], np.int32), w[t:t + n])
        for r, pos in enumerate(dead):
            if len(pos):
                self.pool.evict(np.full(len(pos), self.ids[r], np.int32), pos)
        if reorder:
            self.pool.reorder(self.ids)
        self.pool.sync()

    def slots(self):
        """Position of every (table entry, slot), from the routing rules: a request's tokens of
        one width fill pages of that width in order; INT2 tokens gather in groups of 32."""
        self.pool.slot_pos = {}
        n2 = self.pool.n_int2_pages
        for rid, w in zip(self.ids, self.widths):
            w = np.asarray(w)
            by = {2: list(np.flatnonzero(w == 2)), 3: list(np.flatnonzero(w == 3)), 4: list(np.flatnonzero(w == 4)),
                  0xF4: list(np.flatnonzero(w == 0xF4))}
            ex = self.pool.export(rid, content=False)
            full2 = len(by[2]) // 32 * 32
            stage = by[2][full2:]
            by[2] = by[2][:full2]
            out = {}
            pages = n2
            tail_seen = {2: 0, 3: 0, 4: 0, 0xF4: 0}
            # pages of one width in order of their first token; the staging page is an INT4 page
            cls = [2 if p < n2 else 4 if p < 2 * pages else 3 if p < 3 * pages else 0xF4 for p in ex["ids"]]
            four = [i for i, c in enumerate(cls) if c == 4]
            stage_at = None
            if stage:
                cand = [i for i in four if ex["fill"][i] == len(stage)]
                firsts = {}
                # with both a partial tail and a staging page, table order follows first tokens
                tail_n = len(by[4]) % 32
                tail_first = by[4][len(by[4]) - tail_n] if tail_n else None
                if tail_n:
                    part = [i for i in four if ex["fill"][i] < 32]
                    assert len(part) == 2
                    stage_at = part[0] if stage[0] < tail_first else part[1]
                else:
                    stage_at = [i for i in cand if ex["fill"][i] < 32][0]
            for i, c in enumerate(cls):
                n = int(ex["fill"][i])
                if i == stage_at:
                    toks = stage
                else:
                    toks = by[c][tail_seen[c]:tail_seen[c] + n]
                    tail_seen[c] += n
                assert len(toks) == n, (i, c, n, len(toks))
                for s, t in enumerate(toks):
                    out[(i, s)] = int(t)
            self.pool.slot_pos[rid] = out

    def content(self, r, head_dead=None):
        self.slots()
        return Content(self.pool, self.ids[r], head_dead=head_dead)


def mixed(n, seed, choice=(2, 4)):
    return np.random.default_rng(seed).choice(choice, n).astype(np.uint8)


def check(P, impl, which, n_new, hq, tree=None, with_kv=True, head_dead=None, fp=None, scale=SCALE, q_mult=1.0,
          rows=None):
    """attend() on the requests `which`, every row (or the listed ones of each request) against the plain form."""
    pool, hkv = P.pool, P.hkv
    g = hq // hkv
    N = sum(n_new)
    q = (torch.randn(N, hq, 128, generator=P.gen, device="cuda") * q_mult).bfloat16()
    k, v = (rand((N, hkv, 128), P.gen), rand((N, hkv, 128), P.gen)) if with_kv else (None, None)
    td = None if tree is None else torch.from_numpy(np.asarray(tree, np.uint64).view(np.int64)).cuda()
    pool.set_decode_impl(impl)
    out = pool.attend(q, [P.ids[r] for r in which], n_new, scale, k, v, tree=td)
    pool.sync()
    got = out.double().cpu().numpy()
    assert got.shape == (N, hq, 128)
    qh = q.double().cpu().numpy()
    kh, vh = (k.double().cpu().numpy(), v.double().cpu().numpy()) if with_kv else (None, None)
    first, num, den = 0, 0.0, 0.0
    for b, r in enumerate(which):
        T = n_new[b]
        C = P.content(r, head_dead=(head_dead or {}).get(r))
        for h in range(hkv):
            Kc, Vc = C.K[h], C.V[h]
            if fp is not None and r in fp:
                Kc = np.concatenate([Kc, fp[r][0][:, h]])
                Vc = np.concatenate([Vc, fp[r][1][:, h]])
            for t in range(T) if rows is None else [x for x in rows if x < T]:
                see = []
                if with_kv:
                    see = [j for j in range(T) if ((int(tree[first + t]) >> j) & 1 if tree is not None else j <= t)]
                K = np.concatenate([Kc, kh[first:first + T, h][see]]) if see else Kc
                V = np.concatenate([Vc, vh[first:first + T, h][see]]) if see else Vc
                for j in range(h * g, (h + 1) * g):
                    o, tol = attend_row(qh[first + t, j], K, V, scale, ROUND[impl])
                    d = np.abs(got[first + t, j] - o)
                    assert (d <= tol).all(), (b, t, h, j, float((d / np.maximum(tol, 1e-30)).max()), float(d.max()))
                    num += float((d ** 2).sum())
                    den += float((o ** 2).sum())
        first += T
    if den > 0:
        # bf16 rounds each element by at most 2^-8 of itself, on average by well under half of that
        # (uniform mantissas: 2^-8 / sqrt(3) at most); the rest is the inside, 2^-11 each
        assert (num / den) ** 0.5 <= 2.0 ** -8, (num / den) ** 0.5
    return out


IMPLS = [SIMT, MMA]


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 3), (2, 4), (1, 5), (1, 7), (2, 8)])
def test_ragged_requests(kvq, impl, hkv, g):
    P = Pool(kvq, hkv, [mixed(n, n) for n in (1, 31, 32, 33, 200, 517)], seed=g)
    check(P, impl, [0, 1, 2, 3, 4, 5], [1, 3, 2, 5, 1, 4], hkv * g)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 130])
def test_lengths(kvq, impl, T):
    P = Pool(kvq, 1, [mixed(300, 5), mixed(0, 1)], seed=T)
    check(P, impl, [0, 1], [T, T], 4, rows=[0, 1, T // 2, T - 2, T - 1] if T > 20 else None)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("n", [0, 1, 127, 128, 129, 1000])
@pytest.mark.parametrize("T", [300])
def test_chunks(kvq, impl, n, T):
    P = Pool(kvq, 2, [mixed(n, 9), mixed(40, 2)], seed=n)
    check(P, impl, [0, 1], [T, 129], 16, rows=[0, 1, 31, 32, 63, 64, 127, 128, 129, 255, 256, T - 1])


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("choice", [(2,), (3,), (4,), (0xF4,), (2, 3, 4, 0xF4)])
def test_widths(kvq, impl, choice):
    P = Pool(kvq, 2, [mixed(450, 3, choice), mixed(70, 4, choice)], seed=len(choice) + choice[0])
    check(P, impl, [0, 1], [5, 40], 8, rows=[0, 3, 17, 39])


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [3, 64])
def test_tree(kvq, impl, T):
    """Random masks: bits of ancestors, of later tokens, none at all (with an empty cache the row is 0),
    and bits past the request's tokens, which are ignored."""
    P = Pool(kvq, 2, [mixed(100, 1), mixed(0, 1), mixed(64, 2)], seed=T)
    rng = np.random.default_rng(T)
    n = [T, T, max(1, T - 1)]
    tree = rng.integers(0, 1 << 63, sum(n), dtype=np.uint64) * np.uint64(2) + rng.integers(0, 2, sum(n)).astype(np.uint64)
    tree[0] = 0
    tree[T] = 0
    tree[T + 1] = np.uint64(1) << np.uint64(T - 1)
    if T < 64:
        tree[-1] = np.uint64(0xFFFFFFFFFFFFFFFF)
    out = check(P, impl, [0, 1, 2], n, 8, tree=tree)
    assert (out[T] == 0).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [1, 40])
def test_cache_only(kvq, impl, T):
    P = Pool(kvq, 2, [mixed(150, 1), mixed(0, 1)], seed=T)
    out = check(P, impl, [0, 1], [T, T], 16, with_kv=False)
    assert (out[T:] == 0).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [2, 70])
def test_evicted_and_excluded(kvq, impl, T):
    """Evicted slots, a request with every slot evicted, and slots excluded for one kv head."""
    rng = np.random.default_rng(T)
    dead = [np.sort(rng.choice(260, 60, replace=False)), np.arange(64), []]
    P = Pool(kvq, 2, [mixed(260, 7), mixed(64, 8), mixed(90, 9)], seed=1, dead=dead)
    check(P, impl, [0, 1, 2], [T, T, T], 8, rows=[0, 1, T - 1])
    ex = {0: {(1, int(p)) for p in rng.choice(260, 100, replace=False)}, 2: {(0, p) for p in range(90)}}
    for r, s in ex.items():
        s = sorted(s)
        P.pool.evict_head([P.ids[r]] * len(s), [p for _, p in s], [h for h, _ in s])
    check(P, impl, [0, 1, 2], [T, T, T], 8, rows=[0, 1, T - 1], head_dead=ex)
    check(P, impl, [2, 1], [T, T], 8, rows=[0], head_dead=ex, with_kv=False)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [1, 30, 140])
def test_full_precision_lists(kvq, impl, T):
    P = Pool(kvq, 2, [mixed(100, 7), mixed(0, 8), mixed(50, 3)], seed=2)
    P.pool.fp_configure(300)
    fp = {}
    for r, n in ((0, 5), (1, 131)):
        k, v = rand((n, 2, 128), P.gen), rand((n, 2, 128), P.gen)
        P.pool.fp_append(P.ids[r], k, v)
        fp[r] = (k.double().cpu().numpy(), v.double().cpu().numpy())
    check(P, impl, [0, 1, 2], [T, T, T], 8, fp=fp, rows=[0, T // 2, T - 1])
    check(P, impl, [1, 0], [T, 1], 8, fp=fp, rows=[0, T - 1], with_kv=False)


@pytest.mark.parametrize("impl", IMPLS)
def test_unsorted_tables_outliers_and_steep_softmax(kvq, impl):
    mult = torch.ones(128, device="cuda")
    mult[[3, 40, 77, 127]] = 20.0
    P = Pool(kvq, 2, [mixed(400, 2), mixed(333, 3)], seed=4, reorder=False, mult=mult)
    check(P, impl, [0, 1], [9, 3], 16)
    check(P, impl, [1, 0], [80, 33], 16, q_mult=6.0, rows=[0, 40, 79])      # logits far apart
    check(P, impl, [1, 0], [3, 33], 16, q_mult=1e-3, rows=[0, 2, 32])       # a flat softmax
    check(P, impl, [0], [4], 16, scale=0.0)
    check(P, impl, [0], [4], 16, scale=-SCALE)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("size", [3000.0, 1e-4])
def test_large_and_small_values(kvq, impl, size):
    P = Pool(kvq, 1, [mixed(200, 2)], seed=4, kv_scale=size)
    check(P, impl, [0], [6], 8, scale=SCALE / size, with_kv=False)
    check(P, impl, [0], [100], 8, scale=SCALE / size, with_kv=False, rows=[0, 99])


@pytest.mark.parametrize("impl", IMPLS)
def test_same_request_twice_none_and_empty_calls(kvq, impl):
    P = Pool(kvq, 1, [mixed(70, 1), mixed(64, 2)], seed=6)
    check(P, impl, [0, 0, 1], [2, 3, 0], 4)
    check(P, impl, [1, 0, 1], [0, 70, 1], 4, rows=[0, 69])
    out = P.pool.attend(torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda"), [P.ids[0]], [0], SCALE)
    assert out.shape == (0, 4, 128)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [2, 90])
def test_unaligned_rows_guards_and_out(kvq, impl, T):
    """Inputs and outputs one element past an aligned address; what lies around out stays."""
    P = Pool(kvq, 2, [mixed(140, 1)], seed=8)
    hq, n = 8, T
    base = {}
    for name, h in (("q", hq), ("k", 2), ("v", 2)):
        base[name] = torch.randn(n * h * 128 + 1, generator=P.gen, device="cuda").bfloat16()
    view = {name: base[name][1:].view(n, h, 128) for name, h in (("q", hq), ("k", 2), ("v", 2))}
    flat = torch.full((n * hq * 128 + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    P.pool.set_decode_impl(impl)
    P.pool.attend(view["q"], [P.ids[0]], [n], SCALE, view["k"], view["v"], out=flat[1:1 + n * hq * 128].view(n, hq, 128))
    out = P.pool.attend(view["q"].clone(), [P.ids[0]], [n], SCALE, view["k"].clone(), view["v"].clone())
    P.pool.sync()
    assert torch.equal(flat[1:1 + n * hq * 128].view(n, hq, 128), out)
    assert flat[0] == 7.0 and (flat[1 + n * hq * 128:] == 7.0).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("T", [2, 90])
def test_values_out_of_range_are_reported_and_used_as_zero(kvq, impl, T):
    """A NaN, an Inf or a huge value in a new token's row does not reach the rows that may not
    see it; the next sync reports it once."""
    P = Pool(kvq, 1, [mixed(50, 1)], seed=9)
    q, k, v = (rand((T, h, 128), P.gen) for h in (4, 1, 1))
    k[T - 1, 0, 5], v[T - 1, 0, 7], v[T - 1, 0, 8] = float("nan"), float("inf"), 1e38
    P.pool.set_decode_impl(impl)
    out = P.pool.attend(q, [P.ids[0]], [T], SCALE, k, v)
    with pytest.raises(kvq.KVError) as e:
        P.pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    k0, v0 = k.clone(), v.clone()
    k0[T - 1, 0, 5] = v0[T - 1, 0, 7] = v0[T - 1, 0, 8] = 0
    ref = P.pool.attend(q, [P.ids[0]], [T], SCALE, k0, v0)
    P.pool.sync()
    assert torch.isfinite(out.float()).all() and torch.equal(out, ref)


@pytest.mark.parametrize("impl", IMPLS)
def test_other_stream_and_repeatability(kvq, impl):
    P = Pool(kvq, 2, [mixed(900, 1), mixed(333, 2)], seed=10)
    P.pool.set_decode_impl(impl)
    q, k, v = (rand((68, h, 128), P.gen) for h in (8, 2, 2))
    a = P.pool.attend(q, P.ids, [5, 63], SCALE, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = P.pool.attend(q, P.ids, [5, 63], SCALE, k, v)
    s.synchronize()
    c = P.pool.attend(q, P.ids, [5, 63], SCALE, k, v)
    P.pool.sync()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_simt_and_mma_agree_on_long_caches(kvq):
    """2,000 to 6,000 tokens, split over many CTAs, against the CUDA-core form."""
    P = Pool(kvq, 2, [mixed(6000, 1, (2, 2, 4)), mixed(2049, 2), mixed(4100, 3, (2, 3, 4, 0xF4))], seed=11, chunk=1000,
             dead=[np.arange(100, 900), [], [5]])
    for n_new, hq in (([1, 2, 1], 8), ([4, 8, 3], 16), ([16, 1, 7], 16), ([33, 64, 5], 8), ([200, 1, 77], 16), ([700, 513, 300], 8)):
        N = sum(n_new)
        q, k, v = (rand((N, h, 128), P.gen) for h in (hq, 2, 2))
        o = {}
        for impl in IMPLS:
            P.pool.set_decode_impl(impl)
            o[impl] = P.pool.attend(q, P.ids, n_new, SCALE, k, v).double()
        P.pool.sync()
        # both are rounded to bf16 (2^-8 each at most); the inside of one is binary16
        rel = float((o[SIMT] - o[MMA]).norm() / o[SIMT].norm())
        assert rel <= 2 * 2.0 ** -8, (n_new, rel)


def test_refusals(kvq):
    P = Pool(kvq, 2, [mixed(40, 1)], seed=12)
    pool, r = P.pool, P.ids[0]
    q, k, v = (rand((3, h, 128), P.gen) for h in (8, 2, 2))
    tree = torch.ones(3, dtype=torch.int64, device="cuda")
    for args, kw in [((q, [r], [2], SCALE, k, v), {}), ((q, [r], [3, 0], SCALE, k, v), {}),
                     ((q.float(), [r], [3], SCALE, k, v), {}), ((q.cpu(), [r], [3], SCALE, k, v), {}),
                     ((q[:, :, ::2], [r], [3], SCALE, k, v), {}), ((q, [r], [3], SCALE, k, None), {}),
                     ((q, [r], [3], SCALE, k[:2], v), {}), ((q, [r], [3], SCALE, k, v.float()), {}),
                     ((q, [r], [3], SCALE, k, v), dict(tree=tree[:2])), ((q, [r], [3], SCALE, k, v), dict(tree=tree.int())),
                     ((q, [r], [3], SCALE, k, v), dict(out=torch.empty_like(q, dtype=torch.float32))),
                     ((q, [r], [3], SCALE, k, v), dict(out=q[:2]))]:
        with pytest.raises(ValueError):
            pool.attend(*args, **kw)
    for args, kw in [((q, [r + 1], [3], SCALE, k, v), {}), ((q, [-1], [3], SCALE, k, v), {}),
                     ((q, [r, r], [4, -1], SCALE, k, v), {}), ((q, [r], [3], float("nan"), k, v), {}),
                     ((q[:, :7].contiguous(), [r], [3], SCALE, k, v), {}), ((q, [r], [3], SCALE), dict(tree=tree)),
                     ((torch.cat([q, q, q], 1), [r], [3], SCALE, k, v), {})]:
        with pytest.raises(kvq.KVError) as e:
            pool.attend(*args, **kw)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    big = [rand((65, h, 128), P.gen) for h in (8, 2, 2)]
    with pytest.raises(kvq.KVError) as e:
        pool.attend(big[0], [r], [65], SCALE, big[1], big[2], tree=torch.ones(65, dtype=torch.int64, device="cuda"))
    assert e.value.status == kvq.KV_ERR_INVALID_ARG
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    out = torch.empty_like(q)
    status = []
    with torch.cuda.graph(g, stream=s):
        x = q + 1   # a graph is not empty
        try:
            pool.attend(q, [r], [3], SCALE, k, v, out=out, stream=s)
        except kvq.KVError as err:
            status.append(err.status)
    assert status == [kvq.KV_ERR_STATE]
    check(P, MMA, [0], [3], 8)


@pytest.mark.parametrize("n_new", [[64, 20, 48, 3, 16], [33, 17, 32, 0, 1], [0, 0, 48, 47, 0]])
def test_middle_sizes(kvq, n_new):
    """Units of 136 to 384 rows: next to larger ones, and alone."""
    P = Pool(kvq, 2, [mixed(n, n) for n in (300, 129, 77, 500, 0)], seed=21)
    check(P, MMA, range(5), n_new, 16, rows=[0, 15, 16, 31, 32, 47])


@pytest.mark.parametrize("n_new", [[2, 1], [70, 2], [100, 300]])
def test_expired_wait_reports_timeout_once(kvq, n_new):
    """The first wait for a copy gives up at once: a status at the next sync, and the pool goes on."""
    P = Pool(kvq, 2, [mixed(600, 1), mixed(200, 2)], seed=22)
    q, k, v = (rand((sum(n_new), h, 128), P.gen) for h in (8, 2, 2))
    P.pool.set_decode_impl(MMA)
    good = P.pool.attend(q, P.ids, n_new, SCALE, k, v)
    P.pool.sync()
    P.pool.set_wait_limit(0)
    P.pool.attend(q, P.ids, n_new, SCALE, k, v)
    with pytest.raises(kvq.KVError) as e:
        P.pool.sync()
    assert e.value.status == kvq.KV_ERR_DEVICE_TIMEOUT
    P.pool.sync()
    P.pool.set_wait_limit(-1)
    again = P.pool.attend(q, P.ids, n_new, SCALE, k, v)
    P.pool.sync()
    assert torch.equal(again, good)


def test_more_keys_than_a_pass(kvq):
    """Operand tiles past one pass's workspace (65536 tiles of 128 keys, 4.3 GB): the same request nine
    times, so that every copy of a row has one answer, and the answer of a call that lists it once."""
    n, T, hkv, hq = 131072, 49, 8, 64
    pages = 2 * (n // 32 + 64)
    pool = kvq.KVPool(hkv, pages, pages, 1, n // 32 + 64)
    rid = pool.open()
    gen = torch.Generator("cuda").manual_seed(23)
    for a in range(0, n, 16384):
        pool.append(rand((16384, hkv, 128), gen), rand((16384, hkv, 128), gen), np.full(16384, rid, np.int32),
                    np.full(16384, 2, np.uint8))
    q, k, v = (rand((T, h, 128), gen) for h in (hq, hkv, hkv))
    one = pool.attend(q, [rid], [T], SCALE, k, v).double()
    many = pool.attend(q.repeat(9, 1, 1), [rid] * 9, [T] * 9, SCALE, k.repeat(9, 1, 1), v.repeat(9, 1, 1)).double()
    pool.sync()
    # both are rounded to bf16 (2^-8 each at most) from sums taken in other pieces (far below)
    for x in many.view(9, T, hq, 128):
        assert float((x - one).norm() / one.norm()) <= 2 * 2.0 ** -8


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("size", [1e20, 1e-20])
def test_queries_far_from_one(kvq, impl, size):
    P = Pool(kvq, 1, [mixed(200, 2)], seed=24)
    check(P, impl, [0], [5], 8, scale=SCALE / size, q_mult=size)
    check(P, impl, [0], [100], 8, scale=SCALE / size, q_mult=size, rows=[0, 60, 99])


@pytest.mark.parametrize("n_new", [[3, 2], [70, 50]])
def test_two_pools_from_two_threads(kvq, n_new):
    """Calls on two pools at once, each on its own stream: what one call alone gives."""
    import threading
    pools = [Pool(kvq, 2, [mixed(700, s), mixed(90, s + 1)], seed=s) for s in (31, 33)]
    q, k, v = (rand((sum(n_new), h, 128), pools[0].gen) for h in (8, 2, 2))
    alone = [P.pool.attend(q, P.ids, n_new, SCALE, k, v) for P in pools]
    torch.cuda.synchronize()
    wrong = []

    def work(P, want):
        s = torch.cuda.Stream()
        out = torch.empty_like(want)
        for _ in range(20):
            P.pool.attend(q, P.ids, n_new, SCALE, k, v, out=out, stream=s)
        s.synchronize()
        P.pool.sync()
        if not torch.equal(out, want):
            wrong.append(P)

    t = [threading.Thread(target=work, args=x) for x in zip(pools, alone)]
    [x.start() for x in t]
    [x.join() for x in t]
    assert not wrong
