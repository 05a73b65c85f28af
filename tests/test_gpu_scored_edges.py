"""Scored decode, selection and what they share with the other calls, at the edges: request ids that
are used again, sums of many kv heads, rows of more keys than shared memory holds, capture of a
decode, outputs on another stream, the statistics of the last decode."""
import numpy as np
import pytest

from attend_ref import SCALE
from test_gpu_attend import MMA, Pool, kvq, mixed, rand  # noqa: F401
from test_gpu_scored import check_select, step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("first", [True, False])
def test_a_request_id_used_again_without_pages(kvq, lists, first):
    """A request closed and opened again, empty or with list tokens only, next to one with pages: its
    rows of scores stay, and so does what lies around them (the earlier request had more positions
    than a row holds)."""
    P = Pool(kvq, 2, [mixed(500, 2), mixed(70, 1)] if first else [mixed(70, 1), mixed(500, 2)], seed=7)
    pool, r = P.pool, 0 if first else 1
    flat = torch.rand(2 * 2 * 70 + 8192, device="cuda", generator=P.gen)
    kept = flat.clone()
    scores = flat[4096:4096 + 280].view(2, 2, 70)
    pool.close_request(P.ids[r])
    assert pool.open() == P.ids[r]
    P.widths[r] = []
    fp = None
    if lists:
        pool.fp_configure(20)
        k, v = rand((9, 2, 128), P.gen), rand((9, 2, 128), P.gen)
        pool.fp_append(P.ids[r], k, v)
        fp = {r: k.double().cpu().numpy()}
    for _ in range(2):
        step(P, 8, scores, 0.5, fp=fp)
    assert torch.equal(scores[r], kept[4096:4096 + 280].view(2, 2, 70)[r])
    assert torch.equal(flat[:4096], kept[:4096]) and torch.equal(flat[4376:], kept[4376:])
    for per_head in (False, True):
        got = check_select(P, scores, 30, 0, per_head)
        assert (got[r] == -1).all()
    # the id in use again, with fewer tokens than before
    w = mixed(45, 3)
    pool.append(rand((45, 2, 128), P.gen), rand((45, 2, 128), P.gen), [P.ids[r]] * 45, w)
    P.widths[r] = list(map(int, w))
    step(P, 8, scores, 1.0, fp=fp)
    check_select(P, scores, 30, 3, False)


def summed_keys(scores):
    """The kv heads' sum in fp64, head after head, rounded to fp32; [H][positions]."""
    s = np.zeros(scores.shape[1])
    for row in scores.astype(np.float64):
        s = s + row
    return s.astype(np.float32)


def hard_sums(hkv, n, seed, signs):
    """Scores of many magnitudes, sums at and next to the middle of two fp32 values, cancellation."""
    rng = np.random.default_rng(seed)
    x = np.ldexp(rng.uniform(1, 2, (hkv, n)), rng.integers(-60, 1, (hkv, n)))
    x[:, n // 4:n // 2] = np.ldexp(1.0, rng.integers(-55, 1, (hkv, n // 2 - n // 4)))          # powers of two
    x[:, n // 2:3 * n // 4] = rng.integers(0, 5, (hkv, 3 * n // 4 - n // 2)) / 8.0                # ties and zeros
    # one, half a unit of it, and something far below that decides (or not, where it is zero)
    near = np.arange(3 * n // 4, n)
    x[:, near] = 0.0
    x[0, near] = rng.integers(1, 4, near.size)
    x[1, near] = np.ldexp(x[0, near], -24) * rng.integers(0, 3, near.size)
    if hkv > 2:
        x[2, near] = np.ldexp(rng.integers(-1 if signs else 0, 2, near.size).astype(np.float64), rng.integers(-52, -40, near.size))
    if signs:
        x[:, :near[0]] *= rng.choice([-1.0, 1.0], (hkv, near[0]))
    for col in x.T:
        rng.shuffle(col)
    return x.astype(np.float32)


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("hkv", [2, 3, 7, 8, 9, 17])
def test_selection_by_the_sum_of_many_heads(kvq, hkv, signs):
    n = 4000
    P = Pool(kvq, hkv, [mixed(n, 1)], seed=hkv, chunk=1000, slack=256)
    sc = hard_sums(hkv, n, 10 * hkv + signs, signs)
    key = summed_keys(sc)
    x = torch.from_numpy(sc[None].copy()).cuda()
    order = np.argsort(key + np.float32(0), kind="stable")
    for m in list(range(1, 60)) + [100, 500, 999, 1000, 1001, 1777, 2000, 2500, 3000, 3100, 3500, 3999]:
        got = P.pool.select_lowest(x, P.ids, m).cpu().numpy()[0]
        assert np.array_equal(got, np.sort(order[:m])), m


def test_selection_where_the_third_head_decides(kvq):
    """1 + 2^-24 + 2^-50 rounds up, 1 + 2^-24 does not."""
    P = Pool(kvq, 3, [mixed(40, 1)], seed=1)
    x = torch.full((1, 3, 40), 2.0, device="cuda")
    x[0, :, 0] = torch.tensor([1.0, 2.0 ** -24, 2.0 ** -50])
    x[0, :, 1] = torch.tensor([1.0, 0.0, 0.0])
    x[0, :, 2] = torch.tensor([1.0, 2.0 ** -24, 0.0])
    assert P.pool.select_lowest(x, P.ids, 1).cpu().tolist() == [[1]]
    assert P.pool.select_lowest(x, P.ids, 2).cpu().tolist() == [[1, 2]]


@pytest.mark.parametrize("before", ["default", "other"])
def test_a_decode_is_captured_after_work_on_another_stream(kvq, before):
    """With a standing plan a decode only launches kernels: a graph of it gives what the call gives."""
    P = Pool(kvq, 2, [mixed(900, 1), mixed(333, 2)], seed=4)
    q, out = rand((2, 8, 128), P.gen), torch.empty(2, 8, 128, device="cuda")
    s, o = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(o if before == "other" else torch.cuda.current_stream()):
        want = P.pool.decode(q, P.ids, SCALE).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        P.pool.decode(q, P.ids, SCALE, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    q.neg_()
    g.replay()
    assert torch.equal(out, P.pool.decode(q, P.ids, SCALE))
    P.pool.sync()


def test_operand_tiles_stay_within_their_bound(kvq):
    """kv_attend's workspace grows to what a call needs and at most to 4.3 GB where that is enough."""
    n, T, hkv, hq = 131072, 49, 8, 64
    pages = 2 * (n // 32 + 64)
    pool = kvq.KVPool(hkv, pages, pages, 1, n // 32 + 64)
    rid = pool.open()
    gen = torch.Generator("cuda").manual_seed(23)
    for a in range(0, n, 16384):
        pool.append(rand((16384, hkv, 128), gen), rand((16384, hkv, 128), gen), np.full(16384, rid, np.int32),
                    np.full(16384, 2, np.uint8))
    q, k, v = (rand((6 * T, h, 128), gen) for h in (hq, hkv, hkv))
    out = torch.empty_like(q)
    pool.sync()
    free = torch.cuda.mem_get_info()[0]
    for times in (5, 6):   # 2.7 and 3.2 GB of tiles
        m = times * T
        pool.attend(q[:m], [rid] * times, [T] * times, SCALE, k[:m], v[:m], out=out[:m])
        pool.sync()
    grown = free - torch.cuda.mem_get_info()[0]
    assert 3.2e9 < grown < 4.8e9, grown   # tiles, and 0.1 GB or so of plan and partial sums


def test_a_workspace_without_memory_for_it(kvq):
    """The logits of one request listed 8191 times (314 GB) are KV_ERR_OOM; scores stay, and the pool
    goes on with what it was."""
    n, hkv, hq, times = 150000, 8, 64, 8191
    pages = 2 * (n // 32 + 64)
    pool = kvq.KVPool(hkv, pages, pages, 1, n // 32 + 64)
    rid = pool.open()
    gen = torch.Generator("cuda").manual_seed(23)
    for a in range(0, n, 15000):
        pool.append(rand((15000, hkv, 128), gen), rand((15000, hkv, 128), gen), np.full(15000, rid, np.int32),
                    np.full(15000, 2, np.uint8))
    q = rand((times, hq, 128), gen)
    pool.set_decode_impl(MMA)
    want = pool.decode(q[:2], [rid, rid], SCALE)
    scores = torch.empty(times, hkv, n, device="cuda")   # 39 GB
    out = torch.empty(times, hq, 128, device="cuda")
    scores[:2] = 0
    with pytest.raises(kvq.KVError) as e:
        pool.decode_scored(q, [rid] * times, SCALE, scores, out=out)
    assert e.value.status == kvq.KV_ERR_OOM and "workspace" in str(e.value)
    pool.sync()
    assert (scores[:2] == 0).all()
    got = pool.decode_scored(q[:2], [rid, rid], SCALE, scores[:2], out=out[:2])
    assert torch.equal(got, want) and torch.equal(pool.decode(q[:2], [rid, rid], SCALE), want)
    # 8 weights' sums of 1: a logit is off by 136 roundings of at most 10 (128 products of normal values,
    # scaled), which moves a weight by twice that, 1.6e-4 of itself; the sum's own error is far below
    assert torch.allclose(scores[:2].sum(2), torch.full((2, hkv), 8.0, device="cuda"), rtol=0.0, atol=2e-3)
    pool.sync()
    del scores
    torch.cuda.empty_cache()


def test_statistics_after_a_scored_decode(kvq):
    """Pages without a live slot are not read by the scored decode, and not counted."""
    P = Pool(kvq, 2, [mixed(320, 1, (4,))], seed=2, dead=[np.arange(64)])
    q, sc = rand((1, 8, 128), P.gen), torch.zeros(1, 2, 320, device="cuda")
    P.pool.set_decode_impl(MMA)
    P.pool.decode(q, P.ids, SCALE)
    plain = P.pool.last_decode_stats()
    P.pool.decode_scored(q, P.ids, SCALE, sc)
    scored = P.pool.last_decode_stats()
    P.pool.decode(q, P.ids, SCALE)
    assert P.pool.last_decode_stats() == plain
    page = 32 * 160 * 2   # an INT4 page of two kv heads
    assert plain["kv_bytes"] - scored["kv_bytes"] == 2 * page


def test_outputs_are_blocks_of_the_stream_of_the_call(kvq):
    """Work queued on the current stream may still use a block that it gave back: an output on another
    stream is none of those, and its own block is not given out while the current stream may read it."""
    P = Pool(kvq, 2, [mixed(300, 1), mixed(65, 2)], seed=6)
    pool, ids, s = P.pool, P.ids, torch.cuda.Stream()
    q, k, v = (rand((2, h, 128), P.gen) for h in (8, 2, 2))
    scores = torch.rand(2, 2, 300, device="cuda", generator=P.gen)
    calls = [(lambda **kw: pool.decode(q, ids, SCALE, **kw), (2, 8, 128), torch.float32),
             (lambda **kw: kvq.KVPool.decode_groups([pool], q, [ids], SCALE, **kw), (2, 8, 128), torch.float32),
             (lambda **kw: pool.attend(q, ids, [1, 1], SCALE, k, v, **kw), (2, 8, 128), torch.bfloat16),
             (lambda **kw: pool.decode_scored(q, ids, SCALE, scores, decay=1.0, **kw), (2, 8, 128), torch.float32),
             (lambda **kw: pool.select_lowest(scores, ids, 40, **kw), (2, 40), torch.int32)]
    for call, shape, dtype in calls:
        want = call()
        given = set()
        for _ in range(20):   # blocks of the current stream, given back
            given |= {x.data_ptr() for x in [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(4)]}
            s.wait_stream(torch.cuda.current_stream())
            out = call(stream=s)
            assert out.data_ptr() not in given and out.shape == shape and out.dtype == dtype
        s.synchronize()
        assert torch.equal(out, want)
    pool.sync()


@pytest.mark.parametrize("per_head", [False, True])
def test_selection_of_rows_past_shared_memory(kvq, per_head):
    """More than 393,216 positions: keys are read again for every digit."""
    n, hkv = 400007, 2
    pool = kvq.KVPool(hkv, n // 32 + 16, n // 32 + 16, 1, n // 32 + 32)
    rid = pool.open()
    gen = torch.Generator("cuda").manual_seed(5)
    for a in range(0, n, 50000):
        m = min(50000, n - a)
        pool.append(rand((m, hkv, 128), gen), rand((m, hkv, 128), gen), np.full(m, rid, np.int32), np.full(m, 2, np.uint8))
    dead = np.arange(1000, 390000, 7)
    pool.evict(np.full(dead.size, rid, np.int32), dead)
    x = torch.rand(1, hkv, n + 3, device="cuda", generator=gen)
    x = torch.where(x < 0.2, torch.zeros_like(x), x)
    live = np.setdiff1d(np.arange(n - 100), dead)
    xs = x.cpu().numpy()[0]
    keys = list(xs) if per_head else [summed_keys(xs)]
    for m in (1, 1000, 200000, 399000):
        got = pool.select_lowest(x, [rid], m, protect=100, per_head=per_head).cpu().numpy()[0]
        for row, key in zip(got if per_head else got[None], keys):
            want = np.sort(live[np.argsort(key[live], kind="stable")[:m]])
            assert np.array_equal(row[:want.size], want) and (row[want.size:] == -1).all(), m


def test_evict_lowest_of_every_head_its_own(kvq):
    """The chosen positions are the least of each head and read as dead for that head only."""
    P = Pool(kvq, 2, [mixed(500, 1), mixed(77, 2), mixed(0, 1)], seed=3)
    P.pool.set_decode_impl(MMA)
    x = torch.rand(3, 2, 500, device="cuda", generator=P.gen)
    want = check_select(P, x, [60, 20, 4], 10, True)
    pos = P.pool.evict_lowest(x, P.ids, [60, 20, 4], protect=10, per_head=True)
    assert np.array_equal(pos, want)
    ex = {r: {(h, int(p)) for h in range(2) for p in pos[r, h] if p >= 0} for r in range(2)}
    assert [len(ex[r]) for r in range(2)] == [120, 40]
    step(P, 8, torch.rand(3, 2, 520, device="cuda"), 1.0, head_dead=ex)
    again = check_select(P, x, [60, 20, 4], 10, True, head_dead=ex)
    for r in range(2):
        for h in range(2):
            assert not set(again[r, h].tolist()) & {p for y, p in ex[r] if y == h}
    # everything, and once more with nothing left
    P.pool.evict_lowest(x, P.ids, 500, per_head=True)
    assert (P.pool.evict_lowest(x, P.ids, 500, per_head=True) == -1).all()
    assert (P.pool.evict_lowest(x, P.ids, 500) == -1).all()


def test_scored_decode_of_requests_without_tokens(kvq):
    P = Pool(kvq, 2, [mixed(0, 1), mixed(0, 2)], seed=1)
    scores = torch.rand(2, 2, 5, device="cuda", generator=P.gen)
    kept = scores.clone()
    out = P.pool.decode_scored(rand((2, 8, 128), P.gen), P.ids, SCALE, scores, decay=0.5)
    assert (out == 0).all() and torch.equal(scores, kept)
    assert (P.pool.evict_lowest(scores, P.ids, 3) == -1).all()


class Live:
    """A pool under random calls, and which positions of every request are live for every kv head."""

    def __init__(self, kvq, seed):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.hkv, self.kvq = 2, kvq
        self.pool = kvq.KVPool(self.hkv, 90, 70, 3, 60, n_int3_pages=30, n_fp4_pages=30)
        self.pool.fp_configure(32)
        self.live, self.lists = {}, {}
        for _ in range(3):
            self.open()

    def open(self):
        r = self.pool.open()
        self.live[r], self.lists[r] = np.zeros((self.hkv, 0), bool), 0

    def some(self, r, share):
        n = self.live[r].shape[1]
        return self.rng.choice(n, int(n * share), replace=False) if n else np.zeros(0, np.int64)

    def append(self):
        reqs = [int(x) for x in self.rng.permutation(list(self.live))[:self.rng.integers(1, 4)]]
        n = int(self.rng.choice([1, 3, 31, 33, 64, 130]))
        ids = np.repeat(reqs, n)
        if self.rng.random() < 0.4:
            self.rng.shuffle(ids)
        choice = [(2, 4), (2,), (4,), (2, 3, 4, 0xF4)][self.rng.integers(4)]
        w = self.rng.choice(choice, ids.size).astype(np.uint8)
        k, v = (rand((ids.size, self.hkv, 128), self.gen) for _ in range(2))
        try:
            self.pool.append(k, v, ids, w)
        except self.kvq.KVError as e:
            assert e.status == self.kvq.KV_ERR_OOM
            return
        for r in reqs:
            self.live[r] = np.concatenate([self.live[r], np.ones((self.hkv, n), bool)], 1)

    def evict(self):
        r = int(self.rng.choice(list(self.live)))
        n = self.live[r].shape[1]
        at = self.some(r, 0.1) if self.rng.random() < 0.5 else np.arange(n // 4, n // 4 + min(90, n - n // 4))
        self.pool.evict(np.full(at.size, r, np.int32), at)
        self.live[r][:, at] = False

    def evict_head(self):
        r, h = int(self.rng.choice(list(self.live))), int(self.rng.integers(self.hkv))
        at = self.some(r, 0.3)
        self.pool.evict_head(np.full(at.size, r, np.int32), at, np.full(at.size, h, np.int32))
        self.live[r][h, at] = False

    def reorder(self):
        self.pool.reorder(list(self.live))

    def drop(self):
        self.pool.drop_dead_pages(list(self.live))

    def again(self):
        r = int(self.rng.choice(list(self.live)))
        self.pool.close_request(r)
        del self.live[r], self.lists[r]
        self.open()

    def fp(self):
        r = int(self.rng.choice(list(self.live)))
        if self.lists[r]:
            self.pool.fp_drop(r, 0, self.lists[r])
            self.lists[r] = 0
        else:
            self.pool.fp_append(r, *(rand((5, self.hkv, 128), self.gen) for _ in range(2)))
            self.lists[r] = 5

    def check(self):
        ids = [int(x) for x in self.rng.permutation(list(self.live))]
        S = max(max(x.shape[1] for x in self.live.values()), 1)
        g = int(self.rng.integers(1, 9))
        scores = torch.rand(len(ids), self.hkv, S, device="cuda", generator=self.gen)
        before = scores.cpu().numpy().astype(np.float64)
        # softmax_scale 0: every key weighs the same
        self.pool.decode_scored(rand((len(ids), g * self.hkv, 128), self.gen), ids, 0.0, scores, decay=0.5)
        after = scores.cpu().numpy()
        n_sel = [int(self.rng.integers(0, S + 1)) for _ in ids]
        protect = int(self.rng.integers(0, 40))
        shared = self.pool.select_lowest(scores, ids, n_sel, protect=protect).cpu().numpy()
        own = self.pool.select_lowest(scores, ids, n_sel, protect=protect, per_head=True).cpu().numpy()
        self.pool.sync()
        for b, r in enumerate(ids):
            L, limit = self.live[r], self.live[r].shape[1] - protect
            for h in range(self.hkv):
                n = int(L[h].sum()) + self.lists[r]
                want = before[b, h].copy()
                at = np.flatnonzero(L[h])
                want[at] = 0.5 * want[at] + (g / n if n else 0.0)
                # g weights of 1 / n and their sum, each rounded a few times
                assert np.abs(after[b, h] - want).max() <= 2.0 ** -20 and (np.delete(after[b, h], at) == np.delete(before[b, h], at)).all()
            rows = [(shared[b], L.any(0), summed_keys(after[b]))] + [(own[b, h], L[h], after[b, h]) for h in range(self.hkv)]
            for got, live, key in rows:
                at = np.flatnonzero(live)
                at = at[at < limit]
                pick = np.sort(at[np.argsort(key[at], kind="stable")[:n_sel[b]]])
                assert np.array_equal(got[:pick.size], pick) and (got[pick.size:] == -1).all()


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_positions_follow_tokens_through_random_calls(kvq, seed):
    """Appends of every shape, repacks, evictions, exclusions, reorders, drops, pages and request ids that
    change hands, lists: weights reach every live position's score and no other; selections match."""
    L = Live(kvq, seed)
    calls = [L.append] * 8 + [L.evict] * 2 + [L.evict_head, L.reorder, L.reorder, L.drop, L.drop, L.again, L.fp]
    for step_no in range(150):
        calls[L.rng.integers(len(calls))]()
        if step_no % 3 == 0:
            L.check()
