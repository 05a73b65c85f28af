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
