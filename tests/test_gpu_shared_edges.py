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


def least_us(f, n=6):
    """The shortest of n calls."""
    f()
    t = []
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        t.append(a.elapsed_time(b) * 1e3)
    return min(t)


def test_decode_step_plain_rows_end(kvq):
    """Rows of a decode step that the join takes plainly, over long own caches: a row that is not a number ends at the
    first page that shows it, and pages without a live slot for the head are passed over 32 at a time."""
    n, hkv = 32768, 8
    pool = kvq.KVPool(hkv, 2 * n // 32 + 64, n // 32 + 64, 2, n // 32 + 64)
    gen = torch.Generator("cuda").manual_seed(5)
    ids = [pool.open() for _ in range(2)]
    for r in ids:
        pool.append(rand((n, hkv, 128), gen), rand((n, hkv, 128), gen), [r] * n, [2] * n)
    q = rand((2, 64, 128), gen)
    step = lambda x: pool.attend_shared(x, ids, [-1, -1], [1, 1], SCALE)
    good = step(q)
    pool.sync()
    usual = least_us(lambda: step(q))
    bad = q.clone()
    bad[0, ::9, 3] = float("nan")
    out = step(bad)
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    fin = torch.isfinite(out).all(-1)
    assert not bool(fin[0, ::9].any()) and int(fin.sum()) == 120
    assert torch.equal(out[fin], good[fin])
    took = least_us(lambda: step(bad))
    assert took < usual + 2000.0, (usual, took)    # a walk over all 1024 pages takes 16 ms
    with pytest.raises(kvq.KVError):
        pool.sync()
    pool.evict_head([ids[1]] * n, list(range(n)), [3] * n)
    out = step(q)
    pool.sync()
    assert bool((out[1, 24:32] == 0).all())
    # pages that no worker reads for the head move the other heads' splits, so their fp32 sums (2^-15 of the terms) are
    # taken in other pieces; each result is then rounded to bf16, by at most 2^-9 of itself
    for x, y in ((out[0], good[0]), (out[1, :24], good[1, :24]), (out[1, 32:], good[1, 32:])):
        assert float((x.double() - y.double()).norm()) <= 1.1 * 2 * 2.0 ** -9 * float(y.double().norm())
    took = least_us(lambda: step(q))
    assert took < 2.5 * usual, (usual, took)       # an entry at a time: 4.7 times
    pool.destroy()


def test_long_chunk_without_a_prefix(kvq):
    """A long chunk of a request without a prefix beside one token of a request with one: no partial sums of its rows."""
    P = Pool(kvq, 8, [mixed(256, i) for i in range(3)], seed=6)
    pool, n, hq = P.pool, 4096, 64
    q, k, v = (rand((n + 1, h, 128), P.gen) for h in (hq, 8, 8))
    out = torch.empty_like(q)
    want = pool.attend(q, P.ids[1:], [n, 1], SCALE, k, v)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    pool.attend_shared(q, P.ids[1:], [-1, P.ids[0]], [n, 1], SCALE, k, v, out=out)
    pool.sync()
    grown = free - torch.cuda.mem_get_info()[0]
    assert grown < 32 << 20, grown     # the chunk's rows would be 138 MB
    # the chunk's blocks may be cut elsewhere than in kv_attend: other pieces of the same fp32 sums, each result rounded
    # to bf16, by at most 2^-9 of itself
    a, b = out[:n].double(), want[:n].double()
    assert float((a - b).norm()) <= 1.1 * 2 * 2.0 ** -9 * float(b.norm())
    P.pool.destroy()


@pytest.mark.parametrize("n_new,prefix", [
    ([1, 33, 97, 2], [-1, -1, -1, 0]), ([33, 1, 33], [-1, 0, 0]), ([40, 2, 40, 1], [-1, -1, 0, 1]),
    ([300, 1, 1, 260], [-1, 0, -1, 0]), ([1, 100, 3], [1, -1, -1])])
@pytest.mark.parametrize("with_kv", [True, False])
def test_rows_with_and_without_a_prefix(kvq, n_new, prefix, with_kv):
    """Few, middle and many rows of requests without a prefix beside few and many with one."""
    P = Pool(kvq, 1, [mixed(300, 1), mixed(130, 2)] + [mixed(40 * i, i) for i in range(len(n_new))], seed=len(n_new))
    check(P, range(2, 2 + len(n_new)), prefix, n_new, 4, with_kv, rows=[0, 1, 32, 39, 96, 99, 259, 299])
    P.pool.destroy()


def test_a_chunk_among_single_tokens(kvq):
    """One long chunk and many single tokens over one prefix, in one call."""
    n = 40
    P = Pool(kvq, 2, [mixed(500, 1)] + [mixed(20 + i, i) for i in range(n)], seed=7)
    n_new = [1] * n
    n_new[17] = 700
    check(P, range(1, n + 1), [0] * n, n_new, 8, rows=[0, 1, 350, 699])
    P.pool.destroy()


def test_decode_step_expired_wait(kvq):
    """A first wait of the own caches' scan that gives up is reported once, and the pool goes on."""
    P = step_pool(kvq, seed=8)
    n = len(P.ids) - 1
    q = rand((n, 16, 128), P.gen)
    step = lambda: P.pool.attend_shared(q, P.ids[1:], [P.ids[0]] * n, [1] * n, SCALE)
    good = step()
    P.pool.sync()
    P.pool.set_wait_limit(0)
    step()
    with pytest.raises(kvq.KVError) as e:
        P.pool.sync()
    assert e.value.status == kvq.KV_ERR_DEVICE_TIMEOUT
    P.pool.sync()
    P.pool.set_wait_limit(-1)
    assert torch.equal(step(), good)
    P.pool.sync()
    P.pool.destroy()


def test_the_same_call_again(kvq):
    """Equal bits from equal calls, whatever ran in between: a decode step, drafts, chunks."""
    P = step_pool(kvq, seed=9)
    n = len(P.ids) - 1
    calls = []
    for n_new, kv in (([1] * n, False), ([1 + i % 5 for i in range(n)], True), ([150, 2] + [0] * (n - 3) + [40], True)):
        q = rand((sum(n_new), 16, 128), P.gen)
        k, v = (rand((sum(n_new), 8, 128), P.gen) for _ in range(2)) if kv else (None, None)
        prefix = [P.ids[0] if i % 4 else -1 for i in range(n)]
        calls.append(lambda q=q, k=k, v=v, n_new=n_new, p=prefix: P.pool.attend_shared(q, P.ids[1:], p, n_new, SCALE, k, v))
    first = [f() for f in calls]
    for _ in range(3):
        for f, y in zip(calls, first):
            assert torch.equal(f(), y)
    P.pool.sync()
    P.pool.destroy()


def test_decode_right_after_its_rotation(kvq):
    """q rotated by the kernel before the decode (or the step over a prefix) on the same stream."""
    P = step_pool(kvq, seed=10)
    pool, n = P.pool, len(P.ids) - 1
    rope = kvq.Rope(torch.randn(64, 128, generator=P.gen, device="cuda"))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    x = [rand((n, 16, 128), P.gen) for _ in range(2)]
    turned = [pool.rotate(y, rope, pos) for y in x]
    torch.cuda.synchronize()
    pre = [P.ids[0]] * n
    want = [(pool.decode(y, P.ids[1:], SCALE).clone(), pool.attend_shared(y, P.ids[1:], pre, [1] * n, SCALE)) for y in turned]
    torch.cuda.synchronize()
    q, got = torch.empty_like(x[0]), []
    for i in range(40):
        pool.rotate(x[i & 1], rope, pos, out=q)
        a = pool.decode(q, P.ids[1:], SCALE)
        pool.rotate(x[i & 1], rope, pos, out=q)
        got.append((a, pool.attend_shared(q, P.ids[1:], pre, [1] * n, SCALE)))
    for i, y in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(y, want[i & 1])), i
    pool.sync()
    pool.destroy()
