"""Rotary positions (kv_rotate), appends that rotate (kv_append_rotated) and reading tokens back
(kv_read_tokens) against plain forms: the rotation and the pages bit for bit."""
import numpy as np
import pytest

import rope_ref
from np_ref import dequant_page

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

W4 = (2, 3, 4, 0xF4)


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def make_rope(kvq, rows, rot, axis=None, pairs=False, base=10000.0):
    tab = rope_ref.table(rows, rot, base)
    return kvq.Rope(torch.from_numpy(tab).cuda(), axis=axis, interleaved=pairs), tab


def rand(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).bfloat16()


def host(t):
    return t.float().cpu().numpy()


def small_pool(kvq, hkv=2, pages=64, n_req=4):
    return kvq.KVPool(hkv, pages, pages, n_req, 4 * pages, n_int3_pages=pages, n_fp4_pages=pages)


def axes_of(kind, rot, n_axes):
    half = rot // 2
    return None if n_axes == 1 else (np.arange(half) % n_axes if kind == "mixed" else np.arange(half) * n_axes // half)


# ---- rotate ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,hq,hk,rot,n_axes,kind,pairs", [
    (1, 8, 2, 128, 1, "", False), (1, 1, 0, 16, 1, "", True), (7, 5, 3, 96, 1, "", False), (33, 32, 8, 128, 3, "mixed", False),
    (130, 12, 4, 64, 2, "blocks", True), (513, 64, 8, 128, 4, "mixed", True), (2000, 3, 1, 32, 3, "blocks", False),
    (1999, 28, 4, 128, 1, "", False), (40, 70, 1, 112, 2, "mixed", False)])
def test_rotate(kvq, n, hq, hk, rot, n_axes, kind, pairs):
    gen = torch.Generator("cuda").manual_seed(n)
    rng = np.random.default_rng(n)
    pool = small_pool(kvq)
    rope, tab = make_rope(kvq, 5000, rot, axes_of(kind, rot, n_axes), pairs)
    pos = rng.integers(0, 5000, (n_axes, n)).astype(np.int32)
    pos[0, 0], pos[-1, -1] = 4999, 0
    # q and k as slices of one projection's output
    x = rand(gen, n, hq + hk + 1, 128)
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    dp = torch.from_numpy(pos if n_axes > 1 else pos[0]).cuda()
    got = pool.rotate(q, rope, dp, k=k)
    pool.sync()
    axis = rope.axis
    for g, t in zip(got if hk else (got,), (q, k)):
        want = rope_ref.rotate(host(t), tab, pos, axis, pairs)
        assert np.array_equal(host(g), want)
        exact, tol = rope_ref.rotate_exact(host(t), tab, pos, axis, pairs)
        assert np.all(np.abs(host(g).astype(np.float64) - exact) <= tol)
    # in place, on a stream of its own
    s = torch.cuda.Stream()
    y = x.clone()
    s.wait_stream(torch.cuda.current_stream())
    pool.rotate(y[:, :hq], rope, dp, k=y[:, hq:hq + hk] if hk else None, out=y[:, :hq],
                k_out=y[:, hq:hq + hk] if hk else None, stream=s)
    s.synchronize()
    assert torch.equal(y[:, :hq], got[0] if hk else got)
    assert torch.equal(y[:, hq + hk:], x[:, hq + hk:])
    if hk:
        assert torch.equal(y[:, hq:hq + hk], got[1])
    pool.destroy()


@pytest.mark.parametrize("off", [1, 4])
def test_rotate_unaligned(kvq, off):
    """Rows at any 2-byte alignment, odd strides, outputs apart."""
    gen = torch.Generator("cuda").manual_seed(off)
    pool = small_pool(kvq)
    rope, tab = make_rope(kvq, 100, 128)
    n, h = 9, 3
    step = h * 128 + off
    flat = rand(gen, 2 * n * step + off)
    q = flat.as_strided((n, h, 128), (step, 128, 1), off)
    out = torch.full((n * step + 7,), 5.0, device="cuda").bfloat16()
    o = out.as_strided((n, h, 128), (step, 128, 1), 3)
    pos = np.arange(n, dtype=np.int32)[::-1].copy()
    pool.rotate(q, rope, torch.from_numpy(pos).cuda(), out=o)
    pool.sync()
    assert np.array_equal(host(o), rope_ref.rotate(host(q), tab, pos))
    rest = torch.ones(out.numel(), dtype=torch.bool)
    rest.as_strided((n, h, 128), (step, 128, 1), 3)[:] = False
    assert bool((out.cpu()[rest] == 5.0).all())
    pool.destroy()


def test_rotate_none(kvq):
    pool = small_pool(kvq)
    rope, _ = make_rope(kvq, 10, 64)
    out = pool.rotate(torch.empty(0, 4, 128, device="cuda", dtype=torch.bfloat16), rope,
                      torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 128)
    pool.sync()
    pool.destroy()


def test_position_outside_the_table(kvq):
    """Counts as 0, is reported once, and the pool goes on."""
    gen = torch.Generator("cuda").manual_seed(3)
    pool = small_pool(kvq)
    rope, tab = make_rope(kvq, 50, 128)
    q = rand(gen, 4, 2, 128)
    pos = np.array([3, 50, -1, 49], np.int32)
    got = pool.rotate(q, rope, torch.from_numpy(pos).cuda())
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    pool.sync()
    assert np.array_equal(host(got), rope_ref.rotate(host(q), tab, np.array([3, 0, 0, 49])))
    r = pool.open()
    pool.append_rotated(q, q, [r] * 4, [4] * 4, rope, torch.from_numpy(pos).cuda())
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    pool.sync()
    pool.destroy()


def test_rotate_captured(kvq):
    """A graph of two rotations replayed on new inputs, beside an eager one of another pool."""
    gen = torch.Generator("cuda").manual_seed(4)
    pool, other = small_pool(kvq), small_pool(kvq)
    rope, tab = make_rope(kvq, 300, 128, np.arange(64) % 3)
    q, k = rand(gen, 17, 8, 128), rand(gen, 17, 2, 128)
    pos = torch.randint(0, 300, (3, 17), generator=gen, device="cuda", dtype=torch.int32)
    pool.rotate(q, rope, pos, k=k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.graph(g):
        pool.rotate(q, rope, pos, k=k, out=oq, k_out=ok)
        pool.rotate(oq, rope, pos, out=oq)
    for _ in range(2):
        q.copy_(rand(gen, 17, 8, 128))
        k.copy_(rand(gen, 17, 2, 128))
        pos.copy_(torch.randint(0, 300, (3, 17), generator=gen, device="cuda", dtype=torch.int32))
        g.replay()
        once = other.rotate(q, rope, pos)
        torch.cuda.synchronize()
        p = pos.cpu().numpy()
        one = rope_ref.rotate(host(q), tab, p, rope.axis)
        assert np.array_equal(host(once), one)
        assert np.array_equal(host(oq), rope_ref.rotate(one, tab, p, rope.axis))
        assert np.array_equal(host(ok), rope_ref.rotate(host(k), tab, p, rope.axis))
    pool.sync()
    pool.destroy()
    other.destroy()


# ---- append ---------------------------------------------------------------------------------------------------------

def same_content(a, b, ra, rb):
    x, y = a.export(ra), b.export(rb)
    for key in ("ids", "is_int2", "fill", "live"):
        assert np.array_equal(x[key], y[key]), key
    for i in range(x["ids"].size):   # slots at or past fill hold unspecified content
        f = int(x["fill"][i])
        for key in ("kc", "vc"):
            assert np.array_equal(x[key][i][:, :f], y[key][i][:, :f]), (key, i)
        if x["is_int2"][i]:
            assert np.array_equal(x["km"][i], y["km"][i])
        else:
            assert np.array_equal(x["km"][i].reshape(-1, 32, 8)[:, :f], y["km"][i].reshape(-1, 32, 8)[:, :f])
        assert np.array_equal(x["vm"][i].reshape(-1, 32, 8)[:, :f], y["vm"][i].reshape(-1, 32, 8)[:, :f])


@pytest.mark.parametrize("hkv,rot,n_axes,pairs,widths,lens,packed", [
    (2, 128, 1, False, (4,), (1,), True),                       # one token
    (1, 128, 1, True, (2, 4), (3, 1, 2), False),                # a few, by value
    (8, 64, 3, False, (2, 4), (40, 97, 33), True),              # runs of several requests
    (3, 96, 2, True, (2, 4), (700,), True),                     # bulk, one request
    (2, 32, 1, False, W4, (211, 5), False),                     # every width
    (4, 16, 4, False, (2, 4), (1500,), False),
    (2, 128, 3, True, W4, (350, 64, 31), True)])
def test_append_rotated_is_append_of_rotated(kvq, hkv, rot, n_axes, pairs, widths, lens, packed):
    """Two chunks (the second meets open tail and staging pages): the pages of kv_append_quant on rotated keys, bit for bit."""
    gen = torch.Generator("cuda").manual_seed(sum(lens))
    rng = np.random.default_rng(sum(lens))
    a, b = small_pool(kvq, hkv, pages=160), small_pool(kvq, hkv, pages=160)
    rope, tab = make_rope(kvq, 4000, rot, axes_of("mixed", rot, n_axes), pairs, base=500000.0)
    ra, rb = [a.open() for _ in lens], [b.open() for _ in lens]
    for chunk in range(2):
        n = sum(lens)
        x = rand(gen, n, 2 * hkv + 2, 128, scale=3.0)
        k, v = (x[:, 1:1 + hkv], x[:, 1 + hkv:1 + 2 * hkv]) if packed else (x[:, :hkv].contiguous(), x[:, hkv:2 * hkv].contiguous())
        pos = rng.integers(0, 4000, (n_axes, n)).astype(np.int32)
        dp = torch.from_numpy(pos if n_axes > 1 else pos[0]).cuda()
        which = np.repeat(np.arange(len(lens)), lens)
        bits = rng.choice(widths, n).astype(np.uint8)
        a.append_rotated(k, v, np.array(ra)[which], bits, rope, dp)
        kr = torch.from_numpy(rope_ref.rotate(host(k), tab, pos, rope.axis, pairs)).cuda().bfloat16()
        b.append(kr, v.contiguous(), np.array(rb)[which], bits)
        a.sync()
        b.sync()
        for x_, y_ in zip(ra, rb):
            same_content(a, b, x_, y_)
    # both pools give the same decode (the largest scales, which the scan uses, among the state)
    q = rand(gen, len(lens), hkv, 128)
    assert torch.equal(a.decode(q, ra, 0.1), b.decode(q, rb, 0.1))
    a.destroy()
    b.destroy()


def test_append_rotated_alignment(kvq):
    """8-byte aligned rows at strides that are multiples of 4 elements: the kernels without 16-byte loads."""
    gen = torch.Generator("cuda").manual_seed(9)
    a, b = small_pool(kvq), small_pool(kvq)
    rope, tab = make_rope(kvq, 600, 128)
    n, step = 500, 2 * 128 + 4
    flat = rand(gen, 2 * n * step + 8)
    k = flat.as_strided((n, 2, 128), (step, 128, 1), 4)
    v = flat.as_strided((n, 2, 128), (step, 128, 1), n * step + 4)
    pos = np.arange(n, dtype=np.int32)
    bits = np.random.default_rng(9).choice([2, 4], n).astype(np.uint8)
    ra, rb = a.open(), b.open()
    a.append_rotated(k, v, [ra] * n, bits, rope, torch.from_numpy(pos).cuda())
    b.append(torch.from_numpy(rope_ref.rotate(host(k), tab, pos)).cuda().bfloat16(), v.contiguous(), [rb] * n, bits)
    same_content(a, b, ra, rb)
    a.destroy()
    b.destroy()


def test_int2_groups_alone(kvq):
    """Calls that are whole INT2 groups and nothing else: 16-byte aligned rows (the kernel of large calls) and rows at an
    odd multiple of 8 bytes (a warp per token) give the same pages, positions and values."""
    gen = torch.Generator("cuda").manual_seed(12)
    a, b = small_pool(kvq, 3), small_pool(kvq, 3)
    rope, _ = make_rope(kvq, 700, 128)
    ra, rb = [[p.open() for _ in range(2)] for p in (a, b)]

    def both(which, bits, rotated):
        n = len(which)
        flat = rand(gen, 2 * n * 3 * 128 + 8, scale=2.0)
        off = flat[4:-4].view(2, n, 3, 128)
        k, v = off.clone()
        assert k.data_ptr() % 16 == 0 and off[0].data_ptr() % 16 == 8
        if rotated:
            pos = torch.randint(0, 700, (n,), generator=gen, device="cuda", dtype=torch.int32)
            a.append_rotated(k, v, np.array(ra)[which], bits, rope, pos)
            b.append_rotated(off[0], off[1], np.array(rb)[which], bits, rope, pos)
        else:
            a.append(k, v, np.array(ra)[which], bits)
            b.append(off[0], off[1], np.array(rb)[which], bits)
        for x, y in zip(ra, rb):
            same_content(a, b, x, y)
        for x, y in zip(a.read(ra, dtype=torch.float32), b.read(rb, dtype=torch.float32)):
            assert torch.equal(x, y)

    both([0] * 5 + [1] * 3, [4] * 8, False)   # (the read after it puts the positions on the device)
    for rotated in (False, True):
        for n in (32, 96, 64):
            both([0] * n, [2] * n, rotated)
        both([0] * 32 + [1] * 64, [2] * 96, rotated)    # runs
        both([0, 1] * 64, [2] * 128, rotated)           # token by token
    a.sync()
    b.sync()
    a.destroy()
    b.destroy()


def test_append_rotated_checks_values_after_the_rotation(kvq):
    pool = small_pool(kvq)
    rope, _ = make_rope(kvq, 10, 128)
    r = pool.open()
    pos = torch.ones(1, dtype=torch.int32, device="cuda")
    for bad in (float("nan"), float("inf")):
        k = torch.zeros(1, 2, 128, device="cuda").bfloat16()
        k[0, 1, 77] = bad
        pool.append_rotated(k, torch.zeros_like(k), [r], [4], rope, pos)
        with pytest.raises(kvq.KVError) as e:
            pool.sync()
        assert e.value.status == kvq.KV_ERR_RANGE
    # 60000 in both channels of a pair passes binary16's range once they are turned by one radian
    k = torch.zeros(1, 2, 128, device="cuda").bfloat16()
    k[0, 0, 0] = k[0, 0, 64] = 60000.0
    pool.append(k, torch.zeros_like(k), [r], [4])
    pool.sync()
    pool.append_rotated(k, torch.zeros_like(k), [r], [4], rope, pos)
    with pytest.raises(kvq.KVError) as e:
        pool.sync()
    assert e.value.status == kvq.KV_ERR_RANGE
    pool.destroy()


# ---- read -----------------------------------------------------------------------------------------------------------

def values_of(pool, rid, where, n, n2, nfb):
    """K and V [n][Hkv][128] fp32 of a request from its export; where[(table index, slot)] = position."""
    ex = pool.export(rid)
    H = pool.num_kv_heads
    K, V = np.zeros((n, H, 128), np.float32), np.zeros((n, H, 128), np.float32)
    for i, pid in enumerate(ex["ids"]):
        for h in range(H):
            k, v = dequant_page(ex["kc"][i, h], ex["vc"][i, h], ex["km"][i, h], ex["vm"][i, h], pid < n2, fp4=pid >= nfb)
            for s in range(32):
                if (int(ex["live"][i]) >> s) & 1:
                    p = where[(i, s)]
                    K[p, h], V[p, h] = k[s], v[s]
    return K, V


def build(kvq, hkv, widths_list, seed, chunk=61):
    from test_gpu_attend import Pool
    P = Pool(kvq, hkv, widths_list, seed=seed, chunk=chunk)
    P.slots()
    return P


@pytest.mark.parametrize("hkv,lens,widths", [(1, (1,), (4,)), (2, (31, 33, 64), (2, 4)), (3, (200, 130), W4), (8, (97,), (2,))])
def test_read(kvq, hkv, lens, widths):
    rng = np.random.default_rng(len(lens) + hkv)
    P = build(kvq, hkv, [rng.choice(widths, n).astype(np.uint8) for n in lens], seed=hkv)
    pool = P.pool
    n2 = pool.n_int2_pages
    want = [values_of(pool, rid, pool.slot_pos[rid], n, n2, pool.first_fp4) for rid, n in zip(P.ids, lens)]
    k, v = pool.read(P.ids, dtype=torch.float32)
    pool.sync()
    for g, j in ((k, 0), (v, 1)):
        assert np.array_equal(g.cpu().numpy(), np.concatenate([w[j] for w in want]))
    kb, vb = pool.read(P.ids)
    assert torch.equal(kb, k.bfloat16()) and torch.equal(vb, v.bfloat16())
    # ranges, requests in another order and twice, empty ones among them
    order = list(range(len(lens)))[::-1] + [0, 0]
    first = [int(rng.integers(0, lens[r] + 1)) for r in order]
    count = [int(rng.integers(0, lens[r] - f + 1)) for r, f in zip(order, first)]
    k, v = pool.read([P.ids[r] for r in order], first, count, dtype=torch.float32)
    for g, j in ((k, 0), (v, 1)):
        assert np.array_equal(g.cpu().numpy(), np.concatenate([want[r][j][f:f + c] for r, f, c in zip(order, first, count)]))
    pool.destroy()


def test_read_after_evictions_and_drops(kvq):
    """Evicted, excluded and dropped tokens are zeros; pages used again hold the new tokens."""
    lens = (150, 96, 0)
    P = build(kvq, 2, [np.full(n, 4, np.uint8) for n in lens], seed=2)
    pool = P.pool
    k0, v0 = (x.cpu().numpy() for x in pool.read(P.ids, dtype=torch.float32))
    a, b, r = P.ids
    pool.evict([a] * 40, list(range(20, 60)))                    # page 1 (32..63) loses 32..59
    pool.evict_head([a] * 3, [5, 61, 149], [1, 0, 1])
    pool.evict([a] * 4, [60, 61, 62, 63])
    pool.drop_dead_pages([a])
    alive = np.ones((sum(lens), 2), bool)
    alive[20:64] = False
    for p, h in ((5, 1), (61, 0), (149, 1)):
        alive[p, h] = False
    k, v = (x.cpu().numpy() for x in pool.read(P.ids, dtype=torch.float32))
    assert np.array_equal(k, k0 * alive[:, :, None]) and np.array_equal(v, v0 * alive[:, :, None])
    # the dropped page's id goes to another request
    x = rand(P.gen, 20, 2, 128)
    pool.append(x, x, [r] * 20, [4] * 20)
    k2, _ = pool.read([a, r, b], dtype=torch.float32)
    k2 = k2.cpu().numpy()
    assert np.array_equal(k2[:150], (k0 * alive[:, :, None])[:150])
    assert np.array_equal(k2[170:], k0[150:])
    assert np.abs(k2[150:170] - host(x)).max() <= 0.5 * (host(x).max() - host(x).min()) / 15 * 1.01
    # a request closed and opened again starts empty, then holds its own tokens alone
    pool.close_request(a)
    a2 = pool.open()
    assert pool.read([a2])[0].shape[0] == 0
    y = rand(P.gen, 3, 2, 128)
    pool.append(y, y, [a2] * 3, [4] * 3)
    k3 = pool.read([a2], dtype=torch.float32)[0].cpu().numpy()
    assert np.abs(k3 - host(y)).max() <= 0.5 * (host(y).max() - host(y).min()) / 15 * 1.01
    pool.sync()
    pool.destroy()


def test_read_many_requests(kvq):
    """More requests than fit the launch's parameters."""
    gen = torch.Generator("cuda").manual_seed(8)
    pool = kvq.KVPool(1, 8, 200, 100, 8)
    ids = [pool.open() for _ in range(100)]
    x = rand(gen, 300, 1, 128)
    which = np.repeat(ids, 3)
    pool.append(x, x, which, np.full(300, 4, np.uint8))
    k, v = pool.read(ids, dtype=torch.float32)
    k1 = torch.cat([pool.read([r], dtype=torch.float32)[0] for r in ids])
    assert torch.equal(k, k1)
    assert (k - x.float()).abs().max() <= 0.5 * (x.float().max() - x.float().min()) / 15 * 1.01
    pool.destroy()


# ---- refusals -------------------------------------------------------------------------------------------------------

def test_refusals(kvq):
    pool = small_pool(kvq)
    gen = torch.Generator("cuda").manual_seed(1)
    rope, _ = make_rope(kvq, 100, 128, np.arange(64) % 3)
    q = rand(gen, 4, 2, 128)
    p1, p3 = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    for bad in (dict(positions=p1), dict(positions=p3.long()), dict(positions=p3[:, :3]), dict(positions=p3.cpu()),
                dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q.transpose(0, 1)), dict(k=q[:3]), dict(k_out=q),
                dict(out=q[:3]), dict(out=q.float())):
        a = dict(q=q, rope=rope, positions=p3)
        a.update(bad)
        with pytest.raises(ValueError):
            pool.rotate(**a)
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros(4, 64, device="cuda"), axis=np.zeros(31))
    with pytest.raises(ValueError):
        kvq.Rope(torch.zeros(4, 64, device="cuda"), axis=np.full(32, 4))
    for rot in (8, 24, 144):   # refused when it is used
        with pytest.raises(kvq.KVError) as e:
            pool.rotate(q, kvq.Rope(torch.zeros(4, rot, device="cuda")), p1)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    with pytest.raises(kvq.KVError):   # an output whose tokens overlap
        pool.rotate(q, rope, p3, out=torch.zeros(2, 128, device="cuda").bfloat16().expand(4, 2, 128))
    r = pool.open()
    one, _ = make_rope(kvq, 100, 128)
    off = torch.zeros(4 * 258 + 8, device="cuda").bfloat16()
    for k in (off[1:1 + 4 * 256].view(4, 2, 128), off[:4 * 258].as_strided((4, 2, 128), (258, 128, 1))):
        with pytest.raises(kvq.KVError) as e:
            pool.append_rotated(k, q, [r] * 4, [4] * 4, one, p1)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pool.append_rotated(q, q, [r] * 3, [4] * 3, one, p1)
    with pytest.raises(kvq.KVError):
        pool.append_rotated(q, q, [r + 1] * 4, [4] * 4, one, p1)
    with pytest.raises(kvq.KVError):
        pool.append_rotated(q, q, [r] * 4, [5] * 4, one, p1)
    assert pool.info(r) == (0, 0)
    pool.append_rotated(q, q, [r] * 4, [4] * 4, one, p1)
    for a in (dict(first=5, n=0), dict(first=-1), dict(n=5), dict(first=2, n=3)):
        with pytest.raises(kvq.KVError) as e:
            pool.read([r], **a)
        assert e.value.status == kvq.KV_ERR_INVALID_ARG
    for a in (dict(n=-1), dict(first=5), dict(dtype=torch.float16), dict(first=[0, 0])):
        with pytest.raises(ValueError):
            pool.read([r], **a)
    with pytest.raises(kvq.KVError):
        pool.read([r + 1], 0, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(kvq.KVError) as e:
            pool.read([r], 0, 4)
        assert e.value.status == kvq.KV_ERR_STATE
    pool.sync()
    pool.destroy()
