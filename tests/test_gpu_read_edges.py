"""Reading cached tokens back (kv_read_tokens): short ranges of long requests, and the slots' positions on the device
under random appends, evictions, drops, closes and reorders."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


def tagged(tags, hkv):
    """V rows that every width keeps exactly: each 32-channel group holds one value, 0, 6, .. 252 (a base-43 digit of
    the token's tag), so its range is 0 and its minimum is exact in binary16, and a sixth of it is.  Head h holds
    (tag + h)."""
    t = np.asarray(tags, np.int64)[:, None] + np.arange(hkv)
    d = np.stack([t // 43 ** g % 43 for g in range(4)], -1) * 6
    return np.repeat(d, 32, axis=-1).astype(np.float32)


def test_short_ranges_of_long_requests(kvq):
    """Ranges that start and end inside pages, of requests with thousands of pages, in one call."""
    hkv, n = 2, 70000
    gen = torch.Generator("cuda").manual_seed(1)
    pool = kvq.KVPool(hkv, 2 * n // 32 + 64, 2 * n // 32 + 64, 2, n // 32 + 64)
    ids = [pool.open() for _ in range(2)]
    for r, tag in zip(ids, (0, 10 ** 6)):
        v = torch.from_numpy(tagged(tag + np.arange(n), hkv)).cuda().bfloat16()
        k = torch.randn(n, hkv, 128, generator=gen, device="cuda").bfloat16()
        pool.append(k, v, [r] * n, [2] * (n // 2) + [4] * (n - n // 2))
    whole = pool.read(ids, dtype=torch.float32)
    assert np.array_equal(whole[1].cpu().numpy(), np.concatenate([tagged(t + np.arange(n), hkv) for t in (0, 10 ** 6)]))
    for first, m in (([n - 64, 0], [64, 1]), ([31, 34999], [2, 66]), ([n, n - 1], [0, 1]), ([17, 69000], [33, 1000])):
        for dtype in (torch.float32, torch.bfloat16):
            got = pool.read(ids, first, m, dtype=dtype)
            for x, w in zip(got, whole):
                want = torch.cat([w[b * n + f:b * n + f + c] for b, (f, c) in enumerate(zip(first, m))])
                assert torch.equal(x, want.to(dtype))
    pool.sync()
    pool.destroy()


@pytest.mark.parametrize("seed", range(4))
def test_read_under_random_calls(kvq, seed):
    """Every token of every request, found by its position, after each of a few hundred random calls."""
    rng = np.random.default_rng(seed)
    hkv, W = 2, (2, 3, 4, kvq.KV_WIDTH_FP4)
    pool = kvq.KVPool(hkv, 400, 500, 6, 200, n_int3_pages=200, n_fp4_pages=200)
    gen = torch.Generator("cuda").manual_seed(seed)
    rope = kvq.Rope(torch.randn(50, 128, generator=gen, device="cuda"))
    alive, tags = {}, {}       # per open request: [positions][heads], [positions]
    for _ in range(3):
        r = pool.open()
        alive[r], tags[r] = np.zeros((0, hkv), bool), np.zeros(0, np.int64)
    next_tag, reads = 1, 0
    for step in range(150):
        what = rng.choice(["append", "append", "append", "evict", "head", "drop", "reorder", "close", "open"])
        ids = list(alive)
        if what == "append" and ids:
            kind = rng.integers(0, 4)
            if kind == 0:                                   # a decode step
                req = np.array(ids)
                bits = rng.choice(W[:3:2] if seed % 2 else W, req.size)
            elif kind == 1:                                 # runs
                req = np.repeat(rng.permutation(ids), rng.integers(32, 120))
                bits = np.where(rng.random(req.size) < 0.6, 2, 4) if rng.random() < 0.5 else np.full(req.size, rng.choice([2, 4]))
            else:                                           # anything
                req = rng.choice(ids, rng.integers(1, 200))
                bits = rng.choice(W if rng.random() < 0.4 else (2, 4), req.size)
            bits = bits.astype(np.uint8)
            t = next_tag + np.arange(req.size)
            v = torch.from_numpy(tagged(t, hkv)).cuda().bfloat16()
            k = torch.randn(req.size, hkv, 128, generator=gen, device="cuda").bfloat16()
            try:
                if rng.random() < 0.3:
                    pool.append_rotated(k, v, req, bits, rope, torch.zeros(req.size, dtype=torch.int32, device="cuda"))
                else:
                    pool.append(k, v, req, bits)
            except kvq.KVError as e:
                assert e.status == kvq.KV_ERR_OOM
                pool.close_request(ids[0])
                del alive[ids[0]], tags[ids[0]]
                continue
            next_tag += req.size
            for r in ids:
                mine = t[req == r]
                tags[r] = np.concatenate([tags[r], mine])
                alive[r] = np.concatenate([alive[r], np.ones((mine.size, hkv), bool)])
        elif what in ("evict", "head") and ids:
            r = int(rng.choice(ids))
            n = tags[r].size
            if n == 0:
                continue
            a = int(rng.integers(0, n))
            pos = np.arange(a, min(n, a + int(rng.integers(1, 90)))) if rng.random() < 0.6 else rng.choice(n, max(1, n // 9), replace=False)
            if what == "evict":
                pool.evict([r] * pos.size, pos)
                alive[r][pos] = False
            elif step > 40:
                pool.evict_head([r] * pos.size, pos, [1] * pos.size)
                alive[r][pos, 1] = False
        elif what == "drop" and ids:
            pool.drop_dead_pages(ids)
        elif what == "reorder" and ids:
            pool.reorder(ids)
        elif what == "close" and len(ids) > 1 and rng.random() < 0.5:
            r = int(rng.choice(ids))
            pool.close_request(r)
            del alive[r], tags[r]
        elif what == "open" and len(ids) < 6:
            r = pool.open()
            alive[r], tags[r] = np.zeros((0, hkv), bool), np.zeros(0, np.int64)
        if step < 20 or rng.random() < 0.4 or not alive:   # (the first read puts the positions on the device)
            continue
        ids = list(alive)
        got = pool.read(ids, dtype=torch.float32)[1].cpu().numpy()
        want = np.concatenate([tagged(tags[r], hkv) * alive[r][:, :, None] for r in ids])
        assert np.array_equal(got, want), (step, what)
        reads += 1
    pool.sync()
    assert reads > 40
    pool.destroy()
