"""q written on the same stream right before the call that reads it, by a kernel that lets its successors start early
(matrix products of libraries do): every form of the decode reads the q of its own step."""
import numpy as np
import pytest

from attend_ref import SCALE
from test_gpu_attend import rand

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import __graft_entry__
    __graft_entry__.build()
    import mixed_precision_kv_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("batch,inner", [(16, 65536), (256, 16384), (16, 4096)])
@pytest.mark.parametrize("call", ["decode", "simt", "noalloc", "scored", "groups", "attend", "attend_shared", "prefix"])
def test_projection_then_attention(kvq, call, batch, inner):
    hkv, hq, n, steps = 8, 32, 96, 12
    gen = torch.Generator("cuda").manual_seed(inner)
    pools = [kvq.KVPool(h, 64, batch * 4 + 64, batch, 16) for h in ((4, 4) if call == "groups" else (hkv,))]
    pool = pools[0]
    ids = [[p.open() for _ in range(batch)] for p in pools]
    for p, r in zip(pools, ids):
        k, v = (rand((n * batch, p.num_kv_heads, 128), gen) for _ in range(2))
        p.append(k, v, np.repeat(r, n), np.full(n * batch, 4, np.uint8))
    pool.set_decode_impl(kvq.KV_DECODE_SIMT if call == "simt" else kvq.KV_DECODE_AUTO)
    scores = torch.zeros(batch, hkv, n, device="cuda")

    def run(q):
        if call in ("decode", "simt"):
            return pool.decode(q, ids[0], SCALE)
        if call == "noalloc":
            return pool.decode_noalloc(q, ids[0], SCALE, torch.empty(batch, hq, 128, device="cuda"))
        if call == "scored":
            return pool.decode_scored(q, ids[0], SCALE, scores)
        if call == "groups":
            return kvq.KVPool.decode_groups(pools, q, ids, SCALE)
        if call == "attend":
            return pool.attend(q, ids[0], [1] * batch, SCALE)
        if call == "prefix":
            return pool.attend_shared(q, ids[0], [-1] + ids[0][:1] * (batch - 1), [1] * batch, SCALE)
        return pool.attend_shared(q, ids[0], [-1] * batch, [1] * batch, SCALE)

    W = rand((inner, hq * 128), gen, inner ** -0.5)
    x = [rand((batch, inner), gen) for _ in range(2)]
    qs = [torch.zeros(batch, hq * 128, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    run(qs[0].view(batch, hq, 128))   # workspaces, plans
    torch.cuda.synchronize()
    got = []
    for i in range(steps):
        torch.matmul(x[i & 1], W, out=qs[i])
        got.append(run(qs[i].view(batch, hq, 128)))
    torch.cuda.synchronize()
    for i in range(steps):
        want = run(qs[i].view(batch, hq, 128))
        torch.cuda.synchronize()
        assert torch.equal(got[i], want), i
    for p in pools:
        p.sync()
        p.destroy()


@pytest.mark.parametrize("batch,inner", [(16, 65536), (200, 16384)])
@pytest.mark.parametrize("rotated", [False, True])
def test_steps_without_a_wait(kvq, batch, inner, rotated):
    """Projection, rotation, append, attention, output product, step after step on one stream with nothing waited for in
    between: the bits of the same steps with a wait after every call.  Large batches append by the bulk kernels."""
    hkv, hq, steps = 2, 8, 6
    gen = torch.Generator("cuda").manual_seed(3)
    W = rand((inner, (hq + 2 * hkv) * 128), gen, inner ** -0.5)
    Wo = rand((hq * 128, inner), gen, (hq * 128) ** -0.5)
    x0 = rand((batch, inner), gen)
    rope = kvq.Rope(torch.randn(batch + steps, 128, generator=gen, device="cuda"))

    def trip(wait):
        pool = kvq.KVPool(hkv, 400, 400, 4, 300)
        ids = [pool.open() for _ in range(4)]
        req = np.repeat(ids, batch // 4)
        x, outs = x0.clone(), []
        settle = torch.cuda.synchronize if wait else (lambda: None)
        for i in range(steps):
            qkv = torch.matmul(x, W).view(batch, hq + 2 * hkv, 128)
            settle()
            pos = torch.arange(batch, dtype=torch.int32, device="cuda") + i
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            bits = np.where(np.arange(batch) % 7 < 3, 4, 2) if i % 2 else np.full(batch, 2)
            if rotated:
                pool.append_rotated(k, v, req, bits, rope, pos)
                settle()
                q = pool.rotate(q, rope, pos)
            else:
                k, v, q = k.contiguous(), v.contiguous(), q.contiguous()
                pool.append(k, v, req, bits)
            settle()
            n = [batch // 4] * 4
            if i % 3 == 2:
                a = pool.attend_shared(q, ids, [-1, ids[0], ids[0], ids[1]], n, SCALE)
            else:
                a = pool.attend(q, ids, n, SCALE)
            settle()
            d = pool.decode(q[:4].contiguous(), ids, SCALE)
            settle()
            y = a.reshape(batch, hq * 128)
            y[:4] += d.reshape(4, hq * 128).bfloat16()
            x = torch.matmul(y, Wo)
            settle()
            outs += [a, d, x]
        outs += list(pool.read(ids))
        pool.sync()
        pool.destroy()
        return outs

    want = trip(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(trip(False), want))
