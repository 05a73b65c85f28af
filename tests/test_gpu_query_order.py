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
@pytest.mark.parametrize("call", ["decode", "simt", "noalloc", "scored", "groups", "attend", "attend_shared"])
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
