"""Cases and plain forms of the operators that read a mixed-precision cache for serving:

- attend: several new tokens per request attend to the request's cached tokens and to each other (drafts to be
  verified, in a line or as a tree; a further chunk of a prompt).
- decode_scored: a decode step that also adds every cached token's attention weight to a running score.
- select_lowest: the cached tokens of least score, outside a protected window of recent ones (what to evict).

The cache holds INT4 tokens (K and V by 32-channel groups of a token) and INT2 tokens (groups of 32 tokens of one
request, requantized from their INT4 values; K by channel over the 32 tokens, V by 32-channel groups of a token).  A
scale is half((max - min) / (2^b - 1)), a zero half(min), a code rint((x - zero) / scale), a value code * scale + zero.
"""
import numpy as np
import torch

own = False

D = 128
DEV = "cuda:0"
SCALE = float(np.float32(1.0 / np.sqrt(128.0)))


def listed():
    base = dict(int2=0.6, dead=0.0)
    return [
        # the next token of one 2K-token conversation, before its K/V are quantized: latency
        dict(base, name="attend 1 after 2K", op="attend", hq=8, hkv=2, batch=1, ctx_lo=2048, ctx_hi=2048, new_lo=1,
             new_hi=1, tree=False, int2=0.5),
        # drafts of uneven length, a continuous batch with evicted tokens
        dict(base, name="attend drafts ragged", op="attend", hq=32, hkv=8, batch=24, ctx_lo=1000, ctx_hi=32768,
             new_lo=1, new_hi=7, tree=False, dead=0.05),
        # a tree of 31 draft tokens per request
        dict(base, name="attend tree 31 x 8 x 32K", op="attend", hq=32, hkv=8, batch=8, ctx_lo=32768, ctx_hi=32768,
             new_lo=31, new_hi=31, tree=True),
        # chunks of several prompts that are half way through
        dict(base, name="attend chunks 300-512", op="attend", hq=32, hkv=8, batch=4, ctx_lo=15000, ctx_hi=32768,
             new_lo=300, new_hi=512, tree=False),
        # a large chunk of one long prompt, 64 q heads
        dict(base, name="attend chunk 2048 at 32K", op="attend", hq=64, hkv=8, batch=1, ctx_lo=32768, ctx_hi=32768,
             new_lo=2048, new_hi=2048, tree=False, int2=0.75),
        # first chunks: nothing cached yet
        dict(base, name="attend first chunks", op="attend", hq=32, hkv=8, batch=4, ctx_lo=0, ctx_hi=0, new_lo=700,
             new_hi=1021, tree=False),
        # one 2K-token conversation: latency
        dict(base, name="scored 1 x 2K", op="scored", hq=8, hkv=2, batch=1, ctx_lo=2048, ctx_hi=2048, decay=1.0,
             int2=0.5),
        # a ragged batch with evicted tokens and fading scores
        dict(base, name="scored 8 x 20K-32K", op="scored", hq=32, hkv=8, batch=8, ctx_lo=20000, ctx_hi=32768,
             decay=0.96875, dead=0.05),
        # long agentic contexts, 64 q heads
        dict(base, name="scored 16 x 100K", op="scored", hq=64, hkv=8, batch=16, ctx_lo=100000, ctx_hi=100000,
             decay=1.0, int2=0.75),
        # a few tokens of one short conversation
        dict(base, name="select 1 x 2K", op="select", hkv=2, batch=1, ctx_lo=2048, ctx_hi=2048, share=0.03125,
             protect=128, per_head=False, int2=0.5),
        # every kv head gives up its own tokens
        dict(base, name="select heads 8 x 20K-32K", op="select", hkv=8, batch=8, ctx_lo=20000, ctx_hi=32768,
             share=0.25, protect=1024, per_head=True, dead=0.05),
        # long contexts, tokens chosen for all kv heads together
        dict(base, name="select 16 x 100K", op="select", hkv=8, batch=16, ctx_lo=100000, ctx_hi=100000, share=0.125,
             protect=4000, per_head=False, int2=0.75, dead=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "scored", "select"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.randint(1, 8)
    hi = _log(rng, 60, 100000)
    lo = rng.randint(max(1, hi // 3), hi)
    cost = hkv * hi
    batch = max(1, min(_log(rng, 1, 32), 8 * 16 * 100000 // cost))
    c = dict(op=op, hkv=hkv, batch=batch, ctx_lo=lo, ctx_hi=hi, int2=round(rng.uniform(0.0, 0.95), 3),
             dead=rng.choice([0.0, 0.02, 0.05, 0.3]))
    if op == "attend":
        most = int(2048 * 34000 * 64 / (batch * (hi + 500.0) * hkv * g))   # products no more than the largest case's
        new = max(1, min(_log(rng, 1, 2048), most, 4000 // batch + 1))
        tree = rng.random() < 0.3
        if tree:
            new = min(new, 64)
        c.update(hq=g * hkv, new_lo=rng.randint(1, new), new_hi=new, tree=tree)
    elif op == "scored":
        c.update(hq=g * hkv, decay=rng.choice([1.0, 0.9, 0.5]))
    else:
        c.update(share=round(rng.uniform(0.01, 0.6), 3), protect=rng.randint(0, lo), per_head=rng.random() < 0.5)
    return c


def _structure(case, seed):
    """Lengths, widths, evicted positions: the host side of the cache, from the seed alone."""
    rng = np.random.default_rng([int(seed), 17])
    B = case["batch"]
    lens = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    lens[0] = case["ctx_hi"]
    bits, dead = [], []
    for n in lens:
        runs = rng.integers(16, 257, int(n) // 16 + 1)
        tags = np.where(rng.random(runs.size) < case["int2"], 2, 4).astype(np.uint8)
        bits.append(np.repeat(tags, runs)[:n].copy())
        dead.append(np.flatnonzero(rng.random(int(n)) < case["dead"]))
    return rng, lens, bits, dead


def _quant(x, levels):
    """x [..., 32] -> codes, scale, zero of the last axis."""
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s, z = ((mx - mn) / levels).half(), mn.half()
    c = ((x - z.float()) / s.float()).round().clamp(0, levels)
    return torch.where(s == 0, torch.zeros_like(c), c).to(torch.uint8), s[..., 0], z[..., 0]


def _value(c, s, z):
    return c.float() * s.float().unsqueeze(-1) + z.float().unsqueeze(-1)


def _cache(case, seed):
    """K and V of every request, quantized: the INT2 part (tokens in groups of 32) and the INT4 part, padded over the
    batch.  Codes [B][H][tokens][128]; pos: the tokens' positions, -1 where there is none or it was evicted."""
    rng, lens, bits, dead = _structure(case, seed)
    B, H = case["batch"], case["hkv"]
    gen = torch.Generator(DEV).manual_seed(int(seed))
    outlier = torch.ones(H, D, device=DEV)
    for h in range(H):
        outlier[h, torch.from_numpy(rng.choice(D, 4, replace=False)).to(DEV)] = 20.0
    n2 = [int((b == 2).sum()) // 32 * 32 for b in bits]
    L2, L4 = max(n2), max([int(n) - m for n, m in zip(lens, n2)] + [0])
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    e16 = lambda *s: torch.zeros(s, dtype=torch.float16, device=DEV)  # noqa: E731
    c = dict(k2=e8(B, H, L2, D), v2=e8(B, H, L2, D), k4=e8(B, H, L4, D), v4=e8(B, H, L4, D),
             k2s=e16(B, H, L2 // 32, D), k2z=e16(B, H, L2 // 32, D), v2s=e16(B, H, L2, 4), v2z=e16(B, H, L2, 4),
             k4s=e16(B, H, L4, 4), k4z=e16(B, H, L4, 4), v4s=e16(B, H, L4, 4), v4z=e16(B, H, L4, 4),
             pos2=torch.full((B, L2), -1, device=DEV), pos4=torch.full((B, L4), -1, device=DEV))
    rows = []
    for r, n in enumerate(int(x) for x in lens):
        k = (torch.randn(n, H, D, generator=gen, device=DEV) * outlier).bfloat16()
        v = torch.randn(n, H, D, generator=gen, device=DEV).bfloat16()
        if own:
            rows.append((k, v))
        gone = np.zeros(n, bool)
        gone[dead[r]] = True
        i2 = np.flatnonzero(bits[r] == 2)[:n2[r]]
        rest = np.ones(n, bool)
        rest[i2] = False
        i4 = np.flatnonzero(rest)
        k4, k4s, k4z = _quant(k.float().view(n, H, 4, 32), 15)
        v4, v4s, v4z = _quant(v.float().view(n, H, 4, 32), 15)
        t4 = torch.from_numpy(i4).to(DEV)
        m4 = i4.size
        for name, x in (("k4", k4), ("v4", v4)):
            c[name][r, :, :m4] = x[t4].reshape(m4, H, D).transpose(0, 1)
        for name, x in (("k4s", k4s), ("k4z", k4z), ("v4s", v4s), ("v4z", v4z)):
            c[name][r, :, :m4] = x[t4].transpose(0, 1)
        c["pos4"][r, :m4] = torch.from_numpy(np.where(gone[i4], -1, i4)).to(DEV)
        if i2.size:
            t2 = torch.from_numpy(i2).to(DEV)
            m2 = i2.size
            kh = _value(k4[t2], k4s[t2], k4z[t2]).view(m2 // 32, 32, H, D).permute(2, 0, 3, 1)   # [H][group][128][32]
            k2, c["k2s"][r, :, :m2 // 32], c["k2z"][r, :, :m2 // 32] = _quant(kh, 3)
            c["k2"][r, :, :m2] = k2.transpose(2, 3).reshape(H, m2, D)
            vh = _value(v4[t2], v4s[t2], v4z[t2]).permute(1, 0, 2, 3)                            # [H][token][4][32]
            v2, c["v2s"][r, :, :m2], c["v2z"][r, :, :m2] = _quant(vh, 3)
            c["v2"][r, :, :m2] = v2.reshape(H, m2, D)
            c["pos2"][r, :m2] = torch.from_numpy(np.where(gone[i2], -1, i2)).to(DEV)
    return c, rng, gen, lens, bits, dead, rows


def _pool(case, lens, bits, dead, rows):
    """The framework's pool, filled with the same rows in chunks, evicted and reordered as a serving program does."""
    import mixed_precision_kv_gb300 as kvq

    pages = int(sum(int(n) // 32 + 4 for n in lens)) + 1024
    pool = kvq.KVPool(case["hkv"], pages, pages, case["batch"], int(max(lens)) // 32 + 64, device=0)
    ids = [pool.open() for _ in lens]
    for r, (k, v) in enumerate(rows):
        n = int(lens[r])
        for t in range(0, n, 16384):
            e = min(n, t + 16384)
            pool.append(k[t:e], v[t:e], np.full(e - t, ids[r], np.int32), bits[r][t:e])
        if dead[r].size:
            pool.evict(np.full(dead[r].size, ids[r], np.int32), dead[r])
    pool.reorder(ids)
    pool.sync()
    return pool, np.asarray(ids, np.int32)


def prepare(case, seed):
    c, rng, gen, lens, bits, dead, rows = _cache(case, seed)
    B, H = case["batch"], case["hkv"]
    s = dict(op=case["op"], H=H, lens=lens)
    if case["op"] == "attend":
        # the batch's shape goes by the case alone
        new = np.random.default_rng([B, case["new_lo"], case["new_hi"]]).integers(case["new_lo"], case["new_hi"] + 1, B)
        new[0] = case["new_hi"]
        N, T = int(new.sum()), int(new.max())
        first = np.concatenate([[0], np.cumsum(new)[:-1]])
        s["q"] = torch.randn(N, case["hq"], D, generator=gen, device=DEV).bfloat16()
        s["k"] = torch.randn(N, H, D, generator=gen, device=DEV).bfloat16()
        s["v"] = torch.randn(N, H, D, generator=gen, device=DEV).bfloat16()
        s["new"] = new.astype(np.int32)
        j = np.arange(T)
        s["at"] = torch.from_numpy(np.minimum(first[:, None] + j, N - 1)).to(DEV)       # [B][T] row of a new token
        s["is"] = torch.from_numpy(j[None] < new[:, None]).to(DEV)
        s["tree"] = None
        if case["tree"]:   # a random tree: every token sees itself and its ancestors
            masks = np.zeros(N, np.uint64)
            for b in range(B):
                for t in range(int(new[b])):
                    up = masks[first[b] + rng.integers(max(0, t - 8), t)] if t and rng.random() < 0.9 else np.uint64(0)
                    masks[first[b] + t] = up | np.uint64(1 << t)
            s["tree"] = torch.from_numpy(masks.view(np.int64)).to(DEV)
    elif case["op"] == "scored":
        s["q"] = torch.randn(B, case["hq"], D, generator=gen, device=DEV).bfloat16()
        s["decay"] = case["decay"]
    if case["op"] != "attend":
        # what a run of earlier steps leaves: few tokens with much weight; some exactly equal
        x = torch.exp(2.0 * torch.randn(B, H, int(max(lens)) + 37, generator=gen, device=DEV) - 6.0)
        s["scores"] = torch.where(x < 2.0 ** -13, torch.zeros_like(x), x)
    if case["op"] == "select":
        s["n"] = np.maximum(1, (lens * case["share"]).astype(np.int64)).astype(np.int32)
        s["protect"], s["per_head"] = case["protect"], case["per_head"]
    if own:
        s["pool"], s["ids"] = _pool(case, lens, bits, dead, rows)
    else:
        s["cache"] = c
    return s


def _dequant(c, w):
    """One of K and V of the whole cache, fp32 [B][H][tokens][128]."""
    B, H, L2, _ = c["k2"].shape
    L4 = c["k4"].shape[2]
    if w == "k":
        x2 = c["k2"].view(B, H, L2 // 32, 32, D).float() * c["k2s"].float().unsqueeze(3) + c["k2z"].float().unsqueeze(3)
    else:
        x2 = _value(c["v2"].view(B, H, L2, 4, 32), c["v2s"], c["v2z"])
    x4 = _value(c[w + "4"].view(B, H, L4, 4, 32), c[w + "4s"], c[w + "4z"])
    return torch.cat([x2.reshape(B, H, L2, D), x4.reshape(B, H, L4, D)], 2)


def _softmax(x):
    """Weights of the last axis and their sum; a row with nothing in it is all zero."""
    m = x.amax(-1, keepdim=True).clamp_min(-3.0e38)
    x.sub_(m).exp_()
    return x, x.sum(-1, keepdim=True)


def _attend(s):
    c, q, at = s["cache"], s["q"], s["at"]
    B, T = at.shape
    H, g = s["H"], q.shape[1] // s["H"]
    pos = torch.cat([c["pos2"], c["pos4"]], 1)
    L = pos.shape[1]
    qr = q.float()[at].view(B, T, H, g, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * g, D)
    kn, vn = (x.float()[at].transpose(1, 2) for x in (s["k"], s["v"]))
    x = torch.empty(B, H, T * g, L + T, device=q.device)
    torch.matmul(qr, _dequant(c, "k").transpose(2, 3), out=x[..., :L])
    x[..., L:] = qr @ kn.transpose(2, 3)
    x.mul_(SCALE)
    j = torch.arange(T, device=q.device)
    if s["tree"] is None:
        see = (j[None, :] <= j[:, None]).expand(B, T, T)
    else:
        see = (s["tree"][at].unsqueeze(-1) >> j) & 1 != 0
    see = see & s["is"][:, None, :]
    x[..., :L].masked_fill_((pos < 0)[:, None, None, :], -torch.inf)
    x.view(B, H, T, g, L + T)[..., L:].masked_fill_(~see[:, None, :, None, :], -torch.inf)
    p, l = _softmax(x)
    o = (p @ torch.cat([_dequant(c, "v"), vn], 2)) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.view(B, H, T, g, D).permute(0, 2, 1, 3, 4)[s["is"]]
    return o.reshape(-1, H * g, D).bfloat16()


def _scored(s):
    c, q = s["cache"], s["q"]
    B, H, g = q.shape[0], s["H"], q.shape[1] // s["H"]
    pos = torch.cat([c["pos2"], c["pos4"]], 1)
    x = (q.float().view(B, H, g, D) @ _dequant(c, "k").transpose(2, 3)).mul_(SCALE)
    x.masked_fill_((pos < 0)[:, None, None, :], -torch.inf)
    p, l = _softmax(x)
    l = torch.where(l > 0, l, torch.ones_like(l))
    out = (p @ _dequant(c, "v")) / l
    w = (p / l).sum(2)                                         # [B][H][tokens]
    b, t = (pos >= 0).nonzero(as_tuple=True)
    at = pos[b, t]
    s["scores"][b, :, at] = s["scores"][b, :, at] * s["decay"] + w[b, :, t]
    return dict(out=out.reshape(B, H * g, D), scores=s["scores"])


def _select(s):
    c, scores = s["cache"], s["scores"]
    B, H, S = scores.shape
    can = torch.zeros(B, S, dtype=torch.bool, device=scores.device)
    pos = torch.cat([c["pos2"], c["pos4"]], 1)
    b, t = (pos >= 0).nonzero(as_tuple=True)
    can[b, pos[b, t]] = True
    lens = torch.as_tensor(s["lens"], device=scores.device)
    can &= torch.arange(S, device=scores.device) < (lens - s["protect"])[:, None]
    # all heads together: the sum in 64 bits, rounded once
    key = scores if s["per_head"] else scores.double().sum(1, keepdim=True).float()
    key = key.masked_fill(~can[:, None], torch.inf)
    n = int(s["n"].max())
    at = torch.sort(key, dim=-1, stable=True).indices[..., :n]
    have = torch.minimum(torch.as_tensor(s["n"], device=scores.device), can.sum(1))[:, None, None]
    at = at.masked_fill(torch.arange(at.shape[-1], device=at.device) >= have, S)
    at = torch.sort(at, dim=-1).values
    at = at.masked_fill(at == S, -1).int()
    return at if s["per_head"] else at[:, 0]


def run(s):
    if own:
        if s["op"] == "attend":
            return s["pool"].attend(s["q"], s["ids"], s["new"], SCALE, s["k"], s["v"], tree=s["tree"])
        if s["op"] == "scored":
            out = s["pool"].decode_scored(s["q"], s["ids"], SCALE, s["scores"], decay=s["decay"])
            return dict(out=out, scores=s["scores"])
        return s["pool"].select_lowest(s["scores"], s["ids"], s["n"], protect=s["protect"], per_head=s["per_head"])
    return {"attend": _attend, "scored": _scored, "select": _select}[s["op"]](s)


def exact(case, seed):
    """From the definition, in 64 bits, one request and kv head at a time."""
    if case["op"] == "select":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, q, H = s["cache"], s["q"].double(), case["hkv"]
    g = q.shape[1] // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    scores = s["scores"].double() if "scores" in s else None
    row = 0
    for b in range(case["batch"]):
        T = int(s["new"][b]) if "new" in s else 1
        p2, p4 = c["pos2"][b], c["pos4"][b]
        i2, i4 = (p2 >= 0).nonzero()[:, 0], (p4 >= 0).nonzero()[:, 0]
        for h in range(H):
            def per_token(name, i):
                sc, z = c[name + "s"][b, h, i].double(), c[name + "z"][b, h, i].double()
                return c[name][b, h, i].double() * sc.repeat_interleave(32, -1) + z.repeat_interleave(32, -1)

            k2 = c["k2"][b, h, i2].double() * c["k2s"][b, h, i2 // 32].double() + c["k2z"][b, h, i2 // 32].double()
            K = torch.cat([k2, per_token("k4", i4)])
            V = torch.cat([per_token("v2", i2), per_token("v4", i4)])
            n = K.shape[0]
            Q = q[row:row + T, h * g:(h + 1) * g].reshape(T * g, D)
            if "new" in s:
                K = torch.cat([K, s["k"][row:row + T, h].double()])
                V = torch.cat([V, s["v"][row:row + T, h].double()])
            x = (Q @ K.T) * SCALE
            if "new" in s:
                for t in range(T):
                    if s["tree"] is None:
                        x[t * g:(t + 1) * g, n + t + 1:] = -torch.inf
                    else:
                        m = int(s["tree"][row + t])
                        hide = [n + j for j in range(T) if not (m >> j) & 1]
                        x[t * g:(t + 1) * g, hide] = -torch.inf
            if x.shape[1] == 0:
                continue
            w = torch.softmax(x, -1).nan_to_num(0.0)
            out[row:row + T, h * g:(h + 1) * g] = (w @ V).view(T, g, D)
            if scores is not None:
                at = torch.cat([p2[i2], p4[i4]])
                scores[b, h, at] = scores[b, h, at] * case["decay"] + w.sum(0)
        row += T
    return dict(out=out, scores=scores) if scores is not None else out


def work(case):
    """Every page, q, new row and score read once, every output written once."""
    B, H = case["batch"], case["hkv"]
    ctx = B * (case["ctx_lo"] + case["ctx_hi"]) / 2.0
    token = case["int2"] * 96.0 + (1 - case["int2"]) * 160.0     # codes, scales and zeros of a token and kv head
    if case["op"] == "select":
        n = case["share"] * ctx * (H if case["per_head"] else 1)
        return dict(bytes=4.0 * H * ctx + ctx / 8 + 4.0 * n, flops=H * ctx)
    if case["op"] == "scored":
        return dict(bytes=H * ctx * (token + 8.0) + B * case["hq"] * D * 6.0, flops=4.0 * D * case["hq"] * ctx)
    T = (case["new_lo"] + case["new_hi"]) / 2.0
    pairs = T * ctx + B * T * (T + 1) / 2
    return dict(bytes=H * ctx * token + B * T * D * (case["hq"] * 4.0 + H * 4.0), flops=4.0 * D * case["hq"] * pairs)
