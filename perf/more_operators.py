"""Cases and plain forms of the operators that fill a mixed-precision cache with rotated keys and share what it holds:

- rotate: rotary positions applied to q and k, with one or several position axes (time, height, width).
- append: a prompt's or a step's keys and values quantized into the cache, the keys rotated on the way; then the cached
  values, read back.
- read: cached tokens' values, dequantized, by token position.
- shared: new tokens (or the single tokens of a decode step) of a batch attend to a cached prefix that several of them
  share, to their own cached tokens and to each other.

Rotation: channels (i, i + R / 2), or (2 i, 2 i + 1), of the first R of a head's 128 are a pair (a, b) that becomes
(a cos - b sin, b cos + a sin), with the cosine and sine of frequency i at the token's position on the frequency's axis,
from a table.  A rotated key is rounded to bf16, as q is, before it is quantized.

The cache holds INT4 tokens (K and V by 32-channel groups of a token) and INT2 tokens (groups of 32 tokens of one request,
requantized from their INT4 values; K by channel over the 32 tokens, V by 32-channel groups of a token).  A scale is
half((max - min) / (2^b - 1)), a zero half(min), a code rint((x - zero) / scale), a value code * scale + zero.
"""
import numpy as np
import torch

own = False

D = 128
DEV = "cuda:0"
SCALE = float(np.float32(1.0 / np.sqrt(128.0)))


def listed():
    rot = dict(rot=128, axes=1, pairs=False, mix=False, start=0, packed=True)
    sh = dict(op="shared", int2=0.6, dead=0.0, lone=0.0, new_lo=1, new_hi=1, cached=False, tree=False)
    return [
        # q and k of one token of a conversation, slices of one projection's output: latency
        dict(rot, name="rotate 1 token", op="rotate", hq=8, hkv=2, n=1, start=2048),
        # a chunk of a prompt with images and video: three axes, their frequencies interleaved
        dict(rot, name="rotate 4000, 3 axes", op="rotate", hq=32, hkv=8, n=4000, axes=3, mix=True),
        # a large chunk of a long prompt, 64 q heads, far positions
        dict(rot, name="rotate 16K far", op="rotate", hq=64, hkv=8, n=16384, start=100000, packed=False),
        # the first tokens of short turns, a continuous batch
        dict(rot, name="append 24 x 1-9", op="append", hkv=8, batch=24, lo=1, hi=9, int2=0.3, start=500),
        # prompts with images, half of each head rotated, neighbouring channels paired
        dict(rot, name="append 5 x 300-2000, 3 axes", op="append", hkv=8, batch=5, lo=300, hi=2000, int2=0.6, rot=64,
             axes=3, pairs=True),
        # whole long prompts
        dict(rot, name="append 8 x 32K", op="append", hkv=8, batch=8, lo=32768, hi=32768, int2=0.6, packed=False),
        # the newest tokens of a short conversation
        dict(name="read 64 of 2K", op="read", hkv=2, batch=1, ctx_lo=2048, ctx_hi=2048, share=0.03125, int2=0.5, dead=0.0),
        # whole requests, some tokens evicted (moving them elsewhere)
        dict(name="read 8 x 20K-32K", op="read", hkv=8, batch=8, ctx_lo=20000, ctx_hi=32768, share=1.0, int2=0.6,
             dead=0.05),
        # four samples of one 2K prompt, a few tokens each: latency
        dict(sh, name="shared 4 x 2K", hq=8, hkv=2, batch=4, prefixes=1, pre_lo=2048, pre_hi=2048, ctx_lo=0, ctx_hi=100,
             cached=True, int2=0.5),
        # drafts of uneven length, three system prompts, some requests without one, evicted tokens
        dict(sh, name="shared drafts ragged", hq=32, hkv=8, batch=24, prefixes=3, pre_lo=2000, pre_hi=16000, ctx_lo=50,
             ctx_hi=4000, new_lo=1, new_hi=7, lone=0.15, dead=0.05),
        # 32 samples of one 32K document
        dict(sh, name="shared 32 x 32K", hq=32, hkv=8, batch=32, prefixes=1, pre_lo=32768, pre_hi=32768, ctx_lo=100,
             ctx_hi=2000, cached=True),
        # 64 samples of one 100K context, 64 q heads
        dict(sh, name="shared 64 x 100K", hq=64, hkv=8, batch=64, prefixes=1, pre_lo=100000, pre_hi=100000, ctx_lo=500,
             ctx_hi=1500, cached=True, int2=0.75),
    ]


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "read", "shared", "shared"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.randint(1, 8)
    if op in ("rotate", "append"):
        axes = rng.choice([1, 1, 2, 3])
        c = dict(op=op, hkv=hkv, rot=rng.choice([128, 128, 96, 64, 32, 16]), axes=axes, pairs=rng.random() < 0.3,
                 mix=axes > 1 and rng.random() < 0.5, start=rng.choice([0, 0, _log(rng, 1, 120000)]),
                 packed=rng.random() < 0.6)
        if op == "rotate":
            c.update(hq=g * hkv, n=_log(rng, 1, 16384))
        else:
            batch = _log(rng, 1, 32)
            hi = _log(rng, 1, min(32768, 8 * 32768 // batch))
            c.update(batch=batch, lo=rng.randint(max(1, hi // 3), hi), hi=hi, int2=round(rng.uniform(0.0, 0.95), 3))
        return c
    dead, int2 = rng.choice([0.0, 0.02, 0.05, 0.3]), round(rng.uniform(0.0, 0.95), 3)
    if op == "read":
        hi = _log(rng, 40, 32768)
        batch = _log(rng, 1, max(1, min(32, 8 * 26000 // hi)))
        return dict(op=op, hkv=hkv, batch=batch, ctx_lo=rng.randint(max(1, hi // 3), hi), ctx_hi=hi,
                    share=round(_log(rng, 10, 1000) / 1000.0, 3), int2=int2, dead=dead)
    pre = _log(rng, 60, 100000)
    most = max(1, min(64, int(64 * 100000 * 64 / (pre * hkv * g + 1))))      # no more than the largest case's products
    batch = _log(rng, 1, most)
    ctx = _log(rng, 1, 4000)
    cached = rng.random() < 0.5
    new = 1 if cached else max(1, min(_log(rng, 1, 64), 4 * most // batch))
    return dict(op=op, hq=g * hkv, hkv=hkv, batch=batch, prefixes=rng.randint(1, min(4, batch)), pre_lo=rng.randint(pre // 2, pre),
                pre_hi=pre, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, new_lo=rng.randint(1, new), new_hi=new, cached=cached,
                tree=not cached and rng.random() < 0.3, lone=rng.choice([0.0, 0.0, 0.2]), int2=int2, dead=dead)


# ---- rotation ------------------------------------------------------------------------------------------------------

def _rotation(case, lens, rng, gen):
    """The table [positions][R] (cosines, then sines), the frequencies' axes and the tokens' positions [axes][n]."""
    R, A, half = case["rot"], case["axes"], case["rot"] // 2
    rows = case["start"] + int(max(lens)) + 1
    inv = torch.tensor(500000.0, dtype=torch.float64, device=DEV) ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    axis = np.arange(half) % A if case["mix"] else np.arange(half) * A // half
    pos = np.empty((A, int(sum(lens))), np.int32)
    at = 0
    for n in (int(x) for x in lens):
        j = np.arange(n)
        if A == 1:
            pos[0, at:at + n] = case["start"] + j
        else:   # text and, in every second run of 800 tokens, frames of 20 x 20 patches
            off = int(rng.integers(0, 1600))
            pic = (j + off) // 800 % 2 == 1
            first = np.minimum(j // 800 * 800, n - 1)
            p = (j + off) % 400
            pos[0, at:at + n] = case["start"] + np.where(pic, first // 4, j // 2)
            pos[1, at:at + n] = case["start"] + np.where(pic, np.minimum(first // 4 + p // 20, n - 1), j // 2)
            if A > 2:
                pos[2, at:at + n] = case["start"] + np.where(pic, np.minimum(first // 4 + p % 20, n - 1), j // 2)
        at += n
    return table, axis.astype(np.uint8), torch.from_numpy(pos).to(DEV)


def _factors(s):
    """Cosines and sines of every token and frequency, fp32 [n][1][R / 2]."""
    half = s["table"].shape[1] // 2
    row = s["pos"].long()[torch.from_numpy(s["axis"].astype(np.int64)).to(DEV)].T          # [n][R / 2]
    i = torch.arange(half, device=DEV)
    return s["table"][row, i].unsqueeze(1), s["table"][row, i + half].unsqueeze(1)


def _rotate(x, cos, sin, pairs):
    """bf16 [n][heads][128], its first R channels rotated in fp32 and rounded once."""
    half = cos.shape[-1]
    f = x.float()
    a, b = (f[..., 0:2 * half:2], f[..., 1:2 * half:2]) if pairs else (f[..., :half], f[..., half:2 * half])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([r, f[..., 2 * half:]], -1).bfloat16()


# ---- quantization --------------------------------------------------------------------------------------------------

def _quant(x, levels):
    """x [..., 32] -> codes, scale, zero of the last axis."""
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s, z = ((mx - mn) / levels).half(), mn.half()
    c = ((x - z.float()) / s.float()).round().clamp(0, levels)
    return torch.where(s == 0, torch.zeros_like(c), c).to(torch.uint8), s[..., 0], z[..., 0]


def _value(c, s, z):
    return c.float() * s.float().unsqueeze(-1) + z.float().unsqueeze(-1)


def _widths(rng, lens, share):
    """Bits of every token, by runs."""
    bits = []
    for n in lens:
        runs = rng.integers(16, 257, int(n) // 16 + 1)
        bits.append(np.repeat(np.where(rng.random(runs.size) < share, 2, 4).astype(np.uint8), runs)[:n].copy())
    return bits


def _heads(gen, rng, n, H, outlier=None):
    """A layer's keys (four channels of every head large) or values."""
    x = torch.randn(n, H, D, generator=gen, device=DEV)
    return (x if outlier is None else x * outlier).bfloat16()


def _outlier(rng, H):
    m = torch.ones(H, D, device=DEV)
    for h in range(H):
        m[h, torch.from_numpy(rng.choice(D, 4, replace=False)).to(DEV)] = 20.0
    return m


def _values(k, v, bits, req):
    """The values that a cache of these tokens stands for, bf16 [n][H][128] each: all requests at once."""
    n, H = k.shape[:2]
    two = bits == 2
    rank = np.cumsum(two) - 1                              # among the INT2 tokens of the call
    per = np.bincount(req, two, minlength=int(req.max()) + 1).astype(np.int64)
    rank = rank - (np.cumsum(per) - per)[req]
    i2 = torch.from_numpy(np.flatnonzero(two & (rank < (per // 32 * 32)[req]))).to(DEV)
    out = []
    for x, by_channel in ((k, True), (v, False)):
        y = _value(*_quant(x.float().view(n, H, 4, 32), 15)).view(n, H, D)
        if i2.numel():
            t = y[i2]
            if by_channel:
                t = _value(*_quant(t.view(-1, 32, H, D).permute(0, 2, 3, 1), 3)).permute(0, 3, 1, 2).reshape(-1, H, D)
            else:
                t = _value(*_quant(t.view(-1, H, 4, 32), 3)).view(-1, H, D)
            y[i2] = t
        out.append(y.bfloat16())
    return out


# ---- a cache in hand: codes, scales, zeros and positions -----------------------------------------------------------

def _cache(lens, H, share, dead_share, rng, gen):
    """K and V of every request, quantized: the INT2 part (tokens in groups of 32) and the INT4 part, padded over the
    requests.  Codes [B][H][tokens][128]; pos: the tokens' positions, -1 where there is none or it was evicted."""
    B = len(lens)
    bits = _widths(rng, lens, share)
    dead = [np.flatnonzero(rng.random(int(n)) < dead_share) for n in lens]
    outlier = _outlier(rng, H)
    n2 = [int((b == 2).sum()) // 32 * 32 for b in bits]
    L2, L4 = max(n2 + [0]), max([int(n) - m for n, m in zip(lens, n2)] + [0])
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    e16 = lambda *s: torch.zeros(s, dtype=torch.float16, device=DEV)  # noqa: E731
    c = dict(k2=e8(B, H, L2, D), v2=e8(B, H, L2, D), k4=e8(B, H, L4, D), v4=e8(B, H, L4, D),
             k2s=e16(B, H, L2 // 32, D), k2z=e16(B, H, L2 // 32, D), v2s=e16(B, H, L2, 4), v2z=e16(B, H, L2, 4),
             k4s=e16(B, H, L4, 4), k4z=e16(B, H, L4, 4), v4s=e16(B, H, L4, 4), v4z=e16(B, H, L4, 4),
             pos2=torch.full((B, L2), -1, device=DEV), pos4=torch.full((B, L4), -1, device=DEV))
    rows = []
    for r, n in enumerate(int(x) for x in lens):
        k, v = _heads(gen, rng, n, H, outlier), _heads(gen, rng, n, H)
        if own:
            rows.append((k, v))
        gone = np.zeros(n, bool)
        gone[dead[r]] = True
        i2 = np.flatnonzero(bits[r] == 2)[:n2[r]]
        rest = np.ones(n, bool)
        rest[i2] = False
        i4 = np.flatnonzero(rest)
        k4, k4s, k4z = _quant(k.float().view(n, H, 4, 32), 15) if n else (e8(0, H, 4, 32), e16(0, H, 4), e16(0, H, 4))
        v4, v4s, v4z = _quant(v.float().view(n, H, 4, 32), 15) if n else (e8(0, H, 4, 32), e16(0, H, 4), e16(0, H, 4))
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
    return c, dict(lens=lens, bits=bits, dead=dead, rows=rows)


def _pool(H, *made):
    """The framework's pool, filled with the same rows in chunks, evicted and reordered as a serving program does."""
    import mixed_precision_kv_gb300 as kvq

    lens = [int(n) for m in made for n in m["lens"]]
    pages = sum(n // 32 + 4 for n in lens) + 1024
    pool = kvq.KVPool(H, pages, pages, len(lens), max(lens) // 32 + 64, device=0)
    ids = []
    for m in made:
        here = [pool.open() for _ in m["lens"]]
        for r, (k, v) in enumerate(m["rows"]):
            n = int(m["lens"][r])
            for t in range(0, n, 16384):
                e = min(n, t + 16384)
                pool.append(k[t:e], v[t:e], np.full(e - t, here[r], np.int32), m["bits"][r][t:e])
            if m["dead"][r].size:
                pool.evict(np.full(m["dead"][r].size, here[r], np.int32), m["dead"][r])
        ids.append(np.asarray(here, np.int32))
    pool.reorder(np.concatenate(ids))
    pool.sync()
    return pool, ids


def _lens(rng, lo, hi, n):
    x = rng.integers(lo, hi + 1, n)
    x[0] = hi
    return x


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 29])
    gen = torch.Generator(DEV).manual_seed(int(seed))
    op, H = case["op"], case["hkv"]
    s = dict(op=op, H=H)
    if op in ("rotate", "append"):
        # a batch's lengths go by the case alone
        lens = [case["n"]] if op == "rotate" else _lens(np.random.default_rng([case["batch"], case["hi"]]), case["lo"], case["hi"], case["batch"])
        s["table"], s["axis"], s["pos"] = _rotation(case, lens, rng, gen)
        s["pairs"] = case["pairs"]
        n, hq = int(sum(lens)), case.get("hq", H)
        k, v = _heads(gen, rng, n, H, _outlier(rng, H)), _heads(gen, rng, n, H)
        if case["packed"]:   # one projection's output: q, k and v of a token side by side
            x = torch.cat([torch.randn(n, hq, D, generator=gen, device=DEV).bfloat16(), k, v], 1)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + H], x[:, hq + H:]
        else:
            s["q"], s["k"], s["v"] = torch.randn(n, hq, D, generator=gen, device=DEV).bfloat16(), k, v
        if op == "append":
            s["lens"] = np.asarray(lens, np.int64)
            s["bits"] = np.concatenate(_widths(rng, lens, case["int2"]))
        if own:
            import mixed_precision_kv_gb300 as kvq

            pages = sum(int(x) // 32 + 4 for x in lens) + 16
            s["pool"] = kvq.KVPool(H, pages, pages, len(lens), int(max(lens)) // 32 + 8, device=0)
            s["rope"] = kvq.Rope(s["table"], axis=s["axis"], interleaved=case["pairs"])
        return s
    if op == "read":
        # a batch's lengths go by the case alone
        lens = _lens(np.random.default_rng([case["batch"], case["ctx_hi"]]), case["ctx_lo"], case["ctx_hi"], case["batch"])
        s["lens"] = lens
        s["n"] = np.maximum(1, (lens * case["share"]).astype(np.int64))
        s["first"] = lens - s["n"]                          # the newest tokens
        c, made = _cache(lens, H, case["int2"], case["dead"], rng, gen)
        if own:
            s["pool"], (s["ids"],) = _pool(H, made)
        else:
            s["cache"] = c
        return s
    B, P = case["batch"], case["prefixes"]
    fix = np.random.default_rng([B, P, case["new_lo"], case["new_hi"]])      # the batch's shape goes by the case alone
    pre, lens = _lens(rng, case["pre_lo"], case["pre_hi"], P), _lens(rng, case["ctx_lo"], case["ctx_hi"], B)
    new = _lens(fix, case["new_lo"], case["new_hi"], B)
    of = fix.permutation(np.arange(B) % P)                  # requests of a prefix need not stand together
    of = np.where(fix.random(B) < case["lone"], -1, of)
    of[0] = 0
    N, T = int(new.sum()), int(new.max())
    first = np.concatenate([[0], np.cumsum(new)[:-1]])
    s["q"] = torch.randn(N, case["hq"], D, generator=gen, device=DEV).bfloat16()
    s["k"], s["v"] = (None, None) if case["cached"] else (_heads(gen, rng, N, H), _heads(gen, rng, N, H))
    s["new"], s["of"] = new.astype(np.int32), of
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
    cp, mp = _cache(pre, H, case["int2"], case["dead"], rng, gen)
    co, mo = _cache(lens, H, case["int2"], case["dead"], rng, gen)
    if own:
        s["pool"], (pids, s["ids"]) = _pool(H, mp, mo)
        s["prefix"] = np.where(of < 0, -1, pids[np.maximum(of, 0)]).astype(np.int32)
    else:
        s["pre"], s["cache"] = cp, co
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------------

def _dequant(c, w):
    """One of K and V of a whole cache, fp32 [B][H][tokens][128]."""
    B, H, L2, _ = c["k2"].shape
    L4 = c["k4"].shape[2]
    if w == "k":
        x2 = c["k2"].view(B, H, L2 // 32, 32, D).float() * c["k2s"].float().unsqueeze(3) + c["k2z"].float().unsqueeze(3)
    else:
        x2 = _value(c["v2"].view(B, H, L2, 4, 32), c["v2s"], c["v2z"])
    x4 = _value(c[w + "4"].view(B, H, L4, 4, 32), c[w + "4s"], c[w + "4z"])
    return torch.cat([x2.reshape(B, H, L2, D), x4.reshape(B, H, L4, D)], 2)


def _positions(c):
    return torch.cat([c["pos2"], c["pos4"]], 1)


def _read(s):
    c = s["cache"]
    pos = _positions(c)
    first, n = (torch.from_numpy(s[x]).to(DEV) for x in ("first", "n"))
    b, t = ((pos >= first[:, None]) & (pos < (first + n)[:, None])).nonzero(as_tuple=True)
    to = (torch.cumsum(n, 0) - n)[b] + pos[b, t] - first[b]
    out = {}
    for w in ("k", "v"):
        out[w] = torch.zeros(int(s["n"].sum()), s["H"], D, dtype=torch.bfloat16, device=DEV)
        out[w][to] = _dequant(c, w)[b, :, t].bfloat16()
    return out


def _shared(s):
    """The prefixes' logits for the rows of all their requests in one product each, and the weighted sums too."""
    cp, co, q, H = s["pre"], s["cache"], s["q"], s["H"]
    B, T = s["at"].shape
    g, P = q.shape[1] // H, cp["k2"].shape[0]
    # rows by prefix: request b is the r-th of its prefix
    of = torch.from_numpy(s["of"]).to(DEV)
    has = of >= 0
    one = (of[:, None] == torch.arange(P, device=DEV)) & has[:, None]
    slot = ((torch.cumsum(one, 0) - 1) * one).sum(1)
    M = max(1, int(np.bincount(s["of"][s["of"] >= 0], minlength=1).max()))
    p_at = of.clamp_min(0)
    qr = q.float()[s["at"]].view(B, T, H, g, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * g, D)
    qp = torch.zeros(P, M, H, T * g, D, device=DEV)
    qp[p_at[has], slot[has]] = qr[has]
    Lp, L = cp["k2"].shape[2] + cp["k4"].shape[2], co["k2"].shape[2] + co["k4"].shape[2]
    xp = (qp.transpose(1, 2).reshape(P, H, M * T * g, D) @ _dequant(cp, "k").transpose(2, 3)).mul_(SCALE)
    xp.masked_fill_((_positions(cp) < 0)[:, None, None, :], -torch.inf)
    xo = (qr @ _dequant(co, "k").transpose(2, 3)).mul_(SCALE)
    xo.masked_fill_((_positions(co) < 0)[:, None, None, :], -torch.inf)
    if s["k"] is not None:
        kn, vn = (x.float()[s["at"]].transpose(1, 2) for x in (s["k"], s["v"]))
        j = torch.arange(T, device=DEV)
        see = (j[None, :] <= j[:, None]).expand(B, T, T) if s["tree"] is None else (s["tree"][s["at"]].unsqueeze(-1) >> j) & 1 != 0
        see = see & s["is"][:, None, :]
        xn = ((qr @ kn.transpose(2, 3)) * SCALE).view(B, H, T, g, T).masked_fill(~see[:, None, :, None, :], -torch.inf)
        xo = torch.cat([xo, xn.view(B, H, T * g, T)], 3)
        vo = torch.cat([_dequant(co, "v"), vn], 2)
    else:
        vo = _dequant(co, "v")
    # maxima and sums of both parts, per request
    low = -3.0e38
    mp = xp.amax(-1, keepdim=True).clamp_min(low) if Lp else torch.full((P, H, M * T * g, 1), low, device=DEV)
    xp.sub_(mp).exp_()
    rows = lambda x: torch.where(has[:, None, None, None], x.view(P, H, M, T * g, -1).transpose(1, 2)[p_at, slot], 0.0)  # noqa: E731
    op, lp = rows(xp @ _dequant(cp, "v")), rows(xp.sum(-1, keepdim=True))
    mp = torch.where(has[:, None, None, None], mp.view(P, H, M, T * g, 1).transpose(1, 2)[p_at, slot], low)
    mo = xo.amax(-1, keepdim=True).clamp_min(low) if xo.shape[-1] else torch.full_like(mp, low)
    xo = (xo - mo).exp_()
    m = torch.maximum(mp, mo)
    fp, fo = (mp - m).exp_(), (mo - m).exp_()
    l = lp * fp + xo.sum(-1, keepdim=True) * fo
    o = (op * fp + (xo @ vo) * fo) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.view(B, H, T, g, D).permute(0, 2, 1, 3, 4)[s["is"]]
    return o.reshape(-1, H * g, D).bfloat16()


def run(s):
    if own:
        pool = s["pool"]
        if s["op"] == "rotate":
            q, k = pool.rotate(s["q"], s["rope"], s["pos"], k=s["k"])
            return dict(q=q, k=k)
        if s["op"] == "append":
            ids = np.array([pool.open() for _ in s["lens"]], np.int32)
            pool.append_rotated(s["k"], s["v"], np.repeat(ids, s["lens"]), s["bits"], s["rope"], s["pos"])
            k, v = pool.read(ids)
            for r in ids:
                pool.close_request(r)
            return dict(k=k, v=v)
        if s["op"] == "read":
            k, v = pool.read(s["ids"], s["first"], s["n"])
            return dict(k=k, v=v)
        return pool.attend_shared(s["q"], s["ids"], s["prefix"], s["new"], SCALE, s["k"], s["v"], tree=s["tree"])
    if s["op"] == "rotate":
        cos, sin = _factors(s)
        return dict(q=_rotate(s["q"], cos, sin, s["pairs"]), k=_rotate(s["k"], cos, sin, s["pairs"]))
    if s["op"] == "append":
        k = _rotate(s["k"], *_factors(s), s["pairs"])
        k, v = _values(k, s["v"], s["bits"], np.repeat(np.arange(s["lens"].size), s["lens"]))
        return dict(k=k, v=v)
    return _read(s) if s["op"] == "read" else _shared(s)


# ---- from the definitions, in 64 bits ------------------------------------------------------------------------------

def _exact_rotate(x, s):
    """As complex numbers."""
    half = s["table"].shape[1] // 2
    t = s["table"].double()
    at = s["pos"].long()
    f = torch.empty(x.shape[0], 1, half, dtype=torch.complex128, device=DEV)
    for i in range(half):
        row = t[at[int(s["axis"][i])]]
        f[:, 0, i] = torch.complex(row[:, i], row[:, half + i])
    y = x.double().clone()
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["pairs"] else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * f
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_levels(x, axis, b):
    """Quantized along an axis and back; scale and zero in binary16."""
    top = 2 ** b - 1
    lo, hi = x.amin(axis, keepdim=True), x.amax(axis, keepdim=True)
    step, zero = ((hi - lo) / top).half().double(), lo.half().double()
    code = torch.where(step > 0, ((x - zero) / torch.where(step > 0, step, torch.ones_like(step))).round().clamp(0, top), torch.zeros_like(x))
    return code * step + zero


def _exact_cached(k, v, bits):
    """One request's tokens [n][H][128]: what the cache stands for."""
    out = []
    for x, two_axis in ((k, 1), (v, -1)):
        n, H = x.shape[:2]
        y = _exact_levels(x.double().view(n, H, 4, 32), -1, 4).view(n, H, D)
        i2 = torch.from_numpy(np.flatnonzero(bits == 2)).to(DEV)
        i2 = i2[:i2.numel() // 32 * 32]
        if two_axis == 1:
            y[i2] = _exact_levels(y[i2].view(-1, 32, H, D), 1, 2).view(-1, H, D)
        else:
            y[i2] = _exact_levels(y[i2].view(-1, H, 4, 32), -1, 2).view(-1, H, D)
        out.append(y)
    return out


def _exact_live(c, r, h, w):
    """K or V of a request's live tokens for a head, in the order of the cache, and their positions."""
    i2, i4 = (c["pos2"][r] >= 0).nonzero()[:, 0], (c["pos4"][r] >= 0).nonzero()[:, 0]

    def per_token(name, i):
        sc, z = c[name + "s"][r, h, i].double(), c[name + "z"][r, h, i].double()
        return c[name][r, h, i].double() * sc.repeat_interleave(32, -1) + z.repeat_interleave(32, -1)

    two = c["k2"][r, h, i2].double() * c["k2s"][r, h, i2 // 32].double() + c["k2z"][r, h, i2 // 32].double() if w == "k" else per_token("v2", i2)
    return torch.cat([two, per_token(w + "4", i4)]), torch.cat([c["pos2"][r, i2], c["pos4"][r, i4]])


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, H = case["op"], case["hkv"]
    if op == "rotate":
        return dict(q=_exact_rotate(s["q"], s), k=_exact_rotate(s["k"], s))
    if op == "append":
        ks, vs, at = [], [], 0
        for n in (int(x) for x in s["lens"]):
            e = at + n
            part = dict(s, pos=s["pos"][:, at:e])
            k, v = _exact_cached(_exact_rotate(s["k"][at:e], part).bfloat16(), s["v"][at:e], s["bits"][at:e])
            ks.append(k.float())     # (values of at most 16 bits' precision: nothing is lost beside the result's bf16)
            vs.append(v.float())
            at = e
        return dict(k=torch.cat(ks).double(), v=torch.cat(vs).double())
    if op == "read":
        out = {}
        for w in ("k", "v"):
            parts = []
            for r, (a, n) in enumerate(zip(s["first"], s["n"])):
                y = torch.zeros(int(n), H, D, dtype=torch.float64, device=DEV)
                for h in range(H):
                    x, pos = _exact_live(s["cache"], r, h, w)
                    take = pos >= int(a)
                    y[pos[take] - int(a), h] = x[take]
                parts.append(y)
            out[w] = torch.cat(parts)
        return out
    q = s["q"].double()
    g = q.shape[1] // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    first = np.concatenate([[0], np.cumsum(s["new"])[:-1]])
    for p in sorted(set(int(x) for x in s["of"])):
        mine = [b for b in range(case["batch"]) if s["of"][b] == p]
        for h in range(H):
            Kp, Vp = (_exact_live(s["pre"], p, h, w)[0] if p >= 0 else torch.zeros(0, D, dtype=torch.float64, device=DEV) for w in "kv")
            for b in mine:
                r0, T = int(first[b]), int(s["new"][b])
                K, V = torch.cat([Kp, _exact_live(s["cache"], b, h, "k")[0]]), torch.cat([Vp, _exact_live(s["cache"], b, h, "v")[0]])
                n = K.shape[0]
                if s["k"] is not None:
                    K, V = torch.cat([K, s["k"][r0:r0 + T, h].double()]), torch.cat([V, s["v"][r0:r0 + T, h].double()])
                if K.shape[0] == 0:
                    continue
                x = (q[r0:r0 + T, h * g:(h + 1) * g].reshape(T * g, D) @ K.T) * SCALE
                if s["k"] is not None:
                    for t in range(T):
                        hide = [n + j for j in range(T) if (j > t if s["tree"] is None else not (int(s["tree"][r0 + t]) >> j) & 1)]
                        x[t * g:(t + 1) * g, hide] = -torch.inf
                w = torch.softmax(x, -1).nan_to_num(0.0)
                out[r0:r0 + T, h * g:(h + 1) * g] = (w @ V).view(T, g, D)
    return out


def work(case):
    """Every input, page and table row read once, every output (and page) written once; a prefix once for its requests."""
    H, op = case["hkv"], case["op"]
    if op == "rotate":
        n, heads = case["n"], case["hq"] + H
        return dict(bytes=n * (heads * 2.0 * 2 * D + case["rot"] * 4.0 + 4.0 * case["axes"]), flops=n * heads * case["rot"] * 3.0)
    token = case["int2"] * 96.0 + (1 - case["int2"]) * 160.0     # codes, scales and zeros of a token and kv head
    if op == "append":
        n = case["batch"] * (case["lo"] + case["hi"]) / 2.0
        return dict(bytes=n * (H * (4.0 * D + token + 4.0 * D) + case["rot"] * 4.0 + 4.0 * case["axes"]),
                    flops=n * H * (3.0 * case["rot"] + 16.0 * D))
    if op == "read":
        n = case["share"] * case["batch"] * (case["ctx_lo"] + case["ctx_hi"]) / 2.0
        return dict(bytes=n * H * (token + 4.0 * D), flops=n * H * 4.0 * D)
    B, T = case["batch"], (case["new_lo"] + case["new_hi"]) / 2.0
    pre, ctx = (case["pre_lo"] + case["pre_hi"]) / 2.0, (case["ctx_lo"] + case["ctx_hi"]) / 2.0
    pairs = B * T * ((1 - case["lone"]) * pre + ctx + (0 if case["cached"] else (T + 1) / 2))
    return dict(bytes=H * (case["prefixes"] * pre + B * ctx) * token + B * T * D * (case["hq"] * 4.0 + (0 if case["cached"] else H * 4.0)),
                flops=4.0 * D * case["hq"] * pairs)
