"""Plain 64-bit forms of the operators that read a pool for serving (attention of new
tokens, accumulated attention weight, lowest-score selection), computed from a pool's
exported content (codes and scales, which other tests hold bit-exact against the oracle)."""
import numpy as np

from np_ref import dequant_page

SCALE = float(np.float32(1 / np.sqrt(128)))


def bf16_round(x):
    """fp64 -> nearest bf16 value, as fp64."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


class Content:
    """A request's live slots per kv head: position, K^ and V^ (fp64)."""

    def __init__(self, pool, rid, head_dead=None):
        ex = pool.export(rid)
        n2 = pool.n_int2_pages
        self.n_tokens = pool.info(rid)[1]
        H = pool.num_kv_heads
        nfb = getattr(pool, "first_fp4", 1 << 62)
        self.pos, self.K, self.V = [[] for _ in range(H)], [[] for _ in range(H)], [[] for _ in range(H)]
        where = pool.slot_pos[rid]
        for i, pid in enumerate(ex["ids"]):
            for h in range(H):
                K, V = dequant_page(ex["kc"][i, h], ex["vc"][i, h], ex["km"][i, h], ex["vm"][i, h],
                                    pid < n2, fp4=pid >= nfb)
                for s in range(32):
                    if (int(ex["live"][i]) >> s) & 1:
                        p = where[(i, s)]
                        if head_dead and (h, p) in head_dead:
                            continue
                        self.pos[h].append(p)
                        self.K[h].append(K[s])
                        self.V[h].append(V[s])
        self.pos = [np.array(x, np.int64) for x in self.pos]
        self.K = [np.array(x, np.float64).reshape(-1, 128) for x in self.K]
        self.V = [np.array(x, np.float64).reshape(-1, 128) for x in self.V]


def attend_row(q, K, V, scale, u):
    """One row in fp64 and how far a computation with unit roundoff u of K, V and weights,
    rounded to bf16 at the end, may be off per element."""
    if K.shape[0] == 0:
        return np.zeros(128), np.full(128, 0.0)
    s = scale * (K @ q)
    w = np.exp(s - s.max())
    w /= w.sum()
    o = w @ V
    mag = w @ np.abs(V)
    ds = u * abs(scale) * np.max(np.abs(K) @ np.abs(q))      # rounding K moves a logit by at most this
    # weights move by 2 ds (numerator and sum); V and the weights round once each; fp32 sums of up
    # to ~1e5 terms and the exponential add less than 2^-15; bf16 rounds the result (half a step)
    tol = mag * (2 * ds + 2 * u + 2.0 ** -15) * 1.01 + np.abs(o) * 2.0 ** -8 + 1e-30
    return o, tol
