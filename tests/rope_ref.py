"""Plain forms of the rotation by position: the definition in fp32 steps (bit-exact) and in 64 bits."""
import numpy as np


def table(rows, rot, base=10000.0):
    """[rows][rot] fp32: cosines of rot / 2 frequencies, then sines, angles in 64 bits."""
    half = rot // 2
    ang = np.arange(rows)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def to_bf16(x):
    """fp32 -> nearest bf16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def _parts(x, tab, pos, axis, pairs):
    half = tab.shape[1] // 2
    pos = np.atleast_2d(pos)
    row = pos[np.zeros(half, int) if axis is None else np.asarray(axis, int)]      # [half][n]
    f = np.arange(half)[:, None]
    c, s = tab[row, f].T[:, None], tab[row, f + half].T[:, None]                    # [n][1][half]
    if pairs:
        return x[..., 0:2 * half:2], x[..., 1:2 * half:2], c, s
    return x[..., :half], x[..., half:2 * half], c, s


def _join(x, u, v, pairs):
    half = u.shape[-1]
    y = x.copy()
    if pairs:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, v
    else:
        y[..., :half], y[..., half:2 * half] = u, v
    return y


def rotate(x, tab, pos, axis=None, pairs=False):
    """x fp32 (bf16 values) [n][heads][128] -> the rotated rows, each step rounded to fp32, the result to bf16."""
    x = np.asarray(x, np.float32)
    a, b, c, s = _parts(x, tab, pos, axis, pairs)
    return to_bf16(_join(x, a * c - b * s, b * c + a * s, pairs))


def rotate_exact(x, tab, pos, axis=None, pairs=False):
    """The same in 64 bits, not rounded, and how far the rounded one may be: two products and a sum of
    fp32 (2^-24 of each), then half a step of bf16 (2^-8 of the value; 2^-134 where it is subnormal)."""
    x = np.asarray(x, np.float64)
    a, b, c, s = _parts(x, np.asarray(tab, np.float64), pos, axis, pairs)
    y = _join(x, a * c - b * s, b * c + a * s, pairs)
    mag = _join(np.zeros_like(x), np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s), pairs)
    return y, np.abs(y) * 2.0 ** -8 + mag * 2.0 ** -22 + 2.0 ** -134
