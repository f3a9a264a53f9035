"""CPU oracle of the operators around the layer (float64, numpy): the residual
sum with dropout and root-mean-square norm, MXFP8 and MXFP4 formats, the 4-bit
matrix-vector product and the few-token layer on 4-bit weights.

TEST INFRASTRUCTURE ONLY; shares no code, tables or helpers with the library.
"""
from __future__ import annotations

import numpy as np

__all__ = ["philox4x32_10", "dropout_keep", "dropout", "add_rmsnorm_fwd", "add_rmsnorm_bwd", "e4m3_value",
           "e4m3_round", "mx_scale", "mxfp8", "e2m1_value", "mxfp4", "mxfp4_value", "e8m0_value", "ffn_w4"]


def philox4x32_10(counter, key):
    """Philox4x32 with ten rounds; counter: four and key: two uint32 arrays or
    numbers.  Returns four uint64 arrays of 32-bit words."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    m = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a = c[0] * np.uint64(0xD2511F53)
        b = c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_keep(T, d, p, seed, offset):
    """Boolean [T][d]: which values dropout keeps."""
    nb = -(-d // 8)
    blocks = np.arange(T * nb, dtype=np.uint64)
    lo = np.uint64(0xFFFFFFFF)
    w = philox4x32_10([blocks & lo, blocks >> np.uint64(32), np.full_like(blocks, offset & 0xFFFFFFFF),
                       np.full_like(blocks, offset >> 32)], [seed & 0xFFFFFFFF, seed >> 32])
    halves = np.empty((T * nb, 8), dtype=np.int64)
    for i in range(4):
        halves[:, 2 * i] = (w[i] & np.uint64(0xFFFF)).astype(np.int64)
        halves[:, 2 * i + 1] = (w[i] >> np.uint64(16)).astype(np.int64)
    return halves.reshape(T, nb * 8)[:, :d] >= int(np.rint(np.float32(p) * 65536.0))


def dropout(x, p, seed=0, offset=0):
    x = np.asarray(x, dtype=np.float64)
    if p == 0:
        return x
    drop = int(np.rint(np.float32(p) * 65536.0)) / 65536.0
    keep = dropout_keep(*x.shape, p, seed, offset)
    out = np.zeros_like(x)
    if drop < 1:
        out[keep] = x[keep] / (1 - drop)
    return out


def add_rmsnorm_fwd(x, residual, w, eps, p=0.0, seed=0, offset=0, store=lambda v: v):
    """(sum as stored, y, rstd); store rounds the sum to its dtype."""
    s = dropout(x, p, seed, offset)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float64)
    s = np.asarray(store(s), dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    y = s * rstd[:, None] * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    return s, y, rstd


def add_rmsnorm_bwd(dy, dsum, s, w, rstd, p=0.0, seed=0, offset=0):
    """(dres, dx, dw) for the stored sum s and rstd."""
    dy, s, r = (np.asarray(v, dtype=np.float64) for v in (dy, s, rstd))
    xh = s * r[:, None]
    g = dy if w is None else dy * np.asarray(w, dtype=np.float64)
    c = np.mean(g * xh, axis=1, keepdims=True) if dy.size else np.zeros((dy.shape[0], 1))
    dres = r[:, None] * (g - xh * c)
    if dsum is not None:
        dres = dres + np.asarray(dsum, dtype=np.float64)
    return dres, dropout(dres, p, seed, offset), (dy * xh).sum(axis=0)


# ---------------------------------------------------------------- 8- and 4-bit formats

def e8m0_value(b):
    """2**(b - 127), 255 is NaN."""
    b = np.asarray(b, dtype=np.float64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127))


def e4m3_value(code):
    code = np.asarray(code, dtype=np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


def e4m3_round(v):
    """Nearest e4m3 value (ties to even) of |v| <= 448."""
    v = np.asarray(v, dtype=np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(v / step) * step


def mx_scale(v, top):
    """Scale bytes of groups of 32 columns: the smallest power of two >= 2**-127
    that holds the group within +-top; 255 where a value is not finite."""
    T, d = v.shape
    pad = np.zeros((T, -(-d // 32) * 32))
    pad[:, :d] = v
    g = np.abs(pad).reshape(T, -1, 32).max(axis=2)       # NaN wins
    out = np.zeros(g.shape, dtype=np.int64)
    for i, m in np.ndenumerate(g):
        if not np.isfinite(m):
            out[i] = 255
            continue
        b = 0
        if m > 0:
            b = max(0, int(np.floor(np.log2(m / top))) + 127)
            while b > 0 and m <= top * 2.0 ** (b - 1 - 127):
                b -= 1
            while m > top * 2.0 ** (b - 127):
                b += 1
        out[i] = b
    return out


def _columns(scale, d):
    return np.repeat(e8m0_value(scale), 32, axis=1)[:, :d]


def mxfp8(v):
    """(values that the MXFP8 codes stand for before scaling, scale bytes)."""
    v = np.asarray(v, dtype=np.float64)
    scale = mx_scale(v, 448.0)
    with np.errstate(invalid="ignore"):
        return e4m3_round(v / _columns(scale, v.shape[1])), scale


_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_value(code):
    code = np.asarray(code, dtype=np.int64)
    return np.where(code & 8, -1.0, 1.0) * _E2M1[code & 7]


def mxfp4(w):
    """(codes [N][K], scale bytes [N][K/32]): nearest e2m1 code, ties to the
    even code, by brute force over the eight magnitudes."""
    w = np.asarray(w, dtype=np.float64)
    scale = mx_scale(w, 6.0)
    a = np.abs(w / _columns(scale, w.shape[1]))
    dist = np.abs(a[..., None] - _E2M1)
    best = np.zeros(a.shape, dtype=np.int64)
    for c in range(1, 8):
        cur = np.take_along_axis(dist, best[..., None], -1)[..., 0]
        better = (dist[..., c] < cur) | ((dist[..., c] == cur) & (c % 2 == 0))
        best = np.where(better, c, best)
    return best | np.where(np.signbit(w), 8, 0), scale


def mxfp4_value(codes, scale):
    return e2m1_value(codes) * _columns(scale, codes.shape[1])


def ffn_w4(x, Wg, bg, Wu, Wd):
    """The layer on dequantised weights [F][d]; x [T][d] values."""
    g = x @ Wg.T + (0.0 if bg is None else bg)
    h = np.where(g > 0, g, 0.0)
    return np.where(h > 0, h * (x @ Wu.T), 0.0) @ Wd
