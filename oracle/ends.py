"""fp64 definitions of the model's two ends: token embedding, norm, 8-bit
checkpoints, and their gradients.

TEST INFRASTRUCTURE ONLY (see the package's header).  Plain numpy, written
from the formulas:

  embed       out_i = s T[id_i], zeros for an id outside [0, V)
  embed_grad  dT[v] = s * sum over id_i = v of dout_i
  norm        xhat = (x - mu) / sqrt(var + eps), y = xhat w + b (RMS: mu = 0,
              var = mean of squares)
  norm_grad   with g = dy w: dx = r (g - mean(g) - xhat mean(g xhat)) (RMS:
              without mean(g)), dw = sum dy xhat, db = sum dy
  ckpt8       blocks of 128 entries of a row as e4m3 codes over the least
              power of two 2^e >= 2^-127 that brings the block's largest finite
              magnitude to 448 or less
"""

import math

import numpy as np

NORM_LAYER = 0
NORM_RMS = 1


def embed(ids, table, scale):
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[i] = scale * table[v]
    return out


def embed_grad(ids, d_out, V, scale, start=None):
    """The table's gradient, added to `start` where given; and, entry by entry,
    the sum of the terms' magnitudes (what a tolerance is made of)."""
    d_out = np.asarray(d_out, dtype=np.float64)
    d = np.zeros((V, d_out.shape[1]))
    size = np.zeros_like(d)
    for i, v in enumerate(ids):
        if 0 <= v < V:
            d[v] += d_out[i]
            size[v] += np.abs(d_out[i])
    d, size = scale * d, abs(scale) * size
    if start is not None:
        d = d + start
        size = size + np.abs(start)
    return d, size


def norm(x, kind, weight, bias, eps):
    """y, mean and reciprocal deviation, row by row."""
    x = np.asarray(x, dtype=np.float64)
    mu = x.mean(axis=1) if kind == NORM_LAYER else np.zeros(x.shape[0])
    d = x - mu[:, None]
    r = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * r[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mu, r


def norm_grad(dy, x, kind, weight, mu, r):
    """dx, dw, db for statistics mu and r taken as given."""
    dy = np.asarray(dy, dtype=np.float64)
    xhat = (np.asarray(x, dtype=np.float64) - mu[:, None]) * r[:, None]
    g = dy if weight is None else dy * weight
    dx = g - xhat * (g * xhat).mean(axis=1)[:, None]
    if kind == NORM_LAYER:
        dx = dx - g.mean(axis=1)[:, None]
    return dx * r[:, None], (dy * xhat).sum(axis=0), dy.sum(axis=0)


def e4m3_value(code):
    """The number an e4m3 code stands for: sign, 4 exponent bits (bias 7), 3
    fraction bits, no infinities, all ones = NaN."""
    s = -1.0 if code & 0x80 else 1.0
    e, f = code >> 3 & 15, code & 7
    if e == 15 and f == 7:
        return math.nan
    if e == 0:
        return s * f * 2.0 ** -9
    return s * (1 + f / 8) * 2.0 ** (e - 7)


_CODES = np.array([e4m3_value(c) for c in range(127)])  # 0 .. 448, ascending


def e4m3_code(v):
    """The code nearest to v, |v| <= 448; of two equally near the even one."""
    a = abs(v)
    hi = int(np.searchsorted(_CODES, a))  # first code with a value >= a
    if hi == 0 or _CODES[min(hi, 126)] == a:
        c = min(hi, 126)
    else:
        below, above = a - _CODES[hi - 1], _CODES[hi] - a
        c = hi if above < below or (above == below and hi % 2 == 0) else hi - 1
    return c | (0x80 if math.copysign(1.0, v) < 0 else 0)


def block_exponent(top):
    """The least e >= -127 with top <= 448 * 2^e."""
    e = -127
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def ckpt8_save(x):
    """Codes and exponent bytes of an [n, H] activation; a non-finite entry
    takes a NaN code."""
    x = np.asarray(x, dtype=np.float64)
    n, H = x.shape
    q = np.zeros((n, H), dtype=np.uint8)
    b = np.zeros((n, -(-H // 128)), dtype=np.uint8)
    for i in range(n):
        for j in range(b.shape[1]):
            blk = x[i, 128 * j:128 * j + 128]
            fin = np.abs(blk[np.isfinite(blk)])
            e = block_exponent(float(fin.max()) if fin.size else 0.0)
            b[i, j] = e + 127
            for k, v in enumerate(blk):
                q[i, 128 * j + k] = e4m3_code(v * 2.0 ** -e) if np.isfinite(v) else 0x7F
    return q, b


def ckpt8_load(q, b):
    q = np.asarray(q)
    vals = np.array([e4m3_value(c) for c in range(256)])[q]
    e = np.repeat(np.asarray(b, dtype=np.int64) - 127, 128, axis=1)[:, :q.shape[1]]
    return vals * np.exp2(e.astype(np.float64))
