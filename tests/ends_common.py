"""Helpers of the GPU tests of embedding, norm and 8-bit checkpoint: tensors
behind guard bands and at odd addresses, and elementwise error bounds.

U is fp32's largest relative rounding error (half a step).  Every bound below
counts roundings from the formula and from how a sum is formed; none is
fitted."""

import numpy as np
import torch

DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


class Guarded:
    """A tensor inside a larger buffer whose other entries hold a pattern, at
    `skew` entries past a 256-byte boundary."""

    def __init__(self, shape, dtype, skew=0, fill=None):
        n = int(np.prod(shape)) if len(shape) else 1
        self.front = 64 + skew
        size = self.front + n + 64
        bytes_each = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((size * bytes_each,), 0xA5, dtype=torch.uint8, device=DEV)
        self.whole = self.raw.view(dtype)
        self.t = self.whole[self.front:self.front + n].view(shape)
        if fill is not None:
            self.t.copy_(fill)
        self.lo, self.hi = self.front * bytes_each, (self.front + n) * bytes_each

    def intact(self):
        return bool((self.raw[:self.lo] == 0xA5).all() and (self.raw[self.hi:] == 0xA5).all())


def to_dev(a, dtype, skew=0):
    """An fp64/fp32 array rounded to dtype on the device, and the fp64 values
    that it holds there."""
    t = torch.as_tensor(np.asarray(a)).to(dtype)
    return Guarded(t.shape, dtype, skew, t), t.double().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what=""):
    """|got - want| <= bound, entry by entry; NaN exactly where wanted."""
    got, want = np.asarray(got), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    ok = ~np.isnan(want)
    err = np.abs(got - want)
    bad = ok & ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.max((err / np.maximum(bound, 1e-300))[ok])))


# Roundings on one entry's way into a sum over a row: at most 16 entries in a
# lane, 6 lane exchanges and 16 waves, and the scale by 1/H and its own
# rounding.
ROW_DEPTH = 16 + 6 + 16 + 2


def norm_bounds(x, kind, w, b, eps, dtype):
    """Bounds on the errors of y, mean and rstd, from the formulas: the mean's
    sum, the difference's rounding, the variance's sum, the square root and
    the division, the products, the one rounding to dtype."""
    H = x.shape[1]
    mu = x.mean(axis=1) if kind == 0 else np.zeros(x.shape[0])
    d_mu = (ROW_DEPTH * U * np.abs(x).mean(axis=1)) if kind == 0 else 0.0 * mu
    d = x - mu[:, None]
    d_d = d_mu[:, None] + U * (np.abs(d) + d_mu[:, None])
    var = (d * d).mean(axis=1)
    d_var = (2 * np.abs(d) * d_d + d_d ** 2).mean(axis=1) + (ROW_DEPTH + 2) * U * var
    # relative error of 1/sqrt(var + eps): half of the argument's, eps as a
    # float, the sum, the root and the quotient one rounding each (the second
    # order of the first is covered by the factor 1.1)
    rel = 1.1 * 0.5 * (d_var + 2 * U * (var + eps)) / (var + eps) + 2 * U
    r = 1.0 / np.sqrt(var + eps)
    xhat = np.abs(d) * r[:, None]
    d_xhat = d_d * r[:, None] * (1 + rel[:, None]) + xhat * (rel[:, None] + U)
    aw = 1.0 if w is None else np.abs(w)
    d_y = aw * (d_xhat + U * xhat)
    y = xhat * aw + (0.0 if b is None else np.abs(b))
    d_y = d_y + U * y
    if dtype != torch.float32:
        d_y = d_y + HALF_STEP[dtype] * (y + d_y) + 2.0 ** -133
    return d_y, d_mu + U * np.abs(mu), rel * r


def norm_grad_bounds(dy, x, kind, w, mu, r, dtype):
    """Bounds on the errors of dx, dw and db for given statistics."""
    n = dy.shape[0]
    d = np.abs(x - mu[:, None])
    xhat = d * r[:, None]
    d_xhat = 2.1 * U * xhat  # the difference and the product
    g = np.abs(dy) * (1.0 if w is None else np.abs(w))
    m1 = g.mean(axis=1) if kind == 0 else 0.0 * r
    gx = (g * xhat).mean(axis=1)
    d_m1 = (ROW_DEPTH + 1) * U * m1
    d_m2 = (ROW_DEPTH + 5) * U * gx
    # r (g - m1 - xhat m2): one rounding per product and difference, at most
    # the sum of the terms' magnitudes large
    total = g + m1[:, None] + xhat * gx[:, None]
    d_dx = r[:, None] * (U * g + d_m1[:, None] + xhat * d_m2[:, None] + d_xhat * gx[:, None]
                         + 5 * U * total)
    if dtype != torch.float32:
        d_dx = d_dx + HALF_STEP[dtype] * r[:, None] * total * 1.01 + 2.0 ** -133
    # every row's term takes at most one rounding per later row on its way
    d_dw = (n + 8) * U * (np.abs(dy) * xhat).sum(axis=0)
    d_db = (n + 8) * U * np.abs(dy).sum(axis=0)
    return d_dx, d_dw, d_db
