"""Layer and RMS norm on the GPU, forward and backward, from x and from its
8-bit checkpoint, against the fp64 definitions, with bounds counted from the
formulas (ends_common)."""

import numpy as np
import pytest
import torch

from ends_common import (DEV, Guarded, f64, norm_bounds, norm_grad_bounds, to_dev, within)
from oracle import ends
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
KINDS = [B.MDLM_NORM_LAYER, B.MDLM_NORM_RMS]
EPS = 1e-5
SIZES = [(1, 1), (1, 4096), (3, 64), (5, 130), (4, 511), (7, 512), (2, 513), (9, 1000), (3, 1024),
         (5, 1025), (2, 2048), (3, 2053), (6, 2816), (2, 4100), (3, 8192), (2, 8200), (2, 12296),
         (2, 16384), (1, 16383), (1100, 40), (4500, 9)]


def rows(n, H, seed):
    """Rows of different scales and offsets, the first one all zeros, the
    second one constant."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, H)) * np.exp2(rng.integers(-3, 4, (n, 1)))
    x += rng.choice([0.0, 0.5, -20.0], (n, 1))
    if n > 2:
        x[0], x[1] = 0.0, 0.375
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,H", SIZES)
def test_norm_forward(dtype, kind, n, H):
    skew = 3 if H % 8 else 0
    rng = np.random.default_rng(H)
    x, x64 = to_dev(rows(n, H, n + H), dtype, skew)
    w, w64 = to_dev(rng.standard_normal(H), dtype, skew)
    b, b64 = to_dev(rng.standard_normal(H), dtype, skew)
    for with_w, with_b in ((True, True), (True, False), (False, True), (False, False)):
        y = Guarded((n, H), dtype, skew)
        mean, rstd = Guarded((n,), torch.float32), Guarded((n,), torch.float32)
        B.mdlm_norm_fwd(x.t, kind, w.t if with_w else None, b.t if with_b else None, EPS, y.t,
                        mean.t, rstd.t)
        wa, ba = w64 if with_w else None, b64 if with_b else None
        want, mu, r = ends.norm(x64, kind, wa, ba, EPS)
        d_y, d_mu, d_r = norm_bounds(x64, kind, wa, ba, EPS, dtype)
        within(f64(y.t), want, d_y, ("y", n, H))
        within(f64(rstd.t), r, d_r, ("rstd", n, H))
        if kind == B.MDLM_NORM_LAYER:
            within(f64(mean.t), mu, d_mu, ("mean", n, H))
        assert y.intact() and mean.intact() and rstd.intact()
    if kind == B.MDLM_NORM_RMS:  # the mean is not written
        assert bool((mean.raw == 0xA5).all())
    # without statistics: the same y
    y2 = torch.empty_like(y.t)
    B.mdlm_norm_fwd(x.t, kind, None, None, EPS, y2)
    assert torch.equal(y2, y.t)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,H", SIZES)
def test_norm_backward(dtype, kind, n, H):
    skew = 3 if H % 8 else 0
    rng = np.random.default_rng(H + 1)
    x, x64 = to_dev(rows(n, H, n + H), dtype, skew)
    dy, dy64 = to_dev(rng.standard_normal((n, H)) * 1e-3, dtype, skew)
    w, w64 = to_dev(rng.standard_normal(H), dtype, skew)
    _, mu, r = ends.norm(x64, kind, None, None, EPS)
    mean, mu64 = to_dev(mu, torch.float32)
    rstd, r64 = to_dev(r, torch.float32)
    start = rng.standard_normal((2, H)).astype(np.float32)
    for wt, acc in ((w, False), (None, True)):
        wa = None if wt is None else w64
        dx = Guarded((n, H), dtype, skew)
        dw = Guarded((H,), torch.float32, skew, torch.from_numpy(start[0]))
        db = Guarded((H,), torch.float32, skew, torch.from_numpy(start[1]))
        B.mdlm_norm_bwd(dy.t, x.t, kind, None if wt is None else wt.t,
                        mean.t if kind == B.MDLM_NORM_LAYER else None, rstd.t, dx.t, dw.t, db.t,
                        accumulate=acc)
        want = ends.norm_grad(dy64, x64, kind, wa, mu64, r64)
        bound = norm_grad_bounds(dy64, x64, kind, wa, mu64, r64, dtype)
        add = start.astype(np.float64) if acc else 0.0 * start
        within(f64(dx.t), want[0], bound[0], ("dx", n, H))
        # (the addition to what was there rounds once more)
        within(f64(dw.t), want[1] + add[0],
               bound[1] + 2.0 ** -24 * np.abs(want[1] + add[0]) * 1.01, ("dw", n, H))
        within(f64(db.t), want[2] + add[1],
               bound[2] + 2.0 ** -24 * np.abs(want[2] + add[1]) * 1.01, ("db", n, H))
        assert dx.intact() and dw.intact() and db.intact()
    # each output by itself: the same bits
    alone = torch.empty_like(dx.t)
    B.mdlm_norm_bwd(dy.t, x.t, kind, None, mean.t, rstd.t, alone)
    assert torch.equal(alone, dx.t)
    for at in (0, 1):
        out = torch.from_numpy(start[at].copy()).to(DEV)
        B.mdlm_norm_bwd(dy.t, x.t, kind, None, mean.t, rstd.t, None,
                        *((out, None) if at == 0 else (None, out)), accumulate=True)
        assert torch.equal(out, (dw, db)[at].t)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,H", [(1, 1), (3, 130), (5, 512), (9, 1001), (4, 2816), (3, 4096),
                                 (5, 1000), (3, 5128), (2, 8195), (2, 8200), (2, 16384),
                                 (700, 136)])
def test_norm_with_checkpoint(dtype, kind, n, H):
    """The forward's checkpoint is mdlm_ckpt8_save's, bit for bit, its y that of
    the call without one; the gradients are those at the restored x."""
    rng = np.random.default_rng(H + 2)
    x, _ = to_dev(rows(n, H, n + H), dtype)
    dy, dy64 = to_dev(rng.standard_normal((n, H)) * 1e-3, dtype)
    w, w64 = to_dev(rng.standard_normal(H), dtype)
    y = [torch.empty((n, H), dtype=dtype, device=DEV) for _ in range(2)]
    mean, rstd = (torch.zeros(n, device=DEV) for _ in range(2))
    nb = -(-H // 128)
    q, qe = Guarded((n, H), torch.uint8), Guarded((n, nb), torch.uint8)
    B.mdlm_norm_fwd(x.t, kind, w.t, None, EPS, y[0], mean, rstd)
    B.mdlm_norm_fwd(x.t, kind, w.t, None, EPS, y[1], mean, rstd, q.t, qe.t)
    assert torch.equal(y[0], y[1])
    q2, qe2 = torch.empty_like(q.t), torch.empty_like(qe.t)
    B.mdlm_ckpt8_save(x.t, q2, qe2)
    assert torch.equal(q.t, q2) and torch.equal(qe.t, qe2)
    assert q.intact() and qe.intact()
    held = ends.ckpt8_load(q.t.cpu().numpy(), qe.t.cpu().numpy())
    m64, r64 = f64(mean), f64(rstd)
    dx, dw, db = (Guarded(s, t) for s, t in (((n, H), dtype), ((H,), torch.float32),
                                              ((H,), torch.float32)))
    B.mdlm_norm_bwd_ckpt8(dy.t, q.t, qe.t, kind, w.t,
                          mean if kind == B.MDLM_NORM_LAYER else None, rstd, dx.t, dw.t, db.t)
    want = ends.norm_grad(dy64, held, kind, w64, m64, r64)
    bound = norm_grad_bounds(dy64, held, kind, w64, m64, r64, dtype)
    for t, a, d in zip((dx, dw, db), want, bound):
        within(f64(t.t), a, d, (n, H))
        assert t.intact()


@pytest.mark.parametrize("kind", KINDS)
def test_nonfinite_rows_keep_to_themselves(kind):
    x = torch.randn(6, 300, device=DEV)
    clean = x.clone()
    x[1, 17], x[4, 299] = float("nan"), float("inf")
    y, y0 = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(6, device=DEV)
    mean = torch.empty(6, device=DEV)
    B.mdlm_norm_fwd(clean, kind, None, None, EPS, y0)
    B.mdlm_norm_fwd(x, kind, None, None, EPS, y, mean, rstd)
    good = [0, 2, 3, 5]
    assert torch.equal(y[good], y0[good])
    assert torch.isnan(y[1]).all() and torch.isnan(rstd[1])
    dy = torch.randn_like(x)
    dx, dx0 = torch.empty_like(x), torch.empty_like(x)
    st = mean if kind == B.MDLM_NORM_LAYER else None
    B.mdlm_norm_bwd(dy, x, kind, None, st, rstd, dx)
    B.mdlm_norm_fwd(clean, kind, None, None, EPS, y0, mean, rstd)
    B.mdlm_norm_bwd(dy, clean, kind, None, st, rstd, dx0)
    assert torch.equal(dx[good], dx0[good])
    assert torch.isnan(dx[1]).all()


def test_norm_gradient_against_differences():
    """Central differences of sum(dy * y) through the forward kernel, in
    float32: a step of 2^-4 at values of order 1 has a truncation error of
    about h^2 f''' / 6 ~ 1e-3 and a rounding error of some U |f| / h ~ 1e-5 per
    term; 2e-2 of the gradient's norm covers both with room."""
    for kind in KINDS:
        g = torch.Generator(device=DEV).manual_seed(3)
        x = torch.randn(1, 48, device=DEV, generator=g)
        dy = torch.randn(1, 48, device=DEV, generator=g)
        w = torch.randn(48, device=DEV, generator=g)
        h = 2.0 ** -4
        many = x + torch.cat([torch.eye(48), -torch.eye(48)]).to(DEV) * h
        y = torch.empty_like(many)
        B.mdlm_norm_fwd(many.contiguous(), kind, w, None, EPS, y)
        f = (y.double() * dy.double()).sum(1)
        diff = (f[:48] - f[48:]) / (2 * h)
        y1, mean, rstd = torch.empty_like(x), torch.empty(1, device=DEV), torch.empty(1, device=DEV)
        B.mdlm_norm_fwd(x, kind, w, None, EPS, y1, mean, rstd)
        dx = torch.empty_like(x)
        B.mdlm_norm_bwd(dy, x, kind, w, mean, rstd, dx)
        assert float((dx[0].double() - diff).norm() / diff.norm()) < 2e-2


def test_norm_without_rows():
    x = torch.empty(0, 32, device=DEV)
    dw = torch.full((32,), 3.0, device=DEV)
    stat = torch.empty(0, device=DEV)
    B.mdlm_norm_fwd(x, 0, None, None, EPS, torch.empty_like(x), stat, stat)
    B.mdlm_norm_bwd(x, x, 0, None, stat, stat, None, dw, accumulate=True)
    assert bool((dw == 3.0).all())
    B.mdlm_norm_bwd(x, x, 0, None, stat, stat, None, dw)
    assert not dw.any()


def test_norm_same_bits_every_run():
    n, H = 5000, 328
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(n, H, device=DEV, generator=g).bfloat16()
    dy = torch.randn(n, H, device=DEV, generator=g).bfloat16()
    rstd, y = torch.empty(n, device=DEV), torch.empty_like(x)
    B.mdlm_norm_fwd(x, 1, None, None, EPS, y, None, rstd)
    got = []
    for fill in (0, 255):
        ws = torch.full((B.mdlm_norm_bwd_workspace_bytes(n, H),), fill, dtype=torch.uint8,
                        device=DEV)
        dw, db = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
        B.mdlm_norm_bwd(dy, x, 1, None, None, rstd, None, dw, db, workspace=ws)
        got.append((dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(B.MdlmError, match="workspace"):
        B.mdlm_norm_bwd(dy, x, 1, None, None, rstd, None, dw, db, workspace=ws[:-1])


def test_norm_binding_refusals():
    x = torch.zeros(4, 32, device=DEV)
    s = torch.zeros(4, device=DEV)
    w = torch.zeros(32, device=DEV)
    with pytest.raises(TypeError):
        B.mdlm_norm_fwd(x, 0, w.bfloat16(), None, EPS, torch.empty_like(x))
    with pytest.raises(ValueError):
        B.mdlm_norm_fwd(x, 0, w[:31], None, EPS, torch.empty_like(x))
    with pytest.raises(ValueError):
        B.mdlm_norm_fwd(x.t(), 0, None, None, EPS, torch.empty(32, 4, device=DEV))
    with pytest.raises(ValueError):
        B.mdlm_norm_fwd(x, 0, None, None, EPS, torch.empty_like(x), s[:3])
    with pytest.raises(B.MdlmError, match="eps"):
        B.mdlm_norm_fwd(x, 0, None, None, 0.0, torch.empty_like(x))
    with pytest.raises(B.MdlmError, match="unknown norm"):
        B.mdlm_norm_fwd(x, 5, None, None, EPS, torch.empty_like(x))
    with pytest.raises(B.MdlmError, match="exceeds"):
        big = torch.zeros(1, 16385, device=DEV)
        B.mdlm_norm_fwd(big, 0, None, None, EPS, torch.empty_like(big))
    with pytest.raises(B.MdlmError, match="null input"):
        B.mdlm_norm_bwd(x, x, 0, None, None, s, torch.empty_like(x))
    with pytest.raises(B.MdlmError, match="no gradient"):
        B.mdlm_norm_bwd(x, x, 1, None, None, s, None)
    with pytest.raises(TypeError):
        B.mdlm_norm_bwd(x, x, 1, None, None, s, x.bfloat16())
    with pytest.raises(ValueError):
        B.mdlm_norm_bwd_ckpt8(x, x.to(torch.uint8), torch.zeros(4, 2, device=DEV,
                                                                 dtype=torch.uint8),
                              1, None, None, s, torch.empty_like(x))
