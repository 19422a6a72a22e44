"""The norm near the ends of float32's range: rows whose mean or whose
statistics are large while the results are not, at widths whose last waves or
lanes hold no column.  Bounds as in ends_common."""

import numpy as np
import pytest
import torch

from ends_common import (DEV, Guarded, f64, norm_bounds, norm_grad_bounds, to_dev,
                         within)
from oracle import ends
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
EPS = 1e-5
BIG = 1.5 * 2.0 ** 64  # its square is past float32's largest value


# Widths at which the waves that share a row are more than it fills (2,048: not).
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1280, 1281, 2048, 2100, 2304, 3100, 5000, 7000, 7003])
def test_forward_of_rows_with_a_large_mean(dtype, H):
    """A constant row, and one whose deviations (about 2^56, so that their
    squares sum to less than 2^128) stay far below its mean."""
    rng = np.random.default_rng(H)
    rows = np.full((3, H), BIG)
    rows[1] += rng.standard_normal(H) * 2.0 ** 56
    rows[2] = rng.standard_normal(H)
    x, x64 = to_dev(rows, dtype)
    w, w64 = to_dev(rng.standard_normal(H), dtype)
    b, b64 = to_dev(rng.standard_normal(H), dtype)
    y = Guarded((3, H), dtype)
    mean, rstd = Guarded((3,), torch.float32), Guarded((3,), torch.float32)
    B.mdlm_norm_fwd(x.t, B.MDLM_NORM_LAYER, w.t, b.t, EPS, y.t, mean.t, rstd.t)
    want, mu, r = ends.norm(x64, B.MDLM_NORM_LAYER, w64, b64, EPS)
    d_y, d_mu, d_r = norm_bounds(x64, B.MDLM_NORM_LAYER, w64, b64, EPS, dtype)
    assert all(bool(torch.isfinite(t.t).all()) for t in (y, mean, rstd))
    within(f64(mean.t), mu, d_mu, "mean")
    within(f64(rstd.t), r, d_r, "rstd")
    within(f64(y.t), want, d_y, "y")
    assert y.intact() and mean.intact() and rstd.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", [B.MDLM_NORM_LAYER, B.MDLM_NORM_RMS])
@pytest.mark.parametrize("H", [4, 300, 1280, 1281, 7000, 8200])
def test_forward_of_a_variance_past_the_range(dtype, kind, H):
    """Deviations (RMS: entries) whose squares overflow: rstd is 0, y the bias."""
    x = torch.full((2, H), BIG, device=DEV).to(dtype)
    x[:, ::2] *= -1.0
    b = torch.randn(H, device=DEV).to(dtype)
    y, rstd = torch.empty_like(x), torch.empty(2, device=DEV)
    B.mdlm_norm_fwd(x, kind, None, b, EPS, y, None, rstd)
    assert not rstd.any()
    assert torch.equal(y, b.expand(2, H))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [4, 300, 1280, 1281, 7000, 8200])
def test_forward_of_a_sum_past_the_range(dtype, H):
    """A layer norm's row whose plain sum overflows is NaN, and its neighbours
    are what they are without it."""
    x = torch.randn(3, H, device=DEV).to(dtype)
    y, alone = torch.empty_like(x), torch.empty_like(x)
    B.mdlm_norm_fwd(x, B.MDLM_NORM_LAYER, None, None, EPS, alone)
    x[1] = 3e38
    B.mdlm_norm_fwd(x, B.MDLM_NORM_LAYER, None, None, EPS, y)
    assert torch.isnan(y[1]).all()
    assert torch.equal(y[::2], alone[::2])


# Widths with lanes past the row's end that hold whole eights of no column, or
# an eight that the row only begins.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("source", ["x", "checkpoint"])
@pytest.mark.parametrize("H", [1, 4, 9, 1001, 1100, 2053, 8195])
def test_backward_of_a_row_whose_mean_times_rstd_overflows(dtype, source, H):
    """A constant row of 2^120 with rstd = 1 / sqrt(1e-5): (0 - mean) * rstd is
    infinite, but no entry of the row is 0 and xhat is 0 in all of it.  A row of
    ordinary values beside it."""
    g = torch.Generator(device=DEV).manual_seed(H)
    x = torch.randn(2, H, device=DEV, generator=g)
    if source == "checkpoint":  # values an 8-bit checkpoint holds exactly
        x = x.to(torch.float8_e4m3fn).float()
    x[0] = 2.0 ** 120
    x = x.to(dtype)
    x64 = f64(x)
    dy = torch.randn(2, H, device=DEV, generator=g).to(dtype)
    w = torch.randn(H, device=DEV, generator=g).to(dtype)
    _, mu, r = ends.norm(x64, B.MDLM_NORM_LAYER, None, None, EPS)
    mean, mu64 = to_dev(mu, torch.float32)
    rstd, r64 = to_dev(r, torch.float32)
    assert mu64[0] == 2.0 ** 120 and mu64[0] * r64[0] > torch.finfo(torch.float32).max
    dx = torch.empty_like(x)
    dw, db = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    if source == "checkpoint":
        q = torch.empty(2, H, dtype=torch.uint8, device=DEV)
        q_exp = torch.empty(2, -(-H // 128), dtype=torch.uint8, device=DEV)
        B.mdlm_ckpt8_save(x, q, q_exp)
        x64 = ends.ckpt8_load(q.cpu().numpy(), q_exp.cpu().numpy())
        assert (x64[0] == 2.0 ** 120).all()
        B.mdlm_norm_bwd_ckpt8(dy, q, q_exp, B.MDLM_NORM_LAYER, w, mean.t, rstd.t, dx, dw, db)
    else:
        B.mdlm_norm_bwd(dy, x, B.MDLM_NORM_LAYER, w, mean.t, rstd.t, dx, dw, db)
    want = ends.norm_grad(f64(dy), x64, B.MDLM_NORM_LAYER, f64(w), mu64, r64)
    bound = norm_grad_bounds(f64(dy), x64, B.MDLM_NORM_LAYER, f64(w), mu64, r64, dtype)
    for t, a, d in zip((dx, dw, db), want, bound):
        within(f64(t), a, d, H)


def test_sums_over_no_rows_leave_the_gradients_bits():
    """n = 0, accumulating: not even a zero's sign changes."""
    x, stat = torch.empty(0, 3, device=DEV), torch.empty(0, device=DEV)
    start = torch.tensor([-0.0, 1.5, float("nan")], device=DEV)
    dw, db = start.clone(), start.clone()
    B.mdlm_norm_bwd(x, x, B.MDLM_NORM_RMS, None, None, stat, None, dw, db, accumulate=True)
    for t in (dw, db):
        assert torch.equal(t.view(torch.int32), start.view(torch.int32))
