"""A seeded random sweep over sizes, types, kinds and addresses of the
embedding, the norm and the checkpoint, against the fp64 definitions with the
bounds of ends_common."""

import numpy as np
import pytest
import torch

from ends_common import DEV, Guarded, f64, norm_bounds, norm_grad_bounds, to_dev, within
from oracle import ends
from test_gpu_embed import check_grad, draw_ids
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(40))
def test_embed_grad_sweep(seed):
    rng = np.random.default_rng(1000 + seed)
    n, H = log_int(rng, 1, 12000), log_int(rng, 1, 1500)
    n = max(1, min(n, 2_000_000 // H))
    V = max(1, min(log_int(rng, 1, 20000), 3_000_000 // H))
    kind = rng.choice(["absorb", "one", "distinct", "few", "uniform", "padded", "none"])
    ids = draw_ids(rng, str(kind), n, V)
    check_grad(ids, n, H, V, [torch.bfloat16, torch.float32][seed % 2], bool(rng.integers(2)),
               float(rng.uniform(-3, 3)), seed, skew=int(rng.integers(8)))


@pytest.mark.parametrize("seed", range(40))
def test_norm_sweep(seed):
    rng = np.random.default_rng(2000 + seed)
    H = log_int(rng, 1, 16384)
    if seed % 3:
        H = max(8, H // 8 * 8)
    n = max(1, min(log_int(rng, 1, 3000), 1_500_000 // H))
    dtype = [torch.bfloat16, torch.float32][seed % 2]
    kind = int(rng.integers(2))
    skew = int(rng.integers(8))
    x, x64 = to_dev(rng.standard_normal((n, H)) * 3 + rng.uniform(-2, 2), dtype, skew)
    dy, dy64 = to_dev(rng.standard_normal((n, H)), dtype, skew)
    w, w64 = to_dev(rng.standard_normal(H), dtype, skew)
    b, b64 = to_dev(rng.standard_normal(H), dtype, skew)
    y, dx = (Guarded((n, H), dtype, skew) for _ in range(2))
    mean, rstd = (Guarded((n,), torch.float32, skew) for _ in range(2))
    q, qe = Guarded((n, H), torch.uint8, skew), Guarded((n, -(-H // 128)), torch.uint8, skew)
    dw, db = (Guarded((H,), torch.float32, skew) for _ in range(2))
    B.mdlm_norm_fwd(x.t, kind, w.t, b.t, 1e-5, y.t, mean.t, rstd.t, q.t, qe.t)
    want, mu, r = ends.norm(x64, kind, w64, b64, 1e-5)
    d_y, d_mu, d_r = norm_bounds(x64, kind, w64, b64, 1e-5, dtype)
    within(f64(y.t), want, d_y, (n, H))
    within(f64(rstd.t), r, d_r, (n, H))
    some = np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, 4)]))
    want_q, want_e = ends.ckpt8_save(x64[some])
    assert np.array_equal(q.t.cpu().numpy()[some], want_q)
    assert np.array_equal(qe.t.cpu().numpy()[some], want_e)
    st = mean.t if kind == B.MDLM_NORM_LAYER else None
    m64 = f64(mean.t) if kind == B.MDLM_NORM_LAYER else np.zeros(n)
    held = ends.ckpt8_load(q.t.cpu().numpy(), qe.t.cpu().numpy())
    for source in (x64, held):
        if source is held:
            B.mdlm_norm_bwd_ckpt8(dy.t, q.t, qe.t, kind, w.t, st, rstd.t, dx.t, dw.t, db.t)
        else:
            B.mdlm_norm_bwd(dy.t, x.t, kind, w.t, st, rstd.t, dx.t, dw.t, db.t)
        ref = ends.norm_grad(dy64, source, kind, w64, m64, f64(rstd.t))
        bound = norm_grad_bounds(dy64, source, kind, w64, m64, f64(rstd.t), dtype)
        for t, a, d in zip((dx, dw, db), ref, bound):
            within(f64(t.t), a, d, (n, H))
    assert all(t.intact() for t in (x, dy, w, b, y, dx, mean if st is not None else dx, rstd, q,
                                    qe, dw, db))
    back = Guarded((n, H), dtype, skew)
    B.mdlm_ckpt8_load(q.t, qe.t, back.t)
    assert np.array_equal(f64(back.t), held) and back.intact()


@pytest.mark.parametrize("seed", range(20))
def test_embed_sweep(seed):
    rng = np.random.default_rng(3000 + seed)
    n, H, V = log_int(rng, 1, 3000), log_int(rng, 1, 5000), log_int(rng, 1, 900)
    dtype, skew = [torch.bfloat16, torch.float32][seed % 2], int(rng.integers(8))
    T, T64 = to_dev(rng.standard_normal((V, H)), dtype, skew)
    ids = rng.integers(-1, V + 1, n).astype(np.int32)
    scale = np.float32(rng.uniform(-40, 40))
    out = Guarded((n, H), dtype, skew)
    B.mdlm_embed(torch.from_numpy(ids).to(DEV), T.t, float(scale), out.t)
    prod = torch.from_numpy(T64).float() * scale  # one rounding
    want = torch.zeros(n, H)
    ok = (ids >= 0) & (ids < V)
    want[ok] = prod[torch.from_numpy(ids[ok]).long()]
    assert torch.equal(out.t.cpu(), want.to(dtype))
    assert out.intact()
