"""Tensors of more than 2^32 entries: every offset of the embedding, the norm
and the checkpoint has to be formed in 64 bits.  Rows on both sides of 2^31
and 2^32 entries, and the last ones, are compared; the sums over rows whole."""

import numpy as np
import pytest
import torch

from ends_common import DEV, f64, norm_bounds, norm_grad_bounds, within
from oracle import ends
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu

N, H = 1_050_000, 4096  # 4.3e9 entries
ROWS = [0, 524287, 524288, 524289, 1048575, 1048576, 1048577, N - 2, N - 1]


def big(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(N, H, dtype=torch.bfloat16, device=DEV)
    for i in range(0, N, 150_000):
        x[i:i + 150_000].normal_(generator=g)
    return x


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def test_embed_from_a_large_table():
    table = big(0)
    ids = torch.tensor(ROWS + ROWS[::-1], dtype=torch.int32, device=DEV)
    out = torch.empty(len(ids), H, dtype=torch.bfloat16, device=DEV)
    B.mdlm_embed(ids, table, 2.0, out)
    assert torch.equal(out, table[ids.long()] * 2.0)


def test_embed_grad_of_a_large_table():
    ids = torch.tensor(ROWS + ROWS[::-1], dtype=torch.int32, device=DEV)
    g = torch.randn(len(ids), H, device=DEV)
    d = torch.full((N, H), float("nan"), device=DEV)
    B.mdlm_embed_grad(ids, g, 1.0, d)
    want = g[:len(ROWS)] + g[len(ROWS):].flip(0)  # two terms: one rounding
    assert torch.equal(d[ids[:len(ROWS)].long()], want)
    hit = 0
    for i in range(0, N, 150_000):
        hit += int((d[i:i + 150_000] != 0).any(1).sum())  # (a NaN left over counts)
    assert hit == len(ROWS)


def test_embed_grad_of_many_tokens():
    """1.05 M tokens on 1,000 ids, half of them one: sorted runs merged in LDS
    and twice in memory, a cut run of 16,000 chunks."""
    g = torch.Generator(device=DEV).manual_seed(1)
    V = 1000
    ids = torch.randint(0, V, (N,), device=DEV, generator=g, dtype=torch.int32)
    ids[torch.rand(N, device=DEV, generator=g) < 0.5] = 77
    d_out = big(2)
    d = torch.empty(V, H, device=DEV)
    B.mdlm_embed_grad(ids, d_out, 1.0, d)
    again = torch.empty_like(d)
    B.mdlm_embed_grad(ids, d_out, 1.0, again)
    assert torch.equal(d, again)
    cols = torch.tensor([0, 1, 511, 512, 4095], device=DEV)
    part = torch.cat([d_out[i:i + 150_000][:, cols] for i in range(0, N, 150_000)]).double()
    order = torch.argsort(ids, stable=True)
    ends_at = torch.cumsum(torch.bincount(ids, minlength=V), 0)
    part = torch.cat([torch.zeros(1, len(cols), device=DEV, dtype=torch.float64), part[order]])
    want, size = (torch.cumsum(p, 0)[ends_at] for p in (part, part.abs()))
    want[1:] -= want[:-1].clone()  # (running sums of 1e6 terms in float64: exact to 1e-10)
    size[1:] -= size[:-1].clone()
    # a term meets at most a chunk's and its neighbour's 64 additions, one per
    # partial row a lane group adds up (16,500 / 64) and the 64 groups'
    depth = 64 + 16500 // 64 + 64 + 2
    within(f64(d[:, cols]), f64(want), depth * 2.0 ** -24 * f64(size))


@pytest.mark.parametrize("kind", [B.MDLM_NORM_LAYER, B.MDLM_NORM_RMS])
def test_norm_and_checkpoint_of_many_rows(kind):
    x = big(3)
    y = torch.empty_like(x)
    mean = torch.empty(N, device=DEV) if kind == B.MDLM_NORM_LAYER else None
    rstd = torch.empty(N, device=DEV)
    q = torch.empty(N, H, dtype=torch.uint8, device=DEV)
    qe = torch.empty(N, H // 128, dtype=torch.uint8, device=DEV)
    B.mdlm_norm_fwd(x, kind, None, None, 1e-5, y, mean, rstd, q, qe)
    at = torch.tensor(ROWS, device=DEV)
    x64 = f64(x[at])
    want, mu, r = ends.norm(x64, kind, None, None, 1e-5)
    d_y, _, d_r = norm_bounds(x64, kind, None, None, 1e-5, torch.bfloat16)
    within(f64(y[at]), want, d_y)
    within(f64(rstd[at]), r, d_r)
    want_q, want_e = ends.ckpt8_save(x64)
    assert np.array_equal(q[at].cpu().numpy(), want_q)
    assert np.array_equal(qe[at].cpu().numpy(), want_e)
    B.mdlm_ckpt8_load(q, qe, y)
    held = ends.ckpt8_load(want_q, want_e)
    assert np.array_equal(f64(y[at]), held)
    q.zero_(), qe.zero_()
    B.mdlm_ckpt8_save(x, q, qe)
    assert np.array_equal(q[at].cpu().numpy(), want_q)

    dy, dx = x, y  # (any dy will do: x itself)
    dw, db = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    B.mdlm_norm_bwd_ckpt8(dy, q, qe, kind, None, mean, rstd, dx, dw, db)
    m64 = np.zeros(len(ROWS)) if mean is None else f64(mean[at])
    r64 = f64(rstd[at])
    ref = ends.norm_grad(x64, held, kind, None, m64, r64)
    bound = norm_grad_bounds(x64, held, kind, None, m64, r64, torch.bfloat16)
    within(f64(dx[at]), ref[0], bound[0])
    B.mdlm_norm_bwd(dy, x, kind, None, mean, rstd, dx, dw, db)
    ref = ends.norm_grad(x64, x64, kind, None, m64, r64)
    bound = norm_grad_bounds(x64, x64, kind, None, m64, r64, torch.bfloat16)
    within(f64(dx[at]), ref[0], bound[0])
    sw = torch.zeros(H, dtype=torch.float64, device=DEV)
    sb, aw, ab = torch.zeros_like(sw), torch.zeros_like(sw), torch.zeros_like(sw)
    for i in range(0, N, 75_000):
        v = x[i:i + 75_000].double()
        z = (v if mean is None else v - mean[i:i + 75_000, None].double())
        z = v * z * rstd[i:i + 75_000, None].double()
        sw += z.sum(0)
        aw += z.abs().sum(0)
        sb += v.sum(0)
        ab += v.abs().sum(0)
    # a term meets the additions of one lane (its rows of 512 a step), the two
    # groups', the sum over 256 partial rows, and three roundings of its own
    depth = N // 512 + 1 + 2 + 16 + 16 + 3
    within(f64(dw), f64(sw), depth * 2.0 ** -24 * f64(aw))
    within(f64(db), f64(sb), depth * 2.0 ** -24 * f64(ab))
