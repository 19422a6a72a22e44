"""8-bit activation checkpoints on the GPU against the definition, bit for bit:
every scale, ties, subnormal and non-finite entries, short blocks, odd
addresses."""

import numpy as np
import pytest
import torch

from ends_common import DEV, Guarded, f64, to_dev
from oracle import ends
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def roundtrip(x, dtype, skew=0):
    g, x64 = to_dev(x, dtype, skew)
    n, H = x64.shape
    q = Guarded((n, H), torch.uint8, skew)
    qe = Guarded((n, -(-H // 128)), torch.uint8, skew)
    B.mdlm_ckpt8_save(g.t, q.t, qe.t)
    out = Guarded((n, H), dtype, skew)
    B.mdlm_ckpt8_load(q.t, qe.t, out.t)
    assert q.intact() and qe.intact() and out.intact() and g.intact()
    return x64, q.t.cpu().numpy(), qe.t.cpu().numpy(), out.t


def check(x, dtype, skew=0):
    x64, q, qe, out = roundtrip(x, dtype, skew)
    want_q, want_e = ends.ckpt8_save(x64)
    assert np.array_equal(qe, want_e)
    nan = ~np.isfinite(x64)
    assert np.array_equal(q[~nan], want_q[~nan])
    assert ((q[nan] & 0x7F) == 0x7F).all()
    want = torch.from_numpy(ends.ckpt8_load(want_q, want_e)).float().to(dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.from_numpy(nan))
    keep = torch.from_numpy(~nan)
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,H,skew", [(1, 1, 0), (1, 127, 1), (2, 128, 0), (3, 129, 0), (5, 200, 3),
                                      (2, 1001, 5), (70, 136, 0), (3, 2816, 0), (1, 20000, 0),
                                      (260, 7, 0), (9, 256, 1)])
def test_checkpoint_bits(dtype, n, H, skew):
    rng = np.random.default_rng(n + H)
    x = rng.standard_normal((n, H)) * np.exp2(rng.integers(-6, 7, (n, H)))
    check(x, dtype, skew)


def test_every_scale():
    """Blocks of one magnitude each, from fp32's least subnormal to its largest
    value, at and on both sides of the border where the scale steps."""
    rows = []
    for k in range(-149, 128):
        for m in (1.0, 1.75, 1.75 * (1 + 2.0 ** -23), 1.875, 1.9999998807907104):
            v = np.float32(m * 2.0 ** k) if k > -127 else np.float32(2.0 ** k)
            rows.append(np.concatenate([[v], v * np.linspace(-1, 1, 15)]))
    check(np.array(rows, dtype=np.float32), torch.float32)


def test_ties_round_to_even():
    """Midpoints between neighbouring codes, under a scale of one."""
    vals = np.array([ends.e4m3_value(c) for c in range(127)])
    mid = np.concatenate([(vals[1:] + vals[:-1]) / 2, [448.0, -448.0]])
    check(mid[None, :], torch.float32)
    check(-mid[None, :], torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nonfinite_entries_leave_their_block_alone(dtype):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 384))
    x[0, 3], x[1, 130], x[2, 383] = np.inf, np.nan, -np.inf
    x[3, :128] = np.nan  # nothing finite in the block
    check(x, dtype)


def test_a_checkpoint_of_one_type_restores_into_the_other():
    x, x64 = to_dev(np.random.default_rng(1).standard_normal((6, 300)), torch.float32)
    q = torch.empty(6, 300, dtype=torch.uint8, device=DEV)
    qe = torch.empty(6, 3, dtype=torch.uint8, device=DEV)
    B.mdlm_ckpt8_save(x.t, q, qe)
    a, b = torch.empty(6, 300, device=DEV), torch.empty(6, 300, device=DEV, dtype=torch.bfloat16)
    B.mdlm_ckpt8_load(q, qe, a)
    B.mdlm_ckpt8_load(q, qe, b)
    assert np.array_equal(f64(a), f64(b))  # four significant bits fit both
    assert np.abs(f64(a) - x64).max() <= 2.0 ** -4 * np.abs(x64).max()


def test_every_code_and_scale_byte_restores():
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(256, 1).to(DEV)
    qe = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 2).to(DEV)
    q, qe = q[:248].contiguous(), qe[:248].contiguous()  # a save writes bytes up to 247
    x = torch.empty(248, 256, device=DEV)
    B.mdlm_ckpt8_load(q, qe, x)
    want = ends.ckpt8_load(q.cpu().numpy(), qe.cpu().numpy())
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)  # exact, or past float32's largest value: infinite
    assert np.array_equal(x.cpu().numpy(), want, equal_nan=True)


def test_checkpoint_refusals_and_no_rows():
    x = torch.zeros(3, 130, device=DEV)
    q = torch.zeros(3, 130, dtype=torch.uint8, device=DEV)
    qe = torch.zeros(3, 2, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        B.mdlm_ckpt8_save(x, q, qe[:, :1].contiguous())
    with pytest.raises(TypeError):
        B.mdlm_ckpt8_save(x, q.to(torch.int8), qe)
    with pytest.raises(ValueError):
        B.mdlm_ckpt8_load(q[:, ::2], qe, x[:, :65].contiguous())
    with pytest.raises(TypeError):
        B.mdlm_ckpt8_load(q, qe, x.half())
    e = x[:0]
    B.mdlm_ckpt8_save(e, q[:0], qe[:0])
    B.mdlm_ckpt8_load(q[:0], qe[:0], e)
