"""CPU pins of the fp64 definitions of embedding, norm and 8-bit checkpoint
(oracle/ends.py): one-hot products, torch's own norms and their autograd in
float64, central differences, and torch's e4m3 casts."""

import numpy as np
import pytest
import torch

from oracle import ends

RNG = np.random.default_rng


def test_embedding_is_a_one_hot_product():
    rng = RNG(0)
    ids = np.array([3, 0, 3, -1, 7, 3, 5, 9], dtype=np.int32)  # -1 and 9: outside [0, 7]
    T = rng.standard_normal((8, 5))
    onehot = (ids[:, None] == np.arange(8)).astype(float)
    assert np.allclose(ends.embed(ids, T, 1.5), 1.5 * onehot @ T)
    d = rng.standard_normal((8, 5))
    start = rng.standard_normal((8, 5))
    got, size = ends.embed_grad(ids, d, 8, 1.5, start)
    assert np.allclose(got, start + 1.5 * onehot.T @ d)
    assert np.allclose(size, np.abs(start) + 1.5 * onehot.T @ np.abs(d))


@pytest.mark.parametrize("kind", [ends.NORM_LAYER, ends.NORM_RMS])
def test_norm_matches_torch_and_its_autograd(kind):
    rng = RNG(1)
    x, dy = rng.standard_normal((6, 40)) + 0.5, rng.standard_normal((6, 40))
    w, b = rng.standard_normal(40), rng.standard_normal(40)
    y, mu, r = ends.norm(x, kind, w, b, 1e-5)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    if kind == ends.NORM_LAYER:
        ty = torch.nn.functional.layer_norm(tx, (40,), tw, tb, 1e-5)
    else:
        ty = torch.nn.functional.rms_norm(tx, (40,), tw, 1e-5) + tb
    assert np.allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    ty.backward(torch.tensor(dy))
    dx, dw, db = ends.norm_grad(dy, x, kind, w, mu, r)
    for got, want in ((dx, tx), (dw, tw), (db, tb)):
        assert np.allclose(got, want.grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("kind", [ends.NORM_LAYER, ends.NORM_RMS])
def test_norm_gradient_against_differences(kind):
    rng = RNG(2)
    x, dy, w = rng.standard_normal((3, 9)), rng.standard_normal((3, 9)), rng.standard_normal(9)
    _, mu, r = ends.norm(x, kind, w, None, 1e-5)
    dx, dw, _ = ends.norm_grad(dy, x, kind, w, mu, r)
    h = 1e-6
    for i in range(3):
        for j in range(9):
            e = np.zeros_like(x)
            e[i, j] = h
            d = (dy * (ends.norm(x + e, kind, w, None, 1e-5)[0]
                       - ends.norm(x - e, kind, w, None, 1e-5)[0])).sum() / (2 * h)
            assert abs(d - dx[i, j]) < 1e-7
    for j in range(9):
        e = np.zeros(9)
        e[j] = h
        d = (dy * (ends.norm(x, kind, w + e, None, 1e-5)[0]
                   - ends.norm(x, kind, w - e, None, 1e-5)[0])).sum() / (2 * h)
        assert abs(d - dw[j]) < 1e-7


def test_e4m3_codes_are_torchs():
    all_codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = all_codes.view(torch.float8_e4m3fn).double().numpy()
    got = np.array([ends.e4m3_value(c) for c in range(256)])
    assert np.array_equal(got, want, equal_nan=True)
    # every value, every midpoint between neighbours and its neighbours, both signs
    vals = got[:127]
    mid = (vals[1:] + vals[:-1]) / 2
    v = np.concatenate([vals, mid, np.nextafter(mid.astype(np.float32), np.float32(np.inf)),
                        np.nextafter(mid.astype(np.float32), np.float32(0)), [2.0 ** -20, 0.0]])
    v = np.concatenate([v, -v])
    cast = torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert [ends.e4m3_code(x) for x in v] == list(cast)


def test_checkpoint_scale_is_the_least_and_the_error_bounded():
    rng = RNG(3)
    x = (rng.standard_normal((5, 300)) * np.exp2(rng.integers(-40, 40, (5, 300)))).astype(np.float32)
    x[0, :128] = 0.0
    x[1, 7], x[1, 200], x[2, 5] = np.inf, np.nan, -np.inf
    x[3, 0] = 448.0
    x[3, 1:128] = 0.25
    q, b = ends.ckpt8_save(x)
    y = ends.ckpt8_load(q, b)
    fin = np.isfinite(x)
    assert np.array_equal(np.isfinite(y), fin)
    assert b[3, 0] == 127  # 448 is held over 2^0
    assert b[0, 0] == 0 and not y[0, :128].any()
    for i in range(5):
        for j in range(3):
            blk = x[i, 128 * j:128 * j + 128].astype(np.float64)
            top = np.abs(blk[np.isfinite(blk)]).max()
            e = int(b[i, j]) - 127
            assert top <= 448.0 * 2.0 ** e
            assert e == -127 or top > 448.0 * 2.0 ** (e - 1)
    e = np.repeat(b.astype(int) - 127, 128, axis=1)[:, :300].astype(float)
    bound = np.maximum(np.abs(np.where(fin, x, 0.0).astype(np.float64)) * 2.0 ** -4,
                       2.0 ** -10 * np.exp2(e))
    assert np.all(np.abs(y - x)[fin] <= bound[fin])
