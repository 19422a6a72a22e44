"""mdlm_sample where the draw falls among weights far below the row's: the
first tokens of a row for u = 0 and below, and for u under any share that the
heavy tokens leave."""

import numpy as np
import pytest
import torch

from ends_common import DEV, f64
from oracle import answer
from test_gpu_sample import check, draw

pytestmark = pytest.mark.gpu
RNG = np.random.default_rng
DT = [torch.bfloat16, torch.float32]
V = 20011
FAINT = [0.0, -1.0, np.nan, 1e-45, 1e-30, 1e-19, 1e-12, 2.0 ** -31, 2.0 ** -29, 1e-7]


def light_rows(m, T, dtype, seed, rate=0.4, tops=(9000, 16000)):
    """Logits 45 to 150 T under the top, with what they are mixed with left out
    (-inf), and two equal tops."""
    rng = RNG(seed)
    x = np.where(rng.random((m, V)) < rate, -T * rng.uniform(45, 150, (m, V)), -np.inf)
    x[:, list(tops)] = 0.0
    return torch.from_numpy(x).to(dtype).to(DEV)


def few_and_many(x, u, **kw):
    """Each row against the oracle, few at a time (cut into segments); the same
    rows among so many that each is one block's give the same tokens."""
    check(x, u, **kw)
    m = 300
    big = x.repeat(-(-m // x.shape[0]), 1)[:m].contiguous()
    par = {k: np.broadcast_to(v, (x.shape[0],)) for k, v in dict(kw, u=u).items()}
    par = {k: np.resize(v, m) for k, v in par.items()}
    tok, _ = draw(big, **par)
    want, _ = draw(x, u, **kw)
    assert np.array_equal(tok, np.resize(want, m))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [1.0, 0.3])
@pytest.mark.parametrize("rate", [0.4, 0.002])
def test_first_tokens(dtype, T, rate):
    x = light_rows(len(FAINT), T, dtype, 1, rate)
    few_and_many(x, np.array(FAINT, dtype=np.float32), T=T)


def test_one_light_token():
    x = torch.full((1, 8192), -np.inf, device=DEV)
    x[0, 5], x[0, 5000] = -50.0, 0.0
    for u in (0.0, -1.0, np.nan):
        check(x, np.array([u]))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kw", [dict(), dict(min_p=1e-38), dict(top_k=3), dict(top_k=4000)])
def test_light_tokens_between_equal_tops(dtype, kw):
    """u = 1/2 of two equal tops: the border lies among the light tokens between
    them.  Sums in fp64 place it within 2^-50 of the row; what is drawn there has
    a weight."""
    x = light_rows(4, 1.0, dtype, 2)
    x = x.repeat(75, 1).contiguous()
    for rows in (x[:4], x):
        tok, _ = draw(rows, np.full(len(rows), 0.5), **kw)
        for i in list(range(4)) + [len(rows) - 1]:
            order, w = answer.kept(f64(rows[i]), **kw)
            at = np.argsort(order)
            units = answer._exact(w[at])
            k = int(np.flatnonzero(order[at] == tok[i])[0])
            before, whole = sum(units[:k]), sum(units)
            assert units[k] > 0
            assert 2 * before - whole <= whole >> 49 and whole - 2 * (before + units[k]) <= whole >> 49


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kw", [dict(min_p=1e-38), dict(top_p=0.9), dict(top_p=0.9999999)])
def test_first_tokens_that_are_kept(dtype, kw):
    x = light_rows(len(FAINT), 1.0, dtype, 3)
    few_and_many(x, np.array(FAINT, dtype=np.float32), **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("spread", [150.0, 12.0])
@pytest.mark.parametrize("k", [9000])
def test_first_tokens_of_a_large_top_k(dtype, spread, k):
    """Tokens of all weights down to e^-spread, alone, and with top-p and min-p."""
    rng = RNG(k)
    m = len(FAINT)
    x = -spread * rng.random((m, V)) ** 0.5
    x[:, 3::4] = -np.inf
    x[:, 15000] = 0.0
    x = torch.from_numpy(x).to(dtype).to(DEV)
    u = np.array(FAINT, dtype=np.float32)
    few_and_many(x, u, top_k=np.full(m, k))
    few_and_many(x, u, top_k=np.full(m, k), top_p=np.full(m, 0.999999))
    few_and_many(x, u, top_k=np.full(m, k), min_p=np.full(m, 1e-30))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tops", [2, 8])
@pytest.mark.parametrize("width", [40, 4000, V])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=3000), dict(top_k=9000)])
def test_borders_between_equal_tops(dtype, tops, width, kw):
    """u on the border between two of some equal logits, `width` apart at most, all
    else 180 and more under them: next to those it adds nothing to a sum, and the draw
    is the next of them."""
    rng = RNG(tops + width)
    m = tops - 1
    x = -rng.uniform(180, 600, (m, V))
    x[rng.random((m, V)) < 0.2] = -np.inf
    for i in range(m):
        x[i, rng.integers(0, V - width + 1) + rng.choice(width, tops, replace=False)] = 0.0
    x = torch.from_numpy(x).to(dtype).to(DEV)
    u = (np.arange(1, tops) / tops).astype(np.float32)
    few_and_many(x, u, **{k: np.full(m, v) for k, v in kw.items()})
