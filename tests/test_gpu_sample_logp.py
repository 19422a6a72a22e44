"""mdlm_sample's log-probability does not depend on where a row's logits lie:
its bound counts distances from the largest logit."""

import numpy as np
import pytest
import torch

from ends_common import DEV, U, f64
from test_gpu_sample import draw

pytestmark = pytest.mark.gpu
RNG = np.random.default_rng


def bound(row, rebased, n):
    """Of a softmax term e^-d: 2^y of the exponent y = -d log2(e), whose two
    roundings (log2(e)'s own, at half a step of it, and y's) weigh 1.5 d U, and of
    which d U more may come from an offset's remainder; 2^y and the offset's
    factor, at a step each; three additions of a vector's terms (seven of eight);
    and, with each of `rebased` larger logits met, a factor of one such power more,
    2 U besides its distance, which the term's d counts."""
    d = row.max() - row
    p = np.exp(-d)
    return float((p * U * (2.5 * d + 2 * 4 + n + 2 * rebased)).sum() / p.sum())


@pytest.mark.parametrize("falling", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,m", [(777, 3), (20011, 3), (20011, 300), (126464, 2)])
@pytest.mark.parametrize("offset", [0.0, -30.0, 100.0, 1000.0, -1e4, 1e6, 3e8])
def test_offset(falling, dtype, V, m, offset):
    x = RNG(V + m).standard_normal((min(m, 3), V)) * 2 + offset
    n = 4 if dtype == torch.float32 else 8  # logits of a vector
    # a lane meets a larger one in each of its vectors at most, in a falling row in
    # none but the first; then lanes, waves and segments are joined
    rebased = 3 + (1 if falling else -(-V // (512 * n)) + 1)
    if falling:
        x = -np.sort(-x, axis=1)
    x = torch.from_numpy(x).to(dtype).to(DEV)
    x = x.repeat(-(-m // len(x)), 1)[:m].contiguous()
    u = np.resize(np.array([0.2, 0.5, 0.9], dtype=np.float32), m)
    for kw in (dict(), dict(top_k=9), dict(top_p=0.9), dict(T=0.0)):
        tok, lp = draw(x, u, **kw)
        for i in range(min(m, 3)):
            row = f64(x[i])
            d = row - row.max()
            want = d[tok[i]] - np.log(np.exp(d).sum())
            assert abs(lp[i] - want) <= bound(row, rebased, n) + U * abs(want), (i, lp[i],
                                                                                want)
        assert np.array_equal(lp, np.resize(lp[:min(m, 3)], m))
