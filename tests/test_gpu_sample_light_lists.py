"""mdlm_sample's draws among light tokens where the kept ones are a list's."""

import numpy as np
import pytest
import torch

from ends_common import DEV
from test_gpu_sample_light import DT, FAINT, RNG, V, few_and_many, light_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("spread", [150.0, 12.0])
@pytest.mark.parametrize("k", [3, 60, 255, 300, 3000])
def test_first_tokens_of_top_k(dtype, spread, k):
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
def test_light_lists(dtype):
    """Lists whose other entries are far lighter than the first."""
    m = len(FAINT)
    u = np.array(FAINT, dtype=np.float32)
    x = light_rows(m, 1.0, dtype, 5, 0.01, tops=(19000,))
    for k in (2, 50, 130, 200):  # about 200 are left
        few_and_many(x, u, top_k=np.full(m, k))
    x = light_rows(m, 1.0, dtype, 6, 0.1, tops=(19000,))
    for k in (300, 1500):
        few_and_many(x, u, top_k=np.full(m, k))
        few_and_many(x, u, top_k=np.full(m, k), min_p=np.full(m, 1e-38))
