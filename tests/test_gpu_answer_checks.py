"""Checking mode and the product's row list, with and without a device count."""

import pytest
import torch

from ends_common import DEV
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu


def product(rows, count, n=20, V=70, H=64):
    q, e = B.mx_shapes((n, H), B.MDLM_MX_E4M3)
    a = torch.full(q, 0x38, dtype=torch.uint8, device=DEV)  # ones
    wq, we = B.mx_shapes((V, H), B.MDLM_MX_E2M1)
    w = torch.full(wq, 0x22, dtype=torch.uint8, device=DEV)
    one = dict(dtype=torch.uint8, device=DEV)
    z = torch.full((len(rows), V), 5.0, device=DEV)
    B.mdlm_mx_product(a, torch.full(e, 127, **one), B.MDLM_MX_E4M3, w, torch.full(we, 127, **one), z,
                      row_idx=torch.tensor(rows, dtype=torch.int32, device=DEV),
                      n_rows=None if count is None else torch.tensor([count], dtype=torch.int32,
                                                                     device=DEV))
    return z


@pytest.mark.parametrize("rows,count,bad", [
    ([0, 19, 3, 3], None, False), ([0, 19, 3, 3], 4, False), ([0, 19, 3, 3], 0, False),
    ([-1, 2], None, True), ([2, 20], None, True), ([2] * 300 + [20], None, True),
    ([-1, 2], 2, True), ([2, 20], 2, True), ([2, 20], 1, False),  # (not among the counted)
])
def test_listed_rows(rows, count, bad):
    was = B.mdlm_set_checking(True)
    try:
        if bad:
            with pytest.raises(RuntimeError, match="row_idx"):
                product(rows, count)
        else:
            z = product(rows, count)
            n = len(rows) if count is None else count
            assert (z[:n] == 64.0).all() and (z[n:] == 5.0).all()
    finally:
        B.mdlm_set_checking(was)
    # without checking such a row counts as one of zeros
    z = product(rows, count)
    n = len(rows) if count is None else count
    for j in range(n):
        assert (z[j] == (64.0 if 0 <= rows[j] < 20 else 0.0)).all()
