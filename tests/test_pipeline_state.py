"""The order of MdlmTrainStep's calls, on the CPU with the library's calls
replaced by a record of their names: what is accepted reaches the library, what
is out of turn is refused before it does."""

import os

import pytest
import torch

from uniform_noise_diffusion_amd import binding as B
from uniform_noise_diffusion_amd import pipeline

CALLS = ("mdlm_corrupt", "mdlm_corrupt_mixture", "mdlm_compact_masked", "mdlm_embed",
         "mdlm_embed_grad", "mdlm_norm_fwd", "mdlm_norm_bwd_ckpt8", "mdlm_fused_head_ce_fwd_bwd",
         "mdlm_fused_head_ce_fwd_bwd_dw")
N, H, V = 6, 64, 90


@pytest.fixture
def calls(monkeypatch):
    """The calls that reached the library, as (name, arguments)."""
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmdlm.so not built")
    made = []
    for name in CALLS:
        monkeypatch.setattr(pipeline.B, name,
                            lambda *a, _name=name, **kw: made.append((_name, a, kw)))
    return made


def make(**kw):
    return pipeline.MdlmTrainStep(N, 1, H, V, device="cpu", **kw)


def begin(s):
    s.corrupt(None, None, 1, 0.3, 0, V - 1, V)


def forward(s, weight):
    begin(s)
    s.embed(torch.zeros(V, H))
    s.final_norm(s.embedded, weight)


W = torch.ones(H, dtype=torch.bfloat16)


def test_norm_without_a_weight(calls):
    """A norm whose weight is 1: final_norm() takes it, so norm_grad() does."""
    s = make()
    forward(s, None)
    s.head_ce_dw(torch.zeros(V, H))
    assert s.norm_grad() is s.d_last
    name, args, _ = calls[-1]
    assert name == "mdlm_norm_bwd_ckpt8" and args[4] is None
