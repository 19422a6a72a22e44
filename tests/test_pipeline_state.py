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


def backward(s):
    s.head_ce_dw(torch.zeros(V, H))
    s.embed_grad(s.norm_grad())


@pytest.mark.parametrize("tied", [True, False])
def test_steps_in_order(calls, tied):
    s = make(tied=tied)
    for _ in range(3):
        forward(s, W)
        backward(s)
    names = [c[0] for c in calls]
    assert names == ["mdlm_corrupt", "mdlm_embed", "mdlm_norm_fwd",
                     "mdlm_fused_head_ce_fwd_bwd_dw", "mdlm_norm_bwd_ckpt8",
                     "mdlm_embed_grad"] * 3


def test_tied_gradient_is_added_once(calls):
    """The table's gradient goes into the dW of this step, once."""
    s = make()
    forward(s, W)
    backward(s)
    done = len(calls)
    with pytest.raises(RuntimeError, match="head_ce_dw"):
        s.embed_grad(s.d_last)  # again: dW holds the sum already
    forward(s, W)
    with pytest.raises(RuntimeError, match="head_ce_dw"):
        s.embed_grad(s.d_last)  # dW is the last step's
    assert len(calls) == done + 3
    backward(s)


@pytest.mark.parametrize("corrupt", ["corrupt", "corrupt_mixture"])
@pytest.mark.parametrize("tied", [True, False])
def test_gradient_of_tokens_that_are_gone(calls, corrupt, tied):
    """embed_grad() reads `xt`, which the next corruption overwrites."""
    s = make(tied=tied)
    forward(s, W)
    s.head_ce_dw(torch.zeros(V, H))
    dx = s.norm_grad()
    args = (None, None, 1, 0.3, 0.5, V - 1, V)
    getattr(s, corrupt)(*(args if corrupt == "corrupt_mixture" else args[:4] + (0,) + args[5:]))
    done = len(calls)
    with pytest.raises(RuntimeError, match="embed_grad"):
        s.embed_grad(dx)
    assert len(calls) == done


@pytest.mark.parametrize("skip", ["head_ce_dw", "final_norm", "both"])
def test_norm_gradient_of_an_earlier_step(calls, skip):
    s = make()
    forward(s, W)
    backward(s)
    begin(s)
    s.embed(torch.zeros(V, H))
    if skip == "head_ce_dw":
        s.final_norm(s.embedded, W)
    if skip == "final_norm":
        s.head_ce_dw(torch.zeros(V, H))
    done = len(calls)
    with pytest.raises(RuntimeError, match="head_ce" if skip == "head_ce_dw" else "final_norm"):
        s.norm_grad()
    assert len(calls) == done
    s.final_norm(s.embedded, W)
    backward(s)


def test_norm_gradient_needs_a_gradient(calls):
    """The first step as well: `d_hidden` holds nothing before a head has run,
    and nothing of these hidden states after another final_norm()."""
    s = make()
    forward(s, W)
    with pytest.raises(RuntimeError, match="head_ce"):
        s.norm_grad()
    s.head_ce(s.hidden, torch.zeros(V, H), 0.0, want_grad=False)
    with pytest.raises(RuntimeError, match="head_ce"):
        s.norm_grad()
    s.head_ce(s.hidden, torch.zeros(V, H), 0.0)  # a frozen head leaves one too
    s.norm_grad()
    s.norm_grad()  # (the same once more)
    s.final_norm(s.embedded, W)
    with pytest.raises(RuntimeError, match="head_ce"):
        s.norm_grad()
    mine = torch.zeros(N, H, dtype=torch.bfloat16)
    s.norm_grad(d_hidden=mine)  # the caller's own
    assert calls[-1][1][0] is mine


def test_norm_gradient_after_the_next_corruption(calls):
    """What norm_grad() reads is not overwritten by it."""
    s = make()
    forward(s, W)
    s.head_ce_dw(torch.zeros(V, H))
    begin(s)
    s.norm_grad()


@pytest.mark.parametrize("tied", [True, False])
def test_gradient_without_the_steps_embedding(calls, tied):
    """A caller that embeds `xt` in its own way calls no embed()."""
    s = make(tied=tied)
    for _ in range(2):
        begin(s)
        s.final_norm(s.embedded, W)
        backward(s)


def test_a_refused_call_changes_nothing(calls, monkeypatch):
    def refuse(*a, **kw):
        raise ValueError("shape")

    s = make()
    begin(s)
    with monkeypatch.context() as m:
        m.setattr(pipeline.B, "mdlm_norm_fwd", refuse)
        m.setattr(pipeline.B, "mdlm_fused_head_ce_fwd_bwd_dw", refuse)
        with pytest.raises(ValueError):
            s.final_norm(s.embedded, W)
        with pytest.raises(ValueError):
            s.head_ce_dw(torch.zeros(V, H))
    with pytest.raises(RuntimeError, match="final_norm"):
        s.norm_grad()
    with pytest.raises(RuntimeError, match="head_ce_dw"):
        s.embed_grad(s.d_last)
    s.final_norm(s.embedded, W)
    s.head_ce_dw(torch.zeros(V, H))
    dx = s.norm_grad()
    with monkeypatch.context() as m:
        m.setattr(pipeline.B, "mdlm_embed_grad", refuse)
        with pytest.raises(ValueError):
            s.embed_grad(dx)
    s.embed_grad(dx)


def test_calls_recorded_in_a_graph(calls, monkeypatch):
    """A graph's replays are not seen: once calls of the step are recorded, the
    others may follow them in every step."""
    s = make()
    capturing = [False]
    monkeypatch.setattr(s, "_capturing", lambda stream: capturing[0])
    forward(s, W)  # (a warm-up pass)
    backward(s)
    capturing[0] = True
    forward(s, W)
    s.head_ce_dw(torch.zeros(V, H))
    capturing[0] = False
    for _ in range(3):  # replay, then
        s.embed_grad(s.norm_grad())
    fresh = make()
    monkeypatch.setattr(fresh, "_capturing", lambda stream: True)
    fresh.embed(torch.zeros(V, H))
    with pytest.raises(RuntimeError, match="final_norm"):
        fresh.norm_grad()  # (a graph that records this reads what nothing wrote)
    with pytest.raises(RuntimeError, match="head_ce_dw"):
        fresh.embed_grad(fresh.d_last)
