"""MdlmTrainStep in use on the GPU: a step of which a graph holds a part, on
side streams, and a norm without a weight."""

import pytest
import torch

import uniform_noise_diffusion_amd as M
import workloads as WL
from ends_common import DEV
from gpu_common import dev_float, dev_tokens
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu


def make(wl, **kw):
    return M.MdlmTrainStep(wl.n_tokens, wl.n_docs, wl.H, wl.V, device=DEV, **kw)


def outputs(s):
    return [t.clone() for t in (s.loss, s.d_last, s.d_norm_weight, s.dW, s.d_table)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("tied", [True, False])
def test_part_of_a_step_in_a_graph(tied):
    """The forward pass and the head in a graph that another stream recorded,
    the gradients eagerly behind every replay."""
    inp = WL.small_case(8, n_docs=4, max_len=300, H=192, V=700)
    wl = inp.wl
    x0, cu = dev_tokens(inp)
    _, W = dev_float(inp)
    T = W if tied else torch.randn_like(W)
    w = torch.ones(wl.H, device=DEV, dtype=torch.bfloat16)
    step, ref = make(wl, tied=tied), make(wl, tied=tied)

    def forward(s, stream=None):
        s.corrupt(x0, cu, wl.seed, 0.3, wl.noise, wl.mask_id, wl.rand_vocab, stream)
        s.compact(x0, cu, wl.align, stream)
        s.final_norm(s.embed(T, stream), w, stream=stream)
        s.head_ce_dw(W, stream=stream)

    forward(step)
    step.embed_grad(step.norm_grad())
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(torch.cuda.default_stream()):
            forward(step, side)  # given the stream, another being the current one
    g = torch.Generator(device=DEV).manual_seed(0)
    for rep in range(3):
        W.copy_((torch.randn(W.shape, device=DEV, generator=g) * 0.02 * (1 + rep)).to(W.dtype))
        graph.replay()
        step.embed_grad(step.norm_grad())
        forward(ref)
        ref.embed_grad(ref.norm_grad())
        torch.cuda.synchronize()
        assert same(outputs(step), outputs(ref)), rep


@pytest.mark.parametrize("kind", [B.MDLM_NORM_LAYER, B.MDLM_NORM_RMS])
def test_step_whose_norm_has_no_weight(kind):
    """The same bits as with a weight of ones."""
    inp = WL.small_case(5, n_docs=3, max_len=200, H=192, V=500)
    wl = inp.wl
    x0, cu = dev_tokens(inp)
    _, W = dev_float(inp)
    got = []
    for weight in (None, torch.ones(wl.H, device=DEV, dtype=torch.bfloat16)):
        s = make(wl, norm_kind=kind)
        s.corrupt(x0, cu, wl.seed, 0.3, wl.noise, wl.mask_id, wl.rand_vocab)
        s.compact(x0, cu, wl.align)
        s.final_norm(s.embed(W), weight)
        s.head_ce_dw(W)
        s.embed_grad(s.norm_grad())
        torch.cuda.synchronize()
        got.append(outputs(s))
    assert same(*got)


def test_gradients_refused_out_of_turn_write_nothing():
    inp = WL.small_case(6, n_docs=2, max_len=100, H=64, V=90)
    wl = inp.wl
    x0, cu = dev_tokens(inp)
    _, W = dev_float(inp)
    s = make(wl)
    s.corrupt(x0, cu, wl.seed, 0.3, wl.noise, wl.mask_id, wl.rand_vocab)
    s.compact(x0, cu, wl.align)
    s.final_norm(s.embed(W), None)
    s.head_ce_dw(W)
    s.embed_grad(s.norm_grad())
    torch.cuda.synchronize()
    kept = outputs(s)
    with pytest.raises(RuntimeError, match="head_ce_dw"):
        s.embed_grad(s.d_last)
    s.corrupt(x0, cu, wl.seed + 1, 0.3, wl.noise, wl.mask_id, wl.rand_vocab)
    with pytest.raises(RuntimeError, match="final_norm"):
        s.norm_grad()
    torch.cuda.synchronize()
    assert same(kept, outputs(s))
