"""The two ends in use: a whole training step (corruption, embedding, final
norm with an 8-bit checkpoint, trained tied head, the gradients back into the
table), the differentiable calls, streams and captured graphs."""

import numpy as np
import pytest
import torch

import uniform_noise_diffusion_amd as M
import workloads as WL
from ends_common import DEV, f64
from gpu_common import dev_float, dev_tokens
from oracle import ends
from uniform_noise_diffusion_amd import binding as B

pytestmark = pytest.mark.gpu


def make_step(inp, kind, tied, bias):
    wl = inp.wl
    return M.MdlmTrainStep(wl.n_tokens, wl.n_docs, wl.H, wl.V, norm_kind=kind, norm_bias=bias,
                           embed_scale=1.25, tied=tied, device=DEV)


def run_step(step, inp, table, W, w, b):
    """One step of a model without layers of its own: embedding, norm, head."""
    wl = inp.wl
    x0, cu = dev_tokens(inp)
    step.corrupt(x0, cu, wl.seed, 0.3, wl.noise, wl.mask_id, wl.rand_vocab)
    step.compact(x0, cu, wl.align)
    step.final_norm(step.embed(table), w, b)
    step.head_ce_dw(W, 30.0)
    step.embed_grad(step.norm_grad())
    return step


@pytest.mark.parametrize("kind", [B.MDLM_NORM_LAYER, B.MDLM_NORM_RMS])
@pytest.mark.parametrize("tied", [True, False])
def test_training_step_against_float64(kind, tied):
    """Loss and gradients of the step against the formulas in float64 on the
    values the device holds.  bf16 rounds the norm's output, the head's
    per-logit gradient, d_hidden and dx by up to 2^-8 each: relative norms
    within 1e-2 for the gradients, 1e-3 for the loss, as for the head alone."""
    inp = WL.small_case(5, n_docs=4, max_len=300, H=256, V=900)
    wl = inp.wl
    bias = kind == B.MDLM_NORM_LAYER
    _, W = dev_float(inp)
    table = W if tied else (torch.randn(wl.V, wl.H, device=DEV) * 0.5).bfloat16()
    w = (1 + 0.1 * torch.randn(wl.H, device=DEV)).bfloat16()
    b = (0.1 * torch.randn(wl.H, device=DEV)).bfloat16() if bias else None
    step = run_step(make_step(inp, kind, tied, bias), inp, table, W, w, b)
    m = int(step.n_rows.item())
    assert m > 50

    ids, xt64 = step.xt.cpu().numpy(), f64(table)
    emb = ends.embed(ids, xt64, 1.25)
    assert np.array_equal(f64(step.embedded),
                          torch.from_numpy(emb).float().bfloat16().double().numpy())
    emb = f64(step.embedded)
    w64, b64 = f64(w), None if b is None else f64(b)
    y, mu, r = ends.norm(emb, kind, w64, b64, 1e-5)
    held = ends.ckpt8_load(*(t.cpu().numpy() for t in (step.q, step.q_exp)))
    assert np.linalg.norm(held - emb) < 2.0 ** -4 * np.linalg.norm(emb)

    rows, tgt = (t[:m].cpu().numpy() for t in (step.row_idx, step.tgt))
    wt = f64(step.w[:m])
    h = f64(step.hidden)[rows]
    W64 = f64(W)
    z = 30.0 * np.tanh(h @ W64.T / 30.0)
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    loss = -(wt * np.log(p[np.arange(m), tgt])).sum()
    assert abs(float(step.loss.item()) - loss) < 1e-3 * abs(loss)
    G = p.copy()
    G[np.arange(m), tgt] -= 1.0
    G *= wt[:, None] * (1 - (z / 30.0) ** 2)
    dh = np.zeros_like(emb)
    dh[rows] = G @ W64
    dx, dw, db = ends.norm_grad(dh, held, kind, w64, mu, r)
    d_table, _ = ends.embed_grad(ids, dx, wl.V, 1.25, G.T @ h if tied else None)

    def close(got, want):
        assert np.linalg.norm(f64(got) - want) < 1e-2 * np.linalg.norm(want)

    close(step.hidden, y)
    close(step.d_last, dx)
    close(step.d_norm_weight, dw)
    if bias:
        close(step.d_norm_bias, db)
    close(step.d_table, d_table)
    if not tied:
        close(step.dW, G.T @ h)


def test_step_refuses_what_it_was_not_made_for():
    inp = WL.small_case(6, n_docs=2, max_len=20, H=64, V=90)
    step = make_step(inp, B.MDLM_NORM_RMS, True, False)
    with pytest.raises(RuntimeError, match="final_norm"):
        step.norm_grad()
    x, w = torch.zeros_like(step.embedded), torch.ones(64, device=DEV, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="norm_bias"):
        step.final_norm(x, w, w)
    with pytest.raises(RuntimeError, match="head_ce_dw"):
        step.embed_grad(x)


def test_captured_step_replays_match_eager():
    """A captured step, replayed between eager steps on other weights, gives the
    eager step's bits every time; two graphs that share the step's workspaces
    replay one after the other."""
    inp = WL.small_case(8, n_docs=5, max_len=600, H=192, V=1100)
    wl = inp.wl
    _, W = dev_float(inp)
    w = torch.ones(wl.H, device=DEV, dtype=torch.bfloat16)
    step, ref = (make_step(inp, B.MDLM_NORM_RMS, True, False) for _ in range(2))
    x0, cu = dev_tokens(inp)
    args = (wl.seed, 0.3, wl.noise, wl.mask_id, wl.rand_vocab)

    def go(s):
        s.corrupt(x0, cu, *args)
        s.compact(x0, cu, wl.align)
        s.final_norm(s.embed(W), w)
        s.head_ce_dw(W, 0.0)
        s.embed_grad(s.norm_grad())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(step)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            go(step)
    gen = torch.Generator(device=DEV).manual_seed(0)
    for rep in range(4):
        W.copy_((torch.randn(W.shape, device=DEV, generator=gen) * 0.02 * (1 + rep)).to(W.dtype))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        go(ref)
        torch.cuda.synchronize()
        for a, b in ((step.dW, ref.dW), (step.d_norm_weight, ref.d_norm_weight),
                     (step.loss, ref.loss)):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), rep


def test_side_streams_give_the_same_bits():
    """Two calls at once on two streams, with allocated workspaces, against the
    default stream's results."""
    g = torch.Generator(device=DEV).manual_seed(2)
    n, H, V = 3000, 264, 800
    cases = []
    for k in range(2):
        ids = torch.randint(-1, V, (n,), device=DEV, generator=g, dtype=torch.int32)
        dy = torch.randn(n, H, device=DEV, generator=g).bfloat16()
        x = torch.randn(n, H, device=DEV, generator=g).bfloat16()
        cases.append((ids, dy, x))

    def go(case, stream):
        ids, dy, x = case
        out = [torch.empty(V, H, device=DEV), torch.empty_like(x), torch.empty(n, device=DEV),
               torch.empty_like(x), torch.empty(H, device=DEV), torch.empty(H, device=DEV)]
        q = torch.empty(n, H, dtype=torch.uint8, device=DEV)
        qe = torch.empty(n, 3, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        return out, q, qe, stream

    def enqueue(case, made):
        ids, dy, x = case
        out, q, qe, stream = made
        B.mdlm_embed_grad(ids, dy, 1.0, out[0], stream=stream)
        B.mdlm_norm_fwd(x, 1, None, None, 1e-5, out[1], None, out[2], q, qe, stream=stream)
        B.mdlm_norm_bwd_ckpt8(dy, q, qe, 1, None, None, out[2], out[3], out[4], out[5],
                              stream=stream)

    ref = []
    for c in cases:
        made = go(c, None)
        enqueue(c, made)
        torch.cuda.synchronize()
        ref.append(made[0])
    for _ in range(3):
        made = [go(c, torch.cuda.Stream()) for c in cases]
        for c, m in zip(cases, made):
            enqueue(c, m)
        torch.cuda.synchronize()
        for r, m in zip(ref, made):
            assert all(torch.equal(a, b) for a, b in zip(r, m[0]))


# ---- the differentiable calls -----------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_embed_tokens_gradient(dtype):
    T = torch.randn(50, 24, device=DEV).to(dtype).requires_grad_()
    ids = torch.randint(-1, 50, (3, 40), device=DEV, dtype=torch.int32)
    out = M.embed_tokens(ids, T, 2.0)
    assert out.shape == (3, 40, 24) and out.dtype == dtype
    seen = ids.clone()
    ids.fill_(7)  # a token buffer reused before the backward pass
    out.sum().backward()  # an expanded gradient
    want, _ = ends.embed_grad(seen.cpu().numpy().ravel(), np.ones((120, 24)), 50, 2.0)
    assert np.array_equal(f64(T.grad), want)  # small whole numbers: exact in both types
    with torch.no_grad():
        assert M.embed_tokens(seen, T).grad_fn is None


@pytest.mark.parametrize("kind", [B.MDLM_NORM_LAYER, B.MDLM_NORM_RMS])
@pytest.mark.parametrize("checkpoint8", [False, True])
def test_norm_function_gradients(kind, checkpoint8):
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(2, 9, 136, device=DEV, generator=g)
    if checkpoint8:  # values an 8-bit checkpoint holds exactly
        x = x.to(torch.float8_e4m3fn).float()
    x.requires_grad_()
    w = torch.randn(136, device=DEV, generator=g).requires_grad_()
    b = torch.randn(136, device=DEV, generator=g).requires_grad_()
    dy = torch.randn(9, 2, 136, device=DEV, generator=g).transpose(0, 1)  # not contiguous
    y = M.norm(x, w, b, 1e-5, kind, checkpoint8)
    gx, gw, gb = torch.autograd.grad(y, (x, w, b), dy)
    x64, w64 = (t.detach().double().cpu().requires_grad_() for t in (x, w))
    b64 = b.detach().double().cpu().requires_grad_()
    if kind == B.MDLM_NORM_LAYER:
        y64 = torch.nn.functional.layer_norm(x64, (136,), w64, b64, 1e-5)
    else:
        y64 = torch.nn.functional.rms_norm(x64, (136,), w64, 1e-5) + b64
    want = torch.autograd.grad(y64, (x64, w64, b64), dy.double().cpu())
    # a few dozen fp32 roundings: 1e-5 of the norm
    for got, ref in zip((y, gx, gw, gb), (y64, *want)):
        err = (got.detach().double().cpu() - ref.detach()).norm() / ref.detach().norm()
        assert float(err) < 1e-5


def test_norm_function_saves_no_x_with_a_checkpoint():
    x = torch.randn(8, 256, device=DEV, requires_grad=True)
    y = M.norm(x, checkpoint8=True)
    kept = [t for t in y.grad_fn.saved_tensors if t is not None]
    assert all(t.data_ptr() != x.data_ptr() for t in kept)
    assert sum(t.numel() * t.element_size() for t in kept) < 0.3 * x.numel() * 4
    with torch.no_grad():
        x.mul_(2.0)  # x is not needed any more
    y.sum().backward()
    z = M.norm(x)
    with torch.no_grad():
        x.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        z.sum().backward()


def test_only_the_gradients_asked_for():
    x = torch.randn(4, 64, device=DEV)
    w = torch.ones(64, device=DEV, requires_grad=True)
    y = M.norm(x, w, torch.zeros(64, device=DEV))
    y.sum().backward()
    assert x.grad is None and w.grad is not None
    assert M.norm(x).grad_fn is None
    with pytest.raises(ValueError, match="contiguous"):
        M.norm(x.t())
    with pytest.raises(RuntimeError):  # no second derivative
        xx = x.clone().requires_grad_()
        (gx,) = torch.autograd.grad(M.norm(xx).square().sum(), xx, create_graph=True)
        gx.sum().backward()


def test_chain_of_differentiable_calls():
    """embed_tokens -> norm -> masked_diffusion_loss: the table's gradient
    against the same chain in float64 (the head frozen)."""
    inp = WL.small_case(12, n_docs=3, max_len=150, H=128, V=500)
    wl = inp.wl
    x0, cu = dev_tokens(inp)
    _, W = dev_float(inp)
    step = M.MdlmLossStep(wl.n_tokens, wl.n_docs, wl.H, wl.V, device=DEV, want_grad=False)
    step.corrupt(x0, cu, 3, 0.3, wl.noise, wl.mask_id, wl.rand_vocab)
    step.compact(x0, cu, wl.align)
    T = torch.randn(wl.V, wl.H, device=DEV).bfloat16().requires_grad_()
    h = M.norm(M.embed_tokens(step.xt, T, 0.5), kind=B.MDLM_NORM_RMS)
    loss = M.masked_diffusion_loss(h, W, step.row_idx, step.tgt, step.w, step.n_rows)
    loss.backward()
    m = int(step.n_rows.item())
    T64 = T.detach().double().cpu().requires_grad_()
    e = T64[step.xt.long().cpu()] * 0.5
    h64 = torch.nn.functional.rms_norm(e, (wl.H,), None, 1e-5)
    z = h64[step.row_idx[:m].long().cpu()] @ W.double().cpu().T
    ce = torch.nn.functional.cross_entropy(z, step.tgt[:m].long().cpu(), reduction="none")
    l64 = (ce * step.w[:m].double().cpu()).sum()
    l64.backward()
    assert abs(float(loss) - float(l64)) < 1e-3 * abs(float(l64))
    err = (T.grad.double().cpu() - T64.grad).norm() / T64.grad.norm()
    assert float(err) < 1e-2


def test_each_call_captured_with_its_own_workspace():
    """Every call by itself in one graph, workspaces allocated inside the
    capture; replays on new inputs, with eager calls between, against eager
    results bit for bit."""
    n, H, V = 700, 200, 300
    g = torch.Generator(device=DEV).manual_seed(9)
    ids = torch.randint(-1, V, (n,), device=DEV, generator=g, dtype=torch.int32)
    x, dy = (torch.randn(n, H, device=DEV, generator=g).bfloat16() for _ in range(2))
    T = torch.randn(V, H, device=DEV, generator=g).bfloat16()
    w = torch.randn(H, device=DEV, generator=g).bfloat16()

    def go():
        f32 = dict(device=DEV, dtype=torch.float32)
        emb, y, back, dx = (torch.empty(n, H, device=DEV, dtype=torch.bfloat16)
                            for _ in range(4))
        d_t, dw, db = torch.empty(V, H, **f32), torch.empty(H, **f32), torch.empty(H, **f32)
        mean, rstd = torch.empty(n, **f32), torch.empty(n, **f32)
        q = torch.empty(n, H, device=DEV, dtype=torch.uint8)
        qe = torch.empty(n, 2, device=DEV, dtype=torch.uint8)
        B.mdlm_embed(ids, T, 0.5, emb)
        B.mdlm_norm_fwd(x, B.MDLM_NORM_LAYER, w, None, 1e-6, y, mean, rstd)
        B.mdlm_norm_bwd(dy, x, B.MDLM_NORM_LAYER, w, mean, rstd, dx, dw, db)
        B.mdlm_embed_grad(ids, dy, 0.5, d_t)
        B.mdlm_ckpt8_save(x, q, qe)
        B.mdlm_ckpt8_load(q, qe, back)
        return emb, y, mean, rstd, dx, dw, db, d_t, back

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go()
    for rep in range(4):
        x.copy_((torch.randn(n, H, device=DEV, generator=g) * (rep + 1)).bfloat16())
        dy.copy_(torch.randn(n, H, device=DEV, generator=g).bfloat16())
        ids.copy_(torch.randint(-1, V, (n,), device=DEV, generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, go()):
            assert torch.equal(a, b), rep


def test_captured_gradients_of_the_functions():
    """embed_tokens -> norm forward and backward in one graph, warmed up on a
    side stream whose graphs are gone by then; replays on new inputs, with eager
    passes over the same leaves between, against those bit for bit."""
    n, H, V = 300, 264, 90
    g = torch.Generator(device=DEV).manual_seed(10)
    ids = torch.randint(-1, V, (n,), device=DEV, generator=g, dtype=torch.int32)
    dy = torch.randn(n, H, device=DEV, generator=g).bfloat16()
    T = torch.randn(V, H, device=DEV, generator=g).bfloat16().requires_grad_()
    w, b = (torch.randn(H, device=DEV, generator=g).bfloat16().requires_grad_()
            for _ in range(2))

    def go():
        y = M.norm(M.embed_tokens(ids, T, 0.5), w, b, checkpoint8=True)
        return (y.detach(), *torch.autograd.grad(y, (T, w, b), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            go()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = go()
    for rep in range(4):
        ids.copy_(torch.randint(-1, V, (n,), device=DEV, generator=g, dtype=torch.int32))
        dy.copy_(torch.randn(n, H, device=DEV, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        for t, want in zip(got, go()):
            assert torch.equal(t, want), rep


def test_step_without_tokens():
    step = M.MdlmTrainStep(0, 0, 64, 90, device=DEV)
    T = torch.randn(90, 64, device=DEV).bfloat16()
    w = torch.ones(64, device=DEV, dtype=torch.bfloat16)
    cu, x0 = torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32,
                                                                        device=DEV)
    step.corrupt(x0, cu, 1, 0.3, 0, 89, 90)
    step.compact(x0, cu, 0)
    step.final_norm(step.embed(T), w)
    step.head_ce_dw(T)
    step.embed_grad(step.norm_grad())
    assert float(step.loss) == 0.0 and not step.dW.any() and not step.d_norm_weight.any()
