"""The library's differentiable calls as torch.autograd.Functions: the fused
head + CE (masked_diffusion_loss), the token embedding (embed_tokens) and the
final norm (norm).

LLaDA-8B-MDLM-LoRA card, Training table, "Objective" row: the masked-
diffusion loss is what the trainer backpropagates through (with the output
layer frozen, "LoRA" row).  `masked_diffusion_loss` returns that loss as a
0-dim tensor whose gradient flows into `hidden`, so it can sit inside any
larger expression (a sum with other loss terms, a scale by an accumulation
factor) before `.backward()`.

Marshalling only: the forward is one mdlm_fused_head_ce_fwd_bwd call, which
forms d_hidden for an upstream gradient of 1 along with the loss; the
backward is one mdlm_scale call, d_hidden times the upstream gradient, read
on the device (no host synchronisation).  The head W must be frozen
(requires_grad False); the head-weight gradient is available through
binding.mdlm_fused_head_ce_fwd_bwd_dw.

embed_tokens and norm are the calls before and after the model whose final
hidden states the loss takes (mdlm_embed, mdlm_norm_fwd and their gradients).
"""

import torch
from torch.autograd.function import once_differentiable

from . import binding as B


class FusedHeadCE(torch.autograd.Function):
    """loss = sum_j w_j CE_j over the scored rows (see include/mdlm.h,
    mdlm_fused_head_ce_fwd_bwd); the gradient with respect to `hidden`."""

    @staticmethod
    def forward(ctx, hidden, W, row_idx, tgt, w, n_rows, max_rows, softcap, workspace):
        if W.requires_grad:
            raise ValueError("masked_diffusion_loss takes a frozen head (W.requires_grad "
                             "False); use mdlm_fused_head_ce_fwd_bwd_dw for a trained head")
        want = ctx.needs_input_grad[0]
        n_tokens, H = hidden.shape
        V = W.shape[0]
        if workspace is None:
            need = B.mdlm_head_ce_workspace_bytes(max_rows, H, V, B.dtype_code(hidden))
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=hidden.device)
        loss = torch.empty(1, dtype=torch.float32, device=hidden.device)
        d_hidden = torch.empty_like(hidden) if want else None
        B.mdlm_fused_head_ce_fwd_bwd(hidden, W, row_idx, tgt, w, n_rows, max_rows, softcap,
                                     loss, None, d_hidden, workspace)
        ctx.save_for_backward(d_hidden)
        return loss.view(())

    @staticmethod
    def backward(ctx, grad_loss):
        (d_hidden,) = ctx.saved_tensors
        if d_hidden is None:
            return (None,) * 9
        g = grad_loss.reshape(1)
        if g.dtype != torch.float32:
            g = g.float()
        out = torch.empty_like(d_hidden)
        B.mdlm_scale(d_hidden, out, g.contiguous())
        return (out,) + (None,) * 8


def masked_diffusion_loss(hidden, W, row_idx, tgt, w, n_rows, max_rows=None, softcap=0.0,
                          workspace=None):
    """The weighted CE of the scored rows (row list from mdlm_compact_masked
    or its variants) through the frozen head W, differentiable in `hidden`.

    hidden: [n_tokens, H] bf16 or float32 (contiguous, on the device);
    W: [V, H] of the same dtype; row_idx, tgt, w, n_rows: the row list;
    max_rows: host bound on *n_rows (default n_tokens); workspace: optional
    uint8 device tensor (default: the preferred size, allocated per call).
    Returns a 0-dim float32 tensor."""
    if max_rows is None:
        max_rows = hidden.shape[0]
    return FusedHeadCE.apply(hidden, W, row_idx, tgt, w, n_rows, int(max_rows), float(softcap),
                             workspace)


class TokenEmbedding(torch.autograd.Function):
    """out = scale * table[ids] (mdlm_embed); the gradient with respect to
    `table` (mdlm_embed_grad)."""

    @staticmethod
    def forward(ctx, ids, table, scale):
        out = torch.empty((*ids.shape, table.shape[-1]), dtype=table.dtype, device=table.device)
        B.mdlm_embed(ids, table, scale, out)
        if ctx.needs_input_grad[1]:
            # a step's token buffer is rewritten in place by the next
            # corruption, which autograd does not see: the ids are kept
            ctx.save_for_backward(ids.clone())
            ctx.table = (table.shape, table.dtype, scale)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        (ids,) = ctx.saved_tensors
        shape, dtype, scale = ctx.table
        d_table = torch.empty(shape, dtype=torch.float32, device=d_out.device)
        B.mdlm_embed_grad(ids, d_out.contiguous(), scale, d_table)
        return None, d_table.to(dtype), None


class FinalNorm(torch.autograd.Function):
    """Layer or RMS norm (mdlm_norm_fwd) with its gradients (mdlm_norm_bwd), the
    input kept as it is or as an 8-bit checkpoint (mdlm_norm_bwd_ckpt8)."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, kind, checkpoint8):
        y = torch.empty_like(x)
        want = any(ctx.needs_input_grad[:3])
        stat = dict(dtype=torch.float32, device=x.device)
        mean = torch.empty(x.shape[:-1], **stat) if want and kind == B.MDLM_NORM_LAYER else None
        rstd = torch.empty(x.shape[:-1], **stat) if want else None
        q = q_exp = None
        if want and checkpoint8:
            byte = dict(dtype=torch.uint8, device=x.device)
            q = torch.empty(x.shape, **byte)
            q_exp = torch.empty((*x.shape[:-1], -(-x.shape[-1] // B.MDLM_CKPT8_BLOCK)), **byte)
        B.mdlm_norm_fwd(x, kind, weight, bias, eps, y, mean, rstd, q, q_exp)
        if want:
            ctx.save_for_backward(None if checkpoint8 else x, q, q_exp, weight, mean, rstd)
            ctx.kind = kind
            ctx.param_types = (None if weight is None else weight.dtype,
                               None if bias is None else bias.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, q, q_exp, weight, mean, rstd = ctx.saved_tensors
        want_x, want_w, want_b = ctx.needs_input_grad[:3]
        dy = dy.contiguous()
        dx = torch.empty_like(dy) if want_x else None
        H = dy.shape[-1]
        d_weight = torch.empty(H, dtype=torch.float32, device=dy.device) if want_w else None
        d_bias = torch.empty(H, dtype=torch.float32, device=dy.device) if want_b else None
        if x is None:
            B.mdlm_norm_bwd_ckpt8(dy, q, q_exp, ctx.kind, weight, mean, rstd, dx, d_weight, d_bias)
        else:
            B.mdlm_norm_bwd(dy, x, ctx.kind, weight, mean, rstd, dx, d_weight, d_bias)
        return (dx, d_weight.to(ctx.param_types[0]) if want_w else None,
                d_bias.to(ctx.param_types[1]) if want_b else None, None, None, None)


def embed_tokens(ids, table, scale=1.0):
    """scale * table[ids], differentiable in `table`.

    ids: int32, any shape, on the device (xt of a corruption; a negative id
    stands for no token and gives zeros); table: [V, H] bf16 or float32.
    Returns [*ids.shape, H] of the table's type.  The gradient is summed in
    float32, in a fixed order, and rounded to the table's type; to add it to a
    float32 gradient kept elsewhere, call binding.mdlm_embed_grad."""
    return TokenEmbedding.apply(ids, table, float(scale))


def norm(x, weight=None, bias=None, eps=1e-5, kind=B.MDLM_NORM_LAYER, checkpoint8=False):
    """Layer norm (kind MDLM_NORM_LAYER) or RMS norm (MDLM_NORM_RMS) over the
    last dimension, differentiable in x, weight and bias.

    x: [..., H] bf16 or float32, contiguous, on the device; weight, bias: [H]
    of x's type or None.  checkpoint8: keep x for the backward pass in 8 bits
    (binding.mdlm_ckpt8_save's format) instead of x itself; the gradients are
    then those at the rounded x, with the statistics of the exact one."""
    return FinalNorm.apply(x, weight, bias, float(eps), int(kind), bool(checkpoint8))
