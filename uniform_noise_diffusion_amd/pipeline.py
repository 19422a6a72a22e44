"""Buffers for one training step of the loss path, and the three calls.

Plumbing only: torch allocates the device buffers once; each step enqueues
mdlm_corrupt, mdlm_compact_masked and mdlm_fused_head_ce_fwd_bwd on one
stream with no host synchronisation (the number of scored rows stays on the
device).  The hidden states would come from the model's forward on `xt`; here
they are an input.
"""

import torch

from . import binding as B


class MdlmLossStep:
    """Owns every buffer the three calls write for a stream of `n_tokens`
    tokens in `n_docs` documents, hidden size H and vocabulary V."""

    def __init__(self, n_tokens, n_docs, H, V, dtype=torch.bfloat16, device="cuda",
                 head_workspace_bytes=None, want_grad=True):
        self.n_tokens, self.n_docs, self.H, self.V = n_tokens, n_docs, H, V
        self.dtype = dtype
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.xt = torch.empty(n_tokens, **i32)
        self.corrupted = torch.empty(n_tokens, dtype=torch.uint8, device=dev)
        self.p_doc = torch.empty(n_docs, dtype=torch.float64, device=dev)
        self.doc_counts = torch.empty(n_docs, **i32)
        self.row_idx = torch.empty(max(n_tokens, 1), **i32)
        self.tgt = torch.empty(max(n_tokens, 1), **i32)
        self.w = torch.empty(max(n_tokens, 1), dtype=torch.float32, device=dev)
        self.n_rows = torch.empty(1, **i32)
        self.compact_ws = torch.empty(max(B.mdlm_compact_workspace_bytes(n_tokens), 1),
                                      dtype=torch.uint8, device=dev)
        self.rows_ws = None
        self.loss = torch.empty(1, dtype=torch.float32, device=dev)
        self.row_ce = torch.empty(max(n_tokens, 1), dtype=torch.float32, device=dev)
        self.d_hidden = (torch.empty((n_tokens, H), dtype=dtype, device=dev)
                         if want_grad else None)
        code = B.dtype_code(torch.empty(0, dtype=dtype))
        if head_workspace_bytes is None:
            head_workspace_bytes = B.mdlm_head_ce_workspace_bytes(n_tokens, H, V, code)
        self.head_ws = torch.empty(max(head_workspace_bytes, 1), dtype=torch.uint8, device=dev)

    def corrupt(self, x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, stream=None):
        B.mdlm_corrupt(x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, self.xt,
                       self.corrupted, self.p_doc, self.doc_counts, stream)

    def compact(self, x0, cu_seqlens, align, stream=None):
        B.mdlm_compact_masked(self.corrupted, x0, cu_seqlens, self.p_doc, align, self.row_idx,
                              self.tgt, self.w, self.n_rows, self.compact_ws, stream)

    def corrupt_mixture(self, x0, cu_seqlens, seed, eps, mixture_prob, mask_id, rand_vocab,
                        stream=None):
        """mdlm_corrupt_mixture: `corrupted` then holds the codes (0 clean,
        1 masked, 2 replaced)."""
        B.mdlm_corrupt_mixture(x0, cu_seqlens, seed, eps, mixture_prob, mask_id, rand_vocab,
                               self.xt, self.corrupted, self.p_doc, self.doc_counts, stream)

    def compact_corrective(self, x0, cu_seqlens, align, noise_token_wt, clean_token_wt,
                           stream=None):
        """mdlm_compact_corrective over the codes of the last corrupt_mixture()."""
        B.mdlm_compact_corrective(self.corrupted, x0, cu_seqlens, self.p_doc, align,
                                  noise_token_wt, clean_token_wt, self.row_idx, self.tgt,
                                  self.w, self.n_rows, self.compact_ws, stream)

    def compact_rows(self, x0, cu_seqlens, align, weighting, weight_scale=1.0,
                     weight_clip=float("inf"), corrupted=True, eligible=None, stream=None):
        """mdlm_compact_rows into this step's row buffers: `corrupted` True uses
        the mask of the last corrupt() call, None scores every token;
        `eligible` is an optional uint8 mask."""
        need = B.mdlm_compact_rows_workspace_bytes(self.n_tokens, self.n_docs, weighting)
        if self.rows_ws is None or self.rows_ws.numel() < need:
            self.rows_ws = torch.empty(max(need, 1), dtype=torch.uint8, device=self.xt.device)
        mask = self.corrupted if corrupted is True else corrupted
        B.mdlm_compact_rows(mask, eligible, x0, cu_seqlens, self.p_doc, align, weighting,
                            weight_scale, weight_clip, self.row_idx, self.tgt, self.w,
                            self.n_rows, self.rows_ws, stream)

    def head_ce(self, hidden, W, softcap, stream=None, want_grad=True, row_ce=True):
        B.mdlm_fused_head_ce_fwd_bwd(hidden, W, self.row_idx, self.tgt, self.w, self.n_rows,
                                     self.n_tokens, softcap, self.loss,
                                     self.row_ce if row_ce else None,
                                     self.d_hidden if want_grad else None, self.head_ws,
                                     stream)

    def step(self, x0, cu_seqlens, hidden, W, seed, eps, noise, mask_id, rand_vocab, align,
             softcap, stream=None, want_grad=True, row_ce=True):
        self.corrupt(x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, stream)
        self.compact(x0, cu_seqlens, align, stream)
        self.head_ce(hidden, W, softcap, stream, want_grad, row_ce)


# States of what MdlmTrainStep's calls leave: nothing yet, this step's, an
# earlier step's (or already consumed).
_NEVER, _PRESENT, _OUTDATED = range(3)


class MdlmTrainStep(MdlmLossStep):
    """A training step of a model whose embedding, final norm and head are
    trained, the model's own layers running between embed() and final_norm()
    and between norm_grad() and embed_grad():

        corrupt, compact   ->  embed          ->  the model's layers
        ->  final_norm     ->  head_ce_dw     ->  norm_grad
        ->  the layers' backward              ->  embed_grad

    final_norm() keeps its input as an 8-bit checkpoint, so the caller need not
    hold it until norm_grad().  With a tied head (`tied`) the table is the head:
    embed_grad() adds to the `dW` that head_ce_dw() wrote; otherwise it writes
    `d_table`.  bf16, as the trained head is.

    The buffers are one step's, so a call that would read an earlier step's is
    refused (RuntimeError): norm_grad() takes a final_norm() and, behind it, a
    gradient of its output; embed_grad() takes the tokens that embed() saw (of
    a caller that embeds `xt` in its own way, the present ones) and, tied, adds
    to a dW of this step, once.  corrupt() begins the next step: of the step
    before, only norm_grad() may still follow.  Replays of a captured graph are
    not seen here, so once one of a step's calls is captured only calls that
    nothing has ever preceded are refused."""

    def __init__(self, n_tokens, n_docs, H, V, norm_kind=B.MDLM_NORM_RMS, norm_eps=1e-5,
                 norm_bias=False, embed_scale=1.0, tied=True, device="cuda"):
        dw_bytes = B.mdlm_head_ce_dw_workspace_bytes(n_tokens, H, V)
        super().__init__(n_tokens, n_docs, H, V, device=device, head_workspace_bytes=dw_bytes)
        dev = self.xt.device
        f32 = dict(dtype=torch.float32, device=dev)
        u8 = dict(dtype=torch.uint8, device=dev)
        self.norm_kind, self.norm_eps, self.embed_scale = norm_kind, norm_eps, embed_scale
        self.embedded = torch.empty((n_tokens, H), dtype=self.dtype, device=dev)
        self.hidden = torch.empty_like(self.embedded)
        self.mean = torch.empty(n_tokens, **f32) if norm_kind == B.MDLM_NORM_LAYER else None
        self.rstd = torch.empty(n_tokens, **f32)
        self.q = torch.empty((n_tokens, H), **u8)
        self.q_exp = torch.empty((n_tokens, -(-H // B.MDLM_CKPT8_BLOCK)), **u8)
        self.d_last = torch.empty_like(self.embedded)
        self.d_norm_weight = torch.empty(H, **f32)
        self.d_norm_bias = torch.empty(H, **f32) if norm_bias else None
        self.dW = torch.empty((V, H), **f32)
        self.tied = tied
        self.d_table = self.dW if tied else torch.empty((V, H), **f32)
        self.norm_ws = torch.empty(max(B.mdlm_norm_bwd_workspace_bytes(n_tokens, H), 1), **u8)
        self.embed_ws = torch.empty(max(B.mdlm_embed_grad_workspace_bytes(n_tokens, H), 1), **u8)
        self._norm_weight = None  # (of the last final_norm(): None is a weight of 1)
        # what the step's calls have left in the buffers
        self._left = dict.fromkeys(("embedded", "hidden", "d_hidden", "dW"), _NEVER)
        self._norm_grad_taken = False
        self._recorded = False  # some call was captured into a graph

    def _capturing(self, stream):
        """Whether `stream` (the current one if None) is being captured."""
        dev = self.xt.device
        if dev.type != "cuda":
            return False
        if stream is None and dev.index == torch.cuda.current_device():
            return torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(torch.cuda.current_stream(dev) if stream is None else stream):
            return torch.cuda.is_current_stream_capturing()

    def _begin_call(self, stream):
        self._recorded = self._recorded or self._capturing(stream)

    def _outdate(self, *names):
        for name in names:
            if self._left[name] == _PRESENT:
                self._left[name] = _OUTDATED

    def _has(self, name):
        state = self._left[name]
        return state == _PRESENT or (state == _OUTDATED and self._recorded)

    def _begin_step(self):
        self._outdate("embedded", "dW")
        if self._norm_grad_taken:
            self._outdate("hidden", "d_hidden")

    def corrupt(self, x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, stream=None):
        self._begin_call(stream)
        super().corrupt(x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, stream)
        self._begin_step()

    def corrupt_mixture(self, x0, cu_seqlens, seed, eps, mixture_prob, mask_id, rand_vocab,
                        stream=None):
        """MdlmLossStep.corrupt_mixture()."""
        self._begin_call(stream)
        super().corrupt_mixture(x0, cu_seqlens, seed, eps, mixture_prob, mask_id, rand_vocab,
                                stream)
        self._begin_step()

    def embed(self, table, stream=None):
        """The corrupted tokens' embeddings into `embedded`."""
        self._begin_call(stream)
        B.mdlm_embed(self.xt, table, self.embed_scale, self.embedded, stream)
        self._left["embedded"] = _PRESENT
        return self.embedded

    def final_norm(self, x, weight, bias=None, stream=None):
        """The final norm of the model's last activation into `hidden`; x is kept
        as an 8-bit checkpoint."""
        if (bias is None) != (self.d_norm_bias is None):
            raise ValueError("bias: given exactly when the step was made with norm_bias=True")
        self._begin_call(stream)
        B.mdlm_norm_fwd(x, self.norm_kind, weight, bias, self.norm_eps, self.hidden, self.mean,
                        self.rstd, self.q, self.q_exp, stream)
        self._norm_weight = weight
        self._left["hidden"] = _PRESENT
        self._outdate("d_hidden")
        self._norm_grad_taken = False
        return self.hidden

    def head_ce(self, hidden, W, softcap, stream=None, want_grad=True, row_ce=True):
        """MdlmLossStep.head_ce(): a frozen head's loss and, if wanted,
        `d_hidden`."""
        self._begin_call(stream)
        super().head_ce(hidden, W, softcap, stream, want_grad, row_ce)
        if want_grad:
            self._left["d_hidden"] = _PRESENT

    def head_ce_dw(self, W, softcap=0.0, stream=None):
        """Loss, `d_hidden` and the head's gradient `dW` from `hidden`."""
        self._begin_call(stream)
        B.mdlm_fused_head_ce_fwd_bwd_dw(self.hidden, W, self.row_idx, self.tgt, self.w,
                                        self.n_rows, self.n_tokens, softcap, self.loss,
                                        self.row_ce, self.d_hidden, self.dW, self.head_ws, stream)
        self._left["d_hidden"] = self._left["dW"] = _PRESENT
        return self.loss

    def norm_grad(self, stream=None, d_hidden=None):
        """`d_last` (the gradient that enters the model's layers) and the norm's
        own gradients from the checkpoint of the last final_norm() and the
        gradient of its output: `d_hidden` of the head's call, or the one
        given here."""
        self._begin_call(stream)
        if not self._has("hidden"):
            raise RuntimeError("norm_grad() follows this step's final_norm()")
        if d_hidden is None:
            if not self._has("d_hidden"):
                raise RuntimeError("norm_grad() follows head_ce_dw() or head_ce() on the hidden "
                                   "states of the last final_norm(), or takes another d_hidden")
            d_hidden = self.d_hidden
        B.mdlm_norm_bwd_ckpt8(d_hidden, self.q, self.q_exp, self.norm_kind,
                              self._norm_weight, self.mean, self.rstd, self.d_last,
                              self.d_norm_weight, self.d_norm_bias, workspace=self.norm_ws,
                              stream=stream)
        self._norm_grad_taken = True
        return self.d_last

    def embed_grad(self, d_embedded, stream=None):
        """The table's gradient from the gradient of `embedded`: added to `dW`
        (tied) or written to `d_table`."""
        self._begin_call(stream)
        if self._left["embedded"] == _OUTDATED and not self._recorded:
            raise RuntimeError("embed_grad() reads the tokens that embed() saw, and a later "
                               "corruption has replaced them")
        if self.tied and not self._has("dW"):
            raise RuntimeError("embed_grad() of a tied table follows this step's head_ce_dw(), "
                               "once")
        B.mdlm_embed_grad(self.xt, d_embedded, self.embed_scale, self.d_table,
                          accumulate=self.tied, workspace=self.embed_ws, stream=stream)
        if self.tied:
            self._outdate("dW")
        return self.d_table
