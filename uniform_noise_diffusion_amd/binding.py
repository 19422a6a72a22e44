"""ctypes binding of libmdlm.so (include/mdlm.h).

Argument marshalling only: every computation runs in the HIP library.  The
functions keep the C names and take torch tensors for device memory; the
stream is torch's current stream unless one is given.  A non-zero status from
the library raises MdlmError carrying mdlm_last_error().  If the library has
not been built the first call raises; nothing falls back to another
implementation.
"""

import ctypes
import functools
import operator
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmdlm.so")

MDLM_OK = 0
MDLM_EINVAL = 1
MDLM_EUNSUPPORTED = 2
MDLM_EWORKSPACE = 3
MDLM_EHIP = 4
MDLM_NOISE_ABSORB = 0
MDLM_NOISE_UNIFORM = 1
MDLM_ALIGNED = 0
MDLM_SHIFTED = 1
MDLM_F32 = 0
MDLM_BF16 = 1
MDLM_WEIGHT_INV_P = 0
MDLM_WEIGHT_MEAN = 1
MDLM_WEIGHT_EXAMPLE_MEAN_CLIPPED = 2
MDLM_CODE_CLEAN = 0
MDLM_CODE_MASKED = 1
MDLM_CODE_REPLACED = 2
MDLM_CHECK_OFFSETS = 1
MDLM_CHECK_ROW_COUNT = 2
MDLM_CHECK_ROW_INDEX = 4
MDLM_CHECK_TARGET = 8
MDLM_CHECK_WEIGHT = 16
MDLM_CHECK_PROB = 32
MDLM_CHECK_TOKEN = 64
MDLM_NORM_LAYER = 0
MDLM_NORM_RMS = 1
MDLM_CKPT8_BLOCK = 128

EXPORTED = (
    "mdlm_corrupt",
    "mdlm_corrupt_mixture",
    "mdlm_corrupt_compact_workspace_bytes",
    "mdlm_corrupt_compact",
    "mdlm_compact_workspace_bytes",
    "mdlm_compact_masked",
    "mdlm_compact_masked_noalloc",
    "mdlm_compact_corrective",
    "mdlm_compact_rows_workspace_bytes",
    "mdlm_compact_rows",
    "mdlm_head_ce_workspace_bytes",
    "mdlm_head_ce_workspace_min_bytes",
    "mdlm_fused_head_ce_fwd_bwd",
    "mdlm_head_ce_dw_workspace_bytes",
    "mdlm_head_ce_dw_workspace_min_bytes",
    "mdlm_fused_head_ce_fwd_bwd_dw",
    "mdlm_scale",
    "mdlm_embed",
    "mdlm_embed_grad_workspace_bytes",
    "mdlm_embed_grad",
    "mdlm_norm_fwd",
    "mdlm_norm_bwd_workspace_bytes",
    "mdlm_norm_bwd",
    "mdlm_norm_bwd_ckpt8",
    "mdlm_ckpt8_save",
    "mdlm_ckpt8_load",
    "mdlm_check_offsets",
    "mdlm_check_probs",
    "mdlm_check_rows",
    "mdlm_check_tokens",
    "mdlm_set_checking",
    "mdlm_last_error",
    "mdlm_version",
)

_lib = None

_I32_MAX = 0x7FFFFFFF


class _Int32:
    """Type of the library's int32_t arguments: ctypes' own keeps the low 32
    bits of a larger number and says nothing."""

    @staticmethod
    def from_param(value):
        if -_I32_MAX - 1 <= value <= _I32_MAX:
            return operator.index(value)
        raise ValueError(f"{value} does not fit 32 bits")


class MdlmError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"[mdlm status {code}] {message}")
        self.code = code


def load():
    """Load libmdlm.so once and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m uniform_noise_diffusion_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, f32, f64, sz = (ctypes.c_void_p, _Int32, ctypes.c_int64,
                                       ctypes.c_uint64, ctypes.c_float, ctypes.c_double,
                                       ctypes.c_size_t)
    lib.mdlm_corrupt.argtypes = [vp, i64, vp, i32, u64, f64, i32, i32, i32, vp, vp, vp, vp, vp]
    lib.mdlm_corrupt.restype = ctypes.c_int
    lib.mdlm_corrupt_mixture.argtypes = [vp, i64, vp, i32, u64, f64, f64, i32, i32, vp, vp, vp,
                                         vp, vp]
    lib.mdlm_corrupt_mixture.restype = ctypes.c_int
    lib.mdlm_corrupt_compact_workspace_bytes.argtypes = [i64]
    lib.mdlm_corrupt_compact_workspace_bytes.restype = sz
    lib.mdlm_corrupt_compact.argtypes = [vp, i64, vp, i32, u64, f64, i32, i32, i32, i32, vp, vp,
                                         vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mdlm_corrupt_compact.restype = ctypes.c_int
    lib.mdlm_compact_workspace_bytes.argtypes = [i64]
    lib.mdlm_compact_workspace_bytes.restype = sz
    lib.mdlm_compact_masked.argtypes = [vp, vp, i64, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.mdlm_compact_masked.restype = ctypes.c_int
    lib.mdlm_compact_masked_noalloc.argtypes = [vp, vp, i64, vp, i32, vp, i32, vp, vp, vp, vp,
                                                vp]
    lib.mdlm_compact_masked_noalloc.restype = ctypes.c_int
    lib.mdlm_compact_corrective.argtypes = [vp, vp, i64, vp, i32, vp, i32, f64, f64, vp, vp, vp,
                                            vp, vp, sz, vp]
    lib.mdlm_compact_corrective.restype = ctypes.c_int
    lib.mdlm_compact_rows_workspace_bytes.argtypes = [i64, i32, i32]
    lib.mdlm_compact_rows_workspace_bytes.restype = sz
    lib.mdlm_compact_rows.argtypes = [vp, vp, vp, i64, vp, i32, vp, i32, i32, f64, f64, vp, vp,
                                      vp, vp, vp, sz, vp]
    lib.mdlm_compact_rows.restype = ctypes.c_int
    lib.mdlm_head_ce_workspace_bytes.argtypes = [i64, i32, i32, i32]
    lib.mdlm_head_ce_workspace_bytes.restype = sz
    lib.mdlm_head_ce_workspace_min_bytes.argtypes = [i64, i32, i32, i32]
    lib.mdlm_head_ce_workspace_min_bytes.restype = sz
    lib.mdlm_fused_head_ce_fwd_bwd.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, i64,
                                               f32, vp, vp, vp, vp, sz, vp]
    lib.mdlm_fused_head_ce_fwd_bwd.restype = ctypes.c_int
    lib.mdlm_head_ce_dw_workspace_bytes.argtypes = [i64, i32, i32]
    lib.mdlm_head_ce_dw_workspace_bytes.restype = sz
    lib.mdlm_head_ce_dw_workspace_min_bytes.argtypes = [i64, i32, i32]
    lib.mdlm_head_ce_dw_workspace_min_bytes.restype = sz
    lib.mdlm_fused_head_ce_fwd_bwd_dw.argtypes = [vp, vp, i64, i32, i32, vp, vp, vp, vp, i64,
                                                  f32, vp, vp, vp, vp, vp, sz, vp]
    lib.mdlm_fused_head_ce_fwd_bwd_dw.restype = ctypes.c_int
    lib.mdlm_scale.argtypes = [vp, vp, i32, i64, vp, vp]
    lib.mdlm_scale.restype = ctypes.c_int
    lib.mdlm_embed.argtypes = [vp, i64, vp, i32, i32, i32, f32, vp, vp]
    lib.mdlm_embed.restype = ctypes.c_int
    lib.mdlm_embed_grad_workspace_bytes.argtypes = [i64, i32]
    lib.mdlm_embed_grad_workspace_bytes.restype = sz
    lib.mdlm_embed_grad.argtypes = [vp, i64, vp, i32, i32, i32, f32, vp, i32, vp, sz, vp]
    lib.mdlm_embed_grad.restype = ctypes.c_int
    lib.mdlm_norm_fwd.argtypes = [vp, i32, i64, i32, i32, vp, vp, f64, vp, vp, vp, vp, vp, vp]
    lib.mdlm_norm_fwd.restype = ctypes.c_int
    lib.mdlm_norm_bwd_workspace_bytes.argtypes = [i64, i32]
    lib.mdlm_norm_bwd_workspace_bytes.restype = sz
    lib.mdlm_norm_bwd.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, sz,
                                  vp]
    lib.mdlm_norm_bwd.restype = ctypes.c_int
    lib.mdlm_norm_bwd_ckpt8.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, vp,
                                        i32, vp, sz, vp]
    lib.mdlm_norm_bwd_ckpt8.restype = ctypes.c_int
    lib.mdlm_ckpt8_save.argtypes = [vp, i32, i64, i32, vp, vp, vp]
    lib.mdlm_ckpt8_save.restype = ctypes.c_int
    lib.mdlm_ckpt8_load.argtypes = [vp, vp, i32, i64, i32, vp, vp]
    lib.mdlm_ckpt8_load.restype = ctypes.c_int
    lib.mdlm_check_tokens.argtypes = [vp, i64, i32, vp, vp]
    lib.mdlm_check_tokens.restype = ctypes.c_int
    lib.mdlm_check_offsets.argtypes = [vp, i32, i64, vp, vp]
    lib.mdlm_check_offsets.restype = ctypes.c_int
    lib.mdlm_check_probs.argtypes = [vp, i32, vp, vp]
    lib.mdlm_check_probs.restype = ctypes.c_int
    lib.mdlm_check_rows.argtypes = [vp, vp, vp, vp, i64, i64, i32, vp, vp]
    lib.mdlm_check_rows.restype = ctypes.c_int
    lib.mdlm_set_checking.argtypes = [ctypes.c_int]
    lib.mdlm_set_checking.restype = ctypes.c_int
    lib.mdlm_last_error.argtypes = []
    lib.mdlm_last_error.restype = ctypes.c_char_p
    lib.mdlm_version.argtypes = []
    lib.mdlm_version.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(code):
    if code != MDLM_OK:
        raise MdlmError(code, load().mdlm_last_error().decode())


def _need(t, dtype, name):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


def mdlm_last_error():
    return load().mdlm_last_error().decode()


def mdlm_version():
    return load().mdlm_version()


def mdlm_corrupt(x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, xt, corrupted,
                 p_doc, doc_counts, stream=None):
    """See mdlm_corrupt in include/mdlm.h."""
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(xt, torch.int32, "xt")
    _need(corrupted, torch.uint8, "corrupted")
    _need(p_doc, torch.float64, "p_doc")
    _need(doc_counts, torch.int32, "doc_counts")
    n_docs = cu_seqlens.numel() - 1
    _check(load().mdlm_corrupt(_ptr(x0), x0.numel(), _ptr(cu_seqlens), n_docs,
                               int(seed) & 0xFFFFFFFFFFFFFFFF, float(eps), int(noise),
                               int(mask_id), int(rand_vocab), _ptr(xt), _ptr(corrupted),
                               _ptr(p_doc), _ptr(doc_counts), _stream(stream)))


def mdlm_corrupt_mixture(x0, cu_seqlens, seed, eps, mixture_prob, mask_id, rand_vocab, xt,
                         codes, p_doc, doc_counts, stream=None):
    """See mdlm_corrupt_mixture in include/mdlm.h."""
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(xt, torch.int32, "xt")
    _need(codes, torch.uint8, "codes")
    _need(p_doc, torch.float64, "p_doc")
    _need(doc_counts, torch.int32, "doc_counts")
    n_docs = cu_seqlens.numel() - 1
    _check(load().mdlm_corrupt_mixture(_ptr(x0), x0.numel(), _ptr(cu_seqlens), n_docs,
                                       int(seed) & 0xFFFFFFFFFFFFFFFF, float(eps),
                                       float(mixture_prob), int(mask_id), int(rand_vocab),
                                       _ptr(xt), _ptr(codes), _ptr(p_doc), _ptr(doc_counts),
                                       _stream(stream)))


def mdlm_corrupt_compact_workspace_bytes(n_tokens):
    return load().mdlm_corrupt_compact_workspace_bytes(int(n_tokens))


def mdlm_corrupt_compact(x0, cu_seqlens, seed, eps, noise, mask_id, rand_vocab, align, xt,
                         corrupted, p_doc, doc_counts, row_idx, tgt, w, n_rows, workspace,
                         stream=None):
    """See mdlm_corrupt_compact in include/mdlm.h.  `corrupted` may be None;
    `workspace` is a uint8 tensor."""
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(xt, torch.int32, "xt")
    _need(corrupted, torch.uint8, "corrupted")
    _need(p_doc, torch.float64, "p_doc")
    _need(doc_counts, torch.int32, "doc_counts")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(load().mdlm_corrupt_compact(
        _ptr(x0), x0.numel(), _ptr(cu_seqlens), cu_seqlens.numel() - 1,
        int(seed) & 0xFFFFFFFFFFFFFFFF, float(eps), int(noise), int(mask_id), int(rand_vocab),
        int(align), _ptr(xt), _ptr(corrupted), _ptr(p_doc), _ptr(doc_counts), _ptr(row_idx),
        _ptr(tgt), _ptr(w), _ptr(n_rows), _ptr(workspace), ws_bytes, _stream(stream)))


def mdlm_compact_workspace_bytes(n_tokens):
    return load().mdlm_compact_workspace_bytes(int(n_tokens))


def mdlm_compact_masked(corrupted, x0, cu_seqlens, p_doc, align, row_idx, tgt, w, n_rows,
                        workspace, stream=None):
    """See mdlm_compact_masked in include/mdlm.h.  `workspace` is a uint8 tensor."""
    _need(corrupted, torch.uint8, "corrupted")
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(p_doc, torch.float64, "p_doc")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(load().mdlm_compact_masked(_ptr(corrupted), _ptr(x0), x0.numel(), _ptr(cu_seqlens),
                                      cu_seqlens.numel() - 1, _ptr(p_doc), int(align),
                                      _ptr(row_idx), _ptr(tgt), _ptr(w), _ptr(n_rows),
                                      _ptr(workspace), ws_bytes, _stream(stream)))


def mdlm_compact_masked_noalloc(corrupted, x0, cu_seqlens, p_doc, align, row_idx, tgt, w,
                                n_rows, stream=None):
    """See mdlm_compact_masked_noalloc in include/mdlm.h (no workspace)."""
    _need(corrupted, torch.uint8, "corrupted")
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(p_doc, torch.float64, "p_doc")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _check(load().mdlm_compact_masked_noalloc(
        _ptr(corrupted), _ptr(x0), x0.numel(), _ptr(cu_seqlens), cu_seqlens.numel() - 1,
        _ptr(p_doc), int(align), _ptr(row_idx), _ptr(tgt), _ptr(w), _ptr(n_rows),
        _stream(stream)))


def mdlm_compact_corrective(codes, x0, cu_seqlens, p_doc, align, noise_token_wt,
                            clean_token_wt, row_idx, tgt, w, n_rows, workspace, stream=None):
    """See mdlm_compact_corrective in include/mdlm.h.  `workspace` is a uint8
    tensor of mdlm_compact_workspace_bytes(n_tokens) bytes."""
    _need(codes, torch.uint8, "codes")
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(p_doc, torch.float64, "p_doc")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(load().mdlm_compact_corrective(
        _ptr(codes), _ptr(x0), x0.numel(), _ptr(cu_seqlens), cu_seqlens.numel() - 1,
        _ptr(p_doc), int(align), float(noise_token_wt), float(clean_token_wt), _ptr(row_idx),
        _ptr(tgt), _ptr(w), _ptr(n_rows), _ptr(workspace), ws_bytes, _stream(stream)))


def mdlm_compact_rows_workspace_bytes(n_tokens, n_docs, weighting):
    return load().mdlm_compact_rows_workspace_bytes(int(n_tokens), int(n_docs), int(weighting))


def mdlm_compact_rows(corrupted, eligible, x0, cu_seqlens, p_doc, align, weighting,
                      weight_scale, weight_clip, row_idx, tgt, w, n_rows, workspace,
                      stream=None):
    """See mdlm_compact_rows in include/mdlm.h.  `corrupted`, `eligible` and
    `p_doc` may be None; `workspace` is a uint8 tensor."""
    _need(corrupted, torch.uint8, "corrupted")
    _need(eligible, torch.uint8, "eligible")
    _need(x0, torch.int32, "x0")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(p_doc, torch.float64, "p_doc")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(load().mdlm_compact_rows(
        _ptr(corrupted), _ptr(eligible), _ptr(x0), x0.numel(), _ptr(cu_seqlens),
        cu_seqlens.numel() - 1, _ptr(p_doc), int(align), int(weighting), float(weight_scale),
        float(weight_clip), _ptr(row_idx), _ptr(tgt), _ptr(w), _ptr(n_rows), _ptr(workspace),
        ws_bytes, _stream(stream)))


def dtype_code(t):
    if t.dtype == torch.bfloat16:
        return MDLM_BF16
    if t.dtype == torch.float32:
        return MDLM_F32
    raise TypeError(f"unsupported element type {t.dtype}")


def mdlm_head_ce_workspace_bytes(max_rows, H, V, dtype):
    return load().mdlm_head_ce_workspace_bytes(int(max_rows), int(H), int(V), int(dtype))


def mdlm_head_ce_workspace_min_bytes(max_rows, H, V, dtype):
    return load().mdlm_head_ce_workspace_min_bytes(int(max_rows), int(H), int(V), int(dtype))


def mdlm_fused_head_ce_fwd_bwd(hidden, W, row_idx, tgt, w, n_rows, max_rows, softcap, loss,
                               row_ce, d_hidden, workspace, stream=None):
    """See mdlm_fused_head_ce_fwd_bwd in include/mdlm.h.  `d_hidden` and
    `row_ce` may be None; `workspace` is a uint8 tensor."""
    dt = dtype_code(hidden)
    _need(hidden, hidden.dtype, "hidden")
    _need(W, hidden.dtype, "W")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(loss, torch.float32, "loss")
    _need(row_ce, torch.float32, "row_ce")
    _need(d_hidden, hidden.dtype, "d_hidden")
    _need(workspace, torch.uint8, "workspace")
    n_tokens, H = hidden.shape
    V = W.shape[0]
    if W.shape[1] != H:
        raise ValueError("W must be [V, H] with the hidden size of `hidden`")
    if d_hidden is not None and tuple(d_hidden.shape) != tuple(hidden.shape):
        raise ValueError("d_hidden must have the shape of hidden")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(load().mdlm_fused_head_ce_fwd_bwd(
        _ptr(hidden), _ptr(W), dt, n_tokens, H, V, _ptr(row_idx), _ptr(tgt), _ptr(w),
        _ptr(n_rows), int(max_rows), float(softcap), _ptr(loss), _ptr(row_ce), _ptr(d_hidden),
        _ptr(workspace), ws_bytes, _stream(stream)))


def mdlm_head_ce_dw_workspace_bytes(max_rows, H, V):
    return load().mdlm_head_ce_dw_workspace_bytes(int(max_rows), int(H), int(V))


def mdlm_head_ce_dw_workspace_min_bytes(max_rows, H, V):
    return load().mdlm_head_ce_dw_workspace_min_bytes(int(max_rows), int(H), int(V))


def mdlm_fused_head_ce_fwd_bwd_dw(hidden, W, row_idx, tgt, w, n_rows, max_rows, softcap, loss,
                                  row_ce, d_hidden, dW, workspace, stream=None):
    """See mdlm_fused_head_ce_fwd_bwd_dw in include/mdlm.h (bf16 only).
    `d_hidden` and `row_ce` may be None; `dW` is a float32 [V, H] tensor."""
    if hidden.dtype != torch.bfloat16:
        raise TypeError("mdlm_fused_head_ce_fwd_bwd_dw takes bf16 hidden and W")
    _need(hidden, torch.bfloat16, "hidden")
    _need(W, torch.bfloat16, "W")
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(loss, torch.float32, "loss")
    _need(row_ce, torch.float32, "row_ce")
    _need(d_hidden, torch.bfloat16, "d_hidden")
    _need(dW, torch.float32, "dW")
    _need(workspace, torch.uint8, "workspace")
    n_tokens, H = hidden.shape
    V = W.shape[0]
    if W.shape[1] != H or dW is None or tuple(dW.shape) != (V, H):
        raise ValueError("W and dW must be [V, H] with the hidden size of `hidden`")
    if d_hidden is not None and tuple(d_hidden.shape) != tuple(hidden.shape):
        raise ValueError("d_hidden must have the shape of hidden")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(load().mdlm_fused_head_ce_fwd_bwd_dw(
        _ptr(hidden), _ptr(W), n_tokens, H, V, _ptr(row_idx), _ptr(tgt), _ptr(w), _ptr(n_rows),
        int(max_rows), float(softcap), _ptr(loss), _ptr(row_ce), _ptr(d_hidden), _ptr(dW),
        _ptr(workspace), ws_bytes, _stream(stream)))


def mdlm_scale(x, y, scale, stream=None):
    """See mdlm_scale in include/mdlm.h: y = scale * x for bf16 or float32
    tensors of one size (y may be x); `scale` a one-element float32 device
    tensor."""
    dt = dtype_code(x)
    _need(x, x.dtype, "x")
    _need(y, x.dtype, "y")
    _need(scale, torch.float32, "scale")
    if y.numel() != x.numel():
        raise ValueError("x and y must have as many entries")
    _check(load().mdlm_scale(_ptr(x), _ptr(y), dt, x.numel(), _ptr(scale), _stream(stream)))


# The calls below are made many times a step on small tensors, so their checks
# are one pass over each argument, and the stream is read as the plain handle.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _place(t, name):
    """The device index of the tensor that a call's others must share."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected a device tensor")
    return dev


def _arg(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this type, shape and device (None
    of None)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on device {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _rows(x, name):
    """(n, H) of a tensor [..., H] taken as rows."""
    if x.dim() == 0:
        raise ValueError(f"{name}: expected [..., H]")
    H = x.shape[-1]
    _fits(H, name)
    return (x.numel() // H if H else 0), H


def _fits(size, name):
    if size > _I32_MAX:
        raise ValueError(f"{name}: {size} does not fit 32 bits")


def _table(t, name):
    """(V, H) of a table."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected [V, H]")
    V, H = t.shape
    _fits(max(V, H), name)
    return V, H


def _launch(fn, dev, stream, *args):
    """Calls `fn` with `args` and the stream (torch's current one of the
    device unless one is given), the device being the current one meanwhile."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream: expected a stream of device {dev}, got one of {stream.device}")
    else:
        handle = stream.cuda_stream
    if dev == torch.cuda.current_device():
        code = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, handle)
    if code != MDLM_OK:
        _check(code)


def _scratch(workspace, nbytes, dev, stream):
    """The caller's workspace, or one allocated for the call on the stream it
    will run on; None if none is needed."""
    if workspace is not None:
        _arg(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
        return workspace
    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def mdlm_embed(ids, table, scale, out, stream=None):
    """See mdlm_embed in include/mdlm.h: out[...] = scale * table[ids[...]].
    `ids` int32 of any shape; `table` [V, H] and `out` [*ids.shape, H] bf16 or
    float32."""
    V, H = _table(table, "table")
    dt = dtype_code(table)
    dev = _place(table, "table")
    _launch(load().mdlm_embed, dev, stream, _arg(ids, "ids", torch.int32, ids.shape, dev),
            ids.numel(), _arg(table, "table", table.dtype, table.shape, dev), dt, V, H, float(scale),
            _arg(out, "out", table.dtype, (*ids.shape, H), dev))


@functools.lru_cache(maxsize=256)
def mdlm_embed_grad_workspace_bytes(n_tokens, H):
    return load().mdlm_embed_grad_workspace_bytes(int(n_tokens), int(H))


def mdlm_embed_grad(ids, d_out, scale, d_table, accumulate=False, workspace=None, stream=None):
    """See mdlm_embed_grad in include/mdlm.h: `d_out` [*ids.shape, H] bf16 or
    float32, `d_table` [V, H] float32, overwritten or (accumulate) added to;
    `workspace` a uint8 tensor, allocated for the call if None."""
    V, H = _table(d_table, "d_table")
    n = ids.numel()
    dt = dtype_code(d_out)
    dev = _place(d_out, "d_out")
    a_ids = _arg(ids, "ids", torch.int32, ids.shape, dev)
    a_out = _arg(d_out, "d_out", d_out.dtype, (*ids.shape, H), dev)
    a_table = _arg(d_table, "d_table", torch.float32, d_table.shape, dev)
    ws = _scratch(workspace, mdlm_embed_grad_workspace_bytes(n, H), dev, stream)
    _launch(load().mdlm_embed_grad, dev, stream, a_ids, n, a_out, dt, V, H, float(scale), a_table,
            1 if accumulate else 0, None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel())


def _ckpt8_args(q, q_exp, shape, dev):
    return (_arg(q, "q", torch.uint8, shape, dev),
            _arg(q_exp, "q_exp", torch.uint8,
                 (*shape[:-1], -(-shape[-1] // MDLM_CKPT8_BLOCK)), dev))


def mdlm_norm_fwd(x, kind, weight, bias, eps, y, mean=None, rstd=None, q=None, q_exp=None,
                  stream=None):
    """See mdlm_norm_fwd in include/mdlm.h: `x`, `y` [..., H], `weight` and
    `bias` [H] of x's type or None, `mean` and `rstd` float32 [...] or None,
    `q` [..., H] and `q_exp` [..., ceil(H / 128)] uint8 or both None."""
    n, H = _rows(x, "x")
    T, shape, lead = x.dtype, x.shape, x.shape[:-1]
    dt = dtype_code(x)
    dev = _place(x, "x")
    a_q, a_exp = _ckpt8_args(q, q_exp, shape, dev)
    _launch(load().mdlm_norm_fwd, dev, stream, _arg(x, "x", T, shape, dev), dt, n, H, int(kind),
            _arg(weight, "weight", T, (H,), dev), _arg(bias, "bias", T, (H,), dev), float(eps),
            _arg(y, "y", T, shape, dev), _arg(mean, "mean", torch.float32, lead, dev),
            _arg(rstd, "rstd", torch.float32, lead, dev), a_q, a_exp)


@functools.lru_cache(maxsize=256)
def mdlm_norm_bwd_workspace_bytes(n, H):
    return load().mdlm_norm_bwd_workspace_bytes(int(n), int(H))


def _norm_bwd(fn, rows, dy, source, kind, weight, mean, rstd, dx, d_weight, d_bias, accumulate,
              workspace, stream, dev):
    n, H = rows
    T, lead, f32 = dy.dtype, dy.shape[:-1], torch.float32
    args = (_arg(dy, "dy", T, dy.shape, dev), *source, dtype_code(dy), n, H, int(kind),
            _arg(weight, "weight", T, (H,), dev), _arg(mean, "mean", f32, lead, dev),
            _arg(rstd, "rstd", f32, lead, dev), _arg(dx, "dx", T, dy.shape, dev),
            _arg(d_weight, "d_weight", f32, (H,), dev), _arg(d_bias, "d_bias", f32, (H,), dev),
            1 if accumulate else 0)
    need = (mdlm_norm_bwd_workspace_bytes(n, H)
            if d_weight is not None or d_bias is not None else 0)
    ws = _scratch(workspace, need, dev, stream)
    _launch(fn, dev, stream, *args, None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel())


def mdlm_norm_bwd(dy, x, kind, weight, mean, rstd, dx, d_weight=None, d_bias=None,
                  accumulate=False, workspace=None, stream=None):
    """See mdlm_norm_bwd in include/mdlm.h: `dy`, `x`, `dx` [..., H] of one type,
    `mean` (None for RMS) and `rstd` as mdlm_norm_fwd left them, `d_weight` and
    `d_bias` float32 [H]; outputs not wanted are None; `workspace` a uint8
    tensor, allocated for the call if None."""
    rows, dev = _rows(dy, "dy"), _place(dy, "dy")
    _norm_bwd(load().mdlm_norm_bwd, rows, dy, (_arg(x, "x", dy.dtype, dy.shape, dev),), kind,
              weight, mean, rstd, dx, d_weight, d_bias, accumulate, workspace, stream, dev)


def mdlm_norm_bwd_ckpt8(dy, q, q_exp, kind, weight, mean, rstd, dx, d_weight=None, d_bias=None,
                        accumulate=False, workspace=None, stream=None):
    """See mdlm_norm_bwd_ckpt8 in include/mdlm.h: mdlm_norm_bwd with x as the
    8-bit checkpoint `q`, `q_exp` holds it."""
    rows, dev = _rows(dy, "dy"), _place(dy, "dy")
    _norm_bwd(load().mdlm_norm_bwd_ckpt8, rows, dy, _ckpt8_args(q, q_exp, dy.shape, dev), kind,
              weight, mean, rstd, dx, d_weight, d_bias, accumulate, workspace, stream, dev)


def mdlm_ckpt8_save(x, q, q_exp, stream=None):
    """See mdlm_ckpt8_save in include/mdlm.h: `x` [..., H] bf16 or float32 into
    `q` [..., H] and `q_exp` [..., ceil(H / 128)] uint8."""
    n, H = _rows(x, "x")
    dt = dtype_code(x)
    dev = _place(x, "x")
    _launch(load().mdlm_ckpt8_save, dev, stream, _arg(x, "x", x.dtype, x.shape, dev), dt, n, H,
            *_ckpt8_args(q, q_exp, x.shape, dev))


def mdlm_ckpt8_load(q, q_exp, x, stream=None):
    """See mdlm_ckpt8_load in include/mdlm.h: the checkpoint restored into `x`."""
    n, H = _rows(x, "x")
    dt = dtype_code(x)
    dev = _place(x, "x")
    _launch(load().mdlm_ckpt8_load, dev, stream, *_ckpt8_args(q, q_exp, x.shape, dev), dt, n, H,
            _arg(x, "x", x.dtype, x.shape, dev))


def mdlm_check_offsets(cu_seqlens, n_tokens, status, stream=None):
    """See mdlm_check_offsets in include/mdlm.h: ORs violation bits into the
    one-element int32 device tensor `status`."""
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    _need(status, torch.int32, "status")
    _check(load().mdlm_check_offsets(_ptr(cu_seqlens), cu_seqlens.numel() - 1, int(n_tokens),
                                     _ptr(status), _stream(stream)))


def mdlm_check_probs(p_doc, status, stream=None):
    """See mdlm_check_probs in include/mdlm.h."""
    _need(p_doc, torch.float64, "p_doc")
    _need(status, torch.int32, "status")
    _check(load().mdlm_check_probs(_ptr(p_doc), p_doc.numel(), _ptr(status), _stream(stream)))


def mdlm_check_rows(row_idx, tgt, w, n_rows, max_rows, n_tokens, V, status, stream=None):
    """See mdlm_check_rows in include/mdlm.h; `tgt` and `w` may be None."""
    _need(row_idx, torch.int32, "row_idx")
    _need(tgt, torch.int32, "tgt")
    _need(w, torch.float32, "w")
    _need(n_rows, torch.int32, "n_rows")
    _need(status, torch.int32, "status")
    _check(load().mdlm_check_rows(_ptr(row_idx), _ptr(tgt), _ptr(w), _ptr(n_rows),
                                  int(max_rows), int(n_tokens), int(V), _ptr(status),
                                  _stream(stream)))


def mdlm_check_tokens(ids, V, status, stream=None):
    """See mdlm_check_tokens in include/mdlm.h: `ids` int32 of any shape, `status`
    a one-element int32 tensor on the same device."""
    dev = _place(ids, "ids")
    if status.numel() < 1:
        raise ValueError("status: expected one element")
    _launch(load().mdlm_check_tokens, dev, stream, _arg(ids, "ids", torch.int32, ids.shape, dev),
            ids.numel(), int(V), _arg(status, "status", torch.int32, status.shape, dev))


def mdlm_set_checking(enable):
    """See mdlm_set_checking in include/mdlm.h; returns the previous setting."""
    return bool(load().mdlm_set_checking(1 if enable else 0))
