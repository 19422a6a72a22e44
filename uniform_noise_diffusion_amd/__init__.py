"""Masked-diffusion LM loss on AMD MI355X (gfx950).

The HIP library libmdlm.so (C ABI in include/mdlm.h) implements per-document
noise levels, corruption, ordered compaction of scored rows and the fused
frozen-head + cross-entropy forward and backward, and around the model the
token embedding, the final norm and 8-bit activation checkpoints with their
gradients.  `binding` exposes its entry points under the same names;
`pipeline` owns the buffers of one step; `autograd` wraps the calls as
differentiable functions.
"""

from .binding import (  # noqa: F401
    MdlmError,
    MDLM_OK, MDLM_EINVAL, MDLM_EUNSUPPORTED, MDLM_EWORKSPACE, MDLM_EHIP,
    MDLM_NOISE_ABSORB, MDLM_NOISE_UNIFORM, MDLM_ALIGNED, MDLM_SHIFTED,
    MDLM_F32, MDLM_BF16, MDLM_CODE_CLEAN, MDLM_CODE_MASKED, MDLM_CODE_REPLACED,
    mdlm_corrupt, mdlm_corrupt_mixture, mdlm_compact_workspace_bytes, mdlm_compact_masked,
    mdlm_compact_corrective,
    mdlm_head_ce_workspace_bytes, mdlm_head_ce_workspace_min_bytes,
    mdlm_fused_head_ce_fwd_bwd, mdlm_last_error, mdlm_version,
    MDLM_NORM_LAYER, MDLM_NORM_RMS,
    mdlm_embed, mdlm_embed_grad_workspace_bytes, mdlm_embed_grad,
    mdlm_norm_fwd, mdlm_norm_bwd_workspace_bytes, mdlm_norm_bwd, mdlm_norm_bwd_ckpt8,
    mdlm_ckpt8_save, mdlm_ckpt8_load,
)
from .pipeline import MdlmLossStep, MdlmTrainStep  # noqa: F401
from .autograd import (  # noqa: F401
    FusedHeadCE, masked_diffusion_loss, TokenEmbedding, embed_tokens, FinalNorm, norm,
)
