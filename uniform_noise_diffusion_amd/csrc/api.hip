// C ABI entry points: host-side argument checks, then launches on the
// caller's stream.  A failed check returns before anything is enqueued.
#include "mdlm_internal.h"

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

namespace mdlm {
namespace {
thread_local char g_error[512];
}

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof g_error, fmt, ap);
  va_end(ap);
  return code;
}

void clear_error() { g_error[0] = '\0'; }

int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MDLM_EHIP, "%s: %s", what, hipGetErrorString(e));
  return MDLM_OK;
}

// Checking mode's step for entry points that take document offsets (and,
// with `p`, noise levels).
static int check_docs(const char* fn, const int32_t* cu, int32_t n_docs, int64_t n,
                      const double* p, hipStream_t st) {
  if (!checking_enabled() || n_docs <= 0) return MDLM_OK;
  return run_checks(fn, st, [&](int32_t* word) {
    hipError_t e = launch_check_offsets(cu, n_docs, n, word, st);
    if (e == hipSuccess && p) e = launch_check_probs(p, n_docs, word, st);
    return e;
  });
}

// Checking mode's step for entry points that take a row list.
static int check_row_list(const char* fn, const int32_t* row_idx, const int32_t* tgt,
                          const float* w, const int32_t* n_rows, int64_t max_rows,
                          int64_t n_tokens, int32_t V, hipStream_t st) {
  if (!checking_enabled() || max_rows <= 0) return MDLM_OK;
  return run_checks(fn, st, [&](int32_t* word) {
    return launch_check_rows(row_idx, tgt, w, n_rows, max_rows, n_tokens, V, word, st);
  });
}

// Checking mode's step for entry points that take token ids.
static int check_token_ids(const char* fn, const int32_t* ids, int64_t n, int32_t V,
                           hipStream_t st) {
  if (!checking_enabled() || n <= 0) return MDLM_OK;
  return run_checks(fn, st,
                    [&](int32_t* word) { return launch_check_tokens(ids, n, V, word, st); });
}

static size_t entry_bytes(int32_t dtype) { return dtype == MDLM_BF16 ? 2 : 4; }

static bool misaligned(const void* p, size_t to) {
  return reinterpret_cast<uintptr_t>(p) % to != 0;
}

// Sizes shared by the entry points that work on [n, H] rows.
static int check_row_sizes(const char* fn, int32_t dtype, int64_t n, int32_t H) {
  if (dtype != MDLM_F32 && dtype != MDLM_BF16)
    return fail(MDLM_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (n < 0 || H <= 0) return fail(MDLM_EINVAL, "%s: bad sizes n=%lld H=%d", fn, (long long)n, H);
  if (n > INT32_MAX) return fail(MDLM_EUNSUPPORTED, "%s: n must be below 2^31", fn);
  return MDLM_OK;
}

}  // namespace mdlm

using namespace mdlm;

extern "C" {

int mdlm_version(void) { return (1 << 16) | 1; }

const char* mdlm_last_error(void) { return g_error; }

int mdlm_corrupt(const int32_t* x0, int64_t n_tokens, const int32_t* cu_seqlens,
                 int32_t n_docs, uint64_t seed, double eps, int32_t noise, int32_t mask_id,
                 int32_t rand_vocab, int32_t* xt, uint8_t* corrupted, double* p_doc,
                 int32_t* doc_counts, void* stream) {
  clear_error();
  if (n_tokens < 0) return fail(MDLM_EINVAL, "mdlm_corrupt: n_tokens < 0");
  if (n_tokens > INT32_MAX)
    return fail(MDLM_EUNSUPPORTED, "mdlm_corrupt: n_tokens must be below 2^31");
  if (n_docs < 0) return fail(MDLM_EINVAL, "mdlm_corrupt: n_docs < 0");
  if (n_docs == 0 && n_tokens > 0)
    return fail(MDLM_EINVAL, "mdlm_corrupt: tokens given but n_docs = 0");
  if (!(eps > 0.0 && eps <= 1.0)) return fail(MDLM_EINVAL, "mdlm_corrupt: eps must lie in (0, 1]");
  if (noise != MDLM_NOISE_ABSORB && noise != MDLM_NOISE_UNIFORM)
    return fail(MDLM_EINVAL, "mdlm_corrupt: unknown noise mode %d", noise);
  if (noise == MDLM_NOISE_UNIFORM && rand_vocab < 1)
    return fail(MDLM_EINVAL, "mdlm_corrupt: rand_vocab must be >= 1");
  if (n_tokens > 0 && (!x0 || !xt || !corrupted))
    return fail(MDLM_EINVAL, "mdlm_corrupt: null token pointer");
  if (n_docs > 0 && (!cu_seqlens || !p_doc || !doc_counts))
    return fail(MDLM_EINVAL, "mdlm_corrupt: null document pointer");
  if (const int rc = check_docs("mdlm_corrupt", cu_seqlens, n_docs, n_tokens, nullptr,
                                reinterpret_cast<hipStream_t>(stream)))
    return rc;
  if (launch_corrupt(x0, n_tokens, cu_seqlens, n_docs, seed, eps, noise, mask_id, rand_vocab,
                     xt, corrupted, p_doc, doc_counts,
                     reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch("mdlm_corrupt");
  return MDLM_OK;
}

int mdlm_corrupt_mixture(const int32_t* x0, int64_t n_tokens, const int32_t* cu_seqlens,
                         int32_t n_docs, uint64_t seed, double eps, double mixture_prob,
                         int32_t mask_id, int32_t rand_vocab, int32_t* xt,
                         uint8_t* corrupted, double* p_doc, int32_t* doc_counts,
                         void* stream) {
  clear_error();
  const char* fn = "mdlm_corrupt_mixture";
  if (n_tokens < 0) return fail(MDLM_EINVAL, "%s: n_tokens < 0", fn);
  if (n_tokens > INT32_MAX) return fail(MDLM_EUNSUPPORTED, "%s: n_tokens must be below 2^31", fn);
  if (n_docs < 0) return fail(MDLM_EINVAL, "%s: n_docs < 0", fn);
  if (n_docs == 0 && n_tokens > 0) return fail(MDLM_EINVAL, "%s: tokens given but n_docs = 0", fn);
  if (!(eps > 0.0 && eps <= 1.0)) return fail(MDLM_EINVAL, "%s: eps must lie in (0, 1]", fn);
  if (!(mixture_prob >= 0.0 && mixture_prob <= 1.0))
    return fail(MDLM_EINVAL, "%s: mixture_prob must lie in [0, 1]", fn);
  if (rand_vocab < 1) return fail(MDLM_EINVAL, "%s: rand_vocab must be >= 1", fn);
  if (n_tokens > 0 && (!x0 || !xt || !corrupted))
    return fail(MDLM_EINVAL, "%s: null token pointer", fn);
  if (n_docs > 0 && (!cu_seqlens || !p_doc || !doc_counts))
    return fail(MDLM_EINVAL, "%s: null document pointer", fn);
  if (const int rc = check_docs(fn, cu_seqlens, n_docs, n_tokens, nullptr,
                                reinterpret_cast<hipStream_t>(stream)))
    return rc;
  if (launch_corrupt(x0, n_tokens, cu_seqlens, n_docs, seed, eps, kNoiseMixture, mask_id,
                     rand_vocab, xt, corrupted, p_doc, doc_counts,
                     reinterpret_cast<hipStream_t>(stream), mixture_prob) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

size_t mdlm_corrupt_compact_workspace_bytes(int64_t n_tokens) {
  return corrupt_compact_workspace_bytes(n_tokens);
}

int mdlm_corrupt_compact(const int32_t* x0, int64_t n_tokens, const int32_t* cu_seqlens,
                         int32_t n_docs, uint64_t seed, double eps, int32_t noise,
                         int32_t mask_id, int32_t rand_vocab, int32_t align, int32_t* xt,
                         uint8_t* corrupted, double* p_doc, int32_t* doc_counts,
                         int32_t* row_idx, int32_t* tgt, float* w, int32_t* n_rows,
                         void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  const char* fn = "mdlm_corrupt_compact";
  if (n_tokens < 0) return fail(MDLM_EINVAL, "%s: n_tokens < 0", fn);
  if (n_tokens > INT32_MAX) return fail(MDLM_EUNSUPPORTED, "%s: n_tokens must be below 2^31", fn);
  if (n_docs < 0) return fail(MDLM_EINVAL, "%s: n_docs < 0", fn);
  if (n_docs == 0 && n_tokens > 0) return fail(MDLM_EINVAL, "%s: tokens given but n_docs = 0", fn);
  if (!(eps > 0.0 && eps <= 1.0)) return fail(MDLM_EINVAL, "%s: eps must lie in (0, 1]", fn);
  if (noise != MDLM_NOISE_ABSORB && noise != MDLM_NOISE_UNIFORM)
    return fail(MDLM_EINVAL, "%s: unknown noise mode %d", fn, noise);
  if (noise == MDLM_NOISE_UNIFORM && rand_vocab < 1)
    return fail(MDLM_EINVAL, "%s: rand_vocab must be >= 1", fn);
  if (align != MDLM_ALIGNED && align != MDLM_SHIFTED)
    return fail(MDLM_EINVAL, "%s: unknown alignment %d", fn, align);
  if (!n_rows) return fail(MDLM_EINVAL, "%s: null n_rows", fn);
  if (n_tokens > 0 && (!x0 || !xt || !row_idx || !tgt || !w))
    return fail(MDLM_EINVAL, "%s: null token pointer", fn);
  if (n_docs > 0 && (!cu_seqlens || !p_doc || !doc_counts))
    return fail(MDLM_EINVAL, "%s: null document pointer", fn);
  const size_t need = corrupt_compact_workspace_bytes(n_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes,
                need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) % 8) != 0)
    return fail(MDLM_EINVAL, "%s: workspace must be 8-byte aligned", fn);
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (const int rc = check_docs(fn, cu_seqlens, n_docs, n_tokens, nullptr, st)) return rc;
  if (launch_corrupt_compact(x0, n_tokens, cu_seqlens, n_docs, seed, eps, noise, mask_id,
                             rand_vocab, align, xt, corrupted, p_doc, doc_counts, row_idx, tgt,
                             w, n_rows, workspace, st) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

size_t mdlm_compact_workspace_bytes(int64_t n_tokens) {
  return compact_workspace_bytes(n_tokens, 0, MDLM_WEIGHT_INV_P);
}

size_t mdlm_compact_rows_workspace_bytes(int64_t n_tokens, int32_t n_docs, int32_t weighting) {
  if (n_docs < 0 || weighting < MDLM_WEIGHT_INV_P || weighting > MDLM_WEIGHT_EXAMPLE_MEAN_CLIPPED)
    return 0;
  return compact_workspace_bytes(n_tokens, n_docs, weighting);
}

// Shared checks and launch of both compaction entry points.
static int compact_common(const char* fn, bool need_mask, const uint8_t* corrupted,
                          const uint8_t* eligible,
                          const int32_t* x0, int64_t n_tokens, const int32_t* cu_seqlens,
                          int32_t n_docs, const double* p_doc, int32_t align, int32_t weighting,
                          double scale, double clip, int32_t* row_idx, int32_t* tgt, float* w,
                          int32_t* n_rows, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (n_tokens < 0) return fail(MDLM_EINVAL, "%s: n_tokens < 0", fn);
  if (n_tokens > INT32_MAX)
    return fail(MDLM_EUNSUPPORTED, "%s: n_tokens must be below 2^31", fn);
  if (n_docs < 0 || (n_docs == 0 && n_tokens > 0))
    return fail(MDLM_EINVAL, "%s: bad n_docs %d", fn, n_docs);
  if (align != MDLM_ALIGNED && align != MDLM_SHIFTED)
    return fail(MDLM_EINVAL, "%s: unknown alignment %d", fn, align);
  if (weighting < MDLM_WEIGHT_INV_P || weighting > MDLM_WEIGHT_EXAMPLE_MEAN_CLIPPED)
    return fail(MDLM_EINVAL, "%s: unknown weighting %d", fn, weighting);
  if (!isfinite(scale)) return fail(MDLM_EINVAL, "%s: weight_scale must be finite", fn);
  if (weighting == MDLM_WEIGHT_EXAMPLE_MEAN_CLIPPED && !(clip > 0.0))
    return fail(MDLM_EINVAL, "%s: weight_clip must be > 0", fn);
  if (!n_rows) return fail(MDLM_EINVAL, "%s: null n_rows", fn);
  const bool need_p = weighting != MDLM_WEIGHT_MEAN;
  if (n_tokens > 0 && (!x0 || !cu_seqlens || !row_idx || !tgt || !w || (need_p && !p_doc) ||
                       (need_mask && !corrupted)))
    return fail(MDLM_EINVAL, "%s: null pointer", fn);
  const size_t need = compact_workspace_bytes(n_tokens, n_docs, weighting);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes,
                need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) % 4) != 0)
    return fail(MDLM_EINVAL, "%s: workspace must be 4-byte aligned", fn);
  if (const int rc = check_docs(fn, cu_seqlens, n_docs, n_tokens, need_p ? p_doc : nullptr,
                                reinterpret_cast<hipStream_t>(stream)))
    return rc;
  if (launch_compact(corrupted, eligible, x0, n_tokens, cu_seqlens, n_docs, p_doc, align,
                     weighting, scale, clip, row_idx, tgt, w, n_rows, workspace,
                     reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_compact_masked(const uint8_t* corrupted, const int32_t* x0, int64_t n_tokens,
                        const int32_t* cu_seqlens, int32_t n_docs, const double* p_doc,
                        int32_t align, int32_t* row_idx, int32_t* tgt, float* w,
                        int32_t* n_rows, void* workspace, size_t workspace_bytes,
                        void* stream) {
  clear_error();
  return compact_common("mdlm_compact_masked", true, corrupted, nullptr, x0, n_tokens, cu_seqlens,
                        n_docs, p_doc, align, MDLM_WEIGHT_INV_P, 1.0, 0.0, row_idx, tgt, w,
                        n_rows, workspace, workspace_bytes, stream);
}

int mdlm_compact_masked_noalloc(const uint8_t* corrupted, const int32_t* x0, int64_t n_tokens,
                                const int32_t* cu_seqlens, int32_t n_docs, const double* p_doc,
                                int32_t align, int32_t* row_idx, int32_t* tgt, float* w,
                                int32_t* n_rows, void* stream) {
  clear_error();
  const char* fn = "mdlm_compact_masked_noalloc";
  if (n_tokens > kNoAllocMaxTokens)
    return fail(MDLM_EUNSUPPORTED, "%s: n_tokens = %lld exceeds the %lld tokens its scratch "
                "array serves (use mdlm_compact_masked with a workspace)", fn,
                (long long)n_tokens, (long long)kNoAllocMaxTokens);
  void* scratch = nullptr;
  const size_t need = compact_workspace_bytes(n_tokens, n_docs, MDLM_WEIGHT_INV_P);
  if (need > 0 && compact_scratch(&scratch) != hipSuccess)
    return fail(MDLM_EHIP, "%s: no scratch array on this device", fn);
  if (need > compact_scratch_bytes())
    return fail(MDLM_EUNSUPPORTED, "%s: workspace of %zu bytes exceeds the scratch array", fn,
                need);
  return compact_common(fn, true, corrupted, nullptr, x0, n_tokens, cu_seqlens, n_docs, p_doc,
                        align, MDLM_WEIGHT_INV_P, 1.0, 0.0, row_idx, tgt, w, n_rows, scratch,
                        compact_scratch_bytes(), stream);
}

int mdlm_compact_corrective(const uint8_t* codes, const int32_t* x0, int64_t n_tokens,
                            const int32_t* cu_seqlens, int32_t n_docs, const double* p_doc,
                            int32_t align, double noise_token_wt, double clean_token_wt,
                            int32_t* row_idx, int32_t* tgt, float* w, int32_t* n_rows,
                            void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  const char* fn = "mdlm_compact_corrective";
  if (n_tokens < 0) return fail(MDLM_EINVAL, "%s: n_tokens < 0", fn);
  if (n_tokens > INT32_MAX)
    return fail(MDLM_EUNSUPPORTED, "%s: n_tokens must be below 2^31", fn);
  if (n_docs < 0 || (n_docs == 0 && n_tokens > 0))
    return fail(MDLM_EINVAL, "%s: bad n_docs %d", fn, n_docs);
  if (align != MDLM_ALIGNED && align != MDLM_SHIFTED)
    return fail(MDLM_EINVAL, "%s: unknown alignment %d", fn, align);
  if (!isfinite(noise_token_wt) || !isfinite(clean_token_wt))
    return fail(MDLM_EINVAL, "%s: token weights must be finite", fn);
  if (!n_rows) return fail(MDLM_EINVAL, "%s: null n_rows", fn);
  if (n_tokens > 0 && (!codes || !x0 || !cu_seqlens || !p_doc || !row_idx || !tgt || !w))
    return fail(MDLM_EINVAL, "%s: null pointer", fn);
  const size_t need = compact_workspace_bytes(n_tokens, n_docs, MDLM_WEIGHT_INV_P);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes,
                need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) % 4) != 0)
    return fail(MDLM_EINVAL, "%s: workspace must be 4-byte aligned", fn);
  if (const int rc = check_docs(fn, cu_seqlens, n_docs, n_tokens, p_doc,
                                reinterpret_cast<hipStream_t>(stream)))
    return rc;
  if (launch_compact_corrective(codes, x0, n_tokens, cu_seqlens, n_docs, p_doc, align,
                                noise_token_wt, clean_token_wt, row_idx, tgt, w, n_rows,
                                workspace, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_compact_rows(const uint8_t* corrupted, const uint8_t* eligible, const int32_t* x0,
                      int64_t n_tokens, const int32_t* cu_seqlens, int32_t n_docs,
                      const double* p_doc, int32_t align, int32_t weighting,
                      double weight_scale, double weight_clip, int32_t* row_idx, int32_t* tgt,
                      float* w, int32_t* n_rows, void* workspace, size_t workspace_bytes,
                      void* stream) {
  clear_error();
  return compact_common("mdlm_compact_rows", false, corrupted, eligible, x0, n_tokens, cu_seqlens,
                        n_docs, p_doc, align, weighting, weight_scale, weight_clip, row_idx, tgt,
                        w, n_rows, workspace, workspace_bytes, stream);
}

static bool head_sizes_ok(int64_t max_rows, int32_t H, int32_t V, int32_t dtype) {
  return max_rows >= 0 && max_rows <= INT32_MAX && H > 0 && V > 0 &&
         (dtype == MDLM_F32 || dtype == MDLM_BF16);
}

size_t mdlm_head_ce_workspace_bytes(int64_t max_rows, int32_t H, int32_t V, int32_t dtype) {
  if (!head_sizes_ok(max_rows, H, V, dtype)) return 0;
  return head_ce_workspace_bytes(max_rows, H, V, dtype, false, false);
}

size_t mdlm_head_ce_workspace_min_bytes(int64_t max_rows, int32_t H, int32_t V,
                                        int32_t dtype) {
  if (!head_sizes_ok(max_rows, H, V, dtype)) return 0;
  return head_ce_workspace_bytes(max_rows, H, V, dtype, true, false);
}

size_t mdlm_head_ce_dw_workspace_bytes(int64_t max_rows, int32_t H, int32_t V) {
  if (!head_sizes_ok(max_rows, H, V, MDLM_BF16)) return 0;
  return head_ce_workspace_bytes(max_rows, H, V, MDLM_BF16, false, true);
}

size_t mdlm_head_ce_dw_workspace_min_bytes(int64_t max_rows, int32_t H, int32_t V) {
  if (!head_sizes_ok(max_rows, H, V, MDLM_BF16)) return 0;
  return head_ce_workspace_bytes(max_rows, H, V, MDLM_BF16, true, true);
}

// Shared checks and launch of both fused head + CE entry points.
static int head_common(const char* fn, const void* hidden, const void* W, int32_t dtype,
                       int64_t n_tokens, int32_t H, int32_t V, const int32_t* row_idx,
                       const int32_t* tgt, const float* w, const int32_t* n_rows,
                       int64_t max_rows, float softcap, float* loss, float* row_ce,
                       void* d_hidden, float* dW, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (dtype != MDLM_F32 && dtype != MDLM_BF16)
    return fail(MDLM_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (n_tokens < 0 || H <= 0 || V <= 0)
    return fail(MDLM_EINVAL, "%s: bad sizes n_tokens=%lld H=%d V=%d", fn, (long long)n_tokens,
                H, V);
  if (max_rows < 0 || max_rows > n_tokens)
    return fail(MDLM_EINVAL, "%s: max_rows must lie in [0, n_tokens]", fn);
  if (n_tokens > INT32_MAX) return fail(MDLM_EUNSUPPORTED, "%s: n_tokens must be below 2^31", fn);
  if (H % 64 != 0) return fail(MDLM_EUNSUPPORTED, "%s: H = %d is not a multiple of 64", fn, H);
  // the bf16 kernels address hidden (gathered rows) and W (the dH product)
  // through 32-bit byte offsets
  if (dtype == MDLM_BF16 && (n_tokens * (int64_t)H * 2 >= (int64_t)1 << 32 ||
                             (int64_t)V * H * 2 >= (int64_t)1 << 32))
    return fail(MDLM_EUNSUPPORTED, "%s: bf16 hidden and W must each be below 4 GiB", fn);
  if (!(softcap >= 0.f) || !isfinite(softcap))
    return fail(MDLM_EINVAL, "%s: softcap must be finite and >= 0", fn);
  if (!loss) return fail(MDLM_EINVAL, "%s: null loss", fn);
  if (max_rows > 0 && (!hidden || !W || !row_idx || !tgt || !w || !n_rows))
    return fail(MDLM_EINVAL, "%s: null input pointer", fn);
  if (dtype == MDLM_BF16 && max_rows > 0 &&
      ((reinterpret_cast<uintptr_t>(hidden) | reinterpret_cast<uintptr_t>(W)) % 16) != 0)
    return fail(MDLM_EINVAL, "%s: hidden and W must be 16-byte aligned", fn);
  if (dW && (reinterpret_cast<uintptr_t>(dW) % 16) != 0)
    return fail(MDLM_EINVAL, "%s: dW must be 16-byte aligned", fn);
  if (d_hidden && (reinterpret_cast<uintptr_t>(d_hidden) % 16) != 0)
    return fail(MDLM_EINVAL, "%s: d_hidden must be 16-byte aligned", fn);
  const size_t need =
      max_rows > 0 ? head_ce_workspace_bytes(max_rows, H, V, dtype, true, dW != nullptr) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need at least %zu", fn,
                workspace_bytes, need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) % 256) != 0)
    return fail(MDLM_EINVAL, "%s: workspace must be 256-byte aligned", fn);
  if (const int rc = check_row_list(fn, row_idx, tgt, w, n_rows, max_rows, n_tokens, V,
                                    reinterpret_cast<hipStream_t>(stream)))
    return rc;
  HeadCeArgs a;
  a.hidden = hidden;
  a.W = W;
  a.dtype = dtype;
  a.n_tokens = n_tokens;
  a.H = H;
  a.V = V;
  a.row_idx = row_idx;
  a.tgt = tgt;
  a.w = w;
  a.n_rows = n_rows;
  a.max_rows = max_rows;
  a.softcap = softcap;
  a.loss = loss;
  a.row_ce = row_ce;
  a.d_hidden = d_hidden;
  a.dW = dW;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  if (launch_head_ce(a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_fused_head_ce_fwd_bwd(const void* hidden, const void* W, int32_t dtype,
                               int64_t n_tokens, int32_t H, int32_t V,
                               const int32_t* row_idx, const int32_t* tgt, const float* w,
                               const int32_t* n_rows, int64_t max_rows, float softcap,
                               float* loss, float* row_ce, void* d_hidden, void* workspace,
                               size_t workspace_bytes, void* stream) {
  clear_error();
  return head_common("mdlm_fused_head_ce_fwd_bwd", hidden, W, dtype, n_tokens, H, V, row_idx,
                     tgt, w, n_rows, max_rows, softcap, loss, row_ce, d_hidden, nullptr,
                     workspace, workspace_bytes, stream);
}

int mdlm_fused_head_ce_fwd_bwd_dw(const void* hidden, const void* W, int64_t n_tokens,
                                  int32_t H, int32_t V, const int32_t* row_idx,
                                  const int32_t* tgt, const float* w, const int32_t* n_rows,
                                  int64_t max_rows, float softcap, float* loss, float* row_ce,
                                  void* d_hidden, float* dW, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  clear_error();
  const char* fn = "mdlm_fused_head_ce_fwd_bwd_dw";
  if (!dW) return fail(MDLM_EINVAL, "%s: null dW", fn);
  return head_common(fn, hidden, W, MDLM_BF16, n_tokens, H, V, row_idx, tgt, w, n_rows,
                     max_rows, softcap, loss, row_ce, d_hidden, dW, workspace, workspace_bytes,
                     stream);
}

int mdlm_scale(const void* x, void* y, int32_t dtype, int64_t n, const float* scale,
               void* stream) {
  clear_error();
  const char* fn = "mdlm_scale";
  if (dtype != MDLM_F32 && dtype != MDLM_BF16)
    return fail(MDLM_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (n < 0) return fail(MDLM_EINVAL, "%s: n < 0", fn);
  if (n > 0 && (!x || !y || !scale)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (n > 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % 16) != 0)
    return fail(MDLM_EINVAL, "%s: x and y must be 16-byte aligned", fn);
  if (launch_scale(x, y, dtype, n, scale, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_embed(const int32_t* ids, int64_t n_tokens, const void* table, int32_t dtype, int32_t V,
               int32_t H, float scale, void* out, void* stream) {
  clear_error();
  const char* fn = "mdlm_embed";
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (const int rc = check_row_sizes(fn, dtype, n_tokens, H)) return rc;
  if (H > kEmbedMaxH) return fail(MDLM_EUNSUPPORTED, "%s: H = %d exceeds %d", fn, H, kEmbedMaxH);
  if (V <= 0) return fail(MDLM_EINVAL, "%s: V must be > 0", fn);
  if (!isfinite(scale)) return fail(MDLM_EINVAL, "%s: scale must be finite", fn);
  if (n_tokens > 0 && (!ids || !table || !out)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(ids, 4) || misaligned(table, entry_bytes(dtype)) ||
      misaligned(out, entry_bytes(dtype)))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  if (const int rc = check_token_ids(fn, ids, n_tokens, V, st)) return rc;
  if (launch_embed(ids, n_tokens, table, dtype, V, H, scale, out, st) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

size_t mdlm_embed_grad_workspace_bytes(int64_t n_tokens, int32_t H) {
  if (n_tokens > INT32_MAX || H > kEmbedMaxH) return 0;
  return embed_grad_workspace_bytes(n_tokens, H);
}

int mdlm_embed_grad(const int32_t* ids, int64_t n_tokens, const void* d_out, int32_t dtype,
                    int32_t V, int32_t H, float scale, float* d_table, int32_t accumulate,
                    void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  const char* fn = "mdlm_embed_grad";
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (const int rc = check_row_sizes(fn, dtype, n_tokens, H)) return rc;
  if (H > kEmbedMaxH) return fail(MDLM_EUNSUPPORTED, "%s: H = %d exceeds %d", fn, H, kEmbedMaxH);
  if (V <= 0) return fail(MDLM_EINVAL, "%s: V must be > 0", fn);
  if (!isfinite(scale)) return fail(MDLM_EINVAL, "%s: scale must be finite", fn);
  if (accumulate != 0 && accumulate != 1)
    return fail(MDLM_EINVAL, "%s: accumulate must be 0 or 1", fn);
  if (!d_table || (n_tokens > 0 && (!ids || !d_out)))
    return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(ids, 4) || misaligned(d_out, entry_bytes(dtype)) || misaligned(d_table, 4))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  const size_t need = embed_grad_workspace_bytes(n_tokens, H);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes,
                need);
  if (need > 0 && misaligned(workspace, 256))
    return fail(MDLM_EINVAL, "%s: workspace must be 256-byte aligned", fn);
  if (const int rc = check_token_ids(fn, ids, n_tokens, V, st)) return rc;
  if (launch_embed_grad(ids, n_tokens, d_out, dtype, V, H, scale, d_table, accumulate != 0,
                        workspace, st) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

// Sizes and kind of the norm's entry points.
static int check_norm(const char* fn, int32_t dtype, int64_t n, int32_t H, int32_t kind) {
  if (const int rc = check_row_sizes(fn, dtype, n, H)) return rc;
  if (H > kNormMaxH)
    return fail(MDLM_EUNSUPPORTED, "%s: H = %d exceeds %d", fn, H, kNormMaxH);
  if (kind != MDLM_NORM_LAYER && kind != MDLM_NORM_RMS)
    return fail(MDLM_EINVAL, "%s: unknown norm %d", fn, kind);
  return MDLM_OK;
}

int mdlm_norm_fwd(const void* x, int32_t dtype, int64_t n, int32_t H, int32_t kind,
                  const void* weight, const void* bias, double eps, void* y, float* mean,
                  float* rstd, uint8_t* q, uint8_t* q_exp, void* stream) {
  clear_error();
  const char* fn = "mdlm_norm_fwd";
  if (const int rc = check_norm(fn, dtype, n, H, kind)) return rc;
  if (!(eps > 0.0) || !((float)eps > 0.f) || !isfinite((float)eps))
    return fail(MDLM_EINVAL, "%s: eps must be a positive float", fn);
  if (n > 0 && (!x || !y)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if ((q == nullptr) != (q_exp == nullptr))
    return fail(MDLM_EINVAL, "%s: q and q_exp are given together or not at all", fn);
  const size_t to = entry_bytes(dtype);
  if (misaligned(x, to) || misaligned(weight, to) || misaligned(bias, to) || misaligned(y, to) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  if (launch_norm_fwd(x, dtype, n, H, kind, weight, bias, eps, y, mean, rstd, q, q_exp,
                      reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

size_t mdlm_norm_bwd_workspace_bytes(int64_t n, int32_t H) {
  if (n > INT32_MAX) return 0;
  return norm_bwd_workspace_bytes(n, H);
}

// Shared checks and launch of both backward entry points.
static int norm_bwd_common(const char* fn, const void* dy, bool from_x, const void* x,
                           const uint8_t* q, const uint8_t* q_exp, int32_t dtype, int64_t n,
                           int32_t H, int32_t kind, const void* weight, const float* mean,
                           const float* rstd, void* dx, float* d_weight, float* d_bias,
                           int32_t accumulate, void* workspace, size_t workspace_bytes,
                           void* stream, const void* add = nullptr) {
  if (const int rc = check_norm(fn, dtype, n, H, kind)) return rc;
  if (accumulate != 0 && accumulate != 1)
    return fail(MDLM_EINVAL, "%s: accumulate must be 0 or 1", fn);
  if (n > 0 && (!dy || !rstd || (kind == MDLM_NORM_LAYER && !mean) ||
                (from_x ? !x : !q || !q_exp)))
    return fail(MDLM_EINVAL, "%s: null input pointer", fn);
  if (n > 0 && !dx && !d_weight && !d_bias)
    return fail(MDLM_EINVAL, "%s: no gradient is asked for", fn);
  const size_t to = entry_bytes(dtype);
  if (misaligned(dy, to) || misaligned(x, to) || misaligned(weight, to) || misaligned(mean, 4) ||
      misaligned(rstd, 4) || misaligned(dx, to) || misaligned(d_weight, 4) ||
      misaligned(d_bias, 4))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  const size_t need = d_weight || d_bias ? norm_bwd_workspace_bytes(n, H) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes,
                need);
  if (need > 0 && misaligned(workspace, 256))
    return fail(MDLM_EINVAL, "%s: workspace must be 256-byte aligned", fn);
  if (launch_norm_bwd(dy, x, q, q_exp, dtype, n, H, kind, weight, mean, rstd, dx, d_weight,
                      d_bias, accumulate != 0, workspace,
                      reinterpret_cast<hipStream_t>(stream), add) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_norm_bwd(const void* dy, const void* x, int32_t dtype, int64_t n, int32_t H,
                  int32_t kind, const void* weight, const float* mean, const float* rstd,
                  void* dx, float* d_weight, float* d_bias, int32_t accumulate, void* workspace,
                  size_t workspace_bytes, void* stream) {
  clear_error();
  return norm_bwd_common("mdlm_norm_bwd", dy, true, x, nullptr, nullptr, dtype, n, H, kind,
                         weight, mean, rstd, dx, d_weight, d_bias, accumulate, workspace,
                         workspace_bytes, stream);
}

int mdlm_norm_bwd_ckpt8(const void* dy, const uint8_t* q, const uint8_t* q_exp, int32_t dtype,
                        int64_t n, int32_t H, int32_t kind, const void* weight,
                        const float* mean, const float* rstd, void* dx, float* d_weight,
                        float* d_bias, int32_t accumulate, void* workspace,
                        size_t workspace_bytes, void* stream) {
  clear_error();
  return norm_bwd_common("mdlm_norm_bwd_ckpt8", dy, false, nullptr, q, q_exp, dtype, n, H, kind,
                         weight, mean, rstd, dx, d_weight, d_bias, accumulate, workspace,
                         workspace_bytes, stream);
}

// Checks of both checkpoint entry points; x's end is the output of one.
static int check_ckpt8(const char* fn, const void* x, int32_t dtype, int64_t n, int32_t H,
                       const uint8_t* q, const uint8_t* q_exp) {
  if (const int rc = check_row_sizes(fn, dtype, n, H)) return rc;
  if (H > kCkptMaxH) return fail(MDLM_EUNSUPPORTED, "%s: H = %d exceeds %d", fn, H, kCkptMaxH);
  if (n * (((int64_t)H + 127) / 128) > UINT32_MAX)
    return fail(MDLM_EUNSUPPORTED, "%s: 2^32 or more blocks of 128", fn);
  if (n > 0 && (!x || !q || !q_exp)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(x, entry_bytes(dtype)))
    return fail(MDLM_EINVAL, "%s: x is not aligned to its entries", fn);
  return MDLM_OK;
}

int mdlm_ckpt8_save(const void* x, int32_t dtype, int64_t n, int32_t H, uint8_t* q,
                    uint8_t* q_exp, void* stream) {
  clear_error();
  const char* fn = "mdlm_ckpt8_save";
  if (const int rc = check_ckpt8(fn, x, dtype, n, H, q, q_exp)) return rc;
  if (launch_ckpt8_save(x, dtype, n, H, q, q_exp, reinterpret_cast<hipStream_t>(stream)) !=
      hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_ckpt8_load(const uint8_t* q, const uint8_t* q_exp, int32_t dtype, int64_t n, int32_t H,
                    void* x, void* stream) {
  clear_error();
  const char* fn = "mdlm_ckpt8_load";
  if (const int rc = check_ckpt8(fn, x, dtype, n, H, q, q_exp)) return rc;
  if (launch_ckpt8_load(q, q_exp, dtype, n, H, x, reinterpret_cast<hipStream_t>(stream)) !=
      hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_add_norm_fwd(const void* x, const void* residual, int32_t dtype, int64_t n, int32_t H,
                      const void* weight, double eps, void* sum, void* y, float* rstd,
                      uint8_t* q, uint8_t* q_exp, void* stream) {
  clear_error();
  const char* fn = "mdlm_add_norm_fwd";
  if (const int rc = check_norm(fn, dtype, n, H, MDLM_NORM_RMS)) return rc;
  if (!(eps > 0.0) || !((float)eps > 0.f) || !isfinite((float)eps))
    return fail(MDLM_EINVAL, "%s: eps must be a positive float", fn);
  if ((q == nullptr) != (q_exp == nullptr))
    return fail(MDLM_EINVAL, "%s: q and q_exp are given together or not at all", fn);
  if (n > 0 && (!x || !residual || !sum)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (n > 0 && !y && !q) return fail(MDLM_EINVAL, "%s: no form of the norm is asked for", fn);
  const size_t to = entry_bytes(dtype);
  if (misaligned(x, to) || misaligned(residual, to) || misaligned(weight, to) ||
      misaligned(sum, to) || misaligned(y, to) || misaligned(rstd, 4))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  if (launch_add_norm(x, residual, dtype, n, H, weight, eps, sum, y, rstd, q, q_exp,
                      reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_add_norm_bwd(const void* dy, const void* d_sum, const void* sum, int32_t dtype,
                      int64_t n, int32_t H, const void* weight, const float* rstd, void* dx,
                      float* d_weight, int32_t accumulate, void* workspace,
                      size_t workspace_bytes, void* stream) {
  clear_error();
  const char* fn = "mdlm_add_norm_bwd";
  if (d_sum && misaligned(d_sum, entry_bytes(dtype)))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  return norm_bwd_common(fn, dy, true, sum, nullptr, nullptr, dtype, n, H, MDLM_NORM_RMS, weight,
                         nullptr, rstd, dx, d_weight, nullptr, accumulate, workspace,
                         workspace_bytes, stream, dx ? d_sum : nullptr);
}

// Sizes of the entry points that work on microscaled rows.
static int check_mx(const char* fn, int32_t format, int64_t n, int32_t H) {
  if (format != MDLM_MX_E4M3 && format != MDLM_MX_E2M1)
    return fail(MDLM_EINVAL, "%s: unknown format %d", fn, format);
  if (H > kMxMaxH) return fail(MDLM_EUNSUPPORTED, "%s: H = %d exceeds %d", fn, H, kMxMaxH);
  if (n * (((int64_t)H + 31) / 32) > UINT32_MAX)
    return fail(MDLM_EUNSUPPORTED, "%s: 2^32 or more blocks of 32", fn);
  return MDLM_OK;
}

int mdlm_mx_quantize(const void* x, int32_t dtype, int64_t n, int32_t H, int32_t format,
                     uint8_t* q, uint8_t* q_exp, void* stream) {
  clear_error();
  const char* fn = "mdlm_mx_quantize";
  if (const int rc = check_row_sizes(fn, dtype, n, H)) return rc;
  if (const int rc = check_mx(fn, format, n, H)) return rc;
  if (n > 0 && (!x || !q || !q_exp)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(x, entry_bytes(dtype)))
    return fail(MDLM_EINVAL, "%s: x is not aligned to its entries", fn);
  if (launch_mx_quantize(x, dtype, n, H, format, q, q_exp,
                         reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_mx_dequantize(const uint8_t* q, const uint8_t* q_exp, int32_t format, int64_t n,
                       int32_t H, int32_t dtype, void* x, void* stream) {
  clear_error();
  const char* fn = "mdlm_mx_dequantize";
  if (const int rc = check_row_sizes(fn, dtype, n, H)) return rc;
  if (const int rc = check_mx(fn, format, n, H)) return rc;
  if (n > 0 && (!x || !q || !q_exp)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(x, entry_bytes(dtype)))
    return fail(MDLM_EINVAL, "%s: x is not aligned to its entries", fn);
  if (launch_mx_dequantize(q, q_exp, format, n, H, dtype, x,
                           reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_mx_product(const uint8_t* a, const uint8_t* a_exp, int32_t a_format, int64_t n_tokens,
                    const uint8_t* w, const uint8_t* w_exp, int32_t V, int32_t H,
                    const int32_t* row_idx, const int32_t* n_rows, int64_t max_rows,
                    float softcap, int32_t out_dtype, void* logits, void* stream) {
  clear_error();
  const char* fn = "mdlm_mx_product";
  const hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (const int rc = check_row_sizes(fn, out_dtype, n_tokens, H)) return rc;
  if (const int rc = check_mx(fn, a_format, n_tokens, H)) return rc;
  if (V <= 0) return fail(MDLM_EINVAL, "%s: V must be > 0", fn);
  if (max_rows < 0 || max_rows > INT32_MAX)
    return fail(MDLM_EINVAL, "%s: bad max_rows %lld", fn, (long long)max_rows);
  if (!row_idx && max_rows > n_tokens)
    return fail(MDLM_EINVAL, "%s: max_rows exceeds n_tokens and no rows are listed", fn);
  if (V > kMxMaxRows || max_rows > kMxMaxRows)
    return fail(MDLM_EUNSUPPORTED, "%s: V or max_rows exceeds %d", fn, kMxMaxRows);
  if (!(softcap >= 0.f) || !isfinite(softcap) || (softcap > 0.f && !isfinite(1.f / softcap)))
    return fail(MDLM_EINVAL, "%s: softcap and its inverse must be >= 0 and finite", fn);
  if (max_rows > 0 && (!w || !w_exp || !logits || (n_tokens > 0 && (!a || !a_exp))))
    return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(a, 16) || misaligned(w, 16))
    return fail(MDLM_EINVAL, "%s: codes must be 16-byte aligned", fn);
  if (misaligned(logits, entry_bytes(out_dtype)) || misaligned(row_idx, 4) ||
      misaligned(n_rows, 4))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  const int64_t row_bytes = (a_format == MDLM_MX_E4M3 ? 32 : 16) * (((int64_t)H + 31) / 32);
  if (row_idx && n_tokens * row_bytes >= (int64_t)0xFFFFFFF0)
    return fail(MDLM_EUNSUPPORTED, "%s: listed rows need codes of less than 4 GiB", fn);
  if (row_idx)
    if (const int rc = check_row_list(fn, row_idx, nullptr, nullptr, n_rows, max_rows, n_tokens,
                                      V, st))
      return rc;
  if (launch_mx_product(a, a_exp, a_format, n_tokens, w, w_exp, V, H, row_idx, n_rows, max_rows,
                        softcap, out_dtype, logits, st) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

size_t mdlm_sample_workspace_bytes(int64_t max_rows, int32_t V) {
  if (max_rows > INT32_MAX) return 0;
  return sample_workspace_bytes(max_rows, V);
}

int mdlm_sample(const void* logits, int32_t dtype, int64_t max_rows, int32_t V, int64_t stride,
                const int32_t* n_rows, const float* temperature, const int32_t* top_k,
                const float* top_p, const float* min_p, const float* u, int32_t* token,
                float* logp, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  const char* fn = "mdlm_sample";
  if (const int rc = check_row_sizes(fn, dtype, max_rows, V)) return rc;
  if (V > kSampleMaxV) return fail(MDLM_EUNSUPPORTED, "%s: V = %d exceeds %d", fn, V, kSampleMaxV);
  if (stride < V) return fail(MDLM_EINVAL, "%s: rows overlap (stride %lld)", fn, (long long)stride);
  if (max_rows > 0 && stride > INT64_MAX / 8 / max_rows)
    return fail(MDLM_EINVAL, "%s: stride %lld is too large", fn, (long long)stride);
  if (max_rows > 0 && (!logits || !u || !token)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (misaligned(logits, entry_bytes(dtype)) || misaligned(n_rows, 4) ||
      misaligned(temperature, 4) || misaligned(top_k, 4) || misaligned(top_p, 4) ||
      misaligned(min_p, 4) || misaligned(u, 4) || misaligned(token, 4) || misaligned(logp, 4))
    return fail(MDLM_EINVAL, "%s: a pointer is not aligned to its entries", fn);
  const size_t need = sample_workspace_bytes(max_rows, V);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MDLM_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes,
                need);
  if (need > 0 && misaligned(workspace, 256))
    return fail(MDLM_EINVAL, "%s: workspace must be 256-byte aligned", fn);
  SampleArgs a;
  a.logits = logits, a.dtype = dtype, a.max_rows = max_rows, a.V = V, a.stride = stride;
  a.n_rows = n_rows, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p;
  a.min_p = min_p, a.u = u, a.token = token, a.logp = logp, a.workspace = workspace;
  if (launch_sample(a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_check_offsets(const int32_t* cu_seqlens, int32_t n_docs, int64_t n_tokens,
                       int32_t* status, void* stream) {
  clear_error();
  const char* fn = "mdlm_check_offsets";
  if (n_docs < 0 || n_tokens < 0) return fail(MDLM_EINVAL, "%s: bad sizes", fn);
  if (!cu_seqlens || !status) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (launch_check_offsets(cu_seqlens, n_docs, n_tokens, status,
                           reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_check_probs(const double* p_doc, int32_t n_docs, int32_t* status, void* stream) {
  clear_error();
  const char* fn = "mdlm_check_probs";
  if (n_docs < 0) return fail(MDLM_EINVAL, "%s: n_docs < 0", fn);
  if ((n_docs > 0 && !p_doc) || !status) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (launch_check_probs(p_doc, n_docs, status, reinterpret_cast<hipStream_t>(stream)) !=
      hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_check_rows(const int32_t* row_idx, const int32_t* tgt, const float* w,
                    const int32_t* n_rows, int64_t max_rows, int64_t n_tokens, int32_t V,
                    int32_t* status, void* stream) {
  clear_error();
  const char* fn = "mdlm_check_rows";
  if (max_rows < 0 || n_tokens < 0 || V < 0) return fail(MDLM_EINVAL, "%s: bad sizes", fn);
  if (!n_rows || !status || (max_rows > 0 && !row_idx))
    return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (launch_check_rows(row_idx, tgt, w, n_rows, max_rows, n_tokens, V, status,
                        reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_check_tokens(const int32_t* ids, int64_t n_tokens, int32_t V, int32_t* status,
                      void* stream) {
  clear_error();
  const char* fn = "mdlm_check_tokens";
  if (n_tokens < 0 || V <= 0) return fail(MDLM_EINVAL, "%s: bad sizes", fn);
  if (!status || (n_tokens > 0 && !ids)) return fail(MDLM_EINVAL, "%s: null pointer", fn);
  if (launch_check_tokens(ids, n_tokens, V, status, reinterpret_cast<hipStream_t>(stream)) !=
      hipSuccess)
    return check_launch(fn);
  return MDLM_OK;
}

int mdlm_set_checking(int enable) { return set_checking(enable); }

}  // extern "C"
