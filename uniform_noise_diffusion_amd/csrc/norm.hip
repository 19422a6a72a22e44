// Layer norm and RMS norm of rows, forward and backward, the input optionally
// kept as an 8-bit checkpoint.
//
// Axolotl diffusion docs, "Adapters, merging and inference": the loss is taken
// "from hidden states", which leave the model through its final norm; the
// gradient d_hidden enters the model through it.
//
//   layer:  mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps)
//   RMS:    mu = 0,        r = 1 / sqrt(mean(x^2) + eps)
//   xhat = (x - mu) r,  y = xhat w + b
//   g = dy w,  dx = r (g - [layer] mean(g) - xhat mean(g xhat))
//   d_w = sum over rows of dy xhat,  d_b = sum over rows of dy
//
// A row stays in registers between its statistics and its output, so each
// tensor is read or written once; the variance is a second pass over the
// registers, with nothing subtracted that could cancel.  All sums are fp32.
//
// A row's eights of columns are dealt to W waves, NV eights to a lane:
// column 8 ((k W + wave) 64 + lane) for k < NV.  Sixteen consecutive lanes
// hold one block of 128, so the checkpoint's scale comes from four lane
// exchanges.
#include "row_ops.h"

#include <algorithm>

namespace mdlm {
namespace {

constexpr int64_t kMaxBlocks = 1 << 20;

struct NormFwdArgs {
  const void* x;
  const void* weight;  // null: 1
  const void* bias;    // null: 0
  void* y;
  float* mean;  // null: not wanted
  float* rstd;
  uint8_t* q;  // null: no checkpoint
  uint8_t* q_exp;
  int64_t n;
  int32_t H;
  float eps;
  float inv_h;
  int32_t layer;
};

// Sum over a row's W waves; every thread of the block calls it.  `buf` holds
// one float per wave and is not reused before another barrier.
template <int W>
__device__ __forceinline__ float row_sum(float x, float* buf, int wave) {
  x = wave_sum(x);
  if (W == 1) return x;
  if ((threadIdx.x & 63) == 0) buf[wave] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += buf[wave / W * W + w];
  return s;
}

template <typename T, int W, int NV, bool FULL>
__global__ void __launch_bounds__((W > 4 ? W : 4) * 64)
norm_fwd_kernel(const NormFwdArgs a) {
  constexpr int kWaves = W > 4 ? W : 4;
  constexpr int kRows = kWaves / W;
  __shared__ float s_a[kWaves], s_b[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c0 = 8 * ((wave % W) * 64 + lane);
  const int H = a.H;
  const int per_row = (H + kCkptBlock - 1) / kCkptBlock;
  const T* weight = reinterpret_cast<const T*>(a.weight);
  const T* bias = reinterpret_cast<const T*>(a.bias);
  // (the trip count is the block's: every wave reaches every barrier)
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.n;
       base += (int64_t)gridDim.x * kRows) {
    const int64_t row = base + wave / W;
    const bool live = row < a.n;
    const T* x = reinterpret_cast<const T*>(a.x) + (live ? row : 0) * H;
    float v[NV][8];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) widen(load8<FULL>(x, c0 + 512 * W * k, H), v[k]);
    float mean = 0.f;
    if (a.layer) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[k][i];
      mean = row_sum<W>(s, s_a, wave) * a.inv_h;
    }
    s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // columns past H were read as zero and count for nothing
        const float d = c0 + 512 * W * k + i < H ? v[k][i] - mean : 0.f;
        s += d * d;
      }
    const float var = row_sum<W>(s, s_b, wave) * a.inv_h;
    const float r = 1.f / sqrtf(var + a.eps);
    if (live) {
      if (lane == 0 && wave % W == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = r;
      }
      T* y = reinterpret_cast<T*>(a.y) + row * H;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = c0 + 512 * W * k;
        if (a.q) {
          // all 16 lanes of a block take part, whatever of it the row has
          const uint32_t e = ckpt_exp_byte(row16_max(finite_top8(v[k])));
          store8_codes<FULL>(a.q + row * H, c, H, ckpt_encode8(v[k], ckpt_inv_scale(e)));
          if ((lane & 15) == 0 && c < H) a.q_exp[row * per_row + c / kCkptBlock] = (uint8_t)e;
        }
        float o[8], p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (v[k][i] - mean) * r;
        if (weight) {
          widen(load8<FULL>(weight, c, H), p);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] *= p[i];
        }
        if (bias) {
          widen(load8<FULL>(bias, c, H), p);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += p[i];
        }
        store8<FULL>(y, c, H, o);
      }
    }
    if (W > 1 && !a.layer) __syncthreads();  // s_b is free again
  }
}

struct NormBwdArgs {
  const void* dy;
  const void* x;  // null: from the checkpoint
  const uint8_t* q;
  const uint8_t* q_exp;
  const void* weight;  // null: 1
  const float* mean;   // null: RMS norm
  const float* rstd;
  void* dx;       // null: not wanted
  float* part_w;  // [gridDim.x][H], null: not wanted
  float* part_b;
  int64_t n;
  int32_t H;
  float inv_h;
};

constexpr int kBwdWaves = 8;

// One block walks every gridDim.x-th group of rows and keeps its columns'
// parameter gradients in registers; they leave once, as one partial row per
// block.
template <typename T, int W, int NV, bool FULL, bool CKPT>
__global__ void __launch_bounds__((W > kBwdWaves ? W : kBwdWaves) * 64)
norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int kWaves = W > kBwdWaves ? W : kBwdWaves;
  constexpr int kRows = kWaves / W;
  __shared__ float s_sum[2][2][kWaves];
  __shared__ float s_join[kRows > 1 ? 8 * 64 * W * NV : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / W;
  const int c0 = 8 * ((wave % W) * 64 + lane);
  const int H = a.H;
  const int per_row = (H + kCkptBlock - 1) / kCkptBlock;
  float wt[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (a.weight)
      widen(load8<FULL>(reinterpret_cast<const T*>(a.weight), c0 + 512 * W * k, H), wt[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!a.weight) wt[k][i] = 1.f;
      dw[k][i] = db[k][i] = 0.f;
    }
  }
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.n;
       base += (int64_t)gridDim.x * kRows, flip ^= 1) {
    const int64_t row = base + group;
    const bool live = row < a.n;
    const int64_t off = (live ? row : 0) * H;
    const float mean = live && a.mean ? a.mean[row] : 0.f;
    const float r = live ? a.rstd[row] : 0.f;
    float g[NV][8], xh[NV][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = c0 + 512 * W * k;
      widen(load8<FULL>(reinterpret_cast<const T*>(a.dy) + off, c, H), g[k]);
      if (CKPT) {
        const uint32_t e = c < H ? a.q_exp[(live ? row : 0) * per_row + c / kCkptBlock] : 0;
        ckpt_decode8(load8_codes<FULL>(a.q + off, c, H), ckpt_scale(e), xh[k]);
      } else {
        widen(load8<FULL>(reinterpret_cast<const T*>(a.x) + off, c, H), xh[k]);
      }
    }
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = FULL || c0 + 512 * W * k + i < H;
          xh[k][i] = in ? (xh[k][i] - mean) * r : 0.f;
          dw[k][i] += g[k][i] * xh[k][i];
          db[k][i] += g[k][i];
          g[k][i] *= wt[k][i];
          s1 += g[k][i];
          s2 += g[k][i] * xh[k][i];
        }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (W > 1) {
      if (lane == 0) s_sum[flip][0][wave] = s1, s_sum[flip][1][wave] = s2;
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        s1 += s_sum[flip][0][group * W + w];
        s2 += s_sum[flip][1][group * W + w];
      }
    }
    const float m1 = a.mean ? s1 * a.inv_h : 0.f, m2 = s2 * a.inv_h;
    if (live && a.dx) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * (g[k][i] - m1 - xh[k][i] * m2);
        store8<FULL>(reinterpret_cast<T*>(a.dx) + off, c0 + 512 * W * k, H, o);
      }
    }
  }
  // the groups' sums join in order, then leave
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float* part = t == 0 ? a.part_w : a.part_b;
    if (!part) continue;
    auto& d = t == 0 ? dw : db;
    if (kRows > 1)
      for (int j = 1; j < kRows; ++j) {
        __syncthreads();
        if (group == j)
#pragma unroll
          for (int k = 0; k < NV; ++k)
            store8<true>(s_join, c0 + 512 * W * k, 512 * W * NV, d[k]);
        __syncthreads();
        if (group == 0)
#pragma unroll
          for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) d[k][i] += s_join[c0 + 512 * W * k + i];
      }
    if (group == 0)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store8<FULL>(part + (int64_t)blockIdx.x * H, c0 + 512 * W * k, H, d[k]);
  }
}

// d_w and d_b from the blocks' partial rows: 64 columns per block, 16 waves
// sharing the rows, their sums added in order.  blockIdx.y: d_w or d_b.
constexpr int kSumWaves = 16;

__global__ void __launch_bounds__(kSumWaves * 64)
norm_sum_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int32_t rows,
                int32_t H, float* __restrict__ d_weight, float* __restrict__ d_bias,
                int32_t accumulate) {
  __shared__ float s[kSumWaves][64];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? d_weight : d_bias;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float acc = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int r = wave; r < rows; r += kSumWaves) acc += part[(int64_t)r * H + c];
  }
  s[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && c < H) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWaves; ++w) t += s[w][lane];
    out[c] = accumulate ? out[c] + t : t;
  }
}

// Rows that one block of the backward pass holds at a time.
int rows_at_once(int32_t H) {
  const int w = H <= 1024 ? 1 : H <= 2048 ? 2 : H <= 4096 ? 4 : H <= 8192 ? 8 : 16;
  return std::max(w, kBwdWaves) / w;
}

// Blocks of the backward pass, each of which leaves one partial row.
int64_t bwd_blocks(int64_t n, int32_t H) {
  return std::min<int64_t>((n + rows_at_once(H) - 1) / rows_at_once(H), 512);
}

template <typename T, int W, int NV>
void run_fwd(const NormFwdArgs& a, hipStream_t stream) {
  constexpr int kWaves = W > 4 ? W : 4, kRows = kWaves / W;
  const unsigned grid = (unsigned)std::min<int64_t>((a.n + kRows - 1) / kRows, kMaxBlocks);
  if (a.H % 8 == 0)
    norm_fwd_kernel<T, W, NV, true><<<grid, kWaves * 64, 0, stream>>>(a);
  else
    norm_fwd_kernel<T, W, NV, false><<<grid, kWaves * 64, 0, stream>>>(a);
}

template <typename T>
void pick_fwd(const NormFwdArgs& a, hipStream_t stream) {
  const int H = a.H;
  if (H <= 512) run_fwd<T, 1, 1>(a, stream);
  else if (H <= 1024) run_fwd<T, 1, 2>(a, stream);
  else if (H <= 2048) run_fwd<T, 2, 2>(a, stream);
  else if (H <= 4096) run_fwd<T, 4, 2>(a, stream);
  else if (H <= 8192) run_fwd<T, 8, 2>(a, stream);
  else run_fwd<T, 16, 2>(a, stream);
}

template <typename T, int W, int NV>
void run_bwd(const NormBwdArgs& a, unsigned grid, hipStream_t stream) {
  constexpr int kThreads = (W > kBwdWaves ? W : kBwdWaves) * 64;
  const bool full = a.H % 8 == 0;
  if (a.x) {
    if (full) norm_bwd_kernel<T, W, NV, true, false><<<grid, kThreads, 0, stream>>>(a);
    else norm_bwd_kernel<T, W, NV, false, false><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (full) norm_bwd_kernel<T, W, NV, true, true><<<grid, kThreads, 0, stream>>>(a);
    else norm_bwd_kernel<T, W, NV, false, true><<<grid, kThreads, 0, stream>>>(a);
  }
}

template <typename T>
void pick_bwd(const NormBwdArgs& a, unsigned grid, hipStream_t stream) {
  const int H = a.H;
  if (H <= 512) run_bwd<T, 1, 1>(a, grid, stream);
  else if (H <= 1024) run_bwd<T, 1, 2>(a, grid, stream);
  else if (H <= 2048) run_bwd<T, 2, 2>(a, grid, stream);
  else if (H <= 4096) run_bwd<T, 4, 2>(a, grid, stream);
  else if (H <= 8192) run_bwd<T, 8, 2>(a, grid, stream);
  else run_bwd<T, 16, 2>(a, grid, stream);
}

}  // namespace

hipError_t launch_norm_fwd(const void* x, int32_t dtype, int64_t n, int32_t H, int32_t kind,
                           const void* weight, const void* bias, double eps, void* y, float* mean,
                           float* rstd, uint8_t* q, uint8_t* q_exp, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  NormFwdArgs a;
  a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.rstd = rstd, a.q = q, a.q_exp = q_exp;
  a.layer = kind == MDLM_NORM_LAYER;
  a.mean = a.layer ? mean : nullptr;
  a.n = n, a.H = H, a.eps = (float)eps, a.inv_h = (float)(1.0 / H);
  if (dtype == MDLM_BF16)
    pick_fwd<bf16_t>(a, stream);
  else
    pick_fwd<float>(a, stream);
  return hipGetLastError();
}

size_t norm_bwd_workspace_bytes(int64_t n, int32_t H) {
  if (n <= 0 || H <= 0 || H > kNormMaxH) return 0;
  return (size_t)(bwd_blocks(n, H) * H * 2 * 4);
}

hipError_t launch_norm_bwd(const void* dy, const void* x, const uint8_t* q, const uint8_t* q_exp,
                           int32_t dtype, int64_t n, int32_t H, int32_t kind, const void* weight,
                           const float* mean, const float* rstd, void* dx, float* d_weight,
                           float* d_bias, bool accumulate, void* workspace, hipStream_t stream) {
  const int64_t blocks = bwd_blocks(n, H);
  NormBwdArgs a;
  a.dy = dy, a.x = x, a.q = q, a.q_exp = q_exp, a.weight = weight, a.rstd = rstd, a.dx = dx;
  a.mean = kind == MDLM_NORM_LAYER ? mean : nullptr;
  a.part_w = d_weight ? reinterpret_cast<float*>(workspace) : nullptr;
  a.part_b = d_bias ? reinterpret_cast<float*>(workspace) + blocks * H : nullptr;
  a.n = n, a.H = H, a.inv_h = (float)(1.0 / H);
  if (n > 0) {
    if (dtype == MDLM_BF16)
      pick_bwd<bf16_t>(a, (unsigned)blocks, stream);
    else
      pick_bwd<float>(a, (unsigned)blocks, stream);
  }
  if (d_weight || d_bias)
    norm_sum_kernel<<<dim3((H + 63) / 64, 2), kSumWaves * 64, 0, stream>>>(
        a.part_w, a.part_b, (int32_t)blocks, H, d_weight, d_bias, accumulate);
  return hipGetLastError();
}

}  // namespace mdlm
