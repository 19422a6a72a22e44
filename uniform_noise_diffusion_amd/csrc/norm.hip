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
// exchanges.  A block of up to 16 waves holds several rows at a time and
// walks every gridDim.x-th group of them, weights and sums of parameter
// gradients staying in registers.
//
// What bounds both directions is memory, once nothing else stands in its way:
// the next row's loads are issued before this one is reduced and written, and
// nothing in the loops is conditional, so that a wait for those loads is not
// one for the stores behind them too (with conditions the compiler waits for
// all of it: 2.3 us an iteration, 70 us instead of 61 for the gradient of
// 16,384 x 4,096 bf16 from a checkpoint).  With FULL (H a multiple of 8) the
// lanes past the row's end therefore take columns that other lanes hold: they
// write what those write, and count for nothing in the row's sums.
#include "row_ops.h"

#include <algorithm>
#include <type_traits>

namespace mdlm {
namespace {

constexpr int kBlockWaves = 16;

// Rows of W waves that a block holds at a time.
constexpr int rows_of(int W) { return kBlockWaves / W; }

// The column eight that the lane of column c takes: c, or with FULL, past the
// row's end, one of the same place in the row's last block of 128.
template <bool FULL>
__device__ __forceinline__ int column(int c, int H) {
  if (!FULL) return c;
  if ((c & ~127) >= H) c = ((H - 1) & ~127) + (c & 127);
  return c > H - 8 ? H - 8 : c;
}

// Eight entries of a weight or bias; `none` where there is none.
template <typename T, bool FULL>
__device__ __forceinline__ void load_param(const void* p, int c, int H, float none, float v[8]) {
  if (p) {
    widen(load8_in<FULL>(reinterpret_cast<const T*>(p), c, H), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = none;
  }
}

struct NormFwdArgs {
  const void* x;
  const void* weight;  // null: 1
  const void* bias;    // null: 0
  void* y;
  float* mean;  // null: not wanted
  float* rstd;
  uint8_t* q;
  uint8_t* q_exp;
  int64_t n;
  int32_t H;
  float eps;
  float inv_h;
  int32_t layer;
};

template <typename T, int W, int NV, bool FULL, bool CKPT>
__global__ void __launch_bounds__(rows_of(W) * W * 64)
norm_fwd_kernel(const NormFwdArgs a) {
  constexpr int kRows = rows_of(W);
  // each wave's sum, squares about its mean, mean; its columns
  __shared__ float s_part[2][3][kRows * W], s_cols[kRows * W];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / W;
  const int c0 = 8 * ((wave % W) * 64 + lane);
  const int H = a.H;
  const int per_row = (H + kCkptBlock - 1) / kCkptBlock;
  const int64_t last = a.n - 1;
  int col[NV];
  float wt[NV][8], bi[NV][8];
  int mine = 0;  // this lane's columns
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = c0 + 512 * W * k;
    col[k] = column<FULL>(c, H);
    mine += c + 8 <= H ? 8 : c < H ? H - c : 0;
    if (NV == 1) {
      load_param<T, FULL>(a.weight, col[k], H, 1.f, wt[k]);
      load_param<T, FULL>(a.bias, col[k], H, 0.f, bi[k]);
    }
  }
  // columns of each wave, whose sums are joined below
  const float of_wave = wave_sum((float)mine), inv_wave = of_wave > 0.f ? 1.f / of_wave : 0.f;
  if (lane == 0) s_cols[wave] = of_wave;  // (read behind the loop's barrier)
  const int64_t step = (int64_t)gridDim.x * kRows;
  const int64_t first = (int64_t)blockIdx.x * kRows + group;
  Raw8<T> in[NV] = {};
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      in[k] = load8_in<FULL>(reinterpret_cast<const T*>(a.x) + row * H, col[k], H);
  };
  constexpr bool kPrefetch = NV == 1;  // (two eights to a lane leave no registers for it)
  if (kPrefetch) fetch(first < last ? first : last);
  float means = 0.f, rstds = 0.f;  // of this group's rows of the last 64, one per lane
  int it = 0, flip = 0;

  auto take = [&](auto tail, int64_t row) {
    constexpr bool kTail = decltype(tail)::value;  // rows past the last one
    const bool live = !kTail || row <= last;
    float v[NV][8];
    if (!kPrefetch) fetch(live ? row : last);
#pragma unroll
    for (int k = 0; k < NV; ++k) widen(in[k], v[k]);
    if (CKPT && live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        // (all 16 lanes of a block take part, whatever of it the row has)
        uint32_t top = lanes_max<16>(top8(in[k]));
        uint2 code;
        if (__ballot(top >= kNonFinite) == 0) {
          top = ckpt_exp_byte(top);
          code = ckpt_encode8<false>(v[k], ckpt_inv_scale(top));
        } else {
          top = ckpt_exp_byte(lanes_max<16>(finite_top8(v[k])));
          code = ckpt_encode8<true>(v[k], ckpt_inv_scale(top));
        }
        // (the block's lanes write one byte's one value)
        if (FULL || col[k] < H)
          a.q_exp[row * per_row + col[k] / kCkptBlock] = (uint8_t)top;
        store8_codes_in<FULL>(a.q + row * H, col[k], H, code);
      }
    }
    if (kPrefetch && !kTail) fetch(row + step < last ? row + step : last);
    // each wave's mean and squares about it, then the row's from the waves':
    // squares about the row's mean are those about the wave's plus the
    // distance of the means, squared, once a column; nothing cancels
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += c0 + 512 * W * k + i < H ? v[k][i] : 0.f;
    s = a.layer ? wave_sum(s) : 0.f;
    float mean = s * inv_wave;
    float m2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = c0 + 512 * W * k + i < H ? v[k][i] - mean : 0.f;
        m2 += d * d;
      }
    m2 = wave_sum(m2);
    if (W > 1) {
      if (lane == 0) {
        s_part[flip][0][wave] = s;
        s_part[flip][1][wave] = m2;
        s_part[flip][2][wave] = mean;
      }
      __syncthreads();
      const int w0 = group * W;
      m2 = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) m2 += s_part[flip][1][w0 + w];
      if (a.layer) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += s_part[flip][0][w0 + w];
        mean = s * a.inv_h;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float d = s_part[flip][2][w0 + w] - mean, cols = s_cols[w0 + w];
          // (A wave past the row's end has no columns and a mean of 0: its
          // distance is finite, its square need not be.  A condition here
          // would cost the loop's loads their freedom: 57 us instead of 48 for
          // 16,384 x 4,096.  With two eights to a lane every wave has columns,
          // and this order is the faster one, 120 us to 124 for 8,192 x 12,288.)
          m2 += NV == 1 ? (cols * d) * d : cols * (d * d);
        }
      }
      flip ^= 1;
    }
    const float r = 1.f / sqrtf(m2 * a.inv_h + a.eps);
    means = lane == it ? mean : means;
    rstds = lane == it ? r : rstds;
    ++it;
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[8];
        if (NV > 1) {
          load_param<T, FULL>(a.weight, col[k], H, 1.f, wt[k]);
          load_param<T, FULL>(a.bias, col[k], H, 0.f, bi[k]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (v[k][i] - mean) * r * wt[k][i] + bi[k][i];
        store8_in<FULL>(reinterpret_cast<T*>(a.y) + row * H, col[k], H, o);
      }
    }
  };
  // (the trip counts are the block's: every wave reaches every barrier)
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.n;) {
    const int64_t row0 = base + group;
    it = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) arrived(in[k]);
    if constexpr (NV == 1)  // (two copies of the body want too many registers otherwise)
      for (; it < 64 && base + kRows <= a.n; base += step) take(std::false_type(), base + group);
    for (; it < 64 && base < a.n; base += step) take(std::true_type(), base + group);
    const int64_t row = row0 + lane * step;
    if (wave % W == 0 && lane < it && row <= last) {
      if (a.mean) a.mean[row] = means;
      if (a.rstd) a.rstd[row] = rstds;
    }
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

// One row's dy and x (or its checkpoint) as they lie in memory.
template <typename T, int NV, bool CKPT>
struct BwdRow {
  Raw8<T> dy[NV];
  Raw8<T> x[CKPT ? 1 : NV];
  uint2 q[CKPT ? NV : 1];
  uint32_t e[CKPT ? NV : 1];
};

// One block keeps its columns' parameter gradients in registers; they leave
// once, as one partial row per block.
template <typename T, int W, int NV, bool FULL, bool CKPT, bool DX>
__global__ void __launch_bounds__(rows_of(W) * W * 64)
norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int kRows = rows_of(W);
  // (two eights to a lane leave no registers for the next row)
  constexpr bool kPrefetch = NV == 1;
  __shared__ float s_sum[2][2][kRows * W];
  constexpr int kCols = 512 * W * NV;
  __shared__ float s_join[kRows > 1 ? kRows * kCols : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / W;
  const int c0 = 8 * ((wave % W) * 64 + lane);
  const int H = a.H;
  const int per_row = (H + kCkptBlock - 1) / kCkptBlock;
  const int64_t last = a.n - 1;
  int col[NV];
  float wt[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = c0 + 512 * W * k;
    col[k] = column<FULL>(c, H);
    load_param<T, FULL>(a.weight, col[k], H, 1.f, wt[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.f;
  }
  auto fetch = [&](int64_t row, BwdRow<T, NV, CKPT>& in) {
    const int64_t off = row * H;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      in.dy[k] = load8_in<FULL>(reinterpret_cast<const T*>(a.dy) + off, col[k], H);
      if constexpr (CKPT) {
        in.q[k] = load8_codes_in<FULL>(a.q + off, col[k], H);
        in.e[k] = a.q_exp[row * per_row + (FULL || col[k] < H ? col[k] : H - 1) / kCkptBlock];
      } else {
        in.x[k] = load8_in<FULL>(reinterpret_cast<const T*>(a.x) + off, col[k], H);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  const int64_t first = (int64_t)blockIdx.x * kRows + group;
  // the statistics of this group's next 64 rows, one per lane
  float means = 0.f, rstds = 0.f;
  int it = 0, flip = 0;
  BwdRow<T, NV, CKPT> in = {};
  if (kPrefetch) fetch(first < last ? first : last, in);

  auto take = [&](auto tail, int64_t row) {
    constexpr bool kTail = decltype(tail)::value;  // rows past the last one
    const bool live = !kTail || row <= last;
    const float mean = lane_value(means, it), r = lane_value(rstds, it);
    ++it;
    if (!kPrefetch) fetch(live ? row : last, in);
    float g[NV][8], xh[NV][8];
    float s1 = 0.f, s2 = 0.f;
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        widen(in.dy[k], g[k]);
        if constexpr (CKPT)
          ckpt_decode8(in.q[k], ckpt_scale(in.e[k]), xh[k]);
        else
          widen(in.x[k], xh[k]);
        float t1 = 0.f, t2 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (an entry past the row's end is no part of it: its distance from
          // the mean may be past float's range where every column's is not)
          xh[k][i] = FULL || c0 + 512 * W * k + i < H ? (xh[k][i] - mean) * r : 0.f;
          dw[k][i] += g[k][i] * xh[k][i];
          db[k][i] += g[k][i];
          g[k][i] *= wt[k][i];
          t1 += g[k][i];
          t2 += g[k][i] * xh[k][i];
        }
        // lanes past the row's end: see above, or (not FULL) dy = 0 and
        // xhat = 0, which add nothing
        const bool counts = !FULL || c0 + 512 * W * k < H;
        s1 += counts ? t1 : 0.f;
        s2 += counts ? t2 : 0.f;
      }
    }
    if (kPrefetch && !kTail) fetch(row + step < last ? row + step : last, in);
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
      flip ^= 1;
    }
    const float m1 = a.mean ? s1 * a.inv_h * r : 0.f, m2 = s2 * a.inv_h * r;
    if (DX && live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (r * g[k][i] - m1) - xh[k][i] * m2;
        store8_in<FULL>(reinterpret_cast<T*>(a.dx) + row * H, col[k], H, o);
      }
    }
  };
  // (the trip counts are the block's: every wave reaches every barrier)
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.n;) {
    const int64_t r = base + group + lane * step, at = r < last ? r : last;
    means = a.mean ? a.mean[at] : 0.f;
    rstds = a.rstd[at];
    it = 0;
    // what is on its way arrives before the loop, not at a wait inside it
    arrived(means), arrived(rstds);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      arrived(in.dy[k]);
      if constexpr (CKPT)
        arrived(in.q[k].x), arrived(in.e[k]);
      else
        arrived(in.x[k]);
    }
    if constexpr (NV == 1)  // (two copies of the body want too many registers otherwise)
      for (; it < 64 && base + kRows <= a.n; base += step) take(std::false_type(), base + group);
    for (; it < 64 && base < a.n; base += step) take(std::true_type(), base + group);
  }
  // the groups' sums join in order, then leave
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float* part = t == 0 ? a.part_w : a.part_b;
    if (!part) continue;
    part += (int64_t)blockIdx.x * H;
    auto& d = t == 0 ? dw : db;
    if (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store8<true>(s_join + group * kCols, c0 + 512 * W * k, kCols, d[k]);
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += kRows * W * 64) {
        float sum = s_join[c];
#pragma unroll
        for (int j = 1; j < kRows; ++j) sum += s_join[j * kCols + c];
        part[c] = sum;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) store8_in<FULL>(part, col[k], H, d[k]);
    }
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

// Waves per row: one eight of columns to a lane where 16 waves can hold the
// row so, two beyond.
int waves_for(int32_t H) {
  const int w = (H + 511) / 512;
  return w <= 2 ? w : w <= 4 ? 4 : w <= 6 ? 6 : w <= 8 ? 8 : w <= 12 ? 12 : 16;
}

// Blocks of the forward pass: two per compute unit.
constexpr int64_t kFwdBlocks = 512;

// Blocks of the backward pass, each of which leaves one partial row: one per
// compute unit.  Few rows (up to four steps of one block) take one block, whose
// partial row is the gradient itself: a launch less, 11.8 us a call -> 8.8
// (16,384 columns, whose four rows take the block 11.5: no slower).
int64_t bwd_blocks(int64_t n, int32_t H) {
  const int rows = rows_of(waves_for(H));
  if (n <= 4 * rows) return n > 0 ? 1 : 0;
  return std::min<int64_t>((n + rows - 1) / rows, 256);
}

template <typename T, int W, int NV, bool FULL>
void run_fwd(const NormFwdArgs& a, hipStream_t stream) {
  constexpr int kRows = rows_of(W);
  const unsigned grid = (unsigned)std::min<int64_t>((a.n + kRows - 1) / kRows, kFwdBlocks);
  auto kernel = a.q ? norm_fwd_kernel<T, W, NV, FULL, true> : norm_fwd_kernel<T, W, NV, FULL, false>;
  kernel<<<grid, kRows * W * 64, 0, stream>>>(a);
}

template <typename T, bool FULL>
void pick_fwd(const NormFwdArgs& a, hipStream_t stream) {
  switch (waves_for(a.H)) {
    case 1: return run_fwd<T, 1, 1, FULL>(a, stream);
    case 2: return run_fwd<T, 2, 1, FULL>(a, stream);
    case 4: return run_fwd<T, 4, 1, FULL>(a, stream);
    case 6: return run_fwd<T, 6, 1, FULL>(a, stream);
    case 8: return run_fwd<T, 8, 1, FULL>(a, stream);
    case 12: return run_fwd<T, 12, 1, FULL>(a, stream);
    default:
      return a.H <= 8192 ? run_fwd<T, 16, 1, FULL>(a, stream)
                         : run_fwd<T, 16, 2, FULL>(a, stream);
  }
}

template <typename T, int W, int NV, bool FULL>
void run_bwd(const NormBwdArgs& a, unsigned grid, hipStream_t stream) {
  constexpr int kThreads = rows_of(W) * W * 64;
  auto kernel = a.x ? (a.dx ? norm_bwd_kernel<T, W, NV, FULL, false, true>
                            : norm_bwd_kernel<T, W, NV, FULL, false, false>)
                    : (a.dx ? norm_bwd_kernel<T, W, NV, FULL, true, true>
                            : norm_bwd_kernel<T, W, NV, FULL, true, false>);
  kernel<<<grid, kThreads, 0, stream>>>(a);
}

template <typename T, bool FULL>
void pick_bwd(const NormBwdArgs& a, unsigned grid, hipStream_t stream) {
  switch (waves_for(a.H)) {
    case 1: return run_bwd<T, 1, 1, FULL>(a, grid, stream);
    case 2: return run_bwd<T, 2, 1, FULL>(a, grid, stream);
    case 4: return run_bwd<T, 4, 1, FULL>(a, grid, stream);
    case 6: return run_bwd<T, 6, 1, FULL>(a, grid, stream);
    case 8: return run_bwd<T, 8, 1, FULL>(a, grid, stream);
    case 12: return run_bwd<T, 12, 1, FULL>(a, grid, stream);
    default:
      return a.H <= 8192 ? run_bwd<T, 16, 1, FULL>(a, grid, stream)
                         : run_bwd<T, 16, 2, FULL>(a, grid, stream);
  }
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
  auto run = H % 8 == 0 ? (dtype == MDLM_BF16 ? pick_fwd<bf16_t, true> : pick_fwd<float, true>)
                        : (dtype == MDLM_BF16 ? pick_fwd<bf16_t, false> : pick_fwd<float, false>);
  run(a, stream);
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
  const bool direct = blocks == 1 && !accumulate;
  a.part_w = direct ? d_weight : d_weight ? reinterpret_cast<float*>(workspace) : nullptr;
  a.part_b = direct ? d_bias : d_bias ? reinterpret_cast<float*>(workspace) + blocks * H : nullptr;
  a.n = n, a.H = H, a.inv_h = (float)(1.0 / H);
  if (n > 0) {
    auto run = H % 8 == 0
                   ? (dtype == MDLM_BF16 ? pick_bwd<bf16_t, true> : pick_bwd<float, true>)
                   : (dtype == MDLM_BF16 ? pick_bwd<bf16_t, false> : pick_bwd<float, false>);
    run(a, (unsigned)blocks, stream);
  }
  // (no rows, accumulating: nothing to add, and + 0 would clear a zero's sign)
  if ((d_weight || d_bias) && !direct && (n > 0 || !accumulate))
    norm_sum_kernel<<<dim3((H + 63) / 64, 2), kSumWaves * 64, 0, stream>>>(
        a.part_w, a.part_b, (int32_t)blocks, H, d_weight, d_bias, accumulate);
  return hipGetLastError();
}

}  // namespace mdlm
