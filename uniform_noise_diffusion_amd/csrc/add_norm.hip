// The residual's addition and the RMS norm behind it in one pass over the rows,
// the norm written in the rows' own type, in 8 bits for a microscaled product,
// or both.
//
// Axolotl diffusion docs, "Adapters, merging and inference" (hidden states
// leave the model through its final norm).
//
//   s = x + residual, rounded once to its type;  r = 1 / sqrt(mean(s^2) + eps)
//   y = s r w
//
// The norm is that of s as it is kept, so the gradient formed from s later is
// the gradient of what was computed.  Sums are fp32; y is rounded once, to its
// type or (from fp32) to e4m3 over the power of two of its block of 32.
//
// Memory is the bound: x and the residual are read once, s and y written once
// (16,384 x 4,096 bf16 with 8-bit output: 96 us, 4.9 TB/s; 8,192 x 12,288,
// two eights to a lane and no prefetch, 144 us; one row: 2.8 us).
// The layout is norm.hip's: a row's eights of columns dealt to W waves, NV to a
// lane, the next row's loads issued before this one is reduced and written, and
// no condition in the loop (with FULL, H a multiple of 8, lanes past the row's
// end hold what other lanes hold and write what those write).  Four lanes hold
// a block of 32.
#include "mx.h"

#include <algorithm>
#include <type_traits>

namespace mdlm {
namespace {

struct AddNormArgs {
  const void* x;
  const void* residual;
  const void* weight;  // null: 1
  void* sum;
  void* y;
  uint8_t* q;
  uint8_t* q_exp;
  float* rstd;  // null: not wanted
  int64_t n;
  int32_t H;
  float eps;
  float inv_h;
};

// x + r as the sum's type holds it.
__device__ __forceinline__ Raw8<bf16_t> add8(const Raw8<bf16_t>& x, const Raw8<bf16_t>& r) {
  float a[8], b[8];
  widen(x, a), widen(r, b);
  Raw8<bf16_t> s;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s.w[i] = pack_bf16(a[2 * i] + b[2 * i], a[2 * i + 1] + b[2 * i + 1]);
  return s;
}
__device__ __forceinline__ Raw8<float> add8(const Raw8<float>& x, const Raw8<float>& r) {
  Raw8<float> s;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.w[i] = x.w[i] + r.w[i];
  return s;
}

// WITH_Y, WITH_Q: which forms of the norm are written.
template <typename T, int W, int NV, bool FULL, bool WITH_Y, bool WITH_Q>
__global__ void __launch_bounds__(rows_of(W) * W * 64)
add_norm_kernel(const AddNormArgs a) {
  constexpr int kRows = rows_of(W);
  __shared__ float s_part[2][kRows * W];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / W;
  const int H = a.H;
  const int nb = (H + kMxBlock - 1) / kMxBlock;
  const int64_t last = a.n - 1;
  // each eight's place among the codes, and the column it is read from: past
  // the row's last block of 32, the same place of that block; with FULL, past
  // the row's end, the row's last eight
  int at[NV], col[NV];
  float wt[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (((wave % W) + W * k) * 64 + lane);
    at[k] = FULL && (c & ~31) >= H ? ((H - 1) & ~31) + (c & 31) : c;
    col[k] = FULL && at[k] > H - 8 ? H - 8 : at[k];
    if (NV == 1) load_param<T, FULL>(a.weight, col[k], H, 1.f, wt[k]);
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  const int64_t first = (int64_t)blockIdx.x * kRows + group;
  Raw8<T> in_x[NV] = {}, in_r[NV] = {};
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      in_x[k] = load8_in<FULL>(reinterpret_cast<const T*>(a.x) + row * H, col[k], H);
      in_r[k] = load8_in<FULL>(reinterpret_cast<const T*>(a.residual) + row * H, col[k], H);
    }
  };
  constexpr bool kPrefetch = NV == 1;  // (two eights to a lane leave no registers for it)
  if (kPrefetch) fetch(first < last ? first : last);
  float rstds = 0.f;  // of this group's rows of the last 64, one per lane
  int it = 0, flip = 0;

  auto take = [&](auto tail, int64_t row) {
    constexpr bool kTail = decltype(tail)::value;  // rows past the last one
    const bool live = !kTail || row <= last;
    if (!kPrefetch) fetch(live ? row : last);
    float v[NV][8];
    float m2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Raw8<T> s = add8(in_x[k], in_r[k]);
      widen(s, v[k]);
      if (live) store8_in<FULL>(reinterpret_cast<T*>(a.sum) + row * H, col[k], H, v[k]);
      // (not FULL: entries past the row's end are zeros)
      const bool counts = !FULL || 8 * (((wave % W) + W * k) * 64 + lane) < H;
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += v[k][i] * v[k][i];
      m2 += counts ? t : 0.f;
    }
    if (kPrefetch && !kTail) fetch(row + step < last ? row + step : last);
    m2 = wave_sum(m2);
    if (W > 1) {
      if (lane == 0) s_part[flip][wave] = m2;
      __syncthreads();
      m2 = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) m2 += s_part[flip][group * W + w];
      flip ^= 1;
    }
    const float r = 1.f / sqrtf(m2 * a.inv_h + a.eps);
    rstds = lane == it ? r : rstds;
    ++it;
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[8];
        if (NV > 1) load_param<T, FULL>(a.weight, col[k], H, 1.f, wt[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[k][i] * r * wt[k][i];
        if (WITH_Y) store8_in<FULL>(reinterpret_cast<T*>(a.y) + row * H, col[k], H, o);
        if (WITH_Q) {
          if (!FULL) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = at[k] + i < H ? o[i] : 0.f;
          }
          uint32_t byte;
          uint2 code = mx8_encode(o, byte);
          if (FULL) {  // (places of the row's last block behind its end)
            code.x = at[k] < H ? code.x : 0u;
            code.y = at[k] < H ? code.y : 0u;
          }
          if (FULL || at[k] < kMxBlock * nb) {
            *reinterpret_cast<u32x2_a1*>(a.q + row * (kMxBlock * nb) + at[k]) =
                u32x2_a1{code.x, code.y};
            // (the block's lanes write one byte's one value)
            a.q_exp[row * nb + at[k] / kMxBlock] = (uint8_t)byte;
          }
        }
      }
    }
  };
  // (the trip counts are the block's: every wave reaches every barrier)
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.n;) {
    const int64_t row0 = base + group;
    it = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) arrived(in_x[k]), arrived(in_r[k]);
    if constexpr (NV == 1)  // (two copies of the body want too many registers otherwise)
      for (; it < 64 && base + kRows <= a.n; base += step) take(std::false_type(), base + group);
    for (; it < 64 && base < a.n; base += step) take(std::true_type(), base + group);
    const int64_t row = row0 + lane * step;
    if (a.rstd && wave % W == 0 && lane < it && row <= last) a.rstd[row] = rstds;
  }
}

// Two blocks per compute unit.
constexpr int64_t kBlocks = 512;

template <typename T, int W, int NV, bool FULL>
void run(const AddNormArgs& a, hipStream_t stream) {
  constexpr int kRows = rows_of(W);
  const unsigned grid = (unsigned)std::min<int64_t>((a.n + kRows - 1) / kRows, kBlocks);
  auto kernel = !a.q  ? add_norm_kernel<T, W, NV, FULL, true, false>
                : a.y ? add_norm_kernel<T, W, NV, FULL, true, true>
                      : add_norm_kernel<T, W, NV, FULL, false, true>;
  kernel<<<grid, kRows * W * 64, 0, stream>>>(a);
}

template <typename T, bool FULL>
void pick(const AddNormArgs& a, hipStream_t stream) {
  switch (waves_for(a.H)) {
    case 1: return run<T, 1, 1, FULL>(a, stream);
    case 2: return run<T, 2, 1, FULL>(a, stream);
    case 4: return run<T, 4, 1, FULL>(a, stream);
    case 6: return run<T, 6, 1, FULL>(a, stream);
    case 8: return run<T, 8, 1, FULL>(a, stream);
    case 12: return run<T, 12, 1, FULL>(a, stream);
    default:
      return a.H <= 8192 ? run<T, 16, 1, FULL>(a, stream) : run<T, 16, 2, FULL>(a, stream);
  }
}

}  // namespace

hipError_t launch_add_norm(const void* x, const void* residual, int32_t dtype, int64_t n,
                           int32_t H, const void* weight, double eps, void* sum, void* y,
                           float* rstd, uint8_t* q, uint8_t* q_exp, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  AddNormArgs a;
  a.x = x, a.residual = residual, a.weight = weight, a.sum = sum, a.y = y;
  a.q = q, a.q_exp = q_exp, a.rstd = rstd;
  a.n = n, a.H = H, a.eps = (float)eps, a.inv_h = (float)(1.0 / H);
  auto go = H % 8 == 0 ? (dtype == MDLM_BF16 ? pick<bf16_t, true> : pick<float, true>)
                       : (dtype == MDLM_BF16 ? pick<bf16_t, false> : pick<float, false>);
  go(a, stream);
  return hipGetLastError();
}

}  // namespace mdlm
