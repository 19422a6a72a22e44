// Activation checkpoints in 8 bits: an [n, H] activation kept as e4m3 values
// with one power-of-two scale for each block of 128 entries of a row (the
// last block of a row may be shorter), and read back.
//
// LLaDA-8B-MDLM-LoRA card, "Training" table, "Precision" row: the training
// runs these losses belong to keep activation checkpoints.
//
// Both directions are one pass, bound by memory.  Saving, 8 lanes hold a
// block, 16 entries each, so its largest magnitude is three lane exchanges
// away and the codes leave 16 bytes to a lane.
#include "row_ops.h"

#include <algorithm>

namespace mdlm {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 8;  // blocks of 128 per pass of a thread block
constexpr int64_t kMaxBlocks = 1 << 20;

// FULL: H is a multiple of 128, so the rows' blocks lie end to end.
template <typename T, bool FULL>
__global__ void __launch_bounds__(kThreads)
ckpt_save_kernel(const T* __restrict__ x, int64_t blocks, int32_t H, int32_t per_row,
                 uint8_t* __restrict__ q, uint8_t* __restrict__ q_exp) {
  const int sub = 16 * (threadIdx.x & 7);
  for (int64_t b = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 3); b < blocks;
       b += (int64_t)gridDim.x * kGroups) {
    const int64_t row = FULL ? b : (int64_t)((uint32_t)b / (uint32_t)per_row);
    const int c = FULL ? sub : (int)(b - row * per_row) * kCkptBlock + sub;
    const int64_t off = FULL ? b * kCkptBlock : row * H;
    const int len = FULL ? kCkptBlock : H;
    const Raw8<T> r0 = load8<FULL>(x + off, c, len), r1 = load8<FULL>(x + off, c + 8, len);
    float v0[8], v1[8];
    widen(r0, v0), widen(r1, v1);
    const uint32_t t0 = top8(r0), t1 = top8(r1);
    uint32_t top = lanes_max<8>(t0 > t1 ? t0 : t1);
    uint2 q0, q1;
    if (__ballot(top >= kNonFinite) == 0) {
      top = ckpt_exp_byte(top);
      q0 = ckpt_encode8<false>(v0, ckpt_inv_scale(top));
      q1 = ckpt_encode8<false>(v1, ckpt_inv_scale(top));
    } else {
      const uint32_t f0 = finite_top8(v0), f1 = finite_top8(v1);
      top = ckpt_exp_byte(lanes_max<8>(f0 > f1 ? f0 : f1));
      q0 = ckpt_encode8<true>(v0, ckpt_inv_scale(top));
      q1 = ckpt_encode8<true>(v1, ckpt_inv_scale(top));
    }
    store16_codes<FULL>(q + off, c, len, q0, q1);
    if (sub == 0) q_exp[b] = (uint8_t)top;
  }
}

// Eight entries to a lane here: what a store instruction writes then lies end
// to end (16 entries a lane, 36 -> 41 us for 16,384 x 4,096 bf16).
constexpr int kLoadGroups = kThreads / 16;

template <typename T, bool FULL>
__global__ void __launch_bounds__(kThreads)
ckpt_load_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ q_exp,
                 int64_t blocks, int32_t H, int32_t per_row, T* __restrict__ x) {
  const int sub = 8 * (threadIdx.x & 15);
  for (int64_t b = (int64_t)blockIdx.x * kLoadGroups + (threadIdx.x >> 4); b < blocks;
       b += (int64_t)gridDim.x * kLoadGroups) {
    const int64_t row = FULL ? b : (int64_t)((uint32_t)b / (uint32_t)per_row);
    const int c = FULL ? sub : (int)(b - row * per_row) * kCkptBlock + sub;
    const int64_t off = FULL ? b * kCkptBlock : row * H;
    const int len = FULL ? kCkptBlock : H;
    float v[8];
    ckpt_decode8(load8_codes<FULL>(q + off, c, len), ckpt_scale(q_exp[b]), v);
    store8<FULL>(x + off, c, len, v);
  }
}

template <typename T, bool FULL>
void run_save(const void* x, int64_t n, int32_t H, uint8_t* q, uint8_t* q_exp,
              hipStream_t stream) {
  const int per_row = (H + kCkptBlock - 1) / kCkptBlock;
  const int64_t blocks = n * per_row;
  const unsigned grid = (unsigned)std::min<int64_t>((blocks + kGroups - 1) / kGroups, kMaxBlocks);
  ckpt_save_kernel<T, FULL><<<grid, kThreads, 0, stream>>>(reinterpret_cast<const T*>(x), blocks,
                                                           H, per_row, q, q_exp);
}

template <typename T, bool FULL>
void run_load(const uint8_t* q, const uint8_t* q_exp, int64_t n, int32_t H, void* x,
              hipStream_t stream) {
  const int per_row = (H + kCkptBlock - 1) / kCkptBlock;
  const int64_t blocks = n * per_row;
  const unsigned grid =
      (unsigned)std::min<int64_t>((blocks + kLoadGroups - 1) / kLoadGroups, kMaxBlocks);
  ckpt_load_kernel<T, FULL><<<grid, kThreads, 0, stream>>>(q, q_exp, blocks, H, per_row,
                                                           reinterpret_cast<T*>(x));
}

}  // namespace

hipError_t launch_ckpt8_save(const void* x, int32_t dtype, int64_t n, int32_t H, uint8_t* q,
                             uint8_t* q_exp, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  const bool full = H % kCkptBlock == 0;
  if (dtype == MDLM_BF16)
    full ? run_save<bf16_t, true>(x, n, H, q, q_exp, stream)
         : run_save<bf16_t, false>(x, n, H, q, q_exp, stream);
  else
    full ? run_save<float, true>(x, n, H, q, q_exp, stream)
         : run_save<float, false>(x, n, H, q, q_exp, stream);
  return hipGetLastError();
}

hipError_t launch_ckpt8_load(const uint8_t* q, const uint8_t* q_exp, int32_t dtype, int64_t n,
                             int32_t H, void* x, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  const bool full = H % kCkptBlock == 0;
  if (dtype == MDLM_BF16)
    full ? run_load<bf16_t, true>(q, q_exp, n, H, x, stream)
         : run_load<bf16_t, false>(q, q_exp, n, H, x, stream);
  else
    full ? run_load<float, true>(q, q_exp, n, H, x, stream)
         : run_load<float, false>(q, q_exp, n, H, x, stream);
  return hipGetLastError();
}

}  // namespace mdlm
