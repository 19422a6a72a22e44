// Activation checkpoints in 8 bits: an [n, H] activation kept as e4m3 values
// with one power-of-two scale for each block of 128 entries of a row (the
// last block of a row may be shorter), and read back.
//
// LLaDA-8B-MDLM-LoRA card, "Training" table, "Precision" row: the training
// runs these losses belong to keep activation checkpoints.
//
// Both directions are one pass, bound by memory: 16 lanes hold a block, eight
// entries each, so its largest magnitude is four lane exchanges away.
#include "row_ops.h"

#include <algorithm>

namespace mdlm {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // blocks of 128 per pass of a thread block
constexpr int64_t kMaxBlocks = 1 << 20;

// FULL: H is a multiple of 128, so the rows' blocks lie end to end.
template <typename T, bool FULL>
__global__ void __launch_bounds__(kThreads)
ckpt_save_kernel(const T* __restrict__ x, int64_t blocks, int32_t H, int32_t per_row,
                 uint8_t* __restrict__ q, uint8_t* __restrict__ q_exp) {
  const int sub = 8 * (threadIdx.x & 15);
  for (int64_t b = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4); b < blocks;
       b += (int64_t)gridDim.x * kGroups) {
    const int64_t row = FULL ? b : (int64_t)((uint32_t)b / (uint32_t)per_row);
    const int c = FULL ? sub : (int)(b - row * per_row) * kCkptBlock + sub;
    const int64_t off = FULL ? b * kCkptBlock : row * H;
    const int len = FULL ? kCkptBlock : H;
    float v[8];
    widen(load8<FULL>(x + off, c, len), v);
    const uint32_t e = ckpt_exp_byte(row16_max(finite_top8(v)));
    store8_codes<FULL>(q + off, c, len, ckpt_encode8(v, ckpt_inv_scale(e)));
    if (sub == 0) q_exp[b] = (uint8_t)e;
  }
}

template <typename T, bool FULL>
__global__ void __launch_bounds__(kThreads)
ckpt_load_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ q_exp,
                 int64_t blocks, int32_t H, int32_t per_row, T* __restrict__ x) {
  const int sub = 8 * (threadIdx.x & 15);
  for (int64_t b = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4); b < blocks;
       b += (int64_t)gridDim.x * kGroups) {
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
  const unsigned grid = (unsigned)std::min<int64_t>((blocks + kGroups - 1) / kGroups, kMaxBlocks);
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
