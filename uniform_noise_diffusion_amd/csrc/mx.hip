// Matrices held in 8 or 4 bits with one power of two per 32 entries of a row:
// rows coded, and read back.
//
// Axolotl diffusion docs, "Adapters, merging and inference" (QLoRA: frozen
// matrices kept in 4 bits); GGUF catalog page (quantised copies for
// inference).  The pages fix no format; this one is what the matrix cores
// take as it lies (mx_product.hip).
//
// Both directions are one pass, bound by memory: eight entries to a lane, so
// that what an instruction reads or writes lies end to end, four lanes to a
// block, whose largest magnitude is two lane exchanges away (126,464 x 4,096 bf16
// to 4 bits 235 us, 5.6 TB/s, and back 230 us, 5.8 TB/s; to 8 bits 256 us and
// back 252 us, 6.1 and 6.2 TB/s of their own bytes).
#include "mx.h"

#include <algorithm>

namespace mdlm {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;

// Item i is eight entries, a quarter of block i / 4; a row has nb blocks.
// FULL: H is a multiple of 32, and the rows' blocks lie end to end.
template <typename T, int BITS, bool FULL>
__global__ void __launch_bounds__(kThreads)
mx_quantize_kernel(const T* __restrict__ x, int64_t items, int32_t H, uint32_t nb,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ q_exp) {
  // (items and the stride are multiples of four: a quad's lanes stay together)
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * kThreads) {
    float v[8];
    if (FULL) {
      widen(load8<true>(x + 8 * i, 0, 8), v);
    } else {
      const uint32_t block = (uint32_t)(i >> 2), r = block / nb;
      const int64_t row = r;
      const int c = (int)(kMxBlock * (block - r * nb)) + 8 * (int)(i & 3);
      if (c < H) {
        widen(load8<false>(x + row * H, c, H), v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
      }
    }
    uint32_t byte;
    if (BITS == 8) {
      const uint2 code = mx8_encode(v, byte);
      *reinterpret_cast<u32x2_a1*>(q + 8 * i) = u32x2_a1{code.x, code.y};
    } else {
      typedef uint32_t u32_a1 __attribute__((aligned(1)));
      *reinterpret_cast<u32_a1*>(q + 4 * i) = mx4_encode(v, byte);
    }
    if ((i & 3) == 0) q_exp[i >> 2] = (uint8_t)byte;
  }
}

template <typename T, int BITS, bool FULL>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ q_exp,
                     int64_t items, int32_t H, uint32_t nb, T* __restrict__ x) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * kThreads) {
    const float scale = mx_scale(q_exp[i >> 2]);
    float v[8];
    if (BITS == 8) {
      const u32x2_a1 c = *reinterpret_cast<const u32x2_a1*>(q + 8 * i);
      ckpt_decode8(make_uint2(c.x, c.y), scale, v);
    } else {
      typedef uint32_t u32_a1 __attribute__((aligned(1)));
      mx4_decode(*reinterpret_cast<const u32_a1*>(q + 4 * i), scale, v);
    }
    if (FULL) {
      store8<true>(x + 8 * i, 0, 8, v);
    } else {
      const uint32_t block = (uint32_t)(i >> 2), r = block / nb;
      const int64_t row = r;
      const int c = (int)(kMxBlock * (block - r * nb)) + 8 * (int)(i & 3);
      if (c < H) store8<false>(x + row * H, c, H, v);
    }
  }
}

struct Shape {
  int64_t items;
  uint32_t nb;
  unsigned grid;
  Shape(int64_t n, int32_t H) {
    nb = (uint32_t)(((int64_t)H + kMxBlock - 1) / kMxBlock);
    items = 4 * n * nb;
    grid = (unsigned)std::min<int64_t>((items + kThreads - 1) / kThreads, kMaxBlocks);
  }
};

template <typename T, int BITS>
void run_quantize(const void* x, int64_t n, int32_t H, uint8_t* q, uint8_t* q_exp,
                  hipStream_t stream) {
  const Shape s(n, H);
  auto kernel = H % kMxBlock == 0 ? mx_quantize_kernel<T, BITS, true>
                                  : mx_quantize_kernel<T, BITS, false>;
  kernel<<<s.grid, kThreads, 0, stream>>>(reinterpret_cast<const T*>(x), s.items, H, s.nb, q,
                                          q_exp);
}

template <typename T, int BITS>
void run_dequantize(const uint8_t* q, const uint8_t* q_exp, int64_t n, int32_t H, void* x,
                    hipStream_t stream) {
  const Shape s(n, H);
  auto kernel = H % kMxBlock == 0 ? mx_dequantize_kernel<T, BITS, true>
                                  : mx_dequantize_kernel<T, BITS, false>;
  kernel<<<s.grid, kThreads, 0, stream>>>(q, q_exp, s.items, H, s.nb,
                                          reinterpret_cast<T*>(x));
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int32_t dtype, int64_t n, int32_t H, int32_t format,
                              uint8_t* q, uint8_t* q_exp, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  if (dtype == MDLM_BF16)
    format == MDLM_MX_E4M3 ? run_quantize<bf16_t, 8>(x, n, H, q, q_exp, stream)
                           : run_quantize<bf16_t, 4>(x, n, H, q, q_exp, stream);
  else
    format == MDLM_MX_E4M3 ? run_quantize<float, 8>(x, n, H, q, q_exp, stream)
                           : run_quantize<float, 4>(x, n, H, q, q_exp, stream);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* q_exp, int32_t format, int64_t n,
                                int32_t H, int32_t dtype, void* x, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  if (dtype == MDLM_BF16)
    format == MDLM_MX_E4M3 ? run_dequantize<bf16_t, 8>(q, q_exp, n, H, x, stream)
                           : run_dequantize<bf16_t, 4>(q, q_exp, n, H, x, stream);
  else
    format == MDLM_MX_E4M3 ? run_dequantize<float, 8>(q, q_exp, n, H, x, stream)
                           : run_dequantize<float, 4>(q, q_exp, n, H, x, stream);
  return hipGetLastError();
}

}  // namespace mdlm
