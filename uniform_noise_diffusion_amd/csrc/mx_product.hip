// Logits of microscaled rows through a microscaled 4-bit matrix.
//
// Axolotl diffusion docs, "Adapters, merging and inference" (a bare linear
// head over the final hidden states; QLoRA's frozen 4-bit matrices); "Batching"
// (logits only where a position needs them).
//
//   z[j][v] = sum over blocks b of 2^(ea + ew) * sum over the block's 32 k of a w
//   logits[j][v] = softcap ? softcap * tanh(z / softcap) : z
//
// with the codes and exponents of row row_idx[j] of A (8 or 4 bits) and of row
// v of W (4 bits).  The matrix cores take codes and exponents as they lie and
// accumulate in fp32: v_mfma_scale over 32 x 32 tiles and 64 k, its first
// operand 32 rows of W and its second 32 rows of A.
//
// Its register layout: lane l holds row l % 32 and, of the 64 k, for 4-bit
// codes 32 (l / 32) .. + 31; for 8-bit ones 16 (l / 32) .. + 15 and 32 +
// 16 (l / 32) .. + 15.  The exponent of k 0 .. 31 is taken from lane l % 32's
// byte, that of 32 .. 63 from lane 32 + l % 32's; an immediate picks one of the
// four bytes of a register.  The order of the blocks in the sum being free, the
// product of step s (of four) over a stage of eight blocks takes blocks s and
// 4 + s, so that a lane's four exponents of a stage are one word of LDS.
//
// Sums: 4-bit products of an instruction are added exactly, and to the fp32
// accumulator with one rounding.  8-bit ones are added in groups of eight
// consecutive k, over the power of two of the group's largest product, and what
// lies under 2^-13 of that is cut; the groups and the accumulator are added in
// fp32.  (Measured: 256 + 2^-6 within a group gives 256, across groups 256 +
// 2^-6; random rows of 64 to 4,096 are off by 4e-6 to 5e-6 of the result's
// norm, 4-bit ones by none of it.)  That is three orders under bf16's rounding,
// and five under the rows' own rounding to 8 bits.
//
// A stage is 256 k: 128 bytes of a 4-bit row, 256 of an 8-bit one.  Codes go
// from global memory straight into a two-stage LDS ring, exponents through
// registers (rows of them start at any byte).  Pieces past a row's last block
// read as zeros, with an exponent of 0: they add nothing.
// A persistent block sends for its next tile's first stage before it stores the
// logits of this one, straight from the accumulators, and goes on while they drain.
//
// What bounds it.  Few rows: the reading of W, 56 us for one 8-bit row of 126,464 x
// 4,096 and 54 us for a 4-bit one (275 MB, 309 MB by the counters, 5.5 TB/s; 48 and
// 46 us with the same head again and again, part of which the Infinity Cache then
// holds).  Many rows: waiting.  From registers alone the matrix cores reach 6.7
// Pflop/s with random 4-bit rows, kept busy throughout while their power takes the
// clock from 2.4 to 1.66 GHz, and 4.1 with 8-bit ones (2.0 GHz); 4,096 rows of
// 4,096 by 126,464 take 1,260 us (3.4 Pflop/s), matrix cores busy 45% of the cycles
// at 1.78 GHz, 2,048 8-bit ones 1,014 us (2.1).  Each stage's barrier waits for all
// of the next stage's loads, and the block is the only one on its CU.  8-bit rows
// bring twice the bytes for a product, through LDS too.  Of 1,308 us that the
// first took when its logits still passed through LDS, 860 were left without any
// load and LDS read, 930 with the exponents', 980 with LDS reads but no loads,
// 1,190 with loads but no LDS reads; larger tiles per wave (a third fewer LDS
// reads), exponents four stages at a time, stages of 128 k three deep and loads
// spread over the stage gained nothing.
#include <algorithm>

#include "mx.h"
#include "tile_ops.h"

namespace mdlm {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));

constexpr uint32_t kPastEnd = 0xFFFFFFF0u;  // an offset past every buffer
constexpr uint32_t kUnit4 = 0x7F7F7F7Fu;    // four exponents of 0
__device__ const uint64_t kUnit8 = 0x7F7F7F7F7F7F7F7Full;

struct MxProductArgs {
  const uint8_t* a;
  const uint8_t* a_exp;
  const uint8_t* w;
  const uint8_t* w_exp;
  int64_t n_tokens;
  int V;
  int nb;  // blocks of 32 per row
  const int32_t* row_idx;  // null: row j is j
  const int32_t* n_rows;   // null: max_rows
  int max_rows;
  float softcap;
  float inv_softcap;
  void* out;
};

__device__ __forceinline__ v8i as_operand(v4i x) {
  return __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
}
__device__ __forceinline__ v8i as_operand(v8i x) { return x; }

// c tanh(z / c).  tanh(x) = 1 - 2 / (1 + e^(2 x)), which saturates cleanly; near
// zero, where that difference cancels, its power series up to the 9th power
// (from 1/4 on the next term is under 2^-27 of it).
__device__ __forceinline__ float capped(float z, float c, float inv_c) {
  const float x = z * inv_c, x2 = x * x;
  float p = 62.f / 2835.f;
  p = fmaf(p, x2, -17.f / 315.f);
  p = fmaf(p, x2, 2.f / 15.f);
  p = fmaf(p, x2, -1.f / 3.f);
  const float e = __builtin_amdgcn_exp2f(x * 2.8853900817779268f);
  const float far = 1.f - 2.f * __builtin_amdgcn_rcpf(1.f + e);
  return fabsf(x) < 0.25f ? fmaf(z * x2, p, z) : c * far;
}

template <int AF>
struct AFrag;
template <>
struct AFrag<4> {
  typedef v4i type;
};
template <>
struct AFrag<8> {
  typedef v8i type;
};

// WA x WB waves; a wave's tile is NI blocks of 32 rows of W by NJ blocks
// of 32 rows of A.
template <int AF, int WA, int WB, int NI, int NJ, typename Out>
__global__ void __launch_bounds__(WA * WB * 64, WA * WB == 8 ? 2 : 1)
mx_product_kernel(const MxProductArgs a) {
  constexpr int kWaves = WA * WB, kThreads = 64 * kWaves;
  constexpr int kTW = 32 * NI * WA, kTA = 32 * NJ * WB;  // the tile's rows
  constexpr int kRowA = AF == 4 ? 128 : 256;             // bytes of a row in a stage
  constexpr int kBytesW = kTW * 128, kBytesA = kTA * kRowA, kStage = kBytesW + kBytesA;
  constexpr int kLoadsW = kBytesW / 1024 / kWaves;
  constexpr int kChunksA = kBytesA / 1024;
  constexpr int kLoadsA = (kChunksA + kWaves - 1) / kWaves;
  // stages whose exponents are loaded at once: one, or four where the rows are
  // few and the time is the reading of W
  constexpr int kG = NI * NJ >= 4 ? 1 : 4;
  static_assert(kLoadsW * 1024 * kWaves == kBytesW && kLoadsW % 2 == 0,
                "whole loads of W, whose swizzle alternates");
  constexpr int kE = (kTW + kTA + kThreads - 1) / kThreads;  // a thread's rows of exponents
  static_assert(2 * (kStage + 8 * kE * kThreads) <= 160 * 1024, "two stages in LDS");
  __shared__ __attribute__((aligned(1024))) char smem0[kStage];
  __shared__ __attribute__((aligned(1024))) char smem1[kStage];
  __shared__ __attribute__((aligned(16))) uint2 s_exp[2][kE * kThreads];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wa = wave % WA, wb = wave / WA;
  int n_rows = a.max_rows;
  if (a.n_rows) n_rows = max(0, min(*a.n_rows, n_rows));
  const int n_at = (n_rows + kTA - 1) / kTA;
  const int n_wt = (a.V + kTW - 1) / kTW;
  const int64_t n_tiles = (int64_t)n_at * n_wt;
  const int KT = (a.nb + 7) / 8;
  const int64_t row_w = 16 * (int64_t)a.nb, row_a = (AF == 4 ? 16 : 32) * (int64_t)a.nb;

  // fragment reads: row lane % 32 of a block, swizzled (row blocks are
  // multiples of 16 rows, which the swizzle does not see)
  const int half = lane >> 5, fx = swz_k(lane & 15);
  const int w_off = (wa * NI * 32 + (lane & 31)) * 128;
  const int a_off = kBytesW + (wb * 32 + (lane & 31)) * kRowA;

  // What a tile's loads need, of the tile whose loads are next.
  int v0, m0;
  __amdgpu_buffer_rsrc_t rw, ra;
  uint32_t w_voff[kLoadsW], a_voff[kLoadsA];
  int w_piece[2], a_piece[kLoadsA];
  const uint8_t* ep[kE];
  int e_blocks[kE], e_last[kE];
  uint2 ev[kG][kE];  // exponents of kG stages
  auto place = [&](int64_t t) __attribute__((always_inline)) {
    int wt, at;
    grouped_tile(t, n_wt, n_at, 8, 4, &wt, &at);
    v0 = wt * kTW, m0 = at * kTA;
    // loads: chunk c of 1 KiB is 8 rows of W (8 or 4 of A); lane l supplies
    // its piece of 16 bytes l, which holds the row's piece l ^ swizzle
    rw = make_rsrc(a.w + v0 * row_w, std::min<int64_t>((a.V - v0) * row_w, kPastEnd));
#pragma unroll
    for (int q = 0; q < kLoadsW; ++q) {
      const int r = 8 * (kLoadsW * wave + q) + (lane >> 3);
      const int piece = (lane & 7) ^ swz_k(r);
      if (q < 2) w_piece[q] = piece;
      w_voff[q] = (uint32_t)(r * row_w + 16 * piece);
    }
    const int64_t a_base = a.row_idx ? 0 : m0 * row_a;
    ra = make_rsrc(a.a + a_base, std::min<int64_t>(a.n_tokens * row_a - a_base, kPastEnd));
#pragma unroll
    for (int q = 0; q < kLoadsA; ++q) {
      // (with fewer chunks than waves, some are loaded twice)
      const int c = (kLoadsA * wave + q) % kChunksA;
      const int r = AF == 4 ? 8 * c + (lane >> 3) : 4 * c + (lane >> 4);
      a_piece[q] = (AF == 4 ? lane & 7 : lane & 15) ^ swz_k(r);
      const int m = m0 + r;
      int64_t row = -1;
      if (m < n_rows) row = a.row_idx ? a.row_idx[m] : m;
      a_voff[q] = row < 0 || row >= a.n_tokens
                      ? kPastEnd
                      : (uint32_t)(row * row_a - a_base + 16 * a_piece[q]);
    }
    // exponents: thread tid has rows tid, tid + kThreads of the tile, or none
#pragma unroll
    for (int x = 0; x < kE; ++x) {
      ep[x] = reinterpret_cast<const uint8_t*>(&kUnit8);
      e_blocks[x] = 0;
      const int r = x * kThreads + tid;
      if (r < kTW) {
        if (v0 + r < a.V) ep[x] = a.w_exp + (int64_t)(v0 + r) * a.nb, e_blocks[x] = a.nb;
      } else if (r < kTW + kTA && m0 + r - kTW < n_rows) {
        const int m = m0 + r - kTW;
        const int64_t row = a.row_idx ? a.row_idx[m] : m;
        if (row >= 0 && row < a.n_tokens) ep[x] = a.a_exp + row * a.nb, e_blocks[x] = a.nb;
      }
      if (a.nb < 8) {  // one stage, too short for the loads below
        uint64_t v = 0;
        for (int i = 0; i < e_blocks[x]; ++i)
          v |= (uint64_t)ep[x][i] << (8 * (8 - e_blocks[x] + i));
        ev[0][x] = make_uint2((uint32_t)v, (uint32_t)(v >> 32));
        ep[x] = reinterpret_cast<const uint8_t*>(&kUnit8);
      }
      e_last[x] = a.nb < 8 || e_blocks[x] == 0 ? 0 : e_blocks[x] - 8;
    }
  };
    // The eight exponents of stage kt, or, where the row ends before, the row's
    // last eight, moved to their places when they are written to LDS.  (Without
    // a condition, here and in the loads: a branch in the loop would let the
    // compiler carry products across the stage's barrier.)
    auto load_exp = [&](int kt, int first) __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < kE; ++x)
#pragma unroll
        for (int k = 0; k < kG; ++k) {
          if (k < first) continue;
          const u32x2_u v = *(const __attribute__((address_space(1))) u32x2_u*)(
              ep[x] + min(8 * (kt + k), e_last[x]));
          ev[k][x] = make_uint2(v.x, v.y);
        }
    };
    auto put_exp = [&](int kt, const uint2(&e)[kE]) __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < kE; ++x) {
        const int gone = min(8, max(0, 8 * kt + 8 - e_blocks[x]));  // places past the row
        const uint64_t unit = (uint64_t)kUnit4 << 32 | kUnit4;
        // (shifts by 64 in two steps)
        const uint64_t v = ((uint64_t)e[x].y << 32 | e[x].x) >> (4 * gone) >> (4 * gone);
        const uint64_t fill = unit << (32 - 4 * gone) << (32 - 4 * gone);
        const uint64_t y = v | fill;
        s_exp[kt & 1][x * kThreads + tid] = make_uint2((uint32_t)y, (uint32_t)(y >> 32));
      }
    };
    auto issue_w = [&](char* stage, int kt) __attribute__((always_inline)) {
      const int left = a.nb - 8 * kt;  // blocks from this stage on
      const int at = left > 0 ? kt : 0;
#pragma unroll
      for (int q = 0; q < kLoadsW; ++q)
        buf2l(rw, stage + (kLoadsW * wave + q) * 1024,
              w_piece[q & 1] < left ? w_voff[q] : kPastEnd, (uint32_t)(128 * at));
    };
    auto issue_a = [&](char* stage, int kt) __attribute__((always_inline)) {
      const int left = a.nb - 8 * kt;
      const int at = left > 0 ? kt : 0;
#pragma unroll
      for (int q = 0; q < kLoadsA; ++q)
        buf2l(ra, stage + kBytesW + (kLoadsA * wave + q) % kChunksA * 1024,
              a_piece[q] < (AF == 4 ? left : 2 * left) ? a_voff[q] : kPastEnd,
              (uint32_t)(kRowA * at));
    };
    typedef typename AFrag<AF>::type afrag_t;
    auto read_w = [&](const char* base, int s, v4i(&f)[NI]) __attribute__((always_inline)) {
      const int at16 = ((4 * half + s) ^ fx) * 16;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        f[i] = *reinterpret_cast<const v4i*>(base + w_off + i * 32 * 128 + at16);
    };
    auto read_a = [&](const char* base, int s, afrag_t(&f)[NJ]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const char* p = base + a_off + j * (32 * WB) * kRowA;
        if constexpr (AF == 4) {
          f[j] = *reinterpret_cast<const v4i*>(p + ((4 * half + s) ^ fx) * 16);
        } else {
          const v4i lo = *reinterpret_cast<const v4i*>(p + ((2 * s + half) ^ fx) * 16);
          const v4i hi = *reinterpret_cast<const v4i*>(p + ((8 + 2 * s + half) ^ fx) * 16);
          f[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
      }
    };
    uint32_t we[2][NI], ae[2][NJ];
    auto read_exp = [&](int kt, int buf) __attribute__((always_inline)) {
      const uint32_t* e = reinterpret_cast<const uint32_t*>(s_exp[kt & 1]) + half;
#pragma unroll
      for (int i = 0; i < NI; ++i) we[buf][i] = e[2 * ((wa * NI + i) * 32 + (lane & 31))];
#pragma unroll
      for (int j = 0; j < NJ; ++j) ae[buf][j] = e[2 * (kTW + (j * WB + wb) * 32 + (lane & 31))];
    };
    v4i wf[2][NI];
    afrag_t af[2][NJ];
#define MX_MFMAS(S, BUF)                                                                       \
  _Pragma("unroll") for (int i = 0; i < NI; ++i) _Pragma("unroll") for (int j = 0; j < NJ; ++j) \
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(                             \
          as_operand(wf[(S) & 1][i]), as_operand(af[(S) & 1][j]), acc[i][j], 4,                \
          AF == 4 ? 4 : 0, (S), (int)we[BUF][i], (S), (int)ae[BUF][j])
    constexpr int kMfma = NI * NJ, kReads = NI + NJ * (AF == 4 ? 1 : 2);
  // the first loads of a tile: exponents, stage 0 and W's part of stage 1
  auto start = [&]() __attribute__((always_inline)) {
    load_exp(0, a.nb < 8 ? 1 : 0);
    issue_w(smem0, 0);
    issue_a(smem0, 0);
    issue_w(smem1, 1);
  };
  constexpr int kPer = 16 / (int)sizeof(Out);   // entries of a lane's store
  constexpr int kStores = NI * NJ * 16 / kPer;  // of a wave's tile
  bool stored = false;  // the last tile was whole: kStores stores follow the first loads
  int64_t t = logical_block();
  if (t >= n_tiles) return;
  place(t);
  start();
  while (true) {
    f32x16 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    put_exp(0, ev[0]);
    // Stage 0's loads only: W's part of stage 1 and the last tile's stores, which
    // were issued behind them, may stay in flight (loads and stores of a wave are
    // counted off in the order of their issue).
    if (stored)
      wait_barrier<kLoadsW + kStores>();
    else
      wait_barrier<kLoadsW>();
    if constexpr (kG == 1) load_exp(1, 0);
    read_exp(0, 0);
    read_w(smem0, 0, wf[0]);
    read_a(smem0, 0, af[0]);
    // As in the bf16 head: a stage's barrier sits before its last slice, whose
    // fragments are in registers by then; behind it, the stage two ahead is
    // loaded into the one just finished and the next one's first fragments are
    // read while that slice's products run.
    auto step = [&](char* cur, char* nxt, int kt, auto which) __attribute__((always_inline)) {
      constexpr int Q = decltype(which)::value, B = Q & 1;  // kt % 4, kt % 2
#define MX_SLICE(S)                   \
  read_w(cur, (S) + 1, wf[((S) + 1) & 1]); \
  read_a(cur, (S) + 1, af[((S) + 1) & 1]); \
  MX_MFMAS(S, B);
      issue_a(nxt, kt + 1);
      MX_SLICE(0)
      MX_SLICE(1)
      MX_SLICE(2)
#pragma unroll
      for (int s = 0; s < 3; ++s) {
#pragma unroll
        for (int x = 0; x < kMfma; ++x) {
          if (s == 0 && x < kLoadsA) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (x < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
#pragma unroll
        for (int x = kMfma; x < kReads; ++x) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      sched_fence();
      put_exp(kt + 1, ev[(Q + 1) % kG]);
      wait_barrier<0>();
      constexpr int kExp = kG == 1 ? kE : Q == 2 ? kG * kE : 0;
      if constexpr (kExp > 0) load_exp(kt + 2, 0);
      issue_w(cur, kt + 2);
      read_exp(kt + 1, B ^ 1);
      read_w(nxt, 0, wf[0]);
      read_a(nxt, 0, af[0]);
      MX_MFMAS(3, B);
#pragma unroll
      for (int x = 0; x < kMfma; ++x) {
        if (x < kLoadsW + kExp) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      sched_fence();
    };
    int kt = 0;
    for (; kt + 4 <= KT; kt += 4) {
      step(smem0, smem1, kt, std::integral_constant<int, 0>());
      step(smem1, smem0, kt + 1, std::integral_constant<int, 1>());
      step(smem0, smem1, kt + 2, std::integral_constant<int, 2>());
      step(smem1, smem0, kt + 3, std::integral_constant<int, 3>());
    }
    if (kt < KT) step(smem0, smem1, kt, std::integral_constant<int, 0>());
    if (kt + 1 < KT) step(smem1, smem0, kt + 1, std::integral_constant<int, 1>());
    if (kt + 2 < KT) step(smem0, smem1, kt + 2, std::integral_constant<int, 2>());
#undef MX_SLICE
#undef MX_MFMAS
    wait_vmem();
    __syncthreads();

    // The next tile's first loads go out before this one's stores.
    const int v1 = v0 + wa * NI * 32, m1 = m0 + wb * 32 + (lane & 31);
    const bool whole = v0 + kTW <= a.V && m0 + kTA <= n_rows;
    t += gridDim.x;
    const bool more = t < n_tiles;
    if (more) {
      place(t);
      start();
    }
    sched_fence();
    asm volatile("" ::: "memory");
    // Element e of a lane's block is the entry 8 (e / 4) + 4 (lane / 32) + e % 4
    // for row lane % 32: four 32-bit logits are a store, and so are eight 16-bit
    // ones once the halves of the wave have exchanged every other four.
    auto store = [&](auto all) __attribute__((always_inline)) {
      constexpr bool kAll = decltype(all)::value;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int m = m1 + j * (32 * WB);
        if (!kAll && m >= n_rows) continue;
        const int v2 = v1 + half * kPer;
        Out* const o = reinterpret_cast<Out*>(a.out) + (int64_t)m * a.V + v2;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          f32x16& c = acc[i][j];
          if (a.softcap > 0.f)
#pragma unroll
            for (int e = 0; e < 16; ++e) c[e] = capped(c[e], a.softcap, a.inv_softcap);
#pragma unroll
          for (int e = 0; e < 16; e += kPer) {
            u32x4_a2 x;
            if constexpr (sizeof(Out) == 4) {
              x = u32x4_a2{__float_as_uint(c[e]), __float_as_uint(c[e + 1]),
                           __float_as_uint(c[e + 2]), __float_as_uint(c[e + 3])};
            } else {
              const auto lo = __builtin_amdgcn_permlane32_swap(
                  pack_bf16(c[e], c[e + 1]), pack_bf16(c[e + 4], c[e + 5]), false, false);
              const auto hi = __builtin_amdgcn_permlane32_swap(
                  pack_bf16(c[e + 2], c[e + 3]), pack_bf16(c[e + 6], c[e + 7]), false, false);
              x = u32x4_a2{lo[0], hi[0], lo[1], hi[1]};
            }
            const int at = 32 * i + 2 * e;
            if (kAll || v2 + at + kPer <= a.V) {
              *reinterpret_cast<u32x4_a2*>(o + at) = x;
            } else {
#pragma unroll
              for (int b = 0; b < kPer; ++b)
                if (v2 + at + b < a.V) {
                  if constexpr (sizeof(Out) == 4)
                    reinterpret_cast<uint32_t*>(o)[at + b] = x[b];
                  else
                    reinterpret_cast<uint16_t*>(o)[at + b] = (uint16_t)(x[b / 2] >> (16 * (b % 2)));
                }
            }
          }
        }
      }
    };
    stored = whole;
    if (whole)
      store(std::true_type());
    else
      store(std::false_type());
    if (!more) break;
  }
}

template <int AF, int WA, int WB, int NI, int NJ, typename Out>
void run(const MxProductArgs& a, int per_cu, hipStream_t stream) {
  constexpr int kTW = 32 * NI * WA, kTA = 32 * NJ * WB;
  const int64_t tiles =
      (((int64_t)a.max_rows + kTA - 1) / kTA) * (((int64_t)a.V + kTW - 1) / kTW);
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, 256 * per_cu);
  mx_product_kernel<AF, WA, WB, NI, NJ, Out><<<grid, WA * WB * 64, 0, stream>>>(a);
}

// The tile.  Up to 64 rows the time is the reading of W, and a tile has them
// all: blocks of two waves where W is small, so that every CU has some (4,096 x
// 4,096, 64 rows: 9 us, with eight waves 15), else of eight (1 row, 126,464 x
// 4,096: 56 us, 5.5 TB/s).  Beyond, 256 rows of W by 256 of A (128 of 8-bit ones)
// move the fewest bytes into LDS for a product, but a CU holds one block of them.
// 128 x 128 is taken where one round of blocks does it all, or where half of
// the large tile would be past the last row; both measured, 4,096 x 4,096 but
// for the last, in us:
//   4-bit rows    256: 12 and 28    1024: 17 and 29    2048: 28 and 32
//                 4096 (more than a round): 54 and 42    128 by 126,464: 78 and 86
//   8-bit rows    256: 16 and 25    1024: 22 and 29    2048 (more): 41 and 34
template <int AF, typename Out>
void pick(const MxProductArgs& a, hipStream_t stream) {
  const int64_t m = a.max_rows, V = a.V;
  if (m <= 32) {
    if (V <= 256 * 128)
      run<AF, 2, 1, 1, 1, Out>(a, 5, stream);
    else
      run<AF, 8, 1, 1, 1, Out>(a, 2, stream);
  } else if (m <= 64) {
    if (V <= 256 * 128)
      run<AF, 2, 1, 1, 2, Out>(a, AF == 4 ? 4 : 3, stream);
    else
      run<AF, 8, 1, 1, 2, Out>(a, 1, stream);
  } else {
    constexpr int kFit = AF == 4 ? 2 : 1;  // small tiles that a CU holds
    if (((m + 127) / 128) * ((V + 127) / 128) <= 256 * kFit || (AF == 4 && m <= 128))
      run<AF, 2, 2, 2, 2, Out>(a, kFit, stream);
    else
      run<AF, 2, 4, 4, AF == 4 ? 2 : 1, Out>(a, 1, stream);
  }
}

}  // namespace

hipError_t launch_mx_product(const uint8_t* a, const uint8_t* a_exp, int32_t a_format,
                             int64_t n_tokens, const uint8_t* w, const uint8_t* w_exp, int32_t V,
                             int32_t H, const int32_t* row_idx, const int32_t* n_rows,
                             int64_t max_rows, float softcap, int32_t out_dtype, void* logits,
                             hipStream_t stream) {
  if (max_rows == 0) return hipSuccess;
  MxProductArgs p;
  p.a = a, p.a_exp = a_exp, p.w = w, p.w_exp = w_exp;
  p.n_tokens = n_tokens, p.V = V, p.nb = (H + kMxBlock - 1) / kMxBlock;
  p.row_idx = row_idx, p.n_rows = n_rows, p.max_rows = (int)max_rows;
  p.softcap = softcap, p.inv_softcap = softcap > 0.f ? 1.f / softcap : 0.f;
  p.out = logits;
  if (out_dtype == MDLM_BF16)
    a_format == MDLM_MX_E4M3 ? pick<8, bf16_t>(p, stream) : pick<4, bf16_t>(p, stream);
  else
    a_format == MDLM_MX_E4M3 ? pick<8, float>(p, stream) : pick<4, float>(p, stream);
  return hipGetLastError();
}

}  // namespace mdlm
