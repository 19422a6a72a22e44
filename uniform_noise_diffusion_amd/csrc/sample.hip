// One token for each row of logits: temperature, top-k, top-p and min-p, drawn
// with a given uniform number.
//
// Axolotl diffusion docs, "Adapters, merging and inference" (answers by block
// diffusion); diffusiongemma card, "Finetuning notes" (uniform tokens drawn
// from the vocabulary).
//
//   weight of token i: w_i = exp((x_i - max x) / T)
//   order: falling x, equal ones by index
//   top-k keeps the order's first k; top-p of those the ones whose predecessors
//   weigh less than p of all of them together; min-p of those the ones with
//   w_i >= p
//   the token: the first one, by index, up to which the kept weights sum to
//   more than u times their sum
//
// The token is a whole number, so the weights and their sums have to be right
// far beyond what a comparison with u could tell apart by chance: weights are
// formed in fp64.  Sums over a row are fp64 sums in an order that the sizes
// determine; what is summed with atomics is summed as 64-bit integers, in units
// of about 2^-61 of the whole, whose order does not matter.  The token is looked
// for by fp64 sums alone, from the parts of the row down: a part may be lighter
// than any unit of the whole, and u = 0 asks for the first token that weighs
// anything.
//
// A row is never sorted.  What is read from memory counts (a pass costs what the
// caches cannot hold), so a row takes two passes:
//   1. the largest logit, the sum of the softmax's terms (fp32 terms, fp64 sums:
//      the token's log-probability), a rough sum of the weights and, with top-k
//      or top-p, how many logits lie in each of 4,096 steps of T / 128 downwards
//      from a first guess of the largest.  From these counts follow the steps
//      that the cut lies in, a few at most.
//   2. the logits down to the cut in a list in LDS, which is sorted, cut and drawn
//      from; or, where they do not fit, those of the cut's steps alone, and the
//      weights of what lies above them in each of eight contiguous parts of the
//      row (with top-p alone also the exact sum of all weights).  Without top-k
//      and top-p: the kept weights of the parts.  The part that holds the token
//      is divided again, down to a wave.
// Rows whose cut takes more steps than the list holds, or two cuts that far
// down, are left to a second kernel, which cuts by a histogram of exact weights,
// its bin's logits in the list, and, where they do not fit either, by the bits
// of the logits, up to three times; then they are all equal, and the cut is an
// index.
// Few rows are cut into segments, a block each, for both passes; the second
// kernel then draws from what they leave.
//
// What bounds it.  1,024 rows of 262,144 bf16 logits with min-p take 195 us, for
// two readings of 537 MB that memory gives at 6.0 TB/s; of 126,464 fp32 logits
// with top-k 165 us (as bounded), with top-p 282 us, for the vector units: every
// logit then has a term, a count and an fp64 weight; with temperature alone 186 us
// (an fp64 weight for each); greedy 97 us, in one reading.  Rows whose top-p cut
// lies too deep for the list and that min-p cuts too are the second kernel's: 790
// to 1,040 us.  One row of 126,464 takes 28 us, in four launches, for the latencies
// of the steps from one to the next.  Short rows take a block each for its fixed
// work: 4,096 rows of 1,000 bf16 78 us, with top-p 171 us.
// Every function here is inlined: what calls save of the registers was 64 KB of
// scratch memory a row (1,024 rows with top-k took 205 us and not 170).
#include <math.h>

#include <algorithm>

#include "row_ops.h"

namespace mdlm {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kSteps = 4096;  // of a row's counts
constexpr int kBins = 2048;   // of the last kernel's histogram
constexpr int kCap = 4096;    // tokens in the list
constexpr int kFew = 1024;    // and in a slot of it
constexpr int kShort = 256;   // and in a list that is searched as it lies
constexpr int kMaxSegments = 64;
constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.4426950408889634f;

typedef unsigned long long u64;

// Entries of 16 bytes.
template <typename T>
struct Vec {
  static constexpr int n = 16 / (int)sizeof(T);
};

// Vectors that a pass with fp64 work on every entry has on their way.
template <typename T>
constexpr int kFew64 = 8 / Vec<T>::n;

struct Raw16 {
  uint32_t w[4];
};

template <typename T>
__device__ __forceinline__ Raw16 load16(const T* p) {
  const u32x4_a2 v = *reinterpret_cast<const u32x4_a2*>(p);
  return Raw16{{v.x, v.y, v.z, v.w}};
}

// (A NaN counts as -inf and is never drawn; who takes the entries sees to it.)
template <typename T>
__device__ __forceinline__ void unpack(const Raw16& r, float v[Vec<T>::n]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
  }
}

// Calls f(v, i) for the entries i .. of [lo, hi) that a lane has of each vector
// of a wave, in rising order; entries past hi are -inf.  AHEAD vectors are on
// their way while as many are taken.
template <typename T, int AHEAD, typename F>
__device__ __forceinline__ void each_vec(const T* __restrict__ row, int lo, int hi, F f) {
  constexpr int N = Vec<T>::n, kStep = 64 * N * AHEAD;
  const int lane = threadIdx.x & 63;
  int base = lo;
  if (base + kStep <= hi) {
    const int last = lo + (hi - lo - kStep) / kStep * kStep;
    Raw16 cur[AHEAD], next[AHEAD];
    auto load = [&](Raw16* r, int at) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) r[k] = load16(row + at + (k * 64 + lane) * N);
    };
    load(cur, base);
    for (; base <= last; base += kStep) {
      // (the last ones once more, rather than a condition)
      load(next, min(base + kStep, last));
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        float v[N];
        unpack<T>(cur[k], v);
        f(v, base + (k * 64 + lane) * N);
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) cur[k] = next[k];
    }
  }
  if (base < hi) {
    Raw16 r[AHEAD] = {};
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = base + (k * 64 + lane) * N;
      if (i + N <= hi) r[k] = load16(row + i);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = base + (k * 64 + lane) * N;
      if (base + k * 64 * N >= hi) break;
      float v[N];
      unpack<T>(r[k], v);
      if (i + N > hi) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = i + e < hi ? (float)row[i + e] : -kInf;
      }
      f(v, i);
    }
  }
}

// Floats in their order, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ (((int32_t)key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// 2^(-i / 256), i in [0, 256): the power series of e^f up to its 13th term, f
// taken within ln(2) / 2 of zero, which leaves 5e-18.
__device__ __forceinline__ double table_entry(int i) {
  const double f = (double)(i <= 128 ? -i : 256 - i) * (0.693147180559945309417 / 256.0);
  double p = 1.0 / 6227020800.0;
  p = fma(p, f, 1.0 / 479001600.0);
  p = fma(p, f, 1.0 / 39916800.0);
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  return i <= 128 ? p : 0.5 * p;
}

// What a row's caller asks for.
struct Ask {
  bool greedy, by_k, by_p;
  int k;
  float p, temp, u;
  float per_f;   // log2(e) / T, at most 1e30
  double min_w;  // min-p
  __device__ __forceinline__ Ask(const SampleArgs& a, int64_t j) {
    temp = a.temperature ? a.temperature[j] : 1.f;
    greedy = !(temp > 0.f);
    k = a.top_k ? a.top_k[j] : 0;
    by_k = !greedy && k > 0 && k < a.V;
    p = a.top_p ? a.top_p[j] : 1.f;
    by_p = !greedy && p < 1.f;
    const float m = a.min_p ? a.min_p[j] : 0.f;
    min_w = m > 0.f ? fmin((double)m, 1.0) : 0.0;
    u = fminf(fmaxf(a.u[j], 0.f), 0x1.fffffep-1f);
    per_f = greedy ? 0.f : fminf(kLog2e / temp, 1e30f);
  }
  // u's place is under what units of the whole can tell apart
  __device__ __forceinline__ bool faint() const { return u < 0x1p-30f; }
  // u's place in a sum of units
  __device__ __forceinline__ u64 place(u64 sum) const { return (u64)((double)u * (double)sum); }
  // where top-p's tokens end: the first ones that reach this sum
  __device__ __forceinline__ u64 goal(u64 all) const {
    return min(all, (u64)fmax(1.0, ceil((double)p * (double)all)));
  }
};

// What the passes know of a row.
struct Row {
  float top;      // the largest logit
  double per;     // 256 log2(e) / T
  double far;     // from this distance on a weight is 2^-996
  int shift;      // a weight of 1 is 2^shift units
  double most;    // and none is more units than this
  double min_w;   // min-p
  float below;    // logits under this one are certainly not kept
  uint32_t key;   // the cut: kept are larger keys, and this one up to `index`
  int index;
  bool ties_only; // weights are 1 where the key is `key`, else 0
  const double* table;
  __device__ __forceinline__ Row(const Ask& ask, float top_, int V, const double* table_)
      : top(top_), shift(0), most(0x1p62), min_w(ask.min_w), below(-kInf), key(0), index(V),
        ties_only(false), table(table_) {
    // (T = inf: finite logits weigh 1, and -inf nothing all the same)
    per = ask.greedy ? 1.0 : 256.0 * 1.4426950408889634074 / fmin((double)ask.temp, 1e300);
    far = 256.0 * 996.0 / per;
    if (min_w > 0.0 && !ask.greedy) {
      // T ln(min-p) under the largest logit, and a little
      const double d = -log(min_w) * (double)ask.temp;
      const double low = (double)top - d - (1e-5 * (d + fabs((double)top)) + 1e-30);
      if (low > -0x1.fffffep127) below = (float)low;
    }
  }
  // `sum`: the weights that are summed as units, or a bound of them; they come to
  // 2^60 to 2^61 units at most
  __device__ __forceinline__ void scale(double sum) { shift = 60 - ilogb(fmax(sum, 1.0)); }
  // Units for a draw at t, far under the row's weight: t is 2^40 to 2^41 of them,
  // or kLeast's is the least unit, and a weight beyond t counts for 2^45 (of a
  // list's 4,096 entries the sum is below 2^57).  The units that are to be passed.
  __device__ __forceinline__ u64 refine(double t) {
    shift = t > 0.0 ? min(990, 40 - ilogb(t)) : 990;
    most = 0x1p45;
    return (u64)ldexp(t, shift) + 1;
  }
};

// A weight times 2^shift: 2^(-t / 256), t = (top - x) per, as the table's entry
// for t's nearest whole number n and the power series of 2^(r / 256), r = n - t
// (4e-17 remain after the 4th term).  n is formed by adding 1.5 * 2^52 and taken
// from the sum's low bits, and the power of two is added to the entry's
// exponent: rounding, conversion and ldexp would each take four times as long.
// It never becomes zero, 2^-996 being the least; where a token is looked for, what
// is under kLeast counts as zero.
constexpr double kLeast = 0x1p-990;
__device__ __forceinline__ double scaled_weight(const Row& r, float x, int shift) {
  constexpr double kMagic = 0x1.8p52, c = 0.693147180559945309417 / 256.0;
  const double d = fmin((double)r.top - (double)x, r.far);
  const double m = fma(d, r.per, kMagic);
  const double z = fma(-d, r.per, m - kMagic);
  const int i = (int)(uint32_t)__double_as_longlong(m);
  double p = fma(z, c * c * c * c / 24.0, c * c * c / 6.0);
  p = fma(p, z, c * c / 2.0);
  p = fma(p, z, c);
  p = fma(p, z, 1.0);
  const uint64_t e = (uint64_t)__double_as_longlong(r.table[i & 255]);
  const uint32_t hi = (uint32_t)(e >> 32) + ((uint32_t)shift << 20) - ((uint32_t)(i & ~255) << 12);
  return p * __longlong_as_double((long long)((uint64_t)hi << 32 | (uint32_t)e));
}
__device__ __forceinline__ double weight_of(const Row& r, float x) {
  return scaled_weight(r, x, 0);
}
__device__ __forceinline__ u64 to_units(double s) {  // s below 2^62
  const uint32_t hi = (uint32_t)(s * 0x1p-32);
  const uint32_t lo = (uint32_t)fma((double)hi, -0x1p32, s);
  return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 units_of(const Row& r, float x) {
  return to_units(fmin(scaled_weight(r, x, r.shift), r.most));
}
__device__ __forceinline__ bool within_cut(const Row& r, float x, int i) {
  const uint32_t k = key_of(x);
  return k > r.key || (k == r.key && i <= r.index);
}
__device__ __forceinline__ u64 kept_units(const Row& r, float x, int i) {
  if (!within_cut(r, x, i)) return 0;
  return r.min_w > 0.0 && weight_of(r, x) < r.min_w ? 0 : units_of(r, x);
}
__device__ __forceinline__ double kept_weight(const Row& r, float x, int i) {
  if (r.ties_only) return key_of(x) == r.key ? 1.0 : 0.0;
  if (!within_cut(r, x, i)) return 0.0;
  const double w = weight_of(r, x);
  return w < kLeast || w < r.min_w ? 0.0 : w;
}

template <typename X>
__device__ __forceinline__ X scan64(X x) {  // inclusive, over the wave
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const X y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}
template <typename X>
__device__ __forceinline__ X sum_of(X x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ float wave_most(float x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
  return x;
}

// What pass 1 needs of LDS, and what the rest does.
struct Scan {
  uint32_t count[kSteps];
  float top[kWaves], rough[kWaves];
  double whole[kWaves];
  int at[kWaves];
  uint32_t n[kWaves];
  u64 pick[2];
};
struct Shared {
  union {
    Scan scan;
    u64 list[kCap];
  };
  double table[256];
  u64 slot[kThreads];         // units of the list's entries by slot
  uint32_t slot_n[kThreads];  // how many they are
  __attribute__((aligned(16))) u64 few[kFew];  // a slot's entries
  u64 part[kWaves], part2[kWaves];
  double weigh[kWaves];
  float low[kWaves], high[kWaves];
  u64 pick[2];
  uint32_t n_list, n_few;
};

__device__ __forceinline__ void fill_table(Shared& s) {
  if (threadIdx.x < 256) s.table[threadIdx.x] = table_entry(threadIdx.x);
}

// n entries (room for the next power of two) in rising order.
__device__ __forceinline__ void sort_entries(u64* list, int n) {
  int size = 64;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) list[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int p = threadIdx.x; p < size / 2; p += kThreads) {
        const int i = 2 * p - (p & (j - 1)), l = i + j;
        const u64 a = list[i], b = list[l];
        if ((a > b) == ((i & k) == 0)) list[i] = b, list[l] = a;
      }
      __syncthreads();
    }
}
// Sums of x over the threads before this one; the block's own is in *all.
__device__ __forceinline__ u64 block_scan(u64 x, u64* all, Shared& s) {
  const u64 upto = scan64(x);
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.part2[wave] = upto;
  __syncthreads();
  u64 before = upto - x, sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const u64 p = s.part2[w];
    if (w < wave) before += p;
    sum += p;
  }
  *all = sum;
  return before;
}
__device__ __forceinline__ u64 block_sum(u64 x, Shared& s) {
  x = sum_of(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.part2[threadIdx.x >> 6] = x;
  __syncthreads();
  u64 sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += s.part2[w];
  return sum;
}
// The waves' sums of x into s.weigh; their total.
__device__ __forceinline__ double weigh_waves(double x, Shared& s) {
  x = sum_of(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s.weigh[threadIdx.x >> 6] = x;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) sum += s.weigh[w];
  return sum;
}

// An entry: a logit's key, falling, and its index.
__device__ __forceinline__ u64 entry_of(float x, int i) {
  return (u64)~key_of(x) << 32 | (uint32_t)i;
}
__device__ __forceinline__ float logit_of(u64 entry) { return value_of(~(uint32_t)(entry >> 32)); }

// A wave's contiguous share of [lo, hi).
template <typename T>
__device__ __forceinline__ int share_size(int lo, int hi) {
  constexpr int kVec = 64 * Vec<T>::n;
  return ((hi - lo + kWaves * kVec - 1) / (kWaves * kVec)) * kVec;
}
template <typename T>
__device__ __forceinline__ void share(int wave, int lo, int hi, int* from, int* to) {
  const int per = share_size<T>(lo, hi);
  *from = min(hi, lo + wave * per);
  *to = min(hi, *from + per);
}

template <int N>
__device__ __forceinline__ float most_of(const float* v) {
  float most = v[0];
#pragma unroll
  for (int k = 1; k < N; ++k) most = fmaxf(most, v[k]);
  return most;
}

// ---- pass 1 --------------------------------------------------------------
// Steps of T / 128 downwards from 8 T over a first guess of the largest logit.
struct Steps {
  float from, per_t;  // the guess plus 8 T; steps per logit
  __device__ __forceinline__ Steps(float guess, float temp)
      : from(fmaf(8.f, temp, guess > -kInf && guess < kInf ? guess : 0.f)),
        per_t(fminf(128.f / temp, 1e30f)) {}
  __device__ __forceinline__ int of(float x) const {
    return (int)fmaxf(0.f, fminf((from - x) * per_t, (float)(kSteps - 1)));
  }
  // The least float of a step up to `last`: inf if there is none.
  __device__ float edge(int last) const {
    if (last < 0) return kInf;
    if (last >= kSteps - 1) return -kInf;
    uint32_t out = key_of(-kInf), in = key_of(kInf);  // of(in) <= last < of(out)
    while (in - out > 1) {
      const uint32_t mid = out + (in - out) / 2;
      if (of(value_of(mid)) <= last)
        in = mid;
      else
        out = mid;
    }
    return value_of(in);
  }
};

// The largest of a row's first logits: the same for every wave.
template <typename T>
__device__ __forceinline__ float guess_of(const T* row, int V) {
  constexpr int N = Vec<T>::n;
  const int i = (threadIdx.x & 63) * N;
  float v[N];
  float most = -kInf;
  if (i + N <= V) {
    unpack<T>(load16(row + i), v);
    most = most_of<N>(v);
  } else {
    for (int k = i; k < V; ++k) most = fmaxf(most, (float)row[k]);
  }
  return wave_most(most);
}

// What pass 1 finds in a part of a row.
struct Found {
  float top;     // the largest logit
  float rough;   // with top-p alone, the sum of the weights relative to it
  double whole;  // sum of e^(x - top)
  int at;        // a vector with the first of the largest logits
};

// One lane's share of a wave's part.  A term is one multiply-add and one 2^x (a
// NaN's, also of an infinite distance over an infinite T, becomes 0 by the
// maximum).  A vector's terms are added in fp32, without those of the largest
// logit so far, which are 1, and counted: next to a 1 what a decided row's
// log-probability is made of would be lost.  The multiply-add takes the largest
// logit times log2(e) as fp32 rounds it; what that is off by, which grows with the
// logits and not with their distances, is one power of two for all terms, and is
// taken back where their sum is added.
template <typename T, bool COUNT, bool ROUGH>
__device__ __forceinline__ Found scan_part(const T* row, int lo, int hi, const Ask& ask,
                                           const Steps& steps, Scan& s) {
  constexpr int N = Vec<T>::n;
  Found f = {-kInf, 0.f, 0.0, 0};
  uint32_t ones = 0;
  // log2(e) and the largest logit times it (`back`: the power that undoes the
  // product's rounding); the same over T.  From 2^30 on, no other logit is nearer
  // than 64, and the term is 0 next to a 1; over T, near the end of float's range,
  // perhaps wrongly: the rough sum is then found too small.
  double back = 1.0;
  float mul = kLog2e, ref = 0.f, mul_t = ask.per_f, ref_t = 0.f;
  each_vec<T, 4>(row, lo, hi, [&](const float* v, int i) __attribute__((always_inline)) {
    const float most = most_of<N>(v);
    bool same = false;
    if (most >= f.top && most > -kInf) {
      same = true;
      if (most > f.top) {
        const float d = f.top - most;
        f.whole = (f.whole + (double)ones) * (double)__builtin_amdgcn_exp2f(d * kLog2e);
        if (ROUGH) f.rough *= fmaxf(0.f, __builtin_amdgcn_exp2f(d * ask.per_f));
        ones = 0;
        f.top = most;
        f.at = i;
        const bool near = fabsf(most) < 0x1p30f, near_t = fabsf(most * ask.per_f) < 1e37f;
        mul = near ? kLog2e : 0.f, ref = near ? most * kLog2e : 1000.f;
        back = near ? (double)__builtin_amdgcn_exp2f(-fmaf(most, kLog2e, -ref)) : 1.0;
        mul_t = near_t ? ask.per_f : 0.f, ref_t = near_t ? most * ask.per_f : 1000.f;
      }
    }
    float terms = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float e = fmaxf(0.f, __builtin_amdgcn_exp2f(fmaf(v[k], mul, -ref)));
      if (same && v[k] == f.top) e = 0.f, ++ones;
      terms += e;
      if (ROUGH) f.rough += fmaxf(0.f, __builtin_amdgcn_exp2f(fmaf(v[k], mul_t, -ref_t)));
      if (COUNT && i + k < hi) atomicAdd(&s.count[steps.of(v[k])], 1u);
    }
    f.whole = fma((double)terms, back, f.whole);
  });
  f.whole += (double)ones;
  return f;
}

// A part's findings, its sums relative to `top`.
__device__ __forceinline__ Found rebased(Found f, float top, float per_f) {
  const float d = f.top == -kInf ? -kInf : f.top == top ? 0.f : f.top - top;
  f.whole = d == -kInf ? 0.0 : f.whole * (double)__builtin_amdgcn_exp2f(d * kLog2e);
  f.rough = d == -kInf ? 0.f : f.rough * __builtin_amdgcn_exp2f(d * per_f);
  f.at = f.top == top ? f.at : 0x7FFFFFFF;
  f.top = top;
  return f;
}
// The lanes' findings as one, in every lane.
__device__ __forceinline__ Found join_lanes(Found f, float per_f) {
  f = rebased(f, wave_most(f.top), per_f);
  f.whole = sum_of(f.whole);
  f.rough = sum_of(f.rough);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) f.at = min(f.at, __shfl_xor(f.at, d, 64));
  return f;
}
// The block's, in every thread.
__device__ __forceinline__ Found join_block(Found f, float per_f, Scan& s) {
  f = join_lanes(f, per_f);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane == 0) {
    s.top[wave] = f.top, s.rough[wave] = f.rough, s.whole[wave] = f.whole, s.at[wave] = f.at;
  }
  __syncthreads();
  f = Found{-kInf, 0.f, 0.0, 0};
  if (lane < kWaves) f = Found{s.top[lane], s.rough[lane], s.whole[lane], s.at[lane]};
  return join_lanes(f, per_f);
}

// Pass 1 over [lo, hi) by the block; s.count holds its counts afterwards.
template <typename T>
__device__ __forceinline__ Found first_pass(const T* row, int lo, int hi, const Ask& ask,
                                            const Steps& steps, Scan& s) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int from, to;
  share<T>(wave, lo, hi, &from, &to);
  Found f;
  if (ask.by_k || ask.by_p) {
    for (int b = threadIdx.x; b < kSteps; b += kThreads) s.count[b] = 0;
    __syncthreads();
    f = ask.by_k ? scan_part<T, true, false>(row, from, to, ask, steps, s)
                 : scan_part<T, true, true>(row, from, to, ask, steps, s);
  } else {
    f = scan_part<T, false, false>(row, from, to, ask, steps, s);
  }
  return join_block(f, ask.per_f, s);
}

// The steps that the list takes: those of the cut, or all of them down to it
// (first = 0).  last < 0: the list cannot hold them.
struct Bracket {
  int first, last;
  int before;  // logits in the steps before `first`
};

// With top-k, the cut's step is the one that has the k-th token.  With top-p
// alone it is the first one behind which at most 1 - p of the whole weight lies:
// taking every logit for its step's upper edge, and for its lower one, gives the
// last and the first step that it can be.
__device__ __forceinline__ Bracket bracket_of(const Ask& ask, const Steps& steps, const Found& f, Scan& s) {
  constexpr int kPer = kSteps / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // thread t has the steps kSteps - 1 - (t kPer + k): sums from the far end
  const float inv = 1.f / steps.per_t;
  auto upper = [&](int b, uint32_t n) __attribute__((always_inline)) {
    const float x = fmaf(-(float)b, inv, steps.from);
    return n ? (float)n * __builtin_amdgcn_exp2f(fminf(0.f, x - f.top) * ask.per_f) : 0.f;
  };
  uint32_t n[kPer], c = 0;
  float w[kPer], t = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = kSteps - 1 - (tid * kPer + k);
    n[k] = s.count[b];
    w[k] = upper(b, n[k]);
    c += n[k], t += w[k];
  }
  const float far = upper(kSteps - 1, s.count[kSteps - 1]);  // has no lower edge
  uint32_t cs = c;
  float ts = t;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(cs, d, 64);
    const float z = __shfl_up(ts, d, 64);
    if (lane >= d) cs += y, ts += z;
  }
  __syncthreads();
  if (lane == 63) s.n[wave] = cs, s.rough[wave] = ts;
  if (tid == 0) s.pick[0] = s.pick[1] = 0;
  __syncthreads();
  uint32_t all = 0;
  cs -= c, ts -= t;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) {
    all += s.n[v];
    if (v < wave) cs += s.n[v], ts += s.rough[v];
  }
  // (the rough sum, and these, are good to 1e-5 and what the exponents' rounding,
  // |x| / T in units of 2^-24, makes of them)
  const float limit = (1.f - ask.p) * f.rough;
  const float slack = 1e-4f + fabsf(f.top) * ask.per_f * 0x1p-21f;
  const float under = limit * (1.f - slack), over = limit * (1.f + slack);
  const float shrink = __builtin_amdgcn_exp2f(-ask.per_f * inv);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    // behind this step lie cs logits, which weigh ts at most
    const int b = kSteps - 1 - (tid * kPer + k);
    const uint32_t upto = all - cs, before = upto - n[k];
    const float low = (ts - far) * shrink, low_before = (ts + w[k] - far) * shrink;
    // (the first step has no upper edge, and whatever is left)
    const bool last = ask.by_k ? (int)before < ask.k && ask.k <= (int)upto
                               : ts <= under && (b == 0 || !(ts + w[k] <= under));
    const bool first = ask.by_k ? last : low <= over && (b == 0 || !(low_before <= over));
    if (first) s.pick[0] = (u64)(b + 1) << 32 | before;
    if (last) s.pick[1] = (u64)(b + 1) << 32 | upto;
    cs += n[k], ts += w[k];
  }
  __syncthreads();
  // (Scalars, and known as such: kept in vector registers, what follows from them
  // was once selected on another comparison's result.)
  const u64 p0 = s.pick[0], p1 = s.pick[1];
  const uint32_t upto = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p1);
  Bracket r = {__builtin_amdgcn_readfirstlane((int)(p0 >> 32)) - 1,
               __builtin_amdgcn_readfirstlane((int)(p1 >> 32)) - 1,
               __builtin_amdgcn_readfirstlane((int)(uint32_t)p0)};
  __syncthreads();
  // (logits near the ends of float's range can spoil the rough sum, which is 1 at
  // least)
  if (!ask.by_k && !(f.rough > 0.9f))
    r.last = -1;
  else if (upto <= kCap)
    r.first = r.before = 0;
  else if (r.first < 0 || upto - (uint32_t)r.before > kCap || (ask.by_k && ask.by_p) ||
           ask.min_w > 0.0)
    r.last = -1;
  return r;
}

// ---- pass 2 --------------------------------------------------------------
// Of the logits of a wave's share of [lo, hi), one lane's: calls put(x, i) for
// those in the bracket's steps, and adds up the weights of those above them
// (ABOVE: there are any) and, ALL, of all of them.
template <typename T, bool ALL, bool ABOVE, typename Put>
__device__ __forceinline__ void second_pass(const T* row, const Row& r, int lo, int hi,
                                            const Steps& steps, const Bracket& in, double* above,
                                            double* all, Put put) {
  constexpr int N = Vec<T>::n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int from, to;
  share<T>(wave, lo, hi, &from, &to);
  const float least = steps.edge(in.last), over = steps.edge(in.first - 1);
  double sum = 0.0, upper = 0.0;
  each_vec<T, ALL ? kFew64<T> : 4>(row, from, to, [&](const float* v, int i)
                                   __attribute__((always_inline)) {
    if (ALL) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const double w = weight_of(r, v[k]);
        sum += w;
        if (ABOVE) upper += v[k] >= over ? w : 0.0;
      }
    }
    if (most_of<N>(v) < least) return;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (ABOVE && v[k] >= over) {
        if (!ALL) upper += weight_of(r, v[k]);
      } else if (v[k] >= least && i + k < to) {
        put(v[k], i + k);
      }
    }
  });
  *above = upper;
  *all = sum;
}

// Without cuts: one lane's weights of a wave's share that min-p keeps.
template <typename T>
__device__ __forceinline__ double weigh(const T* row, const Row& r, int lo, int hi) {
  constexpr int N = Vec<T>::n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int from, to;
  share<T>(wave, lo, hi, &from, &to);
  double sum = 0.0;
  if (r.min_w > 0.0) {
    each_vec<T, 4>(row, from, to, [&](const float* v, int) __attribute__((always_inline)) {
      if (most_of<N>(v) < r.below) return;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (v[k] >= r.below) {
          const double w = weight_of(r, v[k]);
          sum += w >= r.min_w ? w : 0.0;
        }
    });
  } else {
    each_vec<T, kFew64<T>>(row, from, to, [&](const float* v, int)
                           __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < N; ++k) sum += weight_of(r, v[k]);
    });
  }
  return sum;
}

// The list's entries are not sorted as a whole either: they are dealt to 512
// slots that follow the order, the slot that holds what is looked for is found
// from the slots' sums, and its entries alone are sorted (all of the list's, if
// they are too many).
//
// Finds the entry where the running sum of units(entry), in order, reaches
// `goal`: order_of(entry) rises in that order, slot_of(entry) in [0, 512) does not
// fall.  False if the sum does not reach it.
template <typename Slot, typename Order, typename Units>
__device__ __forceinline__ bool find_entry(Shared& s, int n, u64 goal, Slot slot_of, Order order_of, Units units,
                           u64* entry) {
  const int tid = threadIdx.x;
  s.slot[tid] = 0, s.slot_n[tid] = 0;
  if (tid == 0) s.n_few = 0, s.pick[0] = ~0ull;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const u64 e = s.list[i];
    const int k = slot_of(e);
    atomicAdd(&s.slot[k], units(e));
    atomicAdd(&s.slot_n[k], 1u);
  }
  __syncthreads();
  const u64 mine = s.slot[tid];
  u64 all, before = block_scan(mine, &all, s);
  if (before < goal && goal <= before + mine) s.pick[0] = (u64)tid, s.pick[1] = before;
  __syncthreads();
  const u64 hit = s.pick[0];
  u64 sum = s.pick[1];
  __syncthreads();
  if (hit == ~0ull) return false;
  const int slot = (int)hit;
  u64* found = s.few;
  int m = (int)s.slot_n[slot];
  if (m <= kFew) {
    for (int i = tid; i < n; i += kThreads) {
      const u64 e = s.list[i];
      if (slot_of(e) == slot) s.few[atomicAdd(&s.n_few, 1u)] = order_of(e);
    }
  } else {
    found = s.list, m = n, sum = 0;
    for (int i = tid; i < n; i += kThreads) s.list[i] = order_of(s.list[i]);
  }
  __syncthreads();
  sort_entries(found, m);
  const int each = (m + kThreads - 1) / kThreads;
  const int from = min(m, tid * each), to = min(m, from + each);
  u64 some = 0;
  for (int i = from; i < to; ++i) some += units(order_of(found[i]));
  before = sum + block_scan(some, &all, s);
  for (int i = from; i < to; ++i) {
    const u64 e = order_of(found[i]), w = units(e);
    if (before < goal && goal <= before + w) s.pick[0] = e;
    before += w;
  }
  __syncthreads();
  *entry = s.pick[0];
  if (found == s.list) {  // (order_of undoes itself)
    for (int i = tid; i < n; i += kThreads) s.list[i] = order_of(s.list[i]);
  }
  __syncthreads();
  return true;
}

// Slots by value: a list's finite logits from the largest to the smallest.
struct ValueSlots {
  float most, per_slot;
  __device__ ValueSlots(int n, Shared& s) {
    float lo = kInf, hi = -kInf;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float x = logit_of(s.list[i]);
      hi = fmaxf(hi, x);
      if (x > -kInf) lo = fminf(lo, x);
    }
    hi = wave_most(hi), lo = -wave_most(-lo);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.high[threadIdx.x >> 6] = hi, s.low[threadIdx.x >> 6] = lo;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) hi = fmaxf(hi, s.high[w]), lo = fminf(lo, s.low[w]);
    most = hi;
    per_slot = hi > lo ? (float)(kThreads - 1) / (hi - lo) : 0.f;
  }
  __device__ __forceinline__ int operator()(u64 e) const {
    return (int)fminf((most - logit_of(e)) * per_slot, (float)(kThreads - 1));
  }
};

// The cut among the list's n entries: where they have `goal` units (by_count:
// tokens).  Sets r.key, r.index and r.below; false if they have fewer.
__device__ __forceinline__ bool cut_list(Row& r, int n, bool by_count, u64 goal, Shared& s) {
  const ValueSlots slots(n, s);
  u64 e;
  const auto same = [](u64 x) { return x; };
  if (!find_entry(s, n, goal, slots, same,
                  [&](u64 x) { return by_count ? 1 : units_of(r, logit_of(x)); }, &e))
    return false;
  r.key = ~(uint32_t)(e >> 32);
  r.index = (int)(uint32_t)e;
  r.below = fmaxf(r.below, value_of(r.key));
  return true;
}
// The same with `above` of the whole row's weight lying above the list, for a
// share p of `all` (or, with top-k, `before` of its tokens).
__device__ __forceinline__ bool cut_within(const Ask& ask, Row& r, int n, int before, double above, double all,
                           Shared& s) {
  if (ask.by_k) return cut_list(r, n, true, (u64)(ask.k - before), s);
  const double need = ldexp((double)ask.p * all - above, r.shift);
  return need > 0.0 && need < 0x1p62 && cut_list(r, n, false, (u64)fmax(1.0, ceil(need)), s);
}
// Units of the list's kept entries.
__device__ __forceinline__ u64 entry_units(const Row& r, u64 e) {
  const float x = logit_of(e);
  return x >= r.below ? kept_units(r, x, (int)(uint32_t)e) : 0;
}
__device__ __forceinline__ u64 list_sum(const Row& r, int n, Shared& s) {
  u64 sum = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += entry_units(r, s.list[i]);
  return block_sum(sum, s);
}

// draw_from_list() for at most kShort entries: an entry's place in the order, what
// lies before it and, of what is kept, what lies before it by index are counted by
// looking at every other one, each entry by as many lanes as there are.  (One row
// of 126,464, top-k and top-p: 32 us then, and 45 where slots are searched, with two
// passes over the list and a sort to each cut.  Looked at in pairs, longer lists
// cost more: up to 512 entries, 256 rows' top-p would take 104 us instead of 75.)
__device__ __forceinline__ int draw_from_few(const Ask& ask, Row r, int n, double all, Shared& s) {
  static_assert(kShort <= kThreads && 2 * kShort <= kFew, "a lane to an entry");
  ulonglong2* const pair = reinterpret_cast<ulonglong2*>(s.few);
  const int lanes = n <= kThreads / 4 ? 4 : n <= kThreads / 2 ? 2 : 1;
  const int i = threadIdx.x / lanes, q = threadIdx.x & (lanes - 1);
  auto joined = [&](auto x) __attribute__((always_inline)) {
    if (lanes > 1) x += __shfl_xor(x, 1, 64);
    if (lanes > 2) x += __shfl_xor(x, 2, 64);
    return x;
  };
  const bool mine = i < n;
  __syncthreads();
  const u64 e = mine ? s.list[i] : ~0ull;
  const u64 units = mine ? units_of(r, logit_of(e)) : 0;
  const double w = mine ? weight_of(r, logit_of(e)) : 0.0;
  if (mine && q == 0) pair[i] = make_ulonglong2(e, units);
  __syncthreads();
  int rank = 0;
  u64 before = 0;
#pragma unroll 8
  for (int k = q; k < n; k += lanes) {
    const ulonglong2 p = pair[k];
    rank += p.x < e ? 1 : 0;
    before += p.x < e ? p.y : 0;
  }
  rank = joined(rank), before = joined(before);
  bool kept = mine && !(ask.by_k && rank >= ask.k);
  if (ask.by_p) {
    const u64 sum = block_sum(kept && q == 0 ? units : 0, s);
    u64 goal = 1;
    if (ask.by_k) {
      goal = ask.goal(sum);
    } else if (ask.p > 0.f) {
      const double need = ldexp((double)ask.p * all, r.shift);
      if (!(need > 0.0 && need < 0x1p62)) return -1;
      goal = (u64)fmax(1.0, ceil(need));
    }
    if (goal == 0 || sum < goal) return -1;
    kept = kept && before < goal;
  }
  kept = kept && !(w < r.min_w);
  u64 left = kept ? units : 0;
  const u64 sum = block_sum(q == 0 ? left : 0, s);
  if (sum == 0) return -1;
  u64 goal = ask.place(sum) + 1;
  if (ask.faint()) {  // (as in draw_from_list())
    goal = r.refine((double)ask.u * ldexp((double)sum, -r.shift));
    left = kept ? units_of(r, logit_of(e)) : 0;
  }
  if (mine && q == 0) pair[i].y = left;
  __syncthreads();
  before = 0;
#pragma unroll 8
  for (int k = q; k < n; k += lanes) {
    const ulonglong2 p = pair[k];
    before += (uint32_t)p.x < (uint32_t)e ? p.y : 0;
  }
  before = joined(before);
  if (mine && before < goal && goal <= before + left) s.pick[0] = (uint32_t)e;
  __syncthreads();
  return (int)s.pick[0];
}

// The token that the list's n entries give, all tokens down to the cut being
// among them: cut, then drawn by index.  `all`: the whole row's weight (top-p
// alone).  -1 if the cut is not among them.
__device__ __forceinline__ int draw_from_list(const Ask& ask, Row r, int n, double all, int V, Shared& s) {
  if (n <= kShort) return draw_from_few(ask, r, n, all, s);
  const double min_w = r.min_w;
  const float below = r.below;
  r.min_w = 0.0, r.below = -kInf;  // (the cuts' weights are those of all tokens)
  if (ask.by_k && n > ask.k && !cut_list(r, n, true, (u64)ask.k, s)) return -1;
  if (ask.by_p && !(ask.by_k ? cut_list(r, n, false, ask.goal(list_sum(r, n, s)), s)
                             : ask.p > 0.f ? cut_within(ask, r, n, 0, 0.0, all, s)
                                           : cut_list(r, n, false, 1, s)))
    return -1;
  r.min_w = min_w, r.below = fmaxf(r.below, below);
  const u64 sum = list_sum(r, n, s);
  if (sum == 0) return -1;
  // (units of the whole are too coarse for a draw among its lightest tokens)
  const u64 goal = ask.faint() ? r.refine((double)ask.u * ldexp((double)sum, -r.shift))
                               : ask.place(sum) + 1;
  u64 e;
  const float per_slot = (float)kThreads / (float)V;
  find_entry(
      s, n, goal,
      [&](u64 x) { return min(kThreads - 1, (int)((float)(uint32_t)x * per_slot)); },
      [](u64 x) { return x << 32 | x >> 32; }, [&](u64 x) { return entry_units(r, x); }, &e);
  return (int)(uint32_t)e;
}

// One lane's sum of f(x, i) over the logits of a wave's share of [lo, hi) that r
// may keep.
template <typename X, typename T, typename F>
__device__ __forceinline__ X share_sum(const T* row, const Row& r, int lo, int hi, F f) {
  constexpr int N = Vec<T>::n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int from, to;
  share<T>(wave, lo, hi, &from, &to);
  X sum = 0;
  each_vec<T, kFew64<T>>(row, from, to, [&](const float* v, int i)
                         __attribute__((always_inline)) {
    if (most_of<N>(v) < r.below) return;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (v[k] >= r.below) sum += f(v[k], i + k);
  });
  return sum;
}
// The waves' kept weights over [lo, hi), into s.weigh; their total.
template <typename T>
__device__ __forceinline__ double part_sums(const T* row, const Row& r, int lo, int hi, Shared& s) {
  return weigh_waves(share_sum<double>(row, r, lo, hi,
                                       [&](float x, int i) __attribute__((always_inline)) {
                                         return kept_weight(r, x, i);
                                       }),
                     s);
}

// The largest number below x > 0.
__device__ __forceinline__ double just_below(double x) {
  return __longlong_as_double(__double_as_longlong(x) - 1);
}

// Where *t falls among `n` parts of these weights, *before lying before them: the
// first one up to which all of it sums to more than *t, and in *before what lies
// before that part.  -1: none weighs anything.  Sums taken in different orders may
// leave *t no less than the whole; it is then taken just below.  (Sums start at the
// row's first token all the way down: were what lies before taken off t, a draw on
// the border between two equal tokens would fall to the least one between them.)
__device__ __forceinline__ int part_at(const double* weight, int n, double* t, double* before) {
  double upto = *before;
  for (int k = 0; k < n; ++k) upto += weight[k];
  *t = fmin(*t, just_below(upto));
  int part = -1;
  upto = *before;
  for (int k = 0; k < n && (part < 0 || !(upto > *t)); ++k) {
    if (!(weight[k] > 0.0)) continue;
    part = k, *before = upto, upto += weight[k];
  }
  return part;
}

// The first token of [lo, hi) up to which the kept weights, and `before`, sum to
// more than t (or to as much as they come to); -1: none is kept.
template <typename T>
__device__ __forceinline__ int descend(const T* row, const Row& r, int lo, int hi, double t,
                                       double before, Shared& s) {
  constexpr int N = Vec<T>::n;
  const int lane = threadIdx.x & 63;
  while (hi - lo > 64 * N) {
    part_sums<T>(row, r, lo, hi, s);
    const int w = part_at(s.weigh, kWaves, &t, &before);
    if (w < 0) {
      __syncthreads();
      return -1;
    }
    int from, to;
    share<T>(w, lo, hi, &from, &to);
    lo = from, hi = to;
  }
  // (every wave does the same)
  double mine[N], sum = 0.0;
  const int i = lo + lane * N;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float x = i + k < hi ? fmaxf((float)row[i + k], -kInf) : -kInf;
    mine[k] = i + k < hi && x >= r.below ? kept_weight(r, x, i + k) : 0.0;
    sum += mine[k];
  }
  const double upto = scan64(sum);
  const double last = __shfl_up(upto, 1, 64);
  if (lane > 0) before += last;
  // (sums round: a token is taken only if it weighs something itself)
  double end = before;
#pragma unroll
  for (int k = 0; k < N; ++k) end += mine[k];
  double most = sum > 0.0 ? end : 0.0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) most = fmax(most, __shfl_xor(most, d, 64));
  t = fmin(t, just_below(most));
  int at = -1;
  bool past = false;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    before += mine[k];
    if (mine[k] > 0.0 && !past) at = i + k, past = before > t;
  }
  const u64 hit = __ballot(past);
  __syncthreads();
  return hit ? __shfl(at, __ffsll(hit) - 1, 64) : -1;
}

// Where u falls among the row's `n` parts of these weights: its place *t, the part,
// and *before, what lies before that.  -1, the whole row, where u's place is so near
// the row's start that what the parts leave out (a list's units, what is
// kLeast or less) could decide.
__device__ __forceinline__ int part_of(const Ask& ask, const double* weight, int n, double* t,
                                       double* before) {
  double all = 0.0;
  for (int k = 0; k < n; ++k) all += weight[k];
  *t = (double)ask.u * all;
  *before = 0.0;
  return ask.faint() ? -1 : part_at(weight, n, t, before);
}

// Writes a row's answer.  n_top: how many logits are infinite, if any is.
template <typename T>
__device__ __forceinline__ void answer(const SampleArgs& a, int64_t j, const T* row, int token,
                                       const Found& f, u64 n_top) {
  if (threadIdx.x != 0) return;
  a.token[j] = token;
  if (!a.logp) return;
  if (token < 0)
    a.logp[j] = -kInf;
  else if (f.top == kInf)
    a.logp[j] = (float)-log((double)n_top);
  else
    a.logp[j] = (float)(((double)fmaxf((float)row[token], -kInf) - (double)f.top) - log(f.whole));
}

// The first index of the largest logit, known to lie among the N from `at` on.
template <typename T>
__device__ __forceinline__ int first_top(const T* row, int at, int V, float top) {
  int i = at;
  while (i < V - 1 && !((float)row[i] == top)) ++i;
  return i;
}

// What the first kernels leave of a row to the later ones: nothing, all of it, a
// list, a list of the cut's steps and the weights above them, weights of the
// segments.
enum { kDone = 0, kGeneral = 1, kList = 2, kCutList = 3, kParts = 4 };
struct RowState {
  Found found;
  int route;
  uint32_t n_list;
  int before;  // logits above the cut's steps
};

// ---- a row by a block ----------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
sample_row_kernel(const SampleArgs a, RowState* __restrict__ states) {
  __shared__ Shared s;
  const int64_t j = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (j >= a.max_rows || (a.n_rows && j >= *a.n_rows)) return;
  const T* const row = reinterpret_cast<const T*>(a.logits) + j * a.stride;
  const Ask ask(a, j);
  const int V = a.V;
  fill_table(s);
  if (threadIdx.x == 0) s.n_list = 0;
  const Steps steps(guess_of<T>(row, V), ask.temp);
  const Found f = first_pass<T>(row, 0, V, ask, steps, s.scan);
  int route = kDone, token = -1;
  if (f.top == kInf) {
    route = kGeneral;
  } else if (f.top > -kInf && ask.greedy) {
    token = first_top<T>(row, f.at, V, f.top);
  } else if (f.top > -kInf) {
    Row r(ask, f.top, V, s.table);
    bool parts = false;  // s.weigh has the waves' kept weights
    if (ask.by_k || ask.by_p) {
      const Bracket in = bracket_of(ask, steps, f, s.scan);
      if (in.last >= 0) {
        // (the counts are read: the list takes their place)
        double above, all;
        auto put = [&](float x, int i) __attribute__((always_inline)) {
          const uint32_t at = atomicAdd(&s.n_list, 1u);
          if (at < kCap) s.list[at] = entry_of(x, i);
        };
        if (in.first == 0)
          ask.by_k ? second_pass<T, false, false>(row, r, 0, V, steps, in, &above, &all, put)
                   : second_pass<T, true, false>(row, r, 0, V, steps, in, &above, &all, put);
        else
          ask.by_k ? second_pass<T, false, true>(row, r, 0, V, steps, in, &above, &all, put)
                   : second_pass<T, true, true>(row, r, 0, V, steps, in, &above, &all, put);
        all = weigh_waves(all, s);
        r.scale(ask.by_k ? (double)max(kCap, ask.k) : all);
        const int n = min((int)s.n_list, kCap);
        if (in.first == 0) {
          token = draw_from_list(ask, r, n, all, V, s);
        } else {
          const double upper = weigh_waves(above, s);
          parts = cut_within(ask, r, n, in.before, upper, all, s);
          if (parts) {
            if (threadIdx.x < kWaves) s.part[threadIdx.x] = 0;
            __syncthreads();
            const int per = share_size<T>(0, V);
            for (int i = threadIdx.x; i < n; i += kThreads)
              atomicAdd(&s.part[(int)(uint32_t)s.list[i] / per], entry_units(r, s.list[i]));
            __syncthreads();
            if (threadIdx.x < kWaves)
              s.weigh[threadIdx.x] += ldexp((double)s.part[threadIdx.x], -r.shift);
            __syncthreads();
          }
        }
      }
    } else {
      r.scale(weigh_waves(weigh<T>(row, r, 0, V), s));
      parts = true;
    }
    if (parts) {
      double t, before;
      int lo = 0, hi = V;
      const int part = part_of(ask, s.weigh, kWaves, &t, &before);
      if (part >= 0) share<T>(part, 0, V, &lo, &hi);
      token = descend<T>(row, r, lo, hi, t, before, s);
    }
    if (token < 0) route = kGeneral;
  }
  if (threadIdx.x == 0) {
    states[j].found = f;
    states[j].route = route;
  }
  if (route == kDone) answer<T>(a, j, row, token, f, 0);
}

// ---- a row by several blocks -----------------------------------------------------
struct Segments {
  int per_row;      // segments of a row
  int size;         // logits of one, below 2^16
  Found* found;     // [rows][per_row]
  uint16_t* count;  // [rows][per_row][kSteps]
  double* part;     // [rows][per_row] weights that are kept, or lie above the list's
  double* all;      // [rows][per_row] weights
  u64* list;        // [rows][kCap]
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
sample_first_kernel(const SampleArgs a, RowState* __restrict__ states, const Segments g) {
  __shared__ Scan s;
  const int64_t j = blockIdx.y;
  if (a.n_rows && j >= *a.n_rows) return;
  const T* const row = reinterpret_cast<const T*>(a.logits) + j * a.stride;
  const Ask ask(a, j);
  const Steps steps(guess_of<T>(row, a.V), ask.temp);
  const int lo = min(a.V, (int)blockIdx.x * g.size), hi = min(a.V, lo + g.size);
  const Found f = first_pass<T>(row, lo, hi, ask, steps, s);
  const int64_t seg = j * g.per_row + blockIdx.x;
  if (threadIdx.x == 0) {
    g.found[seg] = f;
    if (blockIdx.x == 0) states[j].n_list = 0;
  }
  if (ask.by_k || ask.by_p) {
    uint32_t* const to = reinterpret_cast<uint32_t*>(g.count + seg * kSteps);
    for (int b = threadIdx.x; b < kSteps / 2; b += kThreads)
      to[b] = s.count[2 * b] | s.count[2 * b + 1] << 16;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
sample_second_kernel(const SampleArgs a, RowState* __restrict__ states, const Segments g) {
  __shared__ Shared s;
  const int64_t j = blockIdx.y;
  if (a.n_rows && j >= *a.n_rows) return;
  const T* const row = reinterpret_cast<const T*>(a.logits) + j * a.stride;
  const Ask ask(a, j);
  const int V = a.V, lane = threadIdx.x & 63;
  fill_table(s);
  if (threadIdx.x == 0) s.n_list = 0;
  static_assert(kSteps == 8 * kThreads, "eight steps to a thread");
  if (ask.by_k || ask.by_p) {
    const uint4* const counts =
        reinterpret_cast<const uint4*>(g.count + j * g.per_row * kSteps) + threadIdx.x;
    uint32_t n[8] = {};
    constexpr int kAhead = 16;  // segments on their way: the last one again past it
    for (int k0 = 0; k0 < g.per_row; k0 += kAhead) {
      uint4 m[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        m[k] = counts[min(k0 + k, g.per_row - 1) * (kSteps / 8)];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t low = k0 + k < g.per_row ? 0xFFFFu : 0u;
        n[0] += m[k].x & low, n[1] += m[k].x >> 16 & low;
        n[2] += m[k].y & low, n[3] += m[k].y >> 16 & low;
        n[4] += m[k].z & low, n[5] += m[k].z >> 16 & low;
        n[6] += m[k].w & low, n[7] += m[k].w >> 16 & low;
      }
    }
    uint4* const to = reinterpret_cast<uint4*>(s.scan.count) + 2 * threadIdx.x;
    to[0] = make_uint4(n[0], n[1], n[2], n[3]);
    to[1] = make_uint4(n[4], n[5], n[6], n[7]);
  }
  Found f = {-kInf, 0.f, 0.0, 0};
  if (lane < g.per_row) f = g.found[j * g.per_row + lane];
  f = join_lanes(f, ask.per_f);
  __syncthreads();
  const int lo = min(V, (int)blockIdx.x * g.size), hi = min(V, lo + g.size);
  const int64_t seg = j * g.per_row + blockIdx.x;
  const Row r(ask, f.top, V, s.table);
  int route = kDone, before = 0;
  double kept = 0.0, all = 0.0;
  if (f.top == kInf) {
    route = kGeneral;
  } else if (f.top > -kInf && !ask.greedy) {
    if (ask.by_k || ask.by_p) {
      const Steps steps(guess_of<T>(row, V), ask.temp);
      const Bracket in = bracket_of(ask, steps, f, s.scan);
      route = kGeneral;
      if (in.last >= 0) {
        route = in.first == 0 ? kList : kCutList;
        before = in.before;
        // (gathered in LDS, where the counts were, and given a place at once)
        auto put = [&](float x, int i) __attribute__((always_inline)) {
          const uint32_t at = atomicAdd(&s.n_list, 1u);
          if (at < kCap) s.list[at] = entry_of(x, i);
        };
        if (ask.by_k)
          second_pass<T, false, true>(row, r, lo, hi, steps, in, &kept, &all, put);
        else
          second_pass<T, true, true>(row, r, lo, hi, steps, in, &kept, &all, put);
        __syncthreads();
        const uint32_t n = min(s.n_list, (uint32_t)kCap);
        if (threadIdx.x == 0 && n > 0) s.n_few = atomicAdd(&states[j].n_list, n);
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < n; i += kThreads)
          if (s.n_few + i < kCap) g.list[j * kCap + s.n_few + i] = s.list[i];
      }
    } else {
      route = kParts;
      kept = weigh<T>(row, r, lo, hi);
    }
    kept = weigh_waves(kept, s);
    all = weigh_waves(all, s);
  }
  if (threadIdx.x == 0) {
    g.part[seg] = kept;
    g.all[seg] = all;
    if (blockIdx.x == 0) {
      states[j].found = f;
      states[j].route = route;
      states[j].before = before;
    }
  }
  if (route == kDone && blockIdx.x == 0)
    answer<T>(a, j, row, f.top == -kInf ? -1 : first_top<T>(row, f.at, V, f.top), f, 0);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
sample_third_kernel(const SampleArgs a, RowState* __restrict__ states, const Segments g) {
  __shared__ Shared s;
  __shared__ double weight[kMaxSegments];
  __shared__ u64 units[kMaxSegments];
  const int64_t j = blockIdx.x;
  if (a.n_rows && j >= *a.n_rows) return;
  const int route = states[j].route;
  if (route == kDone || route == kGeneral) return;
  const T* const row = reinterpret_cast<const T*>(a.logits) + j * a.stride;
  const Ask ask(a, j);
  const int V = a.V;
  const Found f = states[j].found;
  const int n = route == kParts ? 0 : min((int)states[j].n_list, kCap);
  fill_table(s);
  for (int i = threadIdx.x; i < n; i += kThreads) s.list[i] = g.list[j * kCap + i];
  double part = 0.0, all = 0.0;
  if (threadIdx.x < (unsigned)g.per_row) {
    part = g.part[j * g.per_row + threadIdx.x];
    all = g.all[j * g.per_row + threadIdx.x];
  }
  if (threadIdx.x < kMaxSegments) weight[threadIdx.x] = part, units[threadIdx.x] = 0;
  all = weigh_waves(all, s);
  const double above = weigh_waves(part, s);
  Row r(ask, f.top, V, s.table);
  r.scale(ask.by_k ? (double)max(kCap, ask.k) : route == kParts ? above : all);
  int token = -1;
  if (route == kList) {
    token = draw_from_list(ask, r, n, all, V, s);
  } else if (route == kParts || cut_within(ask, r, n, states[j].before, above, all, s)) {
    for (int i = threadIdx.x; i < n; i += kThreads)
      atomicAdd(&units[(int)(uint32_t)s.list[i] / g.size], entry_units(r, s.list[i]));
    __syncthreads();
    if (threadIdx.x < kMaxSegments)
      weight[threadIdx.x] += ldexp((double)units[threadIdx.x], -r.shift);
    __syncthreads();
    double t, before;
    int lo = 0, hi = V;
    const int k = part_of(ask, weight, g.per_row, &t, &before);
    if (k >= 0) lo = min(V, k * g.size), hi = min(V, lo + g.size);
    token = descend<T>(row, r, lo, hi, t, before, s);
  }
  if (threadIdx.x == 0) states[j].route = token < 0 ? kGeneral : kDone;
  if (token >= 0) answer<T>(a, j, row, token, f, 0);
}

// ---- what is left --------------------------------------------------------------
struct RestShared : Shared {
  u64 weight[kBins];
  uint32_t bins[kBins];
};

// Bins of T / 64 downwards from the largest logit.
__device__ __forceinline__ int bin_of(float x, float top, float per_bin) {
  return (int)fminf((top - x) * per_bin, (float)(kBins - 1));
}

// Of the histogram's bins, in order, the one where the running count (by_count)
// or weight reaches `goal`; what lies before it.
__device__ __forceinline__ void find_bin(RestShared& s, bool by_count, u64 goal, int* bin, u64* before_count,
                         u64* before_weight) {
  constexpr int kPer = kBins / kThreads;
  const int tid = threadIdx.x;
  u64 c = 0, w = 0, all;
#pragma unroll
  for (int k = 0; k < kPer; ++k) c += s.bins[tid * kPer + k], w += s.weight[tid * kPer + k];
  if (tid == 0) s.pick[0] = kBins - 1, s.part[0] = s.part[1] = 0;
  u64 bc = block_scan(c, &all, s), bw = block_scan(w, &all, s);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const u64 nc = s.bins[tid * kPer + k], nw = s.weight[tid * kPer + k];
    const u64 b = by_count ? bc : bw, n = by_count ? nc : nw;
    if (b < goal && goal <= b + n) s.pick[0] = tid * kPer + k, s.part[0] = bc, s.part[1] = bw;
    bc += nc, bw += nw;
  }
  __syncthreads();
  *bin = (int)s.pick[0], *before_count = s.part[0], *before_weight = s.part[1];
  __syncthreads();
}

// Which logits a histogram or a list takes: those of a bin, and of these the
// ones whose key begins with certain bits.
struct Within {
  float top, per_bin;
  int bin;          // -1: all
  int open;         // bits of the key that are not yet decided
  uint32_t prefix;  // the others
  __device__ __forceinline__ bool has(float x) const {
    if (bin >= 0 && bin_of(x, top, per_bin) != bin) return false;
    return open == 32 || (key_of(x) >> open) == prefix;
  }
};

// Counts and units of the logits within, over the bins (bits = 0) or over the
// next bits of their keys, largest first.
template <typename T>
__device__ __forceinline__ void histogram(const T* row, const Row& r, const Within& in, int bits,
                                          int V, RestShared& s) {
  constexpr int N = Vec<T>::n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int b = threadIdx.x; b < kBins; b += kThreads) s.weight[b] = 0, s.bins[b] = 0;
  __syncthreads();
  int lo, hi;
  share<T>(wave, 0, V, &lo, &hi);
  u64 far_w = 0;
  uint32_t far_n = 0;
  each_vec<T, 1>(row, lo, hi, [&](const float* v, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float x = fmaxf(v[k], -kInf);
      if (i + k >= hi || !in.has(x)) continue;
      const uint32_t mask = (1u << bits) - 1;
      const int b = bits == 0 ? bin_of(x, in.top, in.per_bin)
                              : (int)(mask - ((key_of(x) >> (in.open - bits)) & mask));
      const u64 w = units_of(r, x);
      if (bits == 0 && b == kBins - 1) {  // (most logits: not all into one bin)
        far_w += w, ++far_n;
      } else {
        atomicAdd(&s.bins[b], 1u);
        atomicAdd(&s.weight[b], w);
      }
    }
  });
  far_w = sum_of(far_w);
  far_n = sum_of(far_n);
  if ((threadIdx.x & 63) == 0 && far_n) {
    atomicAdd(&s.bins[kBins - 1], far_n);
    atomicAdd(&s.weight[kBins - 1], far_w);
  }
  __syncthreads();
}

// The end of the order's first `goal` tokens (by_count) or of the first ones that
// have `goal` units (0: top-p's share of the whole row), into r.key, r.index and
// r.below.
template <typename T>
__device__ __forceinline__ void cut(const T* row, Row& r, const Ask& ask, bool by_count, u64 goal, int V,
                    RestShared& s) {
  constexpr int N = Vec<T>::n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Within in = {r.top, fminf(64.f / ask.temp, 1e30f), -1, 32, 0};
  u64 bc = 0, bw = 0, inside = 0;
  for (int level = 0; level < 4; ++level) {
    const int bits = level == 0 ? 0 : level == 3 ? 10 : 11;
    histogram<T>(row, r, in, bits, V, s);
    if (goal == 0) {
      u64 all = 0;
      for (int k = threadIdx.x; k < kBins; k += kThreads) all += s.weight[k];
      goal = ask.goal(block_sum(all, s));
    }
    int b;
    u64 c, w;
    find_bin(s, by_count, goal - (by_count ? bc : bw), &b, &c, &w);
    bc += c, bw += w;
    inside = s.bins[b];
    if (level == 0) {
      in.bin = b;
    } else {
      in.open -= bits;
      in.prefix = (level == 1 ? 0u : in.prefix << bits) | ((1u << bits) - 1 - (uint32_t)b);
    }
    __syncthreads();
    if (inside <= (u64)kCap) break;
  }
  const u64 need = goal - (by_count ? bc : bw);
  if (inside > (u64)kCap) {  // equal logits
    Row ties = r;
    ties.ties_only = true;
    ties.key = in.prefix;
    ties.below = value_of(in.prefix);
    const u64 each = by_count ? 1 : units_of(r, value_of(in.prefix));
    const u64 n = each ? (need + each - 1) / each : inside;
    r.index = descend<T>(row, ties, 0, V, (double)(max((u64)1, min(n, inside)) - 1), 0.0,
                         s);
    r.key = in.prefix;
    r.below = fmaxf(r.below, ties.below);
    return;
  }
  if (threadIdx.x == 0) s.n_list = 0;
  __syncthreads();
  int lo, hi;
  share<T>(wave, 0, V, &lo, &hi);
  each_vec<T, 2>(row, lo, hi, [&](const float* v, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float x = fmaxf(v[k], -kInf);
      if (i + k < hi && in.has(x)) {
        const uint32_t at = atomicAdd(&s.n_list, 1u);
        if (at < kCap) s.list[at] = entry_of(x, i + k);
      }
    }
  });
  __syncthreads();
  cut_list(r, min((int)s.n_list, kCap), by_count, need, s);
}

template <typename T>
__device__ __forceinline__ void rest_of_row(const SampleArgs& a, int64_t j, const Found& f,
                                            RestShared& s) {
  const int V = a.V;
  const T* const row = reinterpret_cast<const T*>(a.logits) + j * a.stride;
  const Ask ask(a, j);
  u64 n_top = 0;
  int token;
  Row r(ask, f.top, V, s.table);
  if (f.top == kInf) {
    // infinite logits weigh the same
    r.ties_only = true;
    r.key = key_of(f.top);
    r.below = f.top;
    n_top = (u64)part_sums<T>(row, r, 0, V, s);
    u64 n = ask.greedy ? 1 : n_top;
    if (ask.by_k) n = min(n, (u64)ask.k);
    if (ask.by_p) n = ask.goal(n);
    token = descend<T>(row, r, 0, V, (double)ask.u * (double)n, 0.0, s);
  } else {
    const double min_w = r.min_w;
    const float below = r.below;
    r.min_w = 0.0, r.below = -kInf;  // (the cuts' weights are those of all tokens)
    r.scale(weigh_waves(weigh<T>(row, r, 0, V), s));
    u64 all = 0;
    if (ask.by_k) {
      cut<T>(row, r, ask, true, (u64)ask.k, V, s);
      if (ask.by_p)
        all = block_sum(share_sum<u64>(row, r, 0, V,
                                       [&](float x, int i) __attribute__((always_inline)) {
                                         return kept_units(r, x, i);
                                       }),
                        s);
    }
    if (ask.by_p) cut<T>(row, r, ask, false, ask.by_k ? ask.goal(all) : 0, V, s);
    r.min_w = min_w, r.below = fmaxf(r.below, below);
    const double t = (double)ask.u * part_sums<T>(row, r, 0, V, s);
    token = descend<T>(row, r, 0, V, t, 0.0, s);
  }
  answer<T>(a, j, row, token, f, n_top);
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
sample_rest_kernel(const SampleArgs a, const RowState* __restrict__ states) {
  __shared__ RestShared s;
  int64_t n_rows = a.max_rows;
  if (a.n_rows) n_rows = min((int64_t)*a.n_rows, n_rows);
  bool filled = false;
  // every wave looks at 64 of the block's rows at a time
  const int64_t step = gridDim.x;
  for (int64_t base = blockIdx.x; base < n_rows; base += 64 * step) {
    const int64_t mine = base + (threadIdx.x & 63) * step;
    const bool left = mine < n_rows && states[mine].route == kGeneral;
    for (u64 todo = __ballot(left); todo; todo &= todo - 1) {
      if (!filled) fill_table(s);
      filled = true;
      __syncthreads();
      const int64_t j = base + (__ffsll(todo) - 1) * step;
      rest_of_row<T>(a, j, states[j].found, s);
    }
  }
}

// ---- host ------------------------------------------------------------------------
// Rows are cut into segments where they alone would leave much of the card idle:
// so many that about 512 blocks work, but of at least 4,096 logits each (and
// below 2^16, for the counts' type).
int segments_of(int64_t rows, int32_t V) {
  const int64_t n =
      std::min<int64_t>({(V + 4095) / 4096, 512 / std::max<int64_t>(rows, 1), kMaxSegments});
  return rows > 0 && n >= 2 && V / n < 65000 ? (int)n : 0;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t states, found, count, part, all, list, total;
  Layout(int64_t rows, int32_t V) {
    const size_t r = (size_t)rows, segs = r * (size_t)segments_of(rows, V);
    states = 0;
    found = states + up(r * sizeof(RowState));
    count = found + up(segs * sizeof(Found));
    part = count + up(segs * kSteps * sizeof(uint16_t));
    all = part + up(segs * sizeof(double));
    list = all + up(segs * sizeof(double));
    total = list + (segs ? r * kCap * sizeof(u64) : 0);
  }
};

template <typename T>
void run(const SampleArgs& a, hipStream_t stream) {
  const Layout at(a.max_rows, a.V);
  char* const ws = reinterpret_cast<char*>(a.workspace);
  RowState* const states = reinterpret_cast<RowState*>(ws + at.states);
  const unsigned rows = (unsigned)a.max_rows;
  if (const int per_row = segments_of(a.max_rows, a.V)) {
    Segments g;
    const int vec = Vec<T>::n;
    g.per_row = per_row;
    g.size = ((a.V + per_row - 1) / per_row + vec - 1) / vec * vec;
    g.found = reinterpret_cast<Found*>(ws + at.found);
    g.count = reinterpret_cast<uint16_t*>(ws + at.count);
    g.part = reinterpret_cast<double*>(ws + at.part);
    g.all = reinterpret_cast<double*>(ws + at.all);
    g.list = reinterpret_cast<u64*>(ws + at.list);
    const dim3 grid((unsigned)per_row, rows);
    sample_first_kernel<T><<<grid, kThreads, 0, stream>>>(a, states, g);
    sample_second_kernel<T><<<grid, kThreads, 0, stream>>>(a, states, g);
    sample_third_kernel<T><<<rows, kThreads, 0, stream>>>(a, states, g);
  } else {
    // (a launch takes fewer than 2^32 threads along a dimension)
    const unsigned wide = std::min(rows, 1u << 22);
    const dim3 grid(wide, (rows + wide - 1) / wide);
    sample_row_kernel<T><<<grid, kThreads, 0, stream>>>(a, states);
  }
  sample_rest_kernel<T><<<std::min(rows, 256u), kThreads, 0, stream>>>(a, states);
}

}  // namespace

size_t sample_workspace_bytes(int64_t max_rows, int32_t V) {
  return max_rows > 0 && V > 0 ? Layout(max_rows, V).total : 0;
}

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  if (a.max_rows == 0) return hipSuccess;
  a.dtype == MDLM_BF16 ? run<bf16_t>(a, stream) : run<float>(a, stream);
  return hipGetLastError();
}

}  // namespace mdlm
