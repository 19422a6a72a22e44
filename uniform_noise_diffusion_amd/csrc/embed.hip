// Token embedding with a scale, and the table's gradient by sorted tokens.
//
// DiffusionGemma card, "Finetuning notes", and the LLaDA-8B-MDLM-LoRA card,
// "LoRA" row, name the embeddings that stand before the model whose loss this
// library computes: xt goes in through them, and a tied table's gradient adds
// to the head's.
//
//   out[i]      = scale * T[ids[i]]
//   d_T[v] (+)= scale * sum over i with ids[i] = v of d_out[i]
//
// Forward: a gather, bound by memory; a wave moves 2,048 entries of a row.
//
// Gradient: the tokens are sorted by id (position breaking ties), so each
// table row's terms lie side by side: no atomics, and the same bits whenever
// the sizes and the ids are the same.  Absorbing corruption makes about half of
// all tokens one id (the mask), so the sorted list holds one run of n/2 among
// runs of one or two: the list is cut into chunks of C entries.  A run within
// two neighbouring chunks is summed in ascending position by one wave per 512
// columns; a longer one is summed chunk by chunk into partial rows, which a last
// kernel adds up (where it is cut, and so its rounding, depends on how many
// tokens have lower ids).  Few tokens take one launch without a list, in which
// four groups of lanes, or 16 waves, share a run.
#include "row_ops.h"

#include <algorithm>

namespace mdlm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int64_t kMaxBlocks = 1 << 20;

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// ---- forward ---------------------------------------------------------------

template <typename T, bool FULL>
__global__ void __launch_bounds__(kThreads)
embed_kernel(const int32_t* __restrict__ ids, int64_t n, const T* __restrict__ table, int32_t V,
             int32_t H, float scale, T* __restrict__ out) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c0 = blockIdx.y * 2048 + 8 * (threadIdx.x & 63);
  for (int64_t i = (int64_t)blockIdx.x * kWaves + wave; i < n; i += (int64_t)gridDim.x * kWaves) {
    const int32_t id = ids[i];
    const bool ok = (uint32_t)id < (uint32_t)V;
    const T* src = table + (int64_t)(ok ? id : 0) * H;
    T* dst = out + i * H;
    Raw8<T> r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = load8<FULL>(src, c0 + 512 * k, H);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[8];
      widen(r[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = ok ? v[j] * scale : 0.f;
      store8<FULL>(dst, c0 + 512 * k, H, v);
    }
  }
}

// ---- sorting the tokens ----------------------------------------------------

constexpr int kRankThreads = 1024;
constexpr int kRankWaves = kRankThreads / 64;
constexpr int kRankI = 16;        // tokens ranked by one block
constexpr int64_t kOneRun = 8192;  // up to here the whole list is one run
constexpr int64_t kRun = 1024;     // beyond: runs of this many tokens, merged,
constexpr int kLdsRuns = 32;       // first 32 at a time in LDS,
constexpr int kFan = 16;           // then 16 at a time in memory

__device__ __forceinline__ uint32_t sort_id(int32_t id, int32_t V) {
  return (uint32_t)id < (uint32_t)V ? (uint32_t)id : (uint32_t)V;
}

// Clears n floats: one 16-byte store per thread, the blocks in order.  This
// pattern writes fastest here: 305 us for the 2.07 GB of a 126,464 x 4,096
// table (6.8 TB/s); four stores a thread took 345 us, whole rows by waves that
// first look whether the row is written anyway 350 us.
__device__ __forceinline__ void clear(float* __restrict__ p, int64_t n, int64_t thread,
                                      int64_t threads) {
  // 16-byte words from the first address that is a multiple of 16
  int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) / 4 & 3);
  head = head < n ? head : n;
  const int64_t n4 = (n - head) / 4, tail = n - head - 4 * n4;
  float4* words = reinterpret_cast<float4*>(p + head);
  for (int64_t i = thread; i < n4; i += threads) words[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (thread < head) p[thread] = 0.f;
  if (thread < tail) p[head + 4 * n4 + thread] = 0.f;
}

__global__ void __launch_bounds__(kThreads) clear_kernel(float* __restrict__ p, int64_t n) {
  clear(p, n, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
}

// Of four ids in LDS, the number below `key`.
__device__ __forceinline__ int count_below(const uint32_t* s_id, int q, uint32_t key) {
  const uint4 k = *reinterpret_cast<const uint4*>(&s_id[4 * q]);
  return (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
}

// Sorts each run of `len` tokens by (id, position); an id outside [0, V)
// counts as V and so comes last.  A token's place is the number of its run's
// tokens before it, counted over all of them: a block holds the run's ids in
// LDS and ranks 16 tokens at a time, a lane comparing one of them with every
// 64th group of four ids: two instructions per 64 comparisons, no exchange and
// no barriers inside.  6.3 us at 4,096 tokens, of which the comparisons are
// 1.8; 12 to 13 us at 8,192, where they are four times as many.  (A bitonic network of 1,024 took 14 us and left more
// to merge; counting with ballots, whose bits the scalar unit adds up, 7.5
// and 19 us.)
__global__ void __launch_bounds__(kRankThreads)
rank_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t len, int32_t V,
            int32_t* __restrict__ sid, int32_t* __restrict__ spos, int64_t per_block,
            int32_t rank_blocks, float* __restrict__ fill, int64_t fill_n) {
  if ((int)blockIdx.x >= rank_blocks) {
    clear(fill, fill_n, (int64_t)(blockIdx.x - rank_blocks) * kRankThreads + threadIdx.x,
          (int64_t)(gridDim.x - rank_blocks) * kRankThreads);
    return;
  }
  __shared__ __align__(16) uint32_t s_id[kOneRun];
  __shared__ int s_count[kRankWaves][kRankI];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t per_run = (len + kRankI - 1) / kRankI;  // groups of tokens per run
  const int64_t groups = (n + len - 1) / len * per_run;
  const int64_t g_end = (blockIdx.x + 1) * per_block;
  int64_t held = -1;  // the run whose ids are in LDS
  for (int64_t g = blockIdx.x * per_block; g < g_end && g < groups; ++g) {
    const int64_t run = g / per_run, start = run * len;
    const int m = (int)(n - start < len ? n - start : len);  // tokens of this run
    const int i0 = (int)(g - run * per_run) * kRankI;
    if (i0 >= m) continue;
    const int quads = (m + 3) / 4;
    if (run != held) {
      __syncthreads();  // the run before it is done with
      for (int j = tid; j < 4 * quads; j += kRankThreads)
        s_id[j] = j < m ? sort_id(ids[start + j], V) : 0xFFFFFFFFu;
      held = run;
    }
    __syncthreads();
    const int i = i0 + (lane & 15);
    const uint32_t key = s_id[i < m ? i : i0];
    // fours of ids before the group (an equal id comes first), behind it, and
    // the group's own
    const int g0 = i0 / 4, g1 = g0 + kRankI / 4;
    int count = 0;
    int q = tid / 16;
#pragma unroll 4
    for (; q < g0; q += kRankThreads / 16) count += count_below(s_id, q, key + 1);
    if (q < g1) {
      if (q < quads) {
        const uint4 k = *reinterpret_cast<const uint4*>(&s_id[4 * q]);
        const int j = 4 * q;
        count += k.x < key + (j < i) ? 1 : 0;
        count += k.y < key + (j + 1 < i) ? 1 : 0;
        count += k.z < key + (j + 2 < i) ? 1 : 0;
        count += k.w < key + (j + 3 < i) ? 1 : 0;
      }
      q += kRankThreads / 16;
    }
#pragma unroll 4
    for (; q < quads; q += kRankThreads / 16) count += count_below(s_id, q, key);
    count += __shfl_xor(count, 16);
    count += __shfl_xor(count, 32);
    if (lane < kRankI) s_count[tid >> 6][lane] = count;
    __syncthreads();
    if (tid < kRankI && i0 + tid < m) {
      int64_t at = start;
#pragma unroll
      for (int w = 0; w < kRankWaves; ++w) at += s_count[w][tid];
      sid[at] = (int32_t)s_id[i0 + tid];
      spos[at] = (int32_t)(start + i0 + tid);
    }
  }
}

// Merges up to 32 sorted runs of 1,024 entries into one: an entry's place is
// its place in its run plus, for each other run, the number of that run's
// entries before it (equal ids of an earlier run come first, positions
// ascending with the runs).  A block holds all of the group's ids in LDS and
// places 64 neighbours of one run; each wave searches two of the runs for
// them.
constexpr int kMergeThreads = 1024;
constexpr int kMergeWaves = kMergeThreads / 64;

__global__ void __launch_bounds__(kMergeThreads)
merge_lds_kernel(const int32_t* __restrict__ sid, const int32_t* __restrict__ spos, int64_t n,
                 int64_t per_block, int32_t* __restrict__ out_id, int32_t* __restrict__ out_pos) {
  constexpr int kGroup = kLdsRuns * (int)kRun;
  __shared__ __align__(16) int32_t s_id[kGroup];
  __shared__ int s_count[kMergeWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b_end = (blockIdx.x + 1) * per_block;
  int64_t held = -1;  // the group whose ids are in LDS
  for (int64_t b = blockIdx.x * per_block; b < b_end && b * 64 < n; ++b) {
    const int64_t group = b * 64 / kGroup * kGroup;
    const int m = (int)(n - group < kGroup ? n - group : kGroup);
    const int i = (int)(b * 64 - group) + lane;
    const int run = (int)(b * 64 - group) / (int)kRun;
    __syncthreads();  // the entries before these are placed
    if (group != held) {
      for (int j = tid; j < m; j += kMergeThreads) s_id[j] = sid[group + j];
      held = group;
      __syncthreads();
    }
    const int32_t id = s_id[i < m ? i : m - 1];
    int before = 0;
    for (int r = wave; r * (int)kRun < m; r += kMergeWaves) {
      if (r == run) continue;
      const int start = r * (int)kRun;
      int lo = start, hi = start + (int)kRun < m ? start + (int)kRun : m;
      for (int span = (int)kRun; span > 0; span >>= 1)
        if (lo < hi) {
          const int mid = (lo + hi) >> 1;
          const int32_t v = s_id[mid];
          if (v < id || (v == id && r < run))
            lo = mid + 1;
          else
            hi = mid;
        }
      before += lo - start;
    }
    s_count[wave][lane] = before;
    __syncthreads();
    if (wave == 0 && i < m) {
      int64_t at = group + i - run * (int)kRun;
#pragma unroll
      for (int w = 0; w < kMergeWaves; ++w) at += s_count[w][lane];
      out_id[at] = id;
      out_pos[at] = spos[group + i];
    }
  }
}

// Merges up to kFan sorted runs of `len` entries into one, as above, in
// memory.  A wave holds 64 neighbours of one run, so in another run all their
// places lie between those of its first and its last key: one round of 64
// probes of every run bounds both, and the lanes' own searches are confined to
// what lies between.  (Each lane searching the whole runs is bound by the
// gathers: 27 us at 65,536 tokens.)
__device__ __forceinline__ bool comes_before(int32_t v, int64_t r, int32_t id, int64_t run) {
  return v < id || (v == id && r < run);
}

__global__ void __launch_bounds__(kThreads)
merge_runs_kernel(const int32_t* __restrict__ sid, const int32_t* __restrict__ spos, int64_t n,
                  int64_t len, int32_t* __restrict__ out_id, int32_t* __restrict__ out_pos) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int64_t step = len / 64;
  // (len is a multiple of 4,096: a wave's entries are of one run)
  for (int64_t base = (int64_t)blockIdx.x * kThreads + wave * 64; base < n; base += stride) {
    const int64_t run = base / len, group = run / kFan * kFan;
    const int64_t i = base + lane;
    const int32_t id = sid[i < n ? i : n - 1];
    const int32_t id0 = __builtin_amdgcn_readlane(id, 0);
    const int32_t id63 = __builtin_amdgcn_readlane(id, 63);
    int32_t v[kFan];
#pragma unroll
    for (int r = 0; r < kFan; ++r) {
      const int64_t p = (group + r) * len + step * lane;
      v[r] = sid[p < n ? p : n - 1];
    }
    uint32_t at[kFan], to[kFan], span = 0;
    int64_t rank = i - run * len;
#pragma unroll
    for (int r = 0; r < kFan; ++r) {
      const int64_t b = (group + r) * len, p = b + step * lane;
      // probes before the first key and before the last one: the places lie
      // behind the last of the former and not behind the first past the latter
      const int k0 = __popcll(__ballot(p < n && comes_before(v[r], group + r, id0, run)));
      const int k1 = __popcll(__ballot(p < n && comes_before(v[r], group + r, id63, run)));
      const int64_t a = b + (k0 > 0 ? step * (k0 - 1) + 1 : 0), z = b + step * k1;
      at[r] = (uint32_t)(a < n ? a : n);
      to[r] = (uint32_t)(z < n ? z : n);
      if (group + r == run) {
        to[r] = at[r];
        rank -= at[r];  // (added again below)
      } else {
        rank -= b < n ? b : n;
      }
      span = span > to[r] - at[r] ? span : to[r] - at[r];
    }
    for (; span > 0; span >>= 1) {
#pragma unroll
      for (int r = 0; r < kFan; ++r) {
        const uint32_t mid = (at[r] + to[r]) >> 1;
        v[r] = sid[mid < n ? mid : 0];  // (read but not used where at = to)
      }
#pragma unroll
      for (int r = 0; r < kFan; ++r)
        if (at[r] < to[r]) {
          const uint32_t mid = (at[r] + to[r]) >> 1;
          if (comes_before(v[r], group + r, id, run))
            at[r] = mid + 1;
          else
            to[r] = mid;
        }
    }
#pragma unroll
    for (int r = 0; r < kFan; ++r) rank += at[r];
    if (i < n) {
      out_id[group * len + rank] = id;
      out_pos[group * len + rank] = spos[i];
    }
  }
}

// ---- summing the runs of equal ids ------------------------------------------

// A run of equal ids that starts in chunk c belongs to chunk c's wave when it
// ends in chunk c or c + 1; a longer one is cut at the chunk borders: chunk
// c's part goes to slot 1 of its partial rows, every later chunk's to slot 0,
// and `cut` says of chunk c whether such a run starts there.
enum : uint8_t { kNotCut = 0, kCutShort = 1, kCutLong = 2 };  // long: over kShortParts chunks
constexpr int kShortParts = 32;
constexpr int kMaxChunk = 32;  // a chunk and the one behind it fit one wave's lanes

__device__ __forceinline__ int count_lanes(bool p) { return __popcll(__ballot(p)); }

// One wave sums 512 columns of one chunk's runs.
template <typename T, bool FULL, bool ACC>
__device__ __forceinline__ void sum_chunk(const int32_t* __restrict__ sid,
                                          const int32_t* __restrict__ spos, int64_t n, int32_t V,
                                          int32_t H, int32_t C, int64_t chunk, int c,
                                          const T* __restrict__ d_out, float scale,
                                          float* __restrict__ d_table, float* __restrict__ part,
                                          int64_t part_pitch, uint8_t* __restrict__ cut) {
  constexpr int kBatch = 8;  // rows in flight
  const int lane = threadIdx.x & 63;
  const int64_t e0 = chunk * C;
  // the chunk's entries and those behind it, one per lane, and the ids that
  // say whether its first and last runs go on: all read at once
  const int64_t at = e0 + lane;
  const int32_t id = at < n ? sid[at] : V;
  const int32_t pos = at < n ? spos[at] : 0;
  const int32_t prev = sid[e0 > 0 ? e0 - 1 : 0];
  const int32_t far = sid[e0 > C ? e0 - C - 1 : 0];
  const int32_t next2 = sid[e0 + 2 * C < n ? e0 + 2 * C : 0];
  const int64_t e_long = e0 + (int64_t)kShortParts * C;
  const int32_t beyond = sid[e_long < n ? e_long : 0];
  const int cnt = n - e0 < C ? (int)(n - e0) : C;
  const int32_t first = __builtin_amdgcn_readlane(id, 0);
  const int32_t last = __builtin_amdgcn_readlane(id, cnt - 1);
  const bool before = e0 > 0 && prev == first;
  int begin = 0, end = cnt;
  bool head = false, tail = false;  // the first / last run goes to a slot
  if (e0 + cnt < n && __builtin_amdgcn_readlane(id, cnt) == last && !(before && last == first)) {
    if (e0 + 2 * C < n && next2 == last)
      tail = true;
    else
      end += count_lanes(lane >= cnt && lane < 2 * C && id == last);
  }
  if (before) {
    const bool starts_in_prev = e0 <= C || far != first;
    const bool ends_here = e0 + C >= n || __builtin_amdgcn_readlane(id, C) != first;
    if (starts_in_prev && ends_here)
      begin = count_lanes(lane < C && id == first);
    else
      head = true;
  }
  const int32_t follow = __shfl_down(id, 1);
  const uint64_t ends = __ballot(lane + 1 >= end || follow != id);
  if (c == 0)  // (one wave's first lane: the wave of columns 0 .. 511)
    cut[chunk] = !tail || last >= V ? kNotCut
                 : e_long < n && beyond == last ? kCutLong
                                                : kCutShort;
  const int valid = count_lanes(id < V);  // ids outside the table come last
  const int stop = end < valid ? end : valid;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int j = begin; j < stop; j += kBatch) {
    Raw8<T> r[kBatch];
    Raw8<float> old[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (j + k < stop) {
        const int32_t p = __builtin_amdgcn_readlane(pos, j + k);
        r[k] = load8<FULL>(d_out + (int64_t)p * H, c, H);
        if (ACC && (ends >> (j + k) & 1))
          old[k] = load8<FULL>(d_table + (int64_t)__builtin_amdgcn_readlane(id, j + k) * H, c, H);
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (j + k < stop) {
        float v[8];
        widen(r[k], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
        if (ends >> (j + k) & 1) {
          const int slot = head ? 0 : (tail && j + k + 1 >= end ? 1 : -1);
          head = false;
          if (slot >= 0) {
            store8<true>(part + (2 * chunk + slot) * part_pitch, c, (int)part_pitch, acc);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[i] = ACC ? old[k].w[i] + scale * acc[i] : scale * acc[i];
            store8<FULL>(d_table + (int64_t)__builtin_amdgcn_readlane(id, j + k) * H, c, H, acc);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        }
      }
  }
}

template <typename T, bool FULL, bool ACC>
__global__ void __launch_bounds__(kThreads)
sum_runs_kernel(const int32_t* __restrict__ sid, const int32_t* __restrict__ spos, int64_t n,
                int32_t V, int32_t H, int32_t C, int32_t slabs, int64_t units,
                const T* __restrict__ d_out, float scale, float* __restrict__ d_table,
                float* __restrict__ part, int64_t part_pitch, uint8_t* __restrict__ cut) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < units;
       u += (int64_t)gridDim.x * kWaves) {
    const int64_t chunk = u / slabs;
    const int c = (int)(u - chunk * slabs) * 512 + 8 * lane;
    sum_chunk<T, FULL, ACC>(sid, spos, n, V, H, C, chunk, c, d_out, scale, d_table, part,
                            part_pitch, cut);
  }
}

// Number of lanes from lane 0 on for which `p` holds without a gap.
__device__ __forceinline__ int leading(bool p) {
  const uint64_t b = ~__ballot(p);
  return b ? __ffsll((unsigned long long)b) - 1 : 64;
}

// Adds the partial rows of each run that was cut, 256 columns per block
// column (blockIdx.x).  A run of up to 32 partial rows is one wave's; a longer
// one (the mask token's: 1,024 partial rows at 65,536 tokens) is split over
// four blocks of 64 columns, and within a block over 64 groups of 16 lanes,
// whose sums are added in order.  Each block lists the cut runs for itself,
// 1,024 chunks at a time, and takes its share of either kind in turn.
constexpr int kJoinThreads = 1024;
constexpr int kJoinWaves = kJoinThreads / 64;

// First of the numbers from `seen` on that is `mine` modulo `of`, from `seen`.
__device__ __forceinline__ int first_turn(uint32_t seen, uint32_t mine, uint32_t of) {
  const uint32_t at = seen % of;  // (mine < of)
  return (int)(mine >= at ? mine - at : mine + of - at);
}

template <bool ACC>
__global__ void __launch_bounds__(kJoinThreads)
join_runs_kernel(const int32_t* __restrict__ sid, int64_t n, int32_t V, int32_t H, int32_t C,
                 float scale, float* __restrict__ d_table, const float* __restrict__ part,
                 int64_t part_pitch, const uint8_t* __restrict__ cut) {
  __shared__ int32_t s_short[kJoinThreads], s_long[kJoinThreads];
  __shared__ int32_t s_count[2][kJoinWaves];
  __shared__ __align__(16) float s_sum[64][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t chunks = (n + C - 1) / C;
  uint32_t seen_short = 0, seen_long = 0;  // runs found before this round
  for (int64_t base = 0; base < chunks; base += kJoinThreads) {
    const int64_t m = base + tid;
    const int kind = m < chunks ? cut[m] : kNotCut;
    const bool is_short = kind == kCutShort, is_long = kind == kCutLong;
    const uint64_t lo = __ballot(is_short), hi = __ballot(is_long);
    if (lane == 0) s_count[0][wave] = __popcll(lo), s_count[1][wave] = __popcll(hi);
    __syncthreads();
    int at[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (w < wave) at[k] += s_count[k][w];
        total[k] += s_count[k][w];
      }
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    if (is_short) s_short[at[0] + __popcll(lo & below)] = (int32_t)m;
    if (is_long) s_long[at[1] + __popcll(hi & below)] = (int32_t)m;
    __syncthreads();

    // a run's first chunk wrote slot 1, the chunks behind it slot 0
    for (int o = first_turn(seen_short, blockIdx.y * kJoinWaves + wave, gridDim.y * kJoinWaves);
         o < total[0]; o += gridDim.y * kJoinWaves) {
      const int64_t m0 = s_short[o];
      const int32_t id = sid[(m0 + 1) * C];
      const int64_t probe = m0 + 1 + lane;
      const int parts = 1 + leading(probe < chunks && sid[(probe < chunks ? probe : 0) * C] == id);
      const int c = blockIdx.x * 256 + 4 * lane;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < part_pitch) {
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(
              part + (2 * (m0 + i) + (i == 0 ? 1 : 0)) * part_pitch + c);
          acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        float* d = d_table + (int64_t)id * H;
        const float a[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k < H) d[c + k] = ACC ? d[c + k] + scale * a[k] : scale * a[k];
      }
    }

    for (int o = first_turn(seen_long, blockIdx.y / 4, gridDim.y / 4); o < total[1];
         o += gridDim.y / 4) {
      const int64_t m0 = s_long[o];
      const int32_t id = sid[(m0 + 1) * C];
      // the chunk behind the run's last one: the first from which no entry
      // of the run begins
      int64_t first = m0 + kShortParts, end = chunks;
      while (first < end) {
        const int64_t step = (end - first + 63) / 64, probe = first + step * lane;
        const int k = leading(probe < end && sid[(probe < end ? probe : 0) * C] == id);
        // chunks first, first + step, .. (k of them) begin inside the run
        if (k == 0) break;
        end = first + step * k < end ? first + step * k : end;
        first += step * (k - 1) + 1;
      }
      const int64_t parts = first - m0;
      const int c = blockIdx.x * 256 + (blockIdx.y & 3) * 64 + 4 * (lane & 15);
      const int row = tid / 16;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < part_pitch) {
#pragma unroll 8
        for (int64_t i = row; i < parts; i += 64) {
          const float4 v = *reinterpret_cast<const float4*>(
              part + (2 * (m0 + i) + (i == 0 ? 1 : 0)) * part_pitch + c);
          acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
      }
      *reinterpret_cast<float4*>(&s_sum[row][4 * (lane & 15)]) = acc;
      __syncthreads();
      const int col = blockIdx.x * 256 + (blockIdx.y & 3) * 64 + tid;
      if (tid < 64 && col < H) {
        float sum = 0.f;
#pragma unroll 16
        for (int r = 0; r < 64; ++r) sum += s_sum[r][tid];
        float* d = d_table + (int64_t)id * H + col;
        *d = ACC ? *d + scale * sum : scale * sum;
      }
      __syncthreads();
    }
    seen_short += total[0], seen_long += total[1];
  }
}

// ---- few tokens ----------------------------------------------------------------

// Up to kFewTokens tokens need no sorted list: a wave takes one token, looks
// through all ids (in LDS) for its own and, where it is the first with that
// id, sums the id's rows for 128 columns, four rows side by side.  Ids of more
// than 16 tokens (the mask's) are left to the block's 16 waves together, each
// taking every 16th 64 tokens, their sums added in order; 128 columns to a
// block spread such a run's rows over enough compute units (with 512, one unit
// pulls 800 KB of 388 float32 rows and takes 20 us).  The blocks past
// `sum_blocks` clear the rows without a token, `rows` rows each.
constexpr int kFewTokens = 1024;
constexpr int kFewThreads = 1024;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewRun = 16;
constexpr int kFewCols = 128;

// acc += rows list[0 .. m) (m <= 64, entry l on lane l), lane group lane / 16
// taking every fourth of them.
template <typename T, bool FULL>
__device__ __forceinline__ void add_rows(const T* __restrict__ d_out, int list, int m, int32_t H,
                                         int c, float acc[8]) {
  constexpr int kBatch = 4;  // rows of a group in flight
  const int group = (threadIdx.x & 63) >> 4;
  for (int j = 0; j < m; j += 4 * kBatch) {
    Raw8<T> r[kBatch];
    bool on[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int l = j + 4 * k + group;
      on[k] = l < m;
      const int at = __shfl(list, l < m ? l : 0);
      if (on[k]) r[k] = load8<FULL>(d_out + (int64_t)at * H, c, H);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (on[k]) {
        float v[8];
        widen(r[k], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
      }
  }
}

// The four lane groups' sums, on all of them.
__device__ __forceinline__ void add_groups(float acc[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    acc[i] += __shfl_xor(acc[i], 16);
    acc[i] += __shfl_xor(acc[i], 32);
  }
}

template <typename T, bool FULL, bool ACC>
__global__ void __launch_bounds__(kFewThreads)
few_tokens_kernel(const int32_t* __restrict__ ids, int32_t n, int32_t V, int32_t H,
                  int32_t slabs, const T* __restrict__ d_out, float scale,
                  float* __restrict__ d_table, int32_t sum_blocks, int32_t rows) {
  __shared__ int32_t s_id[kFewTokens];
  __shared__ int32_t s_list[kFewWaves][kFewRun];
  __shared__ int32_t s_many[kFewWaves];
  __shared__ uint32_t s_present[2];
  __shared__ float s_sum[kFewWaves][kFewCols];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int j = tid; j < kFewTokens; j += kFewThreads)
    s_id[j] = j < n && (uint32_t)ids[j] < (uint32_t)V ? ids[j] : -1;
  if (tid < 2) s_present[tid] = 0;
  __syncthreads();

  if ((int)blockIdx.x >= sum_blocks) {
    const int64_t r0 = (int64_t)(blockIdx.x - sum_blocks) * rows;
    for (int j = tid; j < n; j += kFewThreads) {
      const int64_t k = s_id[j] - r0;
      if (k >= 0 && k < rows) atomicOr(&s_present[k / 32], 1u << (k % 32));
    }
    __syncthreads();
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = wave; k < rows && r0 + k < V; k += kFewWaves)
      if (!(s_present[k / 32] >> (k % 32) & 1))
        for (int c = 8 * lane; c < H; c += 512) store8<FULL>(d_table + (r0 + k) * H, c, H, zero);
    return;
  }

  const int token0 = (int)blockIdx.x / slabs * kFewWaves;
  const int c = (int)blockIdx.x % slabs * kFewCols + 8 * (lane & 15);
  const int token = token0 + wave;
  const int32_t id = token < n ? s_id[token] : -1;
  int m = 0, first = -1;  // tokens of this id, and the first of them
  if (id >= 0) {
#pragma unroll 4
    for (int j0 = 0; j0 < n; j0 += 64) {
      const int j = j0 + lane;
      const bool same = s_id[j] == id;  // (behind the last token there is none)
      const uint64_t b = __ballot(same);
      const int at = m + __popcll(b & (((uint64_t)1 << lane) - 1));
      if (same && at < kFewRun) s_list[wave][at] = j;
      first = first < 0 && b ? j0 + __ffsll((unsigned long long)b) - 1 : first;
      m += __popcll(b);
    }
  }
  if (first != token) m = 0;  // another wave's
  __builtin_amdgcn_wave_barrier();  // (the list is read by the lanes that it is for)
  if (lane == 0) s_many[wave] = m > kFewRun ? 1 : 0;
  float* row = d_table + (int64_t)(id >= 0 ? id : 0) * H;
  if (m > 0 && m <= kFewRun) {
    Raw8<float> old;
    if (ACC) old = load8<FULL>(row, c, H);
    const int list = s_list[wave][lane < m ? lane : 0];
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_rows<T, FULL>(d_out, list, m, H, c, acc);
    add_groups(acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = ACC ? old.w[i] + scale * acc[i] : scale * acc[i];
    if (lane < 16) store8<FULL>(row, c, H, acc);
  }
  __syncthreads();
  for (int w = 0; w < kFewWaves; ++w) {
    if (!s_many[w]) continue;
    const int32_t of = s_id[token0 + w];
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 64 * wave; j0 < n; j0 += 64 * kFewWaves) {
      const int j = j0 + lane;
      const bool same = s_id[j] == of;
      uint64_t b = __ballot(same);
      // the k-th lane takes the k-th of them
      const int count = __popcll(b);
      int list = 0;
      for (int k = 0; b; b &= b - 1, ++k)
        if (lane == k) list = j0 + __ffsll((unsigned long long)b) - 1;
      add_rows<T, FULL>(d_out, list, count, H, c, acc);
    }
    add_groups(acc);
    if (lane < 16) store8<true>(s_sum[wave], 8 * lane, kFewCols, acc);
    __syncthreads();
    const int col = (int)blockIdx.x % slabs * kFewCols + tid;
    if (tid < kFewCols && col < H) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kFewWaves; ++v) sum += s_sum[v][tid];
      float* d = d_table + (int64_t)of * H + col;
      *d = ACC ? *d + scale * sum : scale * sum;
    }
    __syncthreads();
  }
}

// Few enough for one launch: up to 2^20 entries it is the faster way at every
// width, at twice that both are even, beyond the sorted list is.  us a call,
// added to a table of 16,384 rows, with uniform ids / half of them one; the list
// takes 14 to 15 in all of these:
//   tokens       H = 8       64        256       1,024       4,096
//      256    6.2/ 7.3   6.2/ 7.3   6.1/ 7.4   6.2/ 7.6    6.5/ 7.8
//      512    6.3/ 7.9   6.2/ 7.9   6.3/ 8.1   6.3/ 8.3   12.8/13.7
//    1,024    6.7/10.4   6.5/10.3   6.6/10.4   9.7/11.1   29.6/30.4
bool is_few(int64_t n, int32_t H) { return n <= kFewTokens && n * H <= (int64_t)1 << 20; }

// Rows and number of the blocks that clear the table beside few tokens' sums:
// 64 KiB to a block, as far as its 64 bits for the rows go.
int few_rows(int32_t H) { return std::max(1, std::min(64, 16384 / H)); }
int64_t few_fills(int32_t V, int32_t H) { return ((int64_t)V + few_rows(H) - 1) / few_rows(H); }

template <typename T, bool FULL>
void run_few(const int32_t* ids, int64_t n, int32_t V, int32_t H, const void* d_out, float scale,
             float* d_table, bool accumulate, bool fill, hipStream_t stream) {
  const T* g = reinterpret_cast<const T*>(d_out);
  const int slabs = (H + kFewCols - 1) / kFewCols;
  const int sums = (int)((n + kFewWaves - 1) / kFewWaves) * slabs;
  const int rows = few_rows(H);
  const int fills = fill ? (int)few_fills(V, H) : 0;
  auto kernel = accumulate ? few_tokens_kernel<T, FULL, true> : few_tokens_kernel<T, FULL, false>;
  kernel<<<(unsigned)(sums + fills), kFewThreads, 0, stream>>>(ids, (int32_t)n, V, H, slabs, g,
                                                               scale, d_table, sums, rows);
}

// Floats of a table that the sorting launch clears, and blocks that may clear
// it beside few tokens' sums (two per compute unit).  A call with one token into
// 16,384 x 64 (256 blocks) takes 5.9 us so and 8.8 with a launch to clear the
// table; into 32,768 x 512 (1,024 blocks) 14.2 and 13.4, into 2,097,152 x 8
// (32,768 blocks of 64 short rows) 153 and 13.4.
constexpr int64_t kSmallTable = (int64_t)16 << 20;
constexpr int64_t kFewFills = 512;

// Entries of the sorted list per chunk: the most, up to 32, that leave 2,048
// waves (two per SIMD) something to do, and four at the least.
int chunk_of(int64_t n, int32_t H) {
  const int64_t slabs = (H + 511) / 512;
  int C = kMaxChunk;
  while (C > 4 && n * slabs < (int64_t)C * 2048) C /= 2;
  return C;
}

int64_t pitch_of(int32_t H) { return round_up(H, 8); }

template <typename T, bool FULL>
void run_sum(const int32_t* sid, const int32_t* spos, int64_t n, int32_t V, int32_t H,
             const void* d_out, float scale, float* d_table, bool accumulate, float* part,
             uint8_t* cut, hipStream_t stream) {
  const T* g = reinterpret_cast<const T*>(d_out);
  const int C = chunk_of(n, H);
  const int slabs = (H + 511) / 512;
  const int64_t units = (n + C - 1) / C * slabs;
  const unsigned grid = (unsigned)std::min<int64_t>((units + kWaves - 1) / kWaves, kMaxBlocks);
  if (accumulate)
    sum_runs_kernel<T, FULL, true><<<grid, kThreads, 0, stream>>>(
        sid, spos, n, V, H, C, slabs, units, g, scale, d_table, part, pitch_of(H),
        cut);
  else
    sum_runs_kernel<T, FULL, false><<<grid, kThreads, 0, stream>>>(
        sid, spos, n, V, H, C, slabs, units, g, scale, d_table, part, pitch_of(H),
        cut);
}

template <typename T, bool FULL>
void run_embed(const int32_t* ids, int64_t n, const void* table, int32_t V, int32_t H,
               float scale, void* out, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>((n + kWaves - 1) / kWaves, kMaxBlocks),
                  (unsigned)((H + 2047) / 2048));
  embed_kernel<T, FULL><<<grid, kThreads, 0, stream>>>(
      ids, n, reinterpret_cast<const T*>(table), V, H, scale, reinterpret_cast<T*>(out));
}

}  // namespace

hipError_t launch_embed(const int32_t* ids, int64_t n, const void* table, int32_t dtype,
                        int32_t V, int32_t H, float scale, void* out, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  const bool full = H % 8 == 0;
  if (dtype == MDLM_BF16)
    full ? run_embed<bf16_t, true>(ids, n, table, V, H, scale, out, stream)
         : run_embed<bf16_t, false>(ids, n, table, V, H, scale, out, stream);
  else
    full ? run_embed<float, true>(ids, n, table, V, H, scale, out, stream)
         : run_embed<float, false>(ids, n, table, V, H, scale, out, stream);
  return hipGetLastError();
}

// Two sorted lists (id and position: the merge goes from one to the other),
// a byte per chunk, then two partial rows per chunk; nothing for few tokens.
size_t embed_grad_workspace_bytes(int64_t n, int32_t H) {
  if (n <= 0 || H <= 0 || is_few(n, H)) return 0;
  const int C = chunk_of(n, H);
  const int64_t chunks = (n + C - 1) / C;
  return (size_t)(4 * round_up(4 * n, 256) + round_up(chunks, 256) +
                  chunks * 2 * pitch_of(H) * 4);
}

hipError_t launch_embed_grad(const int32_t* ids, int64_t n, const void* d_out, int32_t dtype,
                             int32_t V, int32_t H, float scale, float* d_table, bool accumulate,
                             void* workspace, hipStream_t stream) {
  if (n == 0 && accumulate) return hipSuccess;
  char* ws = reinterpret_cast<char*>(workspace);
  const int64_t list = round_up(4 * n, 256);
  int32_t* sid[2] = {reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + 2 * list)};
  int32_t* spos[2] = {reinterpret_cast<int32_t*>(ws + list),
                      reinterpret_cast<int32_t*>(ws + 3 * list)};
  const int C = chunk_of(n, H);
  uint8_t* cut = reinterpret_cast<uint8_t*>(ws + 4 * list);
  float* part = reinterpret_cast<float*>(ws + 4 * list + round_up((n + C - 1) / C, 256));
  const int64_t table_n = (int64_t)V * H;
  const bool apart =
      n == 0 || (is_few(n, H) ? few_fills(V, H) > kFewFills : table_n > kSmallTable);
  if (!accumulate && apart)
    clear_kernel<<<(unsigned)std::min<int64_t>(table_n / 4 / kThreads + 1, (int64_t)1 << 23),
                   kThreads, 0, stream>>>(d_table, table_n);
  if (n == 0) return hipGetLastError();
  if (is_few(n, H)) {
    auto run = H % 8 == 0 ? (dtype == MDLM_BF16 ? run_few<bf16_t, true> : run_few<float, true>)
                          : (dtype == MDLM_BF16 ? run_few<bf16_t, false> : run_few<float, false>);
    run(ids, n, V, H, d_out, scale, d_table, accumulate, !accumulate && !apart, stream);
    return hipGetLastError();
  }
  // Neighbouring tokens share a block where there are more than two blocks per
  // compute unit: they share the ids in LDS.
  const int64_t len = n <= kOneRun ? n : kRun;
  const int64_t groups = (n + len - 1) / len * ((len + kRankI - 1) / kRankI);
  const int64_t per_rank = (groups + 511) / 512;
  const int64_t ranks = (groups + per_rank - 1) / per_rank;
  const int64_t fill_n = accumulate || apart ? 0 : table_n;
  const int64_t fills = fill_n > 0 ? fill_n / 4 / kRankThreads + 1 : 0;
  rank_kernel<<<(unsigned)(ranks + fills), kRankThreads, 0, stream>>>(
      ids, n, len, V, sid[0], spos[0], per_rank, (int32_t)ranks, d_table, fill_n);
  int from = 0;
  if (n > kOneRun) {
    const int64_t sets = (n + 63) / 64, per_merge = (sets + 255) / 256;
    merge_lds_kernel<<<(unsigned)((sets + per_merge - 1) / per_merge), kMergeThreads, 0, stream>>>(
        sid[0], spos[0], n, per_merge, sid[1], spos[1]);
    from = 1;
    for (int64_t l = kRun * kLdsRuns; l < n; l *= kFan, from ^= 1)
      merge_runs_kernel<<<(unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, kMaxBlocks),
                          kThreads, 0, stream>>>(sid[from], spos[from], n, l, sid[from ^ 1],
                                                 spos[from ^ 1]);
  }
  auto sum = H % 8 == 0 ? (dtype == MDLM_BF16 ? run_sum<bf16_t, true> : run_sum<float, true>)
                        : (dtype == MDLM_BF16 ? run_sum<bf16_t, false> : run_sum<float, false>);
  sum(sid[from], spos[from], n, V, H, d_out, scale, d_table, accumulate, part, cut, stream);
  if (n > 2 * C) {  // shorter lists have no run that is cut
    // blocks that share the runs: a multiple of 4, up to 32
    const int64_t share = std::min<int64_t>(32, round_up(n / C, 64) / 16);
    const dim3 grid((unsigned)((H + 255) / 256), (unsigned)share);
    auto join = accumulate ? join_runs_kernel<true> : join_runs_kernel<false>;
    join<<<grid, kJoinThreads, 0, stream>>>(sid[from], n, V, H, C, scale, d_table, part,
                                            pitch_of(H), cut);
  }
  return hipGetLastError();
}

}  // namespace mdlm
