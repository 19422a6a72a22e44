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
// table row's terms lie side by side and are summed in ascending position by
// one wave per 512 columns: no atomics, and the same bits on every run.
// Absorbing corruption makes about half of all tokens one id (the mask), so
// the sorted list holds one run of n/2 among runs of one or two: the list is
// cut into chunks of C entries, runs longer than a chunk are summed chunk by
// chunk into partial rows, and a last kernel adds those in order.
#include "row_ops.h"

#include <algorithm>

namespace mdlm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int64_t kMaxBlocks = 1 << 20;

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

constexpr int kTile = 1024;  // tokens sorted by one block
constexpr int kFan = 16;     // sorted runs merged at a time

// Sorts each tile of 1,024 tokens by (id, position); an id outside [0, V)
// counts as V and so comes last.  The blocks past the tiles clear `fill`
// (fill_words 16-byte words and the odd words behind them), which needs no
// order with the sorting and hides it.
__global__ void __launch_bounds__(kThreads)
sort_tiles_kernel(const int32_t* __restrict__ ids, int64_t n, int32_t V,
                  int32_t* __restrict__ sid, int32_t* __restrict__ spos, int32_t tiles,
                  float* __restrict__ fill, int64_t fill_n) {
  if ((int)blockIdx.x >= tiles) {
    const int64_t n4 = fill_n / 4;
    const int64_t stride = (int64_t)(gridDim.x - tiles) * kThreads;
    const f32x4_a4 zero = {0.f, 0.f, 0.f, 0.f};
    const int64_t t = (int64_t)(blockIdx.x - tiles) * kThreads + threadIdx.x;
    for (int64_t i = t; i < n4; i += stride) reinterpret_cast<f32x4_a4*>(fill)[i] = zero;
    if (t < fill_n - 4 * n4) fill[4 * n4 + t] = 0.f;
    return;
  }
  __shared__ uint64_t key[kTile];
  const int64_t base = (int64_t)blockIdx.x * kTile;
  for (int i = threadIdx.x; i < kTile; i += kThreads) {
    uint64_t k = ~(uint64_t)0;
    if (base + i < n) {
      const int32_t id = ids[base + i];
      k = (uint64_t)((uint32_t)id < (uint32_t)V ? id : V) << 32 | (uint32_t)i;
    }
    key[i] = k;
  }
  // bitonic network: 55 steps of 512 compare-exchanges
  for (int size = 2; size <= kTile; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kTile / 2 / kThreads; ++u) {
        const int t = threadIdx.x + u * kThreads;
        const int a = 2 * t - (t & (stride - 1)), b = a + stride;
        const uint64_t x = key[a], y = key[b];
        if ((x > y) == ((a & size) == 0)) key[a] = y, key[b] = x;
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kTile && base + i < n; i += kThreads) {
    sid[base + i] = (int32_t)(key[i] >> 32);
    spos[base + i] = (int32_t)(base + (uint32_t)key[i]);
  }
}

// Merges up to kFan sorted runs of `len` entries into one: an entry's place
// is its place in its run plus, for each other run, the number of that run's
// entries before it (equal ids of an earlier run come first, positions
// ascending with the runs).  One thread per entry; its searches are
// independent of one another, so they run side by side.
__global__ void __launch_bounds__(kThreads)
merge_runs_kernel(const int32_t* __restrict__ sid, const int32_t* __restrict__ spos, int64_t n,
                  int64_t len, int32_t* __restrict__ out_id, int32_t* __restrict__ out_pos) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += stride) {
    const int64_t run = i / len, group = run / kFan * kFan;
    const int32_t id = sid[i];
    int64_t rank = i - run * len;
    uint32_t lo[kFan], hi[kFan];  // n < 2^31
#pragma unroll
    for (int r = 0; r < kFan; ++r) {
      const int64_t b = (group + r) * len;
      lo[r] = (uint32_t)(b < n ? b : n);
      hi[r] = (uint32_t)(b + len < n ? b + len : n);
      if (group + r == run) hi[r] = lo[r];
    }
    // a search over len entries ends after log2(len) + 1 halvings
    for (int64_t span = len; span > 0; span >>= 1) {
#pragma unroll
      for (int r = 0; r < kFan; ++r)
        if (lo[r] < hi[r]) {
          const uint32_t mid = (lo[r] + hi[r]) >> 1;
          const int32_t v = sid[mid];
          if (v < id || (v == id && group + r < run))
            lo[r] = mid + 1;
          else
            hi[r] = mid;
        }
    }
#pragma unroll
    for (int r = 0; r < kFan; ++r)
      if (group + r != run) {
        const int64_t b = (group + r) * len;
        rank += lo[r] - (b < n ? b : n);
      }
    out_id[group * len + rank] = id;
    out_pos[group * len + rank] = spos[i];
  }
}

// ---- summing the runs --------------------------------------------------------

// A run of equal ids that starts in chunk c belongs to chunk c's wave when it
// ends in chunk c or c + 1; a longer one is cut at the chunk borders: chunk
// c's part goes to slot 1 of its partial rows, every later chunk's to slot 0.

// Number of lanes from lane 0 on for which `p` holds without a gap.
__device__ __forceinline__ int leading(bool p) {
  const uint64_t b = ~__ballot(p);
  return b ? __ffsll((unsigned long long)b) - 1 : 64;
}

// One wave sums 512 columns of one chunk's runs (C <= 64 entries, and the
// part of its last run that lies in the next chunk).
template <typename T, bool FULL, bool ACC>
__global__ void __launch_bounds__(kThreads)
sum_runs_kernel(const int32_t* __restrict__ sid, const int32_t* __restrict__ spos, int64_t n,
                int32_t V, int32_t H, int32_t C, int32_t slabs, int64_t units,
                const T* __restrict__ d_out, float scale, float* __restrict__ d_table,
                float* __restrict__ part, int64_t part_pitch) {
  constexpr int kBatch = 8;  // rows in flight
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < units;
       u += (int64_t)gridDim.x * kWaves) {
    const int64_t chunk = u / slabs;
    const int c = (int)(u - chunk * slabs) * 512 + 8 * lane;
    int64_t e = chunk * C;
    int64_t end = e + C < n ? e + C : n;
    const int32_t first = sid[e], last = sid[end - 1];
    bool head = false, tail = false;  // the first / last run goes to a slot
    const bool before = e > 0 && sid[e - 1] == first;
    const bool through = before && last == first;
    // (everything read below as sid[...] past `end` is checked against n)
    if (end < n && sid[end] == last && !through) {
      if (end + C >= n || sid[end + C] != last)
        end += leading(lane < C && end + lane < n && sid[end + lane < n ? end + lane : 0] == last);
      else
        tail = true;
    }
    if (before) {
      const bool starts_in_prev = e <= C || sid[e - C - 1] != first;
      const bool ends_here = e + C >= n || sid[e + C] != first;
      if (starts_in_prev && ends_here)
        e += leading(lane < C && e + lane < n && sid[e + lane < n ? e + lane : 0] == first);
      else
        head = true;
    }
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (; e < end; e += 64) {
      // 64 entries of the list, one per lane
      const int64_t at = e + lane;
      const int32_t id = at < end ? sid[at] : V;
      const int32_t pos = at < end ? spos[at] : 0;
      const int cnt = leading(id < V);
      if (cnt == 0) break;
      const uint64_t ends =
          __ballot(at < end && (at + 1 >= end || sid[at + 1 < n ? at + 1 : at] != id));
      for (int j = 0; j < cnt; j += kBatch) {
        Raw8<T> r[kBatch];
        Raw8<float> old[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (j + k < cnt) {
            const int32_t p = __builtin_amdgcn_readlane(pos, j + k);
            r[k] = load8<FULL>(d_out + (int64_t)p * H, c, H);
            if (ACC && (ends >> (j + k) & 1))
              old[k] = load8<FULL>(
                  d_table + (int64_t)__builtin_amdgcn_readlane(id, j + k) * H, c, H);
          }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (j + k < cnt) {
            float v[8];
            widen(r[k], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += v[i];
            if (ends >> (j + k) & 1) {
              const int slot = head ? 0 : (tail && e + j + k + 1 >= end ? 1 : -1);
              head = false;
              if (slot >= 0) {
                store8<true>(part + (2 * chunk + slot) * part_pitch, c, (int)part_pitch, acc);
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  acc[i] = ACC ? old[k].w[i] + scale * acc[i] : scale * acc[i];
                store8<FULL>(d_table + (int64_t)__builtin_amdgcn_readlane(id, j + k) * H, c, H,
                             acc);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) acc[i] = 0.f;
            }
          }
      }
      if (cnt < 64) break;
    }
  }
}

// Adds the partial rows of each run that was cut: 16 waves share its chunks,
// 256 columns per block, and one thread per column adds the waves' sums in
// order.  Blocks along y take the cut runs in turn.
constexpr int kJoinThreads = 1024;
constexpr int kJoinWaves = kJoinThreads / 64;

template <bool ACC>
__global__ void __launch_bounds__(kJoinThreads)
join_runs_kernel(const int32_t* __restrict__ sid, int64_t n, int32_t V, int32_t H, int32_t C,
                 float scale, float* __restrict__ d_table, const float* __restrict__ part,
                 int64_t part_pitch) {
  __shared__ int32_t s_owner[kJoinThreads];
  __shared__ int32_t s_count[kJoinWaves];
  __shared__ float s_sum[kJoinWaves][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x * 256 + 4 * lane;
  const int64_t chunks = (n + C - 1) / C;
  int64_t seen = 0;  // cut runs found before this round
  for (int64_t base = 0; base < chunks; base += kJoinThreads) {
    const int64_t m = base + tid;
    bool own = false;
    if (m < chunks) {
      const int64_t e0 = m * C, e1 = e0 + C;
      if (e1 + C < n) {
        const int32_t l = sid[e1 - 1];
        own = l < V && sid[e1] == l && sid[e1 + C] == l && (e0 == 0 || sid[e0 - 1] != l);
      }
    }
    const uint64_t mask = __ballot(own);
    if (lane == 0) s_count[wave] = __popcll(mask);
    __syncthreads();
    int at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) {
      if (w < wave) at += s_count[w];
      total += s_count[w];
    }
    if (own) s_owner[at + __popcll(mask & (((uint64_t)1 << lane) - 1))] = (int32_t)m;
    __syncthreads();
    // this block's share: cut runs whose number is blockIdx.y modulo gridDim.y
    int first = (int)((blockIdx.y + gridDim.y - seen % gridDim.y) % gridDim.y);
    for (int o = first; o < total; o += gridDim.y) {
      const int64_t m0 = s_owner[o];
      const int32_t id = sid[(m0 + 1) * C];
      // the run's last chunk: the chunk before the first one that starts past it
      int64_t lo = m0 + 2, hi = chunks;
      while (lo < hi) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t probe = lo + step * lane;
        const int k = leading(probe < hi && sid[(probe < hi ? probe : lo) * C] == id);
        // chunks lo, lo + step, .. (k of them) start inside the run
        if (k == 0) break;
        hi = lo + step * k < hi ? lo + step * k : hi;
        lo = lo + step * (k - 1) + 1;
      }
      const int64_t parts = lo - m0;  // chunks m0 .. lo - 1
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < part_pitch) {
#pragma unroll 8
        for (int64_t i = wave; i < parts; i += kJoinWaves) {
          const float4 v = *reinterpret_cast<const float4*>(
              part + (2 * (m0 + i) + (i == 0 ? 1 : 0)) * part_pitch + c);
          acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
      }
      *reinterpret_cast<float4*>(&s_sum[wave][4 * lane]) = acc;
      __syncthreads();
      const int col = blockIdx.x * 256 + tid;
      if (tid < 256 && col < H) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWaves; ++w) s += s_sum[w][tid];
        float* d = d_table + (int64_t)id * H + col;
        *d = ACC ? *d + scale * s : scale * s;
      }
      __syncthreads();
    }
    seen += total;
  }
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Entries of the sorted list per chunk.
int chunk_of(int64_t n) { return n <= 16384 ? 16 : 64; }

int64_t pitch_of(int32_t H) { return round_up(H, 8); }

template <typename T, bool FULL>
void run_sum(const int32_t* sid, const int32_t* spos, int64_t n, int32_t V, int32_t H,
             const T* d_out, float scale, float* d_table, bool accumulate, float* part,
             hipStream_t stream) {
  const int C = chunk_of(n);
  const int slabs = (H + 511) / 512;
  const int64_t units = (n + C - 1) / C * slabs;
  const unsigned grid = (unsigned)std::min<int64_t>((units + kWaves - 1) / kWaves, kMaxBlocks);
  if (accumulate)
    sum_runs_kernel<T, FULL, true><<<grid, kThreads, 0, stream>>>(
        sid, spos, n, V, H, C, slabs, units, d_out, scale, d_table, part, pitch_of(H));
  else
    sum_runs_kernel<T, FULL, false><<<grid, kThreads, 0, stream>>>(
        sid, spos, n, V, H, C, slabs, units, d_out, scale, d_table, part, pitch_of(H));
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
// then two partial rows per chunk.
size_t embed_grad_workspace_bytes(int64_t n, int32_t H) {
  if (n <= 0 || H <= 0) return 0;
  const int C = chunk_of(n);
  return (size_t)(4 * round_up(4 * n, 256) + (n + C - 1) / C * 2 * pitch_of(H) * 4);
}

hipError_t launch_embed_grad(const int32_t* ids, int64_t n, const void* d_out, int32_t dtype,
                             int32_t V, int32_t H, float scale, float* d_table, bool accumulate,
                             void* workspace, hipStream_t stream) {
  const int64_t fill_n = accumulate ? 0 : (int64_t)V * H;
  if (n == 0 && fill_n == 0) return hipSuccess;
  char* ws = reinterpret_cast<char*>(workspace);
  const int64_t list = round_up(4 * n, 256);
  int32_t* sid[2] = {reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + 2 * list)};
  int32_t* spos[2] = {reinterpret_cast<int32_t*>(ws + list),
                      reinterpret_cast<int32_t*>(ws + 3 * list)};
  float* part = reinterpret_cast<float*>(ws + 4 * list);
  const int64_t tiles = (n + kTile - 1) / kTile;
  const int64_t fill_blocks =
      std::min<int64_t>((fill_n / 4 + kThreads) / kThreads, fill_n ? 8192 : 0);
  sort_tiles_kernel<<<(unsigned)(tiles + fill_blocks), kThreads, 0, stream>>>(
      ids, n, V, sid[0], spos[0], (int32_t)tiles, d_table, fill_n);
  if (n > 0) {
    int from = 0;
    for (int64_t len = kTile; len < n; len *= kFan, from ^= 1)
      merge_runs_kernel<<<(unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, kMaxBlocks),
                          kThreads, 0, stream>>>(sid[from], spos[from], n, len, sid[from ^ 1],
                                                 spos[from ^ 1]);
    const bool full = H % 8 == 0;
    if (dtype == MDLM_BF16) {
      const bf16_t* g = reinterpret_cast<const bf16_t*>(d_out);
      full ? run_sum<bf16_t, true>(sid[from], spos[from], n, V, H, g, scale, d_table, accumulate,
                                   part, stream)
           : run_sum<bf16_t, false>(sid[from], spos[from], n, V, H, g, scale, d_table, accumulate,
                                    part, stream);
    } else {
      const float* g = reinterpret_cast<const float*>(d_out);
      full ? run_sum<float, true>(sid[from], spos[from], n, V, H, g, scale, d_table, accumulate,
                                  part, stream)
           : run_sum<float, false>(sid[from], spos[from], n, V, H, g, scale, d_table, accumulate,
                                   part, stream);
    }
    const int C = chunk_of(n);
    if (n > 2 * C) {  // shorter lists have no run that is cut
      const dim3 grid((unsigned)((H + 255) / 256),
                      (unsigned)std::min<int64_t>((n + C - 1) / C, 32));
      if (accumulate)
        join_runs_kernel<true><<<grid, kJoinThreads, 0, stream>>>(sid[from], n, V, H, C, scale,
                                                                  d_table, part, pitch_of(H));
      else
        join_runs_kernel<false><<<grid, kJoinThreads, 0, stream>>>(sid[from], n, V, H, C, scale,
                                                                   d_table, part, pitch_of(H));
    }
  }
  return hipGetLastError();
}

}  // namespace mdlm
