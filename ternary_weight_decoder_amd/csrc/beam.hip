// Beam selection: the W best of the W * V continuations of a group's beams.
//
// Within a beam the order of the candidates is that of its logits, so a beam
// contributes at most its W largest logits (ties: the lower token), and the
// log-softmax needs only its sum of exp.  One pass over the logits gives both;
// they are read once and nothing else is large, so the kernel is a stream with
// as little as possible beside it.  (The loads are non-temporal: without any
// selection or join the stream of 256 rows of 151,936 logits runs at 6.5 TB/s
// with them and at 5.8 without.)
//
// A workgroup takes one chunk of a row, 4096 logits at a time in registers.
// Each thread keeps its own running maximum and sum of exp.  A 64-bit key (the
// logit's bits in unsigned order, then the inverted token) makes candidates
// distinct.  A wave lists the keys that may be among its W largest: from the
// first tile those above a bound that W of its lanes' own largest keys reach,
// found from the top bits down with ballots, and no more than a few lanes do;
// from later tiles those above that bound, which rises where many would pass it.
// Nothing in the stream waits for another wave.  The chunk's W largest are then
// found among the waves' lists with a bound of the same kind, and by counting.
//
// The last chunk of a row to finish joins the row's chunks, and the last row of
// a group the rows, in the same way.  Partial results go through
// device-coherent accesses, and the counters that tell the last are left at
// zero.
//
// Measured (151,936 logits a row, inputs rotating, a launch in a graph): 32
// groups of 8 beams 39.6 us (139.5 MB, reads within 0.3% of it; waves wait 47% of
// their time; with a barrier and a ranking in every tile 44.2), one group of 4
// beams 11.8, one greedy row 8.5, of which a launch is 1.8.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"

namespace bitnet {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = kThreads / 64;
constexpr int kQuads = 4;                            // 16-byte loads per thread and tile
constexpr int kPer = 4 * kQuads;                     // logits per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int kMaxChunks = 64;                       // of a row
constexpr int kJoinPer = kMaxChunks * kMaxWidth / kThreads;
constexpr int kCounters = kMaxRows;                  // of rows; as many of groups behind them
constexpr int kHeaderBytes = 2 * 4 * kCounters;
// Workgroups before a workgroup takes more than one tile: four a compute unit.
// 256 rows of 151,936 logits: 39.6 us; 39.9 with 768, 44.4 with 1536, 46.8 with
// 2048.  One group of 32 such rows: 39 us, 55 with 1536 or more.
constexpr int kTargetGroups = 1024;
constexpr int kSimdWaves = 4;

typedef float f32x2 __attribute__((ext_vector_type(2)));
// Rows are only 4-byte aligned.
typedef float f32x4_row __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned long long u64;

// Chunks of a row, each of `tiles` tiles; whether a group's chunks are joined at
// once or by rows first; and the workspace: counters, then per
// row and chunk (max, sum) and W keys, then per row W scores and W keys.
constexpr int kNarrow = 8;            // widths of the smaller kernel
constexpr int kFlat = 640;            // candidates of a group that are joined at once
struct SelectPlan {
  int chunks, tiles, flat;
  int row_stride, group_stride;   // of the counters
  size_t stats, keys, scores, row_keys, total;
};
SelectPlan select_plan(int64_t rows, int64_t W, int64_t V) {
  SelectPlan p;
  const int64_t all = (V + kTile - 1) / kTile;
  int64_t chunks = std::min<int64_t>(std::min<int64_t>(all, kMaxChunks),
                                     (kTargetGroups + rows - 1) / rows);
  p.tiles = (int)((all + chunks - 1) / chunks);
  p.chunks = (int)((all + p.tiles - 1) / p.tiles);
  p.flat = W * W * p.chunks <= kFlat;
  // As far apart as there is room for, up to a cache line's 32: arrivals at
  // counters of one line wait for each other.  (16 greedy rows of 151,936 logits:
  // 11.9 us, 17.1 with the counters side by side.)
  p.row_stride = (int)std::min<int64_t>(32, kCounters / rows);
  p.group_stride = (int)std::min<int64_t>(32, kCounters / (rows / W));
  const size_t n = (size_t)rows * p.chunks;
  p.stats = kHeaderBytes;
  p.keys = p.stats + align256(n * 8);
  p.scores = p.keys + align256(n * W * 8);
  p.row_keys = p.scores + align256((size_t)rows * W * 8);
  p.total = p.row_keys + align256((size_t)rows * W * 8);
  return p;
}

__device__ __forceinline__ float clean(float x) {   // NaN and +inf count as -inf
  return x < INFINITY ? x : -INFINITY;
}
__device__ __forceinline__ u64 key_of(float x, uint32_t token) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);   // -0 as 0
  const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((u64)o << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float logit_of(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// exp2 of the difference of two maxima's exponents, m <= n, n > -inf.
__device__ __forceinline__ bool huge(float m) { return fabsf(m) > 0x1p126f; }
__device__ __forceinline__ float shift(float m, float n) {
  return __builtin_amdgcn_exp2f(huge(n) ? (m - n) * kLog2e : m * kLog2e - n * kLog2e);
}
__device__ __forceinline__ double exponent(float m) {
  return huge(m) ? (double)m * (double)kLog2e : (double)(m * kLog2e);
}
// The bits of a rounded score in unsigned order; above 0 (a score is never NaN).
__device__ __forceinline__ uint32_t order_of(double t) {
  return (uint32_t)(key_of((float)t, 0) >> 32);
}
__device__ __forceinline__ uint32_t token_of(u64 key) { return 0xffffffffu - (uint32_t)key; }

__device__ __forceinline__ void st_device(void *p, u64 v) {
  __hip_atomic_store((BITNET_GLOBAL u64 *)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 ld_device(const void *p) {
  return __hip_atomic_load((const BITNET_GLOBAL u64 *)p, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}

// A candidate of a group: its score and its key (which holds its token).
struct Entry {
  double score;
  u64 key;
};

// By the greatest width a kernel serves: room for the waves' lists (all of which may
// reach the bound of their join) and for a group's candidates (which may all tie).
template <int MAXW>
struct SelectShared {
  static constexpr int kEntries = MAXW == kMaxWidth ? kMaxWidth * kMaxWidth : kFlat;
  // A wave's list: what one tile can add, and what is left of a list that was cut.
  static constexpr int kList = 2 * MAXW * kPer;
  static constexpr int kPerLane = kList / 64;
  static_assert(MAXW * kPerLane + MAXW * kPer <= kList, "room for a tile's keys");
  static constexpr int kWords = std::max(2 * kEntries, kWaves * kList);
  __attribute__((aligned(16))) u64 cand[kWords];   // the waves' lists, then candidates
  u64 best[MAXW];                      // the W largest keys, in order
  double lse[MAXW];
  float from[MAXW];                    // scores of the group's beams, and their flags
  int flag[MAXW];
  u64 bound[kWaves];
  float m[kWaves], s[kWaves];
  uint32_t count, last;
  int winner[MAXW];
  uint8_t beam[kEntries];              // of the entries
};

// The largest prefix v of bits, from the top two at a time, that the keys of W
// lanes reach, until no more than `most` lanes do; `at` lanes do in the end, `above`
// of those counted elsewhere.
__device__ __forceinline__ uint32_t bound_bits(uint32_t key, bool in, int above, int W, int most,
                                               int *at) {
  uint32_t v = 0;
#pragma unroll 1
  for (int top = 30; top >= 0 && *at > most; top -= 4)
#pragma unroll
    for (int b = 0; b < 4; b += 2) {
      uint32_t t[3];
      int n[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        t[q] = v | ((uint32_t)(q + 1) << (top - b));
        n[q] = above + __builtin_popcountll(__ballot(in && key >= t[q]));
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        v = n[q] >= W ? t[q] : v;
        *at = n[q] >= W ? n[q] : *at;
      }
    }
  return v;
}
// Maximum over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(p[0], p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(q[0], q[1]);
}
// The W-th largest key of the lanes (0 where fewer have one), one maximum after the
// other.
__device__ __forceinline__ uint32_t bound_of_max(uint32_t key, int W) {
  uint32_t b = 0;
  for (int n = 0; n < W;) {
    const uint32_t m = __builtin_amdgcn_readfirstlane(wave_max(key));
    if (m == 0) return 0;
    b = m;
    n += __builtin_popcountll(__ballot(key == m));
    key = key == m ? 0 : key;
  }
  return b;
}
// A bound that the keys of W lanes reach, and no more than `most` >= W lanes'
// unless keys are equal; 0 where no more than `most` have a key (or fewer than W).
// One maximum after the other up to kSerial, else by bits.  (One greedy row: 8.5
// us, by bits 9.9; groups of 8 beams: 39.5 by bits, 41.0 by eight maxima.)
constexpr int kSerial = 4;
__device__ __forceinline__ uint32_t bound_32(uint32_t key, int W, int most, int *at) {
  if (W <= kSerial) {
    const uint32_t v = bound_of_max(key, W);
    *at = __builtin_popcountll(__ballot(key != 0 && key >= v));
    return v;
  }
  *at = __builtin_popcountll(__ballot(key != 0));
  return bound_bits(key, true, 0, W, most, at);
}
// The same of keys that differ.
__device__ __forceinline__ u64 wave_bound(u64 key, int W, int most) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  int at;
  const uint32_t v = bound_32(hi, W, most, &at);
  uint32_t low = 0;
  if (v != 0 && at > most)   // lanes share the value
    low = bound_bits(lo, hi == v, __builtin_popcountll(__ballot(hi > v)), W, most, &at);
  return ((u64)v << 32) | low;
}

// sh.best becomes the W largest, in order, of the threads' keys: key(j), j < N <=
// kPer, 0 for none; `mine` is the thread's largest.  Every thread calls it, with
// the workgroup in step, and has its keys in registers.
template <int N, int MAXW, typename Key>
__device__ __forceinline__ void select_largest(SelectShared<MAXW> &sh, int W, u64 mine, Key key) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const u64 b = wave_bound(mine, W, MAXW);
  if (lane == 0) sh.bound[wave] = b;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  u64 bound = 1;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) bound = sh.bound[w] > bound ? sh.bound[w] : bound;
  if (mine >= bound)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const u64 k = key(j);
      if (k >= bound) sh.cand[atomicAdd(&sh.count, 1u)] = k;
    }
  __syncthreads();
  const int all = sh.count;
  for (int i = tid; i < all; i += kThreads) {
    const u64 k = sh.cand[i];
    int r = 0;
#pragma unroll 4
    for (int c = 0; c < all; ++c) r += sh.cand[c] > k ? 1 : 0;
    if (r < W) sh.best[r] = k;
  }
  if (tid >= all && tid < W) sh.best[tid] = 0;
  __syncthreads();
}

// Counts one more arrival; true for the last of n, which leaves zero behind.
// Each wave's device-coherent stores are acknowledged before.
template <int MAXW>
__device__ __forceinline__ bool arrive(SelectShared<MAXW> &sh, uint32_t *counter, int n) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t at =
        __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sh.last = at == (uint32_t)n - 1;
    if (sh.last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return sh.last != 0;
}

// A row's sum of exp from its chunks' (max, sum), a lane each: (exponent, sum).
__device__ __forceinline__ void join_sums(f32x2 st, double *e, double *sum) {
  const float top = across16<true>(across4(st.x));
  *e = exponent(top);
  *sum = wave_total(st.x > -INFINITY ? (double)st.y * (double)shift(st.x, top) : 0.0);
}
__device__ __forceinline__ double log_sum(double e, double sum) {
  return sum > 0.0 ? (e + log2(sum)) / (double)kLog2e : 0.0;
}

// The W best of the group's candidates, this thread's being score, key and beam
// [j], j < N, where the key is not 0; ordered by score, then the lower beam, then
// the larger key.  A bound that W scores reach, both rounded to fp32 (which keeps
// the order: whatever is below it is below W others), then ranks by counting among
// those that do.  Ends with winner r in sh.winner[r].
template <int N, int MAXW>
__device__ __forceinline__ void select_group(SelectShared<MAXW> &sh, int W,
                                             const double (&score)[N], const u64 (&key)[N],
                                             const int (&beam)[N]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Entry *list = reinterpret_cast<Entry *>(sh.cand);
  uint32_t mine = 0, order[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    order[j] = key[j] != 0 ? order_of(score[j]) : 0;
    mine = max(mine, order[j]);
  }
  int at;
  const uint32_t b = bound_32(mine, W, W, &at);
  if (lane == 0) sh.bound[wave] = b;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  u64 bound = 1;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) bound = sh.bound[w] > bound ? sh.bound[w] : bound;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (order[j] >= bound) {
      const uint32_t at = atomicAdd(&sh.count, 1u);
      list[at] = Entry{score[j], key[j]};
      sh.beam[at] = (uint8_t)beam[j];
    }
  __syncthreads();
  const int all = sh.count;
  for (int i = tid; i < all; i += kThreads) {
    const Entry e = list[i];
    const int w = sh.beam[i];
    int r = 0;
#pragma unroll 4
    for (int c = 0; c < all; ++c) {
      const Entry u = list[c];
      bool before = u.score > e.score;
      if (u.score == e.score) before = sh.beam[c] != w ? sh.beam[c] < w : u.key > e.key;
      r += before ? 1 : 0;
    }
    if (r < W) sh.winner[r] = i;
  }
  __syncthreads();
}

template <int MAXW>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(kSimdWaves)))
select_kernel(SelectArgs a, SelectPlan p) {
  __shared__ SelectShared<MAXW> sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x, row = blockIdx.y, W = a.W;
  const bool finished = a.finished_in && a.finished_in[row] != 0;
  uint32_t *counters = reinterpret_cast<uint32_t *>(a.ws);
  f32x2 *stats = reinterpret_cast<f32x2 *>(a.ws + p.stats) + (int64_t)row * p.chunks;
  u64 *keys = reinterpret_cast<u64 *>(a.ws + p.keys) + (int64_t)row * p.chunks * W;
  u64 *scores = reinterpret_cast<u64 *>(a.ws + p.scores);
  u64 *row_keys = reinterpret_cast<u64 *>(a.ws + p.row_keys);

  if (!finished) {
    const float *x = a.logits + row * a.ld;
    const int64_t i0 = (int64_t)chunk * p.tiles * kTile + 4 * tid;
    const int64_t stop = min((int64_t)a.V, (int64_t)(chunk + 1) * p.tiles * kTile);
    f32x4 next[kQuads];
    // The last tile of a row checks every logit; the others go out together and
    // stay in flight while the tile before them is worked on.
    auto load = [&](int64_t at) {
      const int64_t last = at - 4 * tid + kTile;
      if (last <= stop) {
#pragma unroll
        for (int j = 0; j < kQuads; ++j)
          next[j] = __builtin_nontemporal_load(
              (const BITNET_GLOBAL f32x4_row *)(x + at + j * 4 * kThreads));
      } else {
#pragma unroll
        for (int j = 0; j < kQuads; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t i = at + j * 4 * kThreads + e;
            next[j][e] = i < stop ? ld_global<float>(x + i) : NAN;
          }
      }
    };
    load(i0);
    // The wave's list: every key of its W largest so far, and others, all from
    // `least`, which W of them reach once there are more than a few.
    typedef SelectShared<MAXW> Shared;
    u64 *list = sh.cand + wave * Shared::kList;
    u64 least = 1;
    float least_logit = -INFINITY;
    int listed = 0;
    auto add = [&](bool in, u64 k) {
      const u64 m = __ballot(in);
      if (in) list[listed + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                                      __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] = k;
      listed += __builtin_popcountll(m);
    };
    auto cut = [&]() {   // down to the keys of few lanes, W of which are largest
      u64 k[Shared::kPerLane], mine = 0;
#pragma unroll
      for (int j = 0; j < Shared::kPerLane; ++j) {
        k[j] = lane + 64 * j < listed ? list[lane + 64 * j] : 0;
        mine = k[j] > mine ? k[j] : mine;
      }
      __builtin_amdgcn_wave_barrier();
      const u64 b = wave_bound(mine, W, MAXW);
      least = b > least ? b : least;
      least_logit = logit_of(least);
      listed = 0;
#pragma unroll
      for (int j = 0; j < Shared::kPerLane; ++j) add(k[j] >= least, k[j]);
      __builtin_amdgcn_wave_barrier();
    };
    // Sum of exp(x - m), m the running maximum, as exp2(x c - fl(m c)): one fma
    // and one exp2 a logit, and since the join takes the same fl(m c), its
    // rounding cancels.  (Where m c would overflow: exp2((x - m) c).)
    float m = -INFINITY, s = 0.0f;
    for (int tile = 0; tile < p.tiles; ++tile) {
      const int64_t at = i0 + (int64_t)tile * kTile;
      // (Held back: the compiler would otherwise move the first use of each logit
      // up behind its load, into the tile before, and wait for it there.)
#pragma unroll
      for (int j = 0; j < kQuads; ++j) asm volatile("" : "+v"(next[j]));
      float v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = fmaxf(next[j >> 2][j & 3], -INFINITY);   // NaN: -inf
      if (tile + 1 < p.tiles) load(at + kTile);
      float top = v[0];
#pragma unroll
      for (int j = 1; j < kPer; ++j) top = fmaxf(top, v[j]);
      if (__any(top == INFINITY)) {
        top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kPer; ++j) top = fmaxf(top, v[j] = clean(v[j]));
      }
      const float m_new = fmaxf(m, top);
      if (m_new > -INFINITY) {
        float e[kPer];
        const float mc = m_new * kLog2e;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[j], kLog2e, -mc));
        if (huge(m_new))
#pragma unroll
          for (int j = 0; j < kPer; ++j) e[j] = __builtin_amdgcn_exp2f((v[j] - m_new) * kLog2e);
#pragma unroll
        for (int d = kPer / 2; d > 0; d >>= 1)
#pragma unroll
          for (int j = 0; j < d; ++j) e[j] += e[j + d];
        s = s * shift(m, m_new) + e[0];
        m = m_new;
      }
      // Keys that may be among the chunk's W largest go to the wave's list.
      if (!__any(top >= least_logit)) continue;
      auto token = [&](int j) { return at + (j >> 2) * 4 * kThreads + (j & 3); };
      int where = kPer - 1;   // ties: the first of the thread's, which has the lowest token
#pragma unroll
      for (int j = kPer - 2; j >= 0; --j) where = v[j] == top ? j : where;
      const u64 mine = at < stop ? key_of(top, (uint32_t)token(where)) : 0;
      const int above = __builtin_popcountll(__ballot(mine >= least));
      if (above == 0) continue;
      if (above > MAXW) {
        least = wave_bound(mine, W, MAXW);
        least_logit = logit_of(least);
      }
      if (listed + MAXW * kPer > Shared::kList) cut();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (__any(v[j] >= least_logit)) {
          const u64 k = token(j) < stop ? key_of(v[j], (uint32_t)token(j)) : 0;
          add(k >= least, k);
        }
    }
    {
      u64 k[Shared::kPerLane], mine = 0;
#pragma unroll
      for (int j = 0; j < Shared::kPerLane; ++j) {
        k[j] = lane + 64 * j < listed ? list[lane + 64 * j] : 0;
        mine = k[j] > mine ? k[j] : mine;
      }
      select_largest<Shared::kPerLane>(sh, W, mine, [&](int j) { return k[j]; });
    }
    // The chunk's maximum and sum.
    const float top = across16<true>(across4(m));
    if (lane == 0) sh.m[wave] = top;
    __syncthreads();
    float all = sh.m[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) all = fmaxf(all, sh.m[w]);
    s = all > -INFINITY ? s * shift(m, all) : 0.0f;
    s = across16<false>(sum4(s));
    if (lane == 0) sh.s[wave] = s;
    __syncthreads();
    if (tid < W) st_device(keys + chunk * W + tid, sh.best[tid]);
    if (tid == 0)
      st_device(stats + chunk,
                __builtin_bit_cast(u64, f32x2{all, (sh.s[0] + sh.s[1]) + (sh.s[2] + sh.s[3])}));
  }
  const int beam = row % W, g0 = row - beam;
  uint32_t *group = counters + kCounters + row / W * p.group_stride;
  // A finished beam's candidates: eos at the unchanged score, then the other
  // tokens from the lowest.
  auto finished_key = [&](int i) {
    return i == 0 ? key_of(1.0f, (uint32_t)a.eos)
                  : key_of(0.0f, (uint32_t)(i - 1 < a.eos ? i - 1 : i));
  };

  if (p.flat) {
    if (!arrive(sh, group, W * p.chunks)) return;
    // Everything is asked for at once: keys, flags, scores, and a wave per row
    // its sums.
    constexpr int kN = (kFlat + kThreads - 1) / kThreads;
    constexpr int kRows = (MAXW + kWaves - 1) / kWaves;
    const int each = p.chunks * W;
    const float per_each = __builtin_amdgcn_rcpf((float)each);
    const u64 *all_keys = reinterpret_cast<const u64 *>(a.ws + p.keys) + (int64_t)g0 * each;
    u64 k[kN];
    int of[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int i = tid + j * kThreads;
      k[j] = i < W * each ? ld_device(all_keys + i) : 0;
      of[j] = i < W * each ? (int)(((float)i + 0.5f) * per_each) : 0;   // exact: i < 2^10
    }
    if (tid < W) {
      sh.from[tid] = clean(a.scores_in[g0 + tid]);
      sh.flag[tid] = a.finished_in && a.finished_in[g0 + tid] != 0;
    }
    double exps = 0.0, sums = 0.0;   // of row wave + kWaves * lane
    f32x2 st[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int w = wave + r * kWaves;
      st[r] = f32x2{-INFINITY, 0.0f};
      if (w < W && lane < p.chunks)
        st[r] = __builtin_bit_cast(
            f32x2, ld_device(reinterpret_cast<f32x2 *>(a.ws + p.stats) +
                             (int64_t)(g0 + w) * p.chunks + lane));
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      double e, sum;
      join_sums(st[r], &e, &sum);
      exps = lane == r ? e : exps;
      sums = lane == r ? sum : sums;
    }
    const double v = log_sum(exps, sums);
    if (lane < kRows && wave + lane * kWaves < W) sh.lse[wave + lane * kWaves] = v;
    __syncthreads();
    double score[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int i = tid + j * kThreads;
      const double base = (double)sh.from[of[j]];
      if (sh.flag[of[j]] != 0) {
        const int place = i - of[j] * each;
        k[j] = i < W * each && place < W ? finished_key(place) : 0;
        score[j] = place == 0 ? base : (double)-INFINITY;
      } else {
        score[j] = base + ((double)logit_of(k[j]) - sh.lse[of[j]]);
      }
    }
    select_group<kN>(sh, W, score, k, of);
  } else {
    if (!arrive(sh, counters + row * p.row_stride, p.chunks)) return;
    // The row: its W largest keys and their scores.
    const double base = (double)clean(a.scores_in[row]);
    if (finished) {
      if (tid < W) {
        st_device(scores + (int64_t)row * W + tid,
                  __builtin_bit_cast(u64, tid == 0 ? base : (double)-INFINITY));
        st_device(row_keys + (int64_t)row * W + tid, finished_key(tid));
      }
    } else {
      f32x2 st = {-INFINITY, 0.0f};
      if (tid < p.chunks) st = __builtin_bit_cast(f32x2, ld_device(stats + tid));
      const int n = p.chunks * W;
      u64 k[kJoinPer];
      u64 mine = 0;
#pragma unroll
      for (int j = 0; j < kJoinPer; ++j) {
        const int i = tid + j * kThreads;
        k[j] = i < n ? ld_device(keys + i) : 0;
        mine = k[j] > mine ? k[j] : mine;
      }
      if (wave == 0) {   // the chunks are lanes of the first wave
        double e, sum;
        join_sums(st, &e, &sum);
        const double v = log_sum(e, sum);
        if (lane == 0) sh.lse[0] = v;
      }
      select_largest<kJoinPer>(sh, W, mine, [&](int j) { return k[j]; });
      if (tid < W) {
        const u64 key = sh.best[tid];
        const double t = base + ((double)logit_of(key) - sh.lse[0]);
        st_device(scores + (int64_t)row * W + tid, __builtin_bit_cast(u64, t));
        st_device(row_keys + (int64_t)row * W + tid, key);
      }
    }
    if (!arrive(sh, group, W)) return;
    constexpr int kN = (MAXW * MAXW + kThreads - 1) / kThreads;
    double score[kN];
    u64 k[kN];
    int of[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int i = tid + j * kThreads;
      score[j] = 0.0;
      k[j] = 0;
      of[j] = 0;
      if (i < W * W) {
        score[j] = __builtin_bit_cast(double, ld_device(scores + (int64_t)g0 * W + i));
        k[j] = ld_device(row_keys + (int64_t)g0 * W + i);
        of[j] = i / W;
      }
    }
    select_group<kN>(sh, W, score, k, of);
  }

  // finished_out may be finished_in, scores_out scores_in: every row of the
  // group has read its own, and here flags are read before any is written.
  int fin = 0, from_beam = 0;
  Entry e = {0.0, 0};
  if (tid < W) {
    e = reinterpret_cast<const Entry *>(sh.cand)[sh.winner[tid]];
    from_beam = sh.beam[sh.winner[tid]];
    if (a.finished_in) fin = a.finished_in[g0 + from_beam] != 0;
  }
  __syncthreads();
  if (tid < W) {
    const int o = g0 + tid;
    const int token = (int)token_of(e.key);
    a.scores_out[o] = (float)e.score;
    a.tokens[o] = token;
    a.parents[o] = g0 + from_beam;
    if (a.finished_in) a.finished_out[o] = fin || token == a.eos;
  }
}

}  // namespace

size_t select_workspace_bytes(int64_t B, int64_t W, int64_t V) {
  return select_plan(B * W, W, V).total;
}

hipError_t launch_beam_select(const SelectArgs &a, hipStream_t stream) {
  const SelectPlan p = select_plan((int64_t)a.B * a.W, a.W, a.V);
  const dim3 grid(p.chunks, a.B * a.W);
  if (a.W <= kNarrow)
    select_kernel<kNarrow><<<grid, kThreads, 0, stream>>>(a, p);
  else
    select_kernel<kMaxWidth><<<grid, kThreads, 0, stream>>>(a, p);
  return hipGetLastError();
}

}  // namespace bitnet
