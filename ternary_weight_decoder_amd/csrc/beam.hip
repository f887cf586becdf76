// Beam selection: the W best of the W * V continuations of a group's beams.
//
// Within a beam the order of the candidates is that of its logits, so a beam
// contributes at most its W largest logits (ties: the lower token), and the
// log-softmax needs only its sum of exp.  One pass over the logits gives both;
// they are read once and nothing else is large, so the kernel is a stream with
// as little as possible beside it.
//
// A workgroup takes one chunk of a row, 4096 logits at a time in registers.
// Each thread keeps its own running maximum and sum of exp.  A 64-bit key (the
// logit's bits in unsigned order, then the inverted token) makes candidates
// distinct.  For the chunk's W largest keys every wave finds a bound that W of
// its lanes' own largest keys reach, bit by bit with ballots; no more than W
// lanes of any wave reach the largest of the waves' bounds, so the keys that do
// are few, and are ranked by counting.  Later tiles of the chunk start from the
// W-th largest so far and mostly end there.
//
// The last chunk of a row to finish joins the row's chunks, and the last row of
// a group the rows, in the same way.  Partial results go through
// device-coherent accesses, and the counters that tell the last are left at
// zero.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"

namespace bitnet {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kQuads = 4;                            // 16-byte loads per thread and tile
constexpr int kPer = 4 * kQuads;                     // logits per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int kMaxChunks = 64;                       // of a row
constexpr int kJoinPer = kMaxChunks * kMaxWidth / kThreads;
constexpr int kRowCounters = kMaxRows;               // then one counter per group
constexpr int kHeaderBytes = 2 * 4 * kMaxRows;
// Workgroups wanted before a workgroup takes more than one tile: two rounds of
// eight a compute unit (256 rows of 151,936 logits: see below).
#ifndef BITNET_SELECT_GROUPS
#define BITNET_SELECT_GROUPS 2048
#endif
constexpr int kTargetGroups = BITNET_SELECT_GROUPS;

typedef float f32x2 __attribute__((ext_vector_type(2)));
// Rows are only 4-byte aligned.
typedef float f32x4_row __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned long long u64;

// Chunks of a row, each of `tiles` tiles; whether a group's chunks are joined at
// once (up to kFlat candidates) or by rows first; and the workspace: counters, then per
// row and chunk (max, sum) and W keys, then per row W scores and W keys.
constexpr int kFlat = 1024;
struct SelectPlan {
  int chunks, tiles, flat;
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
  const size_t n = (size_t)rows * p.chunks;
  p.stats = kHeaderBytes;
  p.keys = p.stats + align256(n * 8);
  p.scores = p.keys + align256(n * W * 8);
  p.row_keys = p.scores + align256((size_t)rows * W * 8);
  p.total = p.row_keys + align256((size_t)rows * W * 8);
  return p;
}

__device__ __forceinline__ float clean(float x) {   // NaN and +inf count as -inf, -0 as 0
  return x < INFINITY ? x + 0.0f : -INFINITY;
}
__device__ __forceinline__ u64 key_of(float x, uint32_t token) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((u64)o << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float logit_of(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// The bits of a score in unsigned order; above 0 (a score is never NaN).
__device__ __forceinline__ u64 order_of(double t) {
  const u64 b = __builtin_bit_cast(u64, t + 0.0);
  return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ uint32_t token_of(u64 key) { return 0xffffffffu - (uint32_t)key; }

__device__ __forceinline__ void st_device(void *p, u64 v) {
  __hip_atomic_store((BITNET_GLOBAL u64 *)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 ld_device(const void *p) {
  return __hip_atomic_load((const BITNET_GLOBAL u64 *)p, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}

// Room for the keys that reach a bound (kMaxWidth lanes of a wave, and those that
// were there), and for a group's candidates, which may all tie.
constexpr int kCandidates = 3 * kFlat;
static_assert(kCandidates >= kWaves * kMaxWidth * kPer + kMaxWidth, "keys above a bound");
static_assert(kFlat >= kMaxWidth * kMaxWidth, "a list per row");

struct SelectShared {
  u64 cand[kCandidates];
  u64 best[kMaxWidth];                 // the W largest keys, in order
  u64 bound[2][kWaves];
  int above[2][kWaves];
  float m[kWaves], s[kWaves];
  uint32_t count, last;
};

// A bound that W lanes' keys reach, and no more than W unless keys are equal
// (0 where fewer than W lanes have one): the W-th largest key from the top bit
// down, until exactly W lanes are left above.
__device__ __forceinline__ u64 wave_bound(u64 key, int W) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  uint32_t v = 0;
  int at = 64;
#pragma unroll 1
  for (int top = 31; top >= 0 && at != W; top -= 8)
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t t = v | (1u << (top - b));
      const int n = __builtin_popcountll(__ballot(hi >= t));
      v = n >= W ? t : v;
      at = n >= W ? n : at;
    }
  if (v == 0) return 0;
  uint32_t low = 0;
  if (at != W) {   // lanes share the value
    const int above = __builtin_popcountll(__ballot(hi > v));
#pragma unroll 1
    for (int b = 31; b >= 0 && at != W; --b) {
      const uint32_t t = low | (1u << b);
      const int n = above + __builtin_popcountll(__ballot(hi == v && lo >= t));
      if (n >= W) {
        low = t;
        at = n;
      }
    }
  }
  return ((u64)v << 32) | low;
}

// sh.best becomes the W largest of sh.best (`have` keys, 0 or W) and of the
// threads' keys: key(j), j < N <= kPer, 0 for none; `mine` is the thread's
// largest.  Every thread calls it, with the workgroup in step; `flip` alternates
// from call to call.
template <int N, typename Key>
__device__ __forceinline__ void select_largest(SelectShared &sh, int W, int have, int flip, u64 mine,
                                               Key key) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const u64 floor = have ? sh.best[W - 1] : 0;
  // A wave with few keys above what is there already needs no further bound:
  // kMaxWidth lanes of a wave fit the list.
  const int above = __builtin_popcountll(__ballot(mine > floor));
  const u64 b = above > (have ? kMaxWidth : W) ? wave_bound(mine, W) : 0;
  if (lane == 0) {
    sh.bound[flip][wave] = b;
    sh.above[flip][wave] = above;
  }
  if (tid == 0) sh.count = have;
  if (tid < have) sh.cand[tid] = sh.best[tid];
  __syncthreads();
  u64 bound = floor + 1;
  int some = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    bound = sh.bound[flip][w] > bound ? sh.bound[flip][w] : bound;
    some |= sh.above[flip][w];
  }
  if (have && some == 0) return;   // the same for every thread
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
    for (int c = 0; c < all; ++c) r += sh.cand[c] > k ? 1 : 0;
    if (r < W) sh.best[r] = k;
  }
  if (tid >= all && tid < W) sh.best[tid] = 0;
  __syncthreads();
}

// Counts one more arrival; true for the last of n, which leaves zero behind.
// Each wave's device-coherent stores are acknowledged before.
__device__ __forceinline__ bool arrive(SelectShared &sh, uint32_t *counter, int n) {
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

// log(sum of exp) of a row from its chunks' (max, sum), a lane each.
__device__ __forceinline__ double log_sum(f32x2 st) {
  const float top = wave_max(st.x);
  double sum = st.x > -INFINITY ? (double)st.y * exp((double)st.x - (double)top) : 0.0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const u64 u = __builtin_bit_cast(u64, sum);
    const u64 o = ((u64)(uint32_t)__shfl_xor((int)(u >> 32), d, 64) << 32) |
                  (uint32_t)__shfl_xor((int)(uint32_t)u, d, 64);
    sum += __builtin_bit_cast(double, o);
  }
  return top > -INFINITY ? (double)top + log(sum) : 0.0;
}

// A candidate of a group.  Order: the score, then the lower beam, then the key.
struct Entry {
  double score;
  u64 key;
  int beam, pad;
};
static_assert(sizeof(Entry) * kFlat <= 8 * kCandidates, "all candidates may tie");

// The W best of the group's candidates: entry(j) of this thread, j < N, at a
// score of NaN none.  A bound that W scores reach, then ranks by counting among
// those that do.  Ends with winner r in best[r].
template <int N, typename Get>
__device__ __forceinline__ void select_group(SelectShared &sh, int W, const double (&score)[N],
                                             Get entry, int *best) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Entry *list = reinterpret_cast<Entry *>(sh.cand);
  u64 mine = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const u64 k = score[j] == score[j] ? order_of(score[j]) : 0;
    mine = k > mine ? k : mine;
  }
  const u64 b = wave_bound(mine, W);
  if (lane == 0) sh.bound[0][wave] = b;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  u64 bound = 1;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) bound = sh.bound[0][w] > bound ? sh.bound[0][w] : bound;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (score[j] == score[j] && order_of(score[j]) >= bound)
      list[atomicAdd(&sh.count, 1u)] = entry(j);
  __syncthreads();
  const int all = sh.count;
  for (int i = tid; i < all; i += kThreads) {
    const Entry e = list[i];
    int r = 0;
    for (int c = 0; c < all; ++c) {
      const Entry u = list[c];
      const bool before = u.beam != e.beam ? u.beam < e.beam : u.key > e.key;
      r += u.score > e.score || (u.score == e.score && before) ? 1 : 0;
    }
    if (r < W) best[r] = i;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) select_kernel(SelectArgs a, SelectPlan p) {
  __shared__ SelectShared sh;
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
    auto load = [&](int64_t at) {
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const int64_t i = at + j * 4 * kThreads;
        if (i + 4 <= stop) {
          next[j] = *(const BITNET_GLOBAL f32x4_row *)(x + i);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) next[j][e] = i + e < stop ? ld_global<float>(x + i + e) : NAN;
        }
      }
    };
    load(i0);
    float m = -INFINITY, s = 0.0f;
    for (int tile = 0; tile < p.tiles; ++tile) {
      const int64_t at = i0 + (int64_t)tile * kTile;
      float v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = clean(next[j >> 2][j & 3]);
      if (tile + 1 < p.tiles) load(at + kTile);
      // The thread's largest: ties go to the first, which has the lower token.
      float top = v[0];
      int where = 0;
#pragma unroll
      for (int j = 1; j < kPer; ++j)
        if (v[j] > top) {
          top = v[j];
          where = j;
        }
      auto token = [&](int j) { return at + (j >> 2) * 4 * kThreads + (j & 3); };
      const u64 mine = at < stop ? key_of(top, (uint32_t)token(where)) : 0;
      const float m_new = fmaxf(m, top);
      if (m_new > -INFINITY) {
        float e[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) e[j] = __expf(v[j] - m_new);
#pragma unroll
        for (int d = kPer / 2; d > 0; d >>= 1)
#pragma unroll
          for (int j = 0; j < d; ++j) e[j] += e[j + d];
        s = s * __expf(m - m_new) + e[0];
        m = m_new;
      }
      select_largest<kPer>(sh, W, tile ? W : 0, tile & 1, mine, [&](int j) {
        return token(j) < stop ? key_of(v[j], (uint32_t)token(j)) : 0;
      });
    }
    // The chunk's maximum and sum.
    const float top = wave_max(m);
    if (lane == 0) sh.m[wave] = top;
    __syncthreads();
    float all = sh.m[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) all = fmaxf(all, sh.m[w]);
    s = all > -INFINITY ? s * __expf(m - all) : 0.0f;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
    if (lane == 0) sh.s[wave] = s;
    __syncthreads();
    if (tid < W) st_device(keys + chunk * W + tid, sh.best[tid]);
    if (tid == 0)
      st_device(stats + chunk,
                __builtin_bit_cast(u64, f32x2{all, (sh.s[0] + sh.s[1]) + (sh.s[2] + sh.s[3])}));
  }
  const int beam = row % W, g0 = row - beam;
  uint32_t *group = counters + kRowCounters + row / W;
  __shared__ int winner[kMaxWidth];
  __shared__ double lse[kMaxWidth];
  // A finished beam's candidates: eos at the unchanged score, then the other
  // tokens from the lowest.
  auto finished_key = [&](int i) {
    return i == 0 ? key_of(1.0f, (uint32_t)a.eos)
                  : key_of(0.0f, (uint32_t)(i - 1 < a.eos ? i - 1 : i));
  };

  if (p.flat) {
    if (!arrive(sh, group, W * p.chunks)) return;
    for (int w = wave; w < W; w += kWaves) {
      const f32x2 *row_stats = reinterpret_cast<f32x2 *>(a.ws + p.stats) + (int64_t)(g0 + w) * p.chunks;
      f32x2 st = {-INFINITY, 0.0f};
      if (lane < p.chunks && !(a.finished_in && a.finished_in[g0 + w] != 0))
        st = __builtin_bit_cast(f32x2, ld_device(row_stats + lane));
      const double v = log_sum(st);
      if (lane == 0) lse[w] = v;
    }
    constexpr int kN = (kFlat + kThreads - 1) / kThreads;
    const int each = p.chunks * W;
    const u64 *all_keys = reinterpret_cast<const u64 *>(a.ws + p.keys) + (int64_t)g0 * each;
    u64 k[kN];
    int of[kN];
    double base[kN], score[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int i = tid + j * kThreads;
      k[j] = 0;
      of[j] = 0;
      if (i < W * each) {
        of[j] = i / each;
        const int place = i - of[j] * each;
        base[j] = (double)clean(a.scores_in[g0 + of[j]]);
        if (a.finished_in && a.finished_in[g0 + of[j]] != 0) {
          k[j] = place < W ? finished_key(place) : 0;
          if (place != 0) base[j] = -INFINITY;
          of[j] |= 0x100;
        } else {
          k[j] = ld_device(all_keys + i);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      score[j] = NAN;
      if (k[j] != 0)
        score[j] = of[j] & 0x100 ? base[j] : base[j] + ((double)logit_of(k[j]) - lse[of[j]]);
    }
    select_group<kN>(sh, W, score, [&](int j) { return Entry{score[j], k[j], of[j] & 0xff, 0}; },
                     winner);
  } else {
    if (!arrive(sh, counters + row, p.chunks)) return;
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
        const double v = log_sum(st);
        if (lane == 0) lse[0] = v;
      }
      select_largest<kJoinPer>(sh, W, 0, 0, mine, [&](int j) { return k[j]; });
      if (tid < W) {
        const u64 key = sh.best[tid];
        const double t = base + ((double)logit_of(key) - lse[0]);
        st_device(scores + (int64_t)row * W + tid, __builtin_bit_cast(u64, t));
        st_device(row_keys + (int64_t)row * W + tid, key);
      }
    }
    if (!arrive(sh, group, W)) return;
    constexpr int kN = kMaxWidth * kMaxWidth / kThreads;
    double score[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int i = tid + j * kThreads;
      score[j] = i < W * W ? __builtin_bit_cast(double, ld_device(scores + (int64_t)g0 * W + i)) : NAN;
    }
    select_group<kN>(
        sh, W, score,
        [&](int j) {
          const int i = tid + j * kThreads;
          return Entry{score[j], ld_device(row_keys + (int64_t)g0 * W + i), i / W, 0};
        },
        winner);
  }

  // finished_out may be finished_in, scores_out scores_in: every row of the
  // group has read its own, and here flags are read before any is written.
  int fin = 0;
  Entry e = {0.0, 0, 0, 0};
  if (tid < W) {
    e = reinterpret_cast<const Entry *>(sh.cand)[winner[tid]];
    if (a.finished_in) fin = a.finished_in[g0 + e.beam] != 0;
  }
  __syncthreads();
  if (tid < W) {
    const int o = g0 + tid;
    const int token = (int)token_of(e.key);
    a.scores_out[o] = (float)e.score;
    a.tokens[o] = token;
    a.parents[o] = g0 + e.beam;
    if (a.finished_in) a.finished_out[o] = fin || token == a.eos;
  }
}

}  // namespace

size_t select_workspace_bytes(int64_t B, int64_t W, int64_t V) {
  return select_plan(B * W, W, V).total;
}

hipError_t launch_beam_select(const SelectArgs &a, hipStream_t stream) {
  const SelectPlan p = select_plan((int64_t)a.B * a.W, a.W, a.V);
  select_kernel<<<dim3(p.chunks, a.B * a.W), kThreads, 0, stream>>>(a, p);
  return hipGetLastError();
}

}  // namespace bitnet
