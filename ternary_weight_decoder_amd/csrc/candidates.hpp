// The largest of a row of logits, streamed by workgroups: keys, bounds, lists of
// the waves, and the sum of exp.  Shared by beam selection and token log
// probabilities.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bitnet_device.hpp"
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

typedef float f32x2 __attribute__((ext_vector_type(2)));
// Rows are only 4-byte aligned.
typedef float f32x4_row __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned long long u64;

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
// The exponent that a maximum m stands for in units of log 2, whose exp2 its sum of
// exp is relative to: the rounded product, as one fma a logit takes it; of a large
// m, whose product's rounding would be a factor of its own (2^(m / 2^24)), the
// exact one, which goes with exp2((x - m) c).
__device__ __forceinline__ bool huge(float m) { return fabsf(m) > 0x1p20f; }
__device__ __forceinline__ double exponent(float m) {
  return huge(m) ? (double)m * (double)kLog2e : (double)(m * kLog2e);
}
// The difference of two maxima's exponents, m <= n, n > -inf, and its exp2.  An fma
// gives a rounded product's difference to an exact one; of two large maxima the
// difference itself is exact where its exp2 is not zero.  (Selects: with a branch to
// fp64 32 groups of 32 beams of 40,000 logits take 66.2 us, 65.3 so; one group of 4 beams
// of 151,936 11.4 and 11.1.)
__device__ __forceinline__ float rise(float m, float n) {
  const float mc = m * kLog2e, nc = n * kLog2e;
  const float to_near = huge(m) ? __builtin_fmaf(m, kLog2e, -nc) : mc - nc;
  const float to_far = huge(m) ? (m - n) * kLog2e : -__builtin_fmaf(n, kLog2e, -mc);
  return huge(n) ? to_far : to_near;
}
__device__ __forceinline__ float shift(float m, float n) {
  return __builtin_amdgcn_exp2f(rise(m, n));
}
__device__ __forceinline__ uint32_t token_of(u64 key) { return 0xffffffffu - (uint32_t)key; }

__device__ __forceinline__ void st_device(void *p, u64 v) {
  __hip_atomic_store((BITNET_GLOBAL u64 *)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 ld_device(const void *p) {
  return __hip_atomic_load((const BITNET_GLOBAL u64 *)p, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}

// By the greatest width a kernel serves: room for the waves' lists (all of which may
// reach the bound of their join), or for WORDS words of what follows.
template <int MAXW, int WORDS = 0>
struct CandidateShared {
  // A wave's list: what one tile can add, and what is left of a list that was cut.
  static constexpr int kList = 2 * MAXW * kPer;
  static constexpr int kPerLane = kList / 64;
  static_assert(MAXW * kPerLane + MAXW * kPer <= kList, "room for a tile's keys");
  static constexpr int kWords = std::max(WORDS, kWaves * kList);
  __attribute__((aligned(16))) u64 cand[kWords];   // the waves' lists, then candidates
  u64 best[MAXW];                      // the W largest keys, in order
  u64 bound[kWaves];
  uint32_t share[kWaves];
  float m[kWaves], s[kWaves];
  uint32_t count, last;
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
template <int N, int MAXW, int WORDS, typename Key>
__device__ __forceinline__ void select_largest(CandidateShared<MAXW, WORDS> &sh, int W, u64 mine, Key key) {
  // What every wave reaches with its share of W lanes is a bound too, below which are
  // most of the keys that reach a wave's own for all W: the ranking reads the square
  // of what is left (32 of a row of 151,936: 26.8 us without, 14.5 with; 20: 13.0 and
  // 12.2).
  constexpr bool kShares = MAXW > 8;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const u64 b = wave_bound(mine, W, MAXW);
  if (lane == 0) sh.bound[wave] = b;
  if constexpr (kShares) {
    const int n = (W + kWaves - 1) / kWaves;
    int at;
    const uint32_t share = bound_32((uint32_t)(mine >> 32), n, n + 2, &at);
    if (lane == 0) sh.share[wave] = share;
  }
  if (tid == 0) sh.count = 0;
  __syncthreads();
  u64 bound = 1;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) bound = sh.bound[w] > bound ? sh.bound[w] : bound;
  if constexpr (kShares) {
    uint32_t least = sh.share[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) least = min(least, sh.share[w]);
    bound = max(bound, (u64)least << 32);
  }
  if (mine >= bound)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const u64 k = key(j);
      if (k >= bound) sh.cand[atomicAdd(&sh.count, 1u)] = k;
    }
  __syncthreads();
  const int all = sh.count;
  // Four threads count for each (one: 20 of a row 0.5 us more).
  for (int i = tid >> 2; i < all; i += kThreads / 4) {
    const u64 k = sh.cand[i];
    int r = 0;
#pragma unroll 4
    for (int c = tid & 3; c < all; c += 4) r += sh.cand[c] > k ? 1 : 0;
    r += __builtin_amdgcn_update_dpp(0, r, 0xB1, 0xF, 0xF, false);
    r += __builtin_amdgcn_update_dpp(0, r, 0x4E, 0xF, 0xF, false);
    if (r < W && (tid & 3) == 0) sh.best[r] = k;
  }
  if (tid >= all && tid < W) sh.best[tid] = 0;
  __syncthreads();
}

// Counts one more arrival; true for the last of n, which leaves zero behind.
// Each wave's device-coherent stores are acknowledged before.
template <int MAXW, int WORDS>
__device__ __forceinline__ bool arrive(CandidateShared<MAXW, WORDS> &sh, uint32_t *counter, int n) {
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

}  // namespace
}  // namespace bitnet
