// Log probabilities of given tokens, the entropy of each row and its likeliest
// tokens, in one pass over the logits:
//
//   lse = log sum exp x,  logprob = x[token] - lse,  H = lse - sum p x
//
// With m the largest logit and d = x - m (in units of log 2, from one fma), a
// thread sums e = exp2(d) and e d; H = ln 2 (log2 S - (sum e d) / S), whose two
// terms are not negative, so that nothing cancels.  When m grows by -D to m',
// the sums become S f and f (sum e d + S D) with f = exp2(D).  The
// likeliest tokens come from lists of the waves as in beam selection.
//
// A row is cut into chunks when rows are few, which the last to finish joins;
// from 1024 rows on a workgroup takes a whole row.
//
// Bound by HBM: 1800 rows of 151,936 in 174 us, 6.3 TB/s.  A few rows wait for what
// follows one another: a row's lse alone takes 4.9 us (launch, load, arrival of 38
// chunks, their join), 5 likeliest tokens 4.6 us more, 20 of them 7.3, in the bounds
// and ranks of the chunks' and the join's candidates; 16 rows 6.3, 11.0 and 14.3 us.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "candidates.hpp"
#include "kv.hpp"
#include "rows.hpp"

namespace bitnet {
namespace {

constexpr int kMaxTop = 32, kNarrow = 8;
constexpr int kTargetGroups = 1024;
constexpr int kLine = 32;                                // counters a cache line apart
constexpr int kHeaderBytes = 4 * kLine * kTargetGroups;  // rows that are cut are fewer
constexpr float kFar = -16384.0f;                        // exponents below this add nothing
constexpr double kLn2 = 0.69314718055994530942;

struct LogprobPlan {
  int chunks, tiles;
  size_t stats, keys, total;
};
LogprobPlan logprob_plan(int64_t R, int64_t V, int64_t top) {
  LogprobPlan p;
  const int64_t all = (V + kTile - 1) / kTile;
  const int64_t chunks = std::min<int64_t>(std::min<int64_t>(all, kMaxChunks),
                                           (kTargetGroups + R - 1) / R);
  p.tiles = (int)((all + chunks - 1) / chunks);
  p.chunks = (int)((all + p.tiles - 1) / p.tiles);
  const size_t n = p.chunks > 1 ? (size_t)R * p.chunks : 0;
  p.stats = kHeaderBytes;
  p.keys = p.stats + align256(n * 16);
  p.total = p.keys + align256(n * top * 8);
  return p;
}

template <int MAXW>
struct LogprobShared : CandidateShared<MAXW == 0 ? kNarrow : MAXW> {
  float t[kWaves];
  double lse;
};

template <int MAXW>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4)))
logprobs_kernel(LogprobArgs a, LogprobPlan p) {
  __shared__ LogprobShared<MAXW> sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x, row = blockIdx.y, W = a.top;
  const float *x = a.logits + row * a.ld;
  const int token = a.tokens ? ld_global<int>(a.tokens + row) : -1;

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
  // The wave's list of keys, as in beam selection: every key of its W largest so
  // far, and others, all from `least`.
  typedef LogprobShared<MAXW> Shared;
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
  float m = -INFINITY, s = 0.0f, t = 0.0f;
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
      float e[kPer], d[kPer];
      const float mc = m_new * kLog2e;
#pragma unroll
      for (int j = 0; j < kPer; ++j) d[j] = __builtin_fmaf(v[j], kLog2e, -mc);
      if (huge(m_new))
#pragma unroll
        for (int j = 0; j < kPer; ++j) d[j] = (v[j] - m_new) * kLog2e;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        d[j] = fmaxf(d[j], kFar);
        e[j] = __builtin_amdgcn_exp2f(d[j]);
        d[j] *= e[j];
      }
#pragma unroll
      for (int n = kPer / 2; n > 0; n >>= 1)
#pragma unroll
        for (int j = 0; j < n; ++j) {
          e[j] += e[j + n];
          d[j] += d[j + n];
        }
      const float up = fmaxf(rise(m, m_new), kFar), f = __builtin_amdgcn_exp2f(up);
      t = (t + s * up) * f + d[0];
      s = s * f + e[0];
      m = m_new;
    }
    if constexpr (MAXW > 0) {
      auto number = [&](int j) { return at + (j >> 2) * 4 * kThreads + (j & 3); };
      auto key = [&](int j) { return number(j) < stop ? key_of(v[j], (uint32_t)number(j)) : 0; };
      // Keys that may be among the chunk's W largest go to the wave's list.
      if (p.tiles > 1 && !__any(top >= least_logit)) continue;
      int where = kPer - 1;   // ties: the first of the thread's, which has the lowest token
#pragma unroll
      for (int j = kPer - 2; j >= 0; --j) where = v[j] == top ? j : where;
      const u64 mine = at < stop ? key_of(top, (uint32_t)number(where)) : 0;
      if (p.tiles == 1) {   // (no tile comes behind it: no list; 8 of a row 0.4 us less)
        select_largest<kPer>(sh, W, mine, key);
        break;
      }
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
          const u64 k = key(j);
          add(k >= least, k);
        }
    }
  }
  if constexpr (MAXW > 0) if (p.tiles > 1) {
    u64 k[Shared::kPerLane], mine = 0;
#pragma unroll
    for (int j = 0; j < Shared::kPerLane; ++j) {
      k[j] = lane + 64 * j < listed ? list[lane + 64 * j] : 0;
      mine = k[j] > mine ? k[j] : mine;
    }
    select_largest<Shared::kPerLane>(sh, W, mine, [&](int j) { return k[j]; });
  }
  // The chunk's maximum and sums.
  const float most = across16<true>(across4(m));
  if (lane == 0) sh.m[wave] = most;
  __syncthreads();
  float all = sh.m[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) all = fmaxf(all, sh.m[w]);
  if (all > -INFINITY) {
    const float up = fmaxf(rise(m, all), kFar), f = __builtin_amdgcn_exp2f(up);
    t = (t + s * up) * f;
    s *= f;
  }
  s = across16<false>(sum4(s));
  t = across16<false>(sum4(t));
  if (lane == 0) {
    sh.s[wave] = s;
    sh.t[wave] = t;
  }
  __syncthreads();
  s = (sh.s[0] + sh.s[1]) + (sh.s[2] + sh.s[3]);
  t = (sh.t[0] + sh.t[1]) + (sh.t[2] + sh.t[3]);

  // The row's results, in the first wave: its exponent and sums.
  const bool given = (uint32_t)token < (uint32_t)a.V;
  auto finish = [&](double e, double sum, double weighted, float logit) {
    const double lse = log_sum(e, sum);
    if (tid == 0) {
      if (a.logprobs)
        a.logprobs[row] = given ? (float)((double)clean(logit) - lse) : 0.0f;
      if (a.entropy)
        a.entropy[row] =
            sum > 0.0 ? (float)fmax(kLn2 * (log2(sum) - weighted / sum), 0.0) : 0.0f;
      sh.lse = lse;
    }
  };
  if (p.chunks == 1) {
    if (wave == 0)
      finish(exponent(all), (double)s, (double)t, tid == 0 && given ? ld_global<float>(x + token) : 0.0f);
  } else {
    u64 *stats = reinterpret_cast<u64 *>(a.ws + p.stats) + (int64_t)row * p.chunks * 2;
    u64 *keys = reinterpret_cast<u64 *>(a.ws + p.keys) + (int64_t)row * p.chunks * W;
    if (MAXW > 0 && tid < W) st_device(keys + chunk * W + tid, sh.best[tid]);
    if (tid == 0) {
      st_device(stats + 2 * chunk, __builtin_bit_cast(u64, f32x2{all, s}));
      st_device(stats + 2 * chunk + 1, __builtin_bit_cast(u64, f32x2{t, 0.0f}));
    }
    if (!arrive(sh, reinterpret_cast<uint32_t *>(a.ws) + row * kLine, p.chunks)) return;
    f32x2 st = {-INFINITY, 0.0f}, wt = {0.0f, 0.0f};
    float logit = 0.0f;
    if (tid < p.chunks) {
      st = __builtin_bit_cast(f32x2, ld_device(stats + 2 * tid));
      wt = __builtin_bit_cast(f32x2, ld_device(stats + 2 * tid + 1));
    }
    if (tid == 0 && given) logit = ld_global<float>(x + token);
    if constexpr (MAXW > 0) {
      constexpr int kN = (kMaxChunks * MAXW + kThreads - 1) / kThreads;
      u64 k[kN], mine = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int i = tid + j * kThreads;
        k[j] = i < p.chunks * W ? ld_device(keys + i) : 0;
        mine = k[j] > mine ? k[j] : mine;
      }
      select_largest<kN>(sh, W, mine, [&](int j) { return k[j]; });
    }
    if (wave == 0) {   // the chunks are its lanes
      const float top = across16<true>(across4(st.x));
      double sum = 0.0, weighted = 0.0;
      if (st.x > -INFINITY) {
        const float up = fmaxf(rise(st.x, top), kFar);
        const double f = (double)__builtin_amdgcn_exp2f(up);
        sum = (double)st.y * f;
        weighted = ((double)wt.x + (double)st.y * (double)up) * f;
      }
      sum = wave_total(sum);
      weighted = wave_total(weighted);
      finish(exponent(top), sum, weighted, logit);
    }
  }
  if constexpr (MAXW > 0) {
    __syncthreads();
    if (tid < W) {
      const u64 k = sh.best[tid];
      a.top_tokens[(int64_t)row * W + tid] = (int)token_of(k);
      a.top_logprobs[(int64_t)row * W + tid] = (float)((double)logit_of(k) - sh.lse);
    }
  }
}

}  // namespace

size_t logprobs_workspace_bytes(int64_t R, int64_t V, int64_t top) {
  return logprob_plan(R, V, top).total;
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t stream) {
  const LogprobPlan p = logprob_plan(a.R, a.V, a.top);
  const dim3 grid(p.chunks, a.R);
  if (a.top == 0)
    logprobs_kernel<0><<<grid, kThreads, 0, stream>>>(a, p);
  else if (a.top <= kNarrow)
    logprobs_kernel<kNarrow><<<grid, kThreads, 0, stream>>>(a, p);
  else
    logprobs_kernel<kMaxTop><<<grid, kThreads, 0, stream>>>(a, p);
  return hipGetLastError();
}

}  // namespace bitnet
