// Beam selection: the W best of the W * V continuations of a group's beams.
//
// Within a beam the order of the candidates is that of its logits, so each
// beam contributes at most its W largest logits (ties: the lower token), and
// the log-softmax needs only the beam's sum of exp.  Both come from one pass
// over the logits: a workgroup takes a chunk of a row into registers, sums its
// exps against the chunk's maximum and picks the chunk's W largest.  A 64-bit
// key (order-preserving bits of the logit, then the inverted token) makes the
// entries of a chunk distinct.  The W-th largest of the threads' own largest
// keys bounds the chunk's W-th largest from below, and exactly W threads hold
// keys at or above it, so at most W * (keys per thread) candidates are left,
// which are ranked by counting.
//
// The second kernel joins the chunks of a group's rows.
#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"

namespace bitnet {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;                     // logits per thread
constexpr int kChunk = kThreads * kPer;      // logits per workgroup
constexpr int kHeaderBytes = 16384;

__host__ __device__ inline int chunks_of(int V) { return (V + kChunk - 1) / kChunk; }

// Workspace: header, then per row and chunk (max, sum) and W keys.
struct SelectWs {
  size_t stats, keys, total;
};
__host__ __device__ inline SelectWs select_ws(int64_t rows, int64_t W, int64_t V) {
  const int64_t n = rows * ((V + kChunk - 1) / kChunk);
  SelectWs w;
  w.stats = kHeaderBytes;
  w.keys = w.stats + align256((size_t)n * 8);
  w.total = w.keys + align256((size_t)n * W * 8);
  return w;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float clean(float x) {   // NaN and +inf count as -inf
  return x < INFINITY ? x + 0.0f : -INFINITY;
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((uint64_t)o << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint32_t token_of(uint64_t key) { return 0xffffffffu - (uint32_t)key; }

__global__ void __launch_bounds__(kThreads) select_chunk_kernel(SelectArgs a) {
  __shared__ uint64_t best[kThreads];
  __shared__ uint64_t cand[kMaxWidth * kPer];
  __shared__ float red[2][kThreads / 64];
  __shared__ uint64_t bound;
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x, row = blockIdx.y;
  if (a.finished_in && a.finished_in[row] != 0) return;
  const float *x = a.logits + row * a.ld;
  float v[kPer];
  float m = -INFINITY;
  uint64_t mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t i = (int64_t)chunk * kChunk + j * kThreads + tid;
    v[j] = -INFINITY;
    if (i < a.V) {
      v[j] = clean(ld_global<float>(x + i));
      const uint64_t k = key_of(v[j], (uint32_t)i);
      mine = k > mine ? k : mine;
    }
    m = fmaxf(m, v[j]);
  }
  m = wave_max(m);
  if (lane == 0) red[0][wave] = m;
  best[tid] = mine;
  if (tid == 0) count = 0;
  __syncthreads();
  for (int w = 0; w < kThreads / 64; ++w) m = fmaxf(m, red[0][w]);
  float s = 0.0f;
  if (m > -INFINITY)
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += __expf(v[j] - m);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
  if (lane == 0) red[1][wave] = s;
  int above = 0;   // threads with a larger best key
  for (int i = 0; i < kThreads; ++i) above += best[i] > mine ? 1 : 0;
  if (above == a.W - 1 && mine != 0) bound = mine;
  __syncthreads();
  // Fewer threads with a key than beams: take every key.
  const int64_t left = a.V - (int64_t)chunk * kChunk;
  const uint64_t low = left < a.W ? 1 : bound;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t i = (int64_t)chunk * kChunk + j * kThreads + tid;
    if (i < a.V) {
      const uint64_t k = key_of(v[j], (uint32_t)i);
      if (k >= low) cand[atomicAdd(&count, 1)] = k;
    }
  }
  __syncthreads();
  const int n = count;
  const SelectWs ws = select_ws(a.B * a.W, a.W, a.V);
  const int64_t at = (int64_t)row * chunks_of(a.V) + chunk;
  uint64_t *keys = reinterpret_cast<uint64_t *>(a.ws + ws.keys) + at * a.W;
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t k = cand[i];
    int r = 0;
    for (int c = 0; c < n; ++c) r += cand[c] > k ? 1 : 0;
    if (r < a.W) keys[r] = k;
  }
  if (tid >= n && tid < a.W) keys[tid] = 0;
  if (tid == 0) {
    f32x2 st = {m, (red[1][0] + red[1][1]) + (red[1][2] + red[1][3])};
    reinterpret_cast<f32x2 *>(a.ws + ws.stats)[at] = st;
  }
}

__global__ void __launch_bounds__(kThreads) select_join_kernel(SelectArgs a) {
  __shared__ double score[kMaxWidth * kMaxWidth];
  __shared__ int32_t token[kMaxWidth * kMaxWidth];
  __shared__ uint64_t red[kThreads / 64];
  __shared__ double lse_sh;
  __shared__ int win[kMaxWidth];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int W = a.W, g0 = blockIdx.x * W, nch = chunks_of(a.V);
  const SelectWs ws = select_ws(a.B * a.W, a.W, a.V);
  for (int w = 0; w < W; ++w) {
    const int row = g0 + w;
    const double base = (double)clean(a.scores_in[row]);
    if (a.finished_in && a.finished_in[row] != 0) {
      // eos at the unchanged score, then the other tokens from the lowest
      if (tid < W) {
        const int other = tid - 1 < a.eos ? tid - 1 : tid;
        token[w * W + tid] = tid == 0 ? a.eos : other;
        score[w * W + tid] = tid == 0 ? base : (double)-INFINITY;
      }
      continue;
    }
    const f32x2 *st = reinterpret_cast<const f32x2 *>(a.ws + ws.stats) + (int64_t)row * nch;
    if (tid == 0) {
      float m = -INFINITY;
      for (int c = 0; c < nch; ++c) m = fmaxf(m, st[c].x);
      double s = 0.0;
      for (int c = 0; c < nch; ++c)
        if (st[c].x > -INFINITY) s += (double)st[c].y * exp((double)st[c].x - (double)m);
      lse_sh = m > -INFINITY ? (double)m + log(s) : 0.0;
    }
    __syncthreads();
    const double lse = lse_sh;
    const uint64_t *keys = reinterpret_cast<const uint64_t *>(a.ws + ws.keys) + (int64_t)row * nch * W;
    uint64_t last = ~0ull;
    for (int k = 0; k < W; ++k) {   // the next largest key below the last one
      uint64_t b = 0;
      for (int i = tid; i < nch * W; i += kThreads) {
        const uint64_t v = keys[i];
        if (v < last && v > b) b = v;
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        const uint64_t o = ((uint64_t)(uint32_t)__shfl_xor((int)(b >> 32), d, 64) << 32) |
                           (uint32_t)__shfl_xor((int)(uint32_t)b, d, 64);
        b = o > b ? o : b;
      }
      if (lane == 0) red[wave] = b;
      __syncthreads();
      for (int i = 0; i < kThreads / 64; ++i) b = red[i] > b ? red[i] : b;
      last = b;
      if (tid == 0) {
        token[w * W + k] = (int32_t)token_of(b);
        score[w * W + k] = base + ((double)logit_of(b) - lse);
      }
      __syncthreads();
    }
  }
  __syncthreads();
  // Rank by (score, then place in the list: beams in order, each descending).
  for (int i = tid; i < W * W; i += kThreads) {
    const double s = score[i];
    int r = 0;
    for (int c = 0; c < W * W; ++c) r += (score[c] > s || (score[c] == s && c < i)) ? 1 : 0;
    if (r < W) win[r] = i;
  }
  __syncthreads();
  // finished_out may be finished_in, scores_out scores_in: read, then write.
  int fin = 0;
  if (tid < W && a.finished_in) fin = a.finished_in[g0 + win[tid] / W] != 0;
  __syncthreads();
  if (tid < W) {
    const int i = win[tid], o = g0 + tid;
    a.scores_out[o] = (float)score[i];
    a.tokens[o] = token[i];
    a.parents[o] = g0 + i / W;
    if (a.finished_in) a.finished_out[o] = fin || token[i] == a.eos;
  }
}

}  // namespace

size_t select_workspace_bytes(int64_t B, int64_t W, int64_t V) {
  return select_ws(B * W, W, V).total;
}

hipError_t launch_beam_select(const SelectArgs &a, hipStream_t stream) {
  select_chunk_kernel<<<dim3(chunks_of(a.V), a.B * a.W), kThreads, 0, stream>>>(a);
  select_join_kernel<<<a.B, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace bitnet
