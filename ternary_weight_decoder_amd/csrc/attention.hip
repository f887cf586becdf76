// Attention of one new token per row over the paged key-value cache.
//
// One workgroup per row and query head walks the length in steps of 256
// tokens: a thread scores one token, the workgroup takes the running maximum
// and sum of the softmax, and the threads then share the channels of the
// weighted sum.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"

namespace bitnet {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

template <int DT> struct KvElem;
template <> struct KvElem<BITNET_KV_BF16> { typedef __bf16 T; };
template <> struct KvElem<BITNET_KV_FP16> { typedef _Float16 T; };
template <> struct KvElem<BITNET_KV_INT8> { typedef int8_t T; };

__device__ __forceinline__ float block_max(float v, float *red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kWaves; ++w) v = fmaxf(v, red[w]);
  __syncthreads();
  return v;
}

__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kWaves; ++w) v += red[w];
  __syncthreads();
  return v;
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(AttendArgs a) {
  typedef typename KvElem<DT>::T E;
  __shared__ float q[D], p[kThreads], red[kWaves], part[kThreads];
  __shared__ int pages[kThreads];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int kvh = h / (a.q_heads / a.c.kv_heads);
  const int r = a.rows ? a.rows[t] : t;
  const int len = r >= 0 && r < a.table_rows ? min(max(a.lens[t], 0), a.max_len) : 0;
  const int ps = 1 << a.c.page_shift;
  if (tid < D) q[tid] = a.q[t * a.q_stride + h * D + tid] * a.scale;
  __syncthreads();
  constexpr int kParts = kThreads / D > 0 ? kThreads / D : 1;
  const int d = tid % D, sub = tid / D;
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int j0 = 0; j0 < len; j0 += kThreads) {
    const int j = j0 + tid;
    float s = -INFINITY;
    int page = -1;
    if (j < len) {
      page = a.tables[(int64_t)r * a.max_pages + (j >> a.c.page_shift)];
      if (page < 0 || page >= a.c.pages) page = -1;
    }
    pages[tid] = page;
    if (page >= 0) {
      const E *k = reinterpret_cast<const E *>(a.c.k) + page * a.c.page_stride +
                   kvh * a.c.head_stride + (j & (ps - 1)) * a.c.token_stride;
      s = 0.0f;
      for (int i = 0; i < D; ++i) s += q[i] * (float)k[i];
      if (DT == BITNET_KV_INT8)
        s *= a.c.k_scale[(((int64_t)page * a.c.kv_heads + kvh) << a.c.page_shift) + (j & (ps - 1))];
    }
    const float mn = fmaxf(m, block_max(s, red));
    const float w = mn == -INFINITY ? 0.0f : __expf(s - mn);
    const float keep = mn == -INFINITY ? 0.0f : __expf(m - mn);
    l = l * keep + block_sum(w, red);
    m = mn;
    p[tid] = w;
    __syncthreads();
    o *= keep;
    const int n = min(kThreads, len - j0);
    for (int i = sub; i < n; i += kParts) {
      const int64_t pg = pages[i];
      if (pg < 0) continue;
      const int tok = (j0 + i) & (ps - 1);
      float x = (float)reinterpret_cast<const E *>(a.c.v)[pg * a.c.page_stride +
                                                          kvh * a.c.head_stride +
                                                          tok * a.c.token_stride + d];
      if (DT == BITNET_KV_INT8)
        x *= a.c.v_scale[((pg * a.c.kv_heads + kvh) << a.c.page_shift) + tok];
      o += p[i] * x;
    }
    __syncthreads();
  }
  part[tid] = o;
  __syncthreads();
  if (tid < D) {
    for (int i = 1; i < kParts; ++i) o += part[tid + i * D];
    a.out[((int64_t)t * a.q_heads + h) * D + tid] = l > 0.0f ? o / l : 0.0f;
  }
  if (tid == 0 && a.lse) a.lse[(int64_t)t * a.q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

template <int DT>
void attend_dim(const AttendArgs &a, int D, hipStream_t stream) {
  const dim3 grid(a.T, a.q_heads);
  if (D == 64)
    attend_kernel<DT, 64><<<grid, kThreads, 0, stream>>>(a);
  else if (D == 128)
    attend_kernel<DT, 128><<<grid, kThreads, 0, stream>>>(a);
  else
    attend_kernel<DT, 256><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

size_t attend_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16384; }

hipError_t launch_attend(const AttendArgs &a, int dtype, int head_dim, hipStream_t stream) {
  if (dtype == BITNET_KV_BF16)
    attend_dim<BITNET_KV_BF16>(a, head_dim, stream);
  else if (dtype == BITNET_KV_FP16)
    attend_dim<BITNET_KV_FP16>(a, head_dim, stream);
  else
    attend_dim<BITNET_KV_INT8>(a, head_dim, stream);
  return hipGetLastError();
}

}  // namespace bitnet
