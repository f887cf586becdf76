// Row operators between the projections: the residual addition with the
// root-mean-square norm, and the gated activation.  Both end in fp32 rows, in
// 8-bit rows with a scale each (the same codes as the quantization of the fp32
// row gives), or in both.
//
//   norm   h = fl32(x + residual),  y = fl32(h w / sqrt(mean h^2 + eps))
//   gate   y = fl32(g u / (1 + exp(-g)))
//   codes  s = fl32(127 / max|y|),  rint(fl32(y s))
//
// A code is decided by the bits of y, so y is computed in fp64 and rounded once:
// whatever the order of a sum, y and with it the code come out the same but for
// the few values in 2^29 that lie that near a border.  fp64 is as fast as fp32
// here, and a value needs few operations: the kernels are bound by memory, and
// read each row once, all of its loads in flight together.
#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"
#include "rows.hpp"

namespace bitnet {
namespace {

constexpr int kAxis = 1 << 20;   // workgroups of a grid's first axis

__device__ __forceinline__ double shared_sum(double v, double *part, int waves) {
  v = wave_total(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < waves; ++w) v += part[w];
  return v;
}
__device__ __forceinline__ float shared_max(float v, float *part, int waves) {
  v = across16<true>(across4(v));
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < waves; ++w) v = fmaxf(v, part[w]);
  return v;
}

// Rows of a workgroup: one, shared by WAVES waves, or with WAVES == 1 four, a
// wave each.
template <int WAVES>
struct RowShared {
  double sum[WAVES];
  float max[WAVES];
};
template <int WAVES>
constexpr int row_threads() { return WAVES == 1 ? 256 : 64 * WAVES; }

// The 8-bit row of y[0..VEC) quads, thread t of a row holding quads t, t + n, ...
template <int WAVES, int VEC>
__device__ __forceinline__ void store_codes(const f32x4 (&y)[VEC], int t, int quads, int8_t *xq,
                                            float *x_scale, RowShared<WAVES> &sh) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) top = fmaxf(top, absmax4(y[j]));
  const float s = scale_of(shared_max(top, sh.max, WAVES));
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = t + j * 64 * WAVES;
    if (i < quads)
      st_global<uint32_t>(xq + 4 * i, pack4_i8(quant_one(y[j].x, s), quant_one(y[j].y, s),
                                               quant_one(y[j].z, s), quant_one(y[j].w, s)));
  }
  if (t == 0) st_global<float>(x_scale, s);
}

template <int WAVES, int VEC>
__global__ void __launch_bounds__(row_threads<WAVES>()) norm_kernel(NormArgs a) {
  __shared__ RowShared<WAVES> sh;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = WAVES == 1 ? block * 4 + (threadIdx.x >> 6) : block;
  if (row >= a.M) return;
  const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int quads = a.K >> 2;
  const float *x = a.x + row * a.x_stride;
  const float *res = a.residual ? a.residual + row * a.r_stride : nullptr;
  constexpr f32x4 kZero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 h[VEC], r[VEC], w[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = t + j * 64 * WAVES;
    h[j] = i < quads ? ld_global<f32x4>(x + 4 * i) : kZero;
    r[j] = res && i < quads ? ld_global<f32x4>(res + 4 * i) : kZero;
    w[j] = i < quads ? ld_global<f32x4>(a.weight + 4 * i) : kZero;
  }
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = t + j * 64 * WAVES;
    if (res) h[j] += r[j];
    if (a.sum && i < quads) st_global<f32x4>(a.sum + row * a.K + 4 * i, h[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) ss += (double)h[j][e] * (double)h[j][e];
  }
  const double d = shared_sum(ss, sh.sum, WAVES) / (double)a.K + (double)a.eps;
  const double inv = d > 0.0 ? 1.0 / sqrt(d) : 0.0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = t + j * 64 * WAVES;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[j][e] = (float)((double)h[j][e] * inv * (double)w[j][e]);
    if (a.y && i < quads) st_global<f32x4>(a.y + row * a.K + 4 * i, h[j]);
  }
  if (a.xq) store_codes<WAVES, VEC>(h, t, quads, a.xq + row * a.K, a.x_scale + row, sh);
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  const double d = (double)g;
  return (float)(d / (1.0 + exp(-d)) * (double)u);
}

template <int WAVES, int VEC>
__global__ void __launch_bounds__(row_threads<WAVES>()) gate_kernel(GateArgs a) {
  __shared__ RowShared<WAVES> sh;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t row = WAVES == 1 ? block * 4 + (threadIdx.x >> 6) : block;
  if (row >= a.M) return;
  const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int quads = a.K >> 2;
  const float *gate = a.gate + row * a.g_stride, *up = a.up + row * a.u_stride;
  constexpr f32x4 kZero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 y[VEC], u[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = t + j * 64 * WAVES;
    y[j] = i < quads ? ld_global<f32x4>(gate + 4 * i) : kZero;
    u[j] = i < quads ? ld_global<f32x4>(up + 4 * i) : kZero;
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int i = t + j * 64 * WAVES;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[j][e] = silu_mul(y[j][e], u[j][e]);
    if (a.y && i < quads) st_global<f32x4>(a.y + row * a.K + 4 * i, y[j]);
  }
  if (a.xq) store_codes<WAVES, VEC>(y, t, quads, a.xq + row * a.K, a.x_scale + row, sh);
}

dim3 row_grid(int64_t blocks) {
  const int64_t axes = (blocks + kAxis - 1) / kAxis;
  return dim3((unsigned)((blocks + axes - 1) / axes), (unsigned)axes);
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t stream) {
  if (a.K <= 64 * 4 * 8)
    norm_kernel<1, 8><<<row_grid((a.M + 3) / 4), row_threads<1>(), 0, stream>>>(a);
  else if (a.K <= 256 * 4 * 10)
    norm_kernel<4, 10><<<row_grid(a.M), row_threads<4>(), 0, stream>>>(a);
  else
    norm_kernel<16, 8><<<row_grid(a.M), row_threads<16>(), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_silu_mul(const GateArgs &a, hipStream_t stream) {
  if (a.K <= 64 * 4 * 8)
    gate_kernel<1, 8><<<row_grid((a.M + 3) / 4), row_threads<1>(), 0, stream>>>(a);
  else if (a.K <= 256 * 4 * 10)
    gate_kernel<4, 10><<<row_grid(a.M), row_threads<4>(), 0, stream>>>(a);
  else
    gate_kernel<16, 8><<<row_grid(a.M), row_threads<16>(), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace bitnet
