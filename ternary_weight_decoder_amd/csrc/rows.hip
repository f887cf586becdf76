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
// here.  A row is read once, all of its loads in flight together, and held in
// registers between its sum, its maximum and its codes.
//
// Measured (a launch in a graph, inputs rotating): norm of 28,800 rows of 1536 with
// sum and fp32 rows 120 us, 708 MB, 5.9 TB/s; of 1800 with 8-bit rows 8.8 us, 36 MB;
// of 16 rows 2.7 us.  Gated rows of 8960 in 8 bits, 1800 of them, 33.3 us, 145 MB, 4.4
// TB/s, beside 60% of the vector units' cycles; 16 rows 2.4 us.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"
#include "rows.hpp"

namespace bitnet {
namespace {

constexpr int kAxis = 1 << 20;   // workgroups of a grid's first axis

__device__ __forceinline__ double shared_sum(double v, double *part, int waves) {
  v = wave_total(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < waves; ++w) v += part[w];
  return v;
}
__device__ __forceinline__ float shared_max(float v, float *part, int waves) {
  v = across16<true>(across4(v));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < waves; ++w) v = fmaxf(v, part[w]);
  return v;
}

template <int WAVES>
struct RowShared {
  double sum[WAVES];
  float max[WAVES];
};

// Four codes rint(fl32(y s)).  |y| <= max|y|, so |y s| rounds to 127 at most, and the
// sum with 3 * 2^22 rounds it to a whole number, half to even, in its lowest byte.
__device__ __forceinline__ uint32_t codes_of(f32x4 y, float s) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = __builtin_bit_cast(uint32_t, y[e] * s + 0x1.8p23f);
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u),
                               __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u), 0x05040100u);
}

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
    if (i >= quads) continue;
    uint32_t q;
    if (s > 0.0f && s < INFINITY)
      q = codes_of(y[j], s);
    else   // 127 / max overflows, or y did: as the quantization of the fp32 row has it
      q = pack4_i8(quant_one(y[j].x, s), quant_one(y[j].y, s), quant_one(y[j].z, s),
                   quant_one(y[j].w, s));
    st_global<uint32_t>(xq + 4 * i, q);
  }
  if (t == 0) st_global<float>(x_scale, s);
}

template <int WAVES, int VEC>
__global__ void __launch_bounds__(64 * WAVES) norm_kernel(NormArgs a) {
  __shared__ RowShared<WAVES> sh;
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.M) return;
  const int t = threadIdx.x, quads = a.K >> 2;
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

// g u / (1 + 2^t), t = -g log2 e = n + f: 2^f by the polynomial of degree 9 whose
// relative error on [-1/2, 1/2] is smallest (2^-46.1, by Remez exchange on values of
// 45 digits), n in the exponent's bits, the quotient by the reciprocal's estimate and
// one Newton step: off by less than 2^-44 before the one rounding to fp32.  (The
// operations count here: 1800 rows of 8960 took 42 us with the library's exp and a
// division.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr double kLog2e = 0x1.71547652b82fep+0;
  constexpr double kRound = 0x1.8p52;   // t + kRound holds n in its low bits
  const double x = (double)g, top = x * (double)u;
  const double d = -fmin(fmax(x, -700.0), 700.0);   // (beyond, the result is 0 or g u)
  const double shifted = __builtin_fma(d, kLog2e, kRound), n = shifted - kRound;
  const double f = __builtin_fma(d, kLog2e, -n);
  double e = 0x1.b3f42370feb32p-24;
  e = __builtin_fma(e, f, 0x1.63edf108fa336p-20);
  e = __builtin_fma(e, f, 0x1.ffce245eb98ddp-17);
  e = __builtin_fma(e, f, 0x1.43088fca981a8p-13);
  e = __builtin_fma(e, f, 0x1.5d87fd9012c5bp-10);
  e = __builtin_fma(e, f, 0x1.3b2ab72a10992p-7);
  e = __builtin_fma(e, f, 0x1.c6b08d70d1ffdp-5);
  e = __builtin_fma(e, f, 0x1.ebfbdff81570dp-3);
  e = __builtin_fma(e, f, 0x1.62e42fefa3752p-1);
  e = __builtin_fma(e, f, 0x1.0000000000039p+0);
  const uint64_t scaled = __builtin_bit_cast(uint64_t, e) +
                          ((uint64_t)(uint32_t)__builtin_bit_cast(uint64_t, shifted) << 52);
  const double under = 1.0 + __builtin_bit_cast(double, scaled);
  double r = __builtin_amdgcn_rcp(under);
  r = __builtin_fma(__builtin_fma(-under, r, 1.0), r, r);
  return (float)(top * r);
}

template <int WAVES, int VEC>
__global__ void __launch_bounds__(64 * WAVES) gate_kernel(GateArgs a) {
  __shared__ RowShared<WAVES> sh;
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.M) return;
  const int t = threadIdx.x, quads = a.K >> 2;
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

// fp32 rows alone: no row has to be held, a quad a thread, as many threads a row as it
// has quads, up to 256 (always 256: 100,000 rows of 64 34 us, 13 so).
__global__ void __launch_bounds__(256) gate_flat_kernel(GateArgs a) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.K >> 2) return;
  for (int64_t row = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; row < a.M;
       row += (int64_t)gridDim.y * blockDim.y) {
    const f32x4 g = ld_global<f32x4>(a.gate + row * a.g_stride + 4 * i);
    const f32x4 u = ld_global<f32x4>(a.up + row * a.u_stride + 4 * i);
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = silu_mul(g[e], u[e]);
    st_global<f32x4>(a.y + row * a.K + 4 * i, y);
  }
}

dim3 row_grid(int64_t blocks) {
  const int64_t axes = (blocks + kAxis - 1) / kAxis;
  return dim3((unsigned)((blocks + axes - 1) / axes), (unsigned)axes);
}

}  // namespace

// A row's values are held by as few waves as their registers allow at full
// occupancy: 1, 2 and 4 waves with 2 quads a lane up to 512, 1024 and 2048 values, 8
// with 5 up to 10240, 16 with 8 beyond.  (1800 rows of 1536: 8.8 us, 10.6 with a wave a
// row and 6 quads a lane; 16 of them 2.7 against 4.3.  1800 gated rows of 8960: 33.3
// us, 35 with 4 waves and 9 quads, 40 with 16 waves and 3.  With 4 waves a row 16,571
// rows of 100 take 24.7 us, 9.3 with one; 30,000 gated rows of 1000 in 8 bits 64, 41
// with two.)
hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t stream) {
  if (a.K <= 512)
    norm_kernel<1, 2><<<row_grid(a.M), 64, 0, stream>>>(a);
  else if (a.K <= 1024)
    norm_kernel<2, 2><<<row_grid(a.M), 128, 0, stream>>>(a);
  else if (a.K <= 2048)
    norm_kernel<4, 2><<<row_grid(a.M), 256, 0, stream>>>(a);
  else if (a.K <= 10240)
    norm_kernel<8, 5><<<row_grid(a.M), 512, 0, stream>>>(a);
  else
    norm_kernel<16, 8><<<row_grid(a.M), 1024, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_silu_mul(const GateArgs &a, hipStream_t stream) {
  const int quads = a.K / 4;
  int across = 1;
  while (across < quads && across < 256) across *= 2;
  const int rows = 256 / across;
  if (!a.xq)
    gate_flat_kernel<<<dim3((quads + across - 1) / across, std::min((a.M + rows - 1) / rows, 65535)),
                       dim3(across, rows), 0, stream>>>(a);
  else if (a.K <= 512)
    gate_kernel<1, 2><<<row_grid(a.M), 64, 0, stream>>>(a);
  else if (a.K <= 1024)
    gate_kernel<2, 2><<<row_grid(a.M), 128, 0, stream>>>(a);
  else if (a.K <= 2048)
    gate_kernel<4, 2><<<row_grid(a.M), 256, 0, stream>>>(a);
  else if (a.K <= 10240)
    gate_kernel<8, 5><<<row_grid(a.M), 512, 0, stream>>>(a);
  else
    gate_kernel<16, 8><<<row_grid(a.M), 1024, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace bitnet
