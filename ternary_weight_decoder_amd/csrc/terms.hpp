// What the attention kernels share: fp32 values as sums of 16-bit terms, 8-bit
// codes as fp16, powers of two, partial results across the chip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bitnet_device.hpp"

namespace bitnet {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

#define BITNET_LDS __attribute__((address_space(3)))

// Partial results cross the chip through device-coherent accesses (cache
// policy sc1), so that no workgroup has to write back or invalidate a cache,
// as a fence of device scope does.
constexpr int kDeviceAux = 16;
__device__ __forceinline__ void st_device(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, f32x4 v,
                                          uint32_t base = 0) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, off, base, kDeviceAux);
}
__device__ __forceinline__ f32x4 ld_device(__amdgpu_buffer_rsrc_t rsrc, uint32_t off,
                                           uint32_t base = 0) {
  return __builtin_bit_cast(f32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, base, kDeviceAux));
}

// x as the sum of three bf16 terms (8 bits each), the largest first.
__device__ __forceinline__ void terms_bf16(const float (&x)[8], bf16x8 (&u)[3]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    f32x2 r = {x[e], x[e + 1]};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const bf16x2 b = __builtin_convertvector(r, bf16x2);
      u[i][e] = b.x;
      u[i][e + 1] = b.y;
      r.x -= (float)b.x;
      r.y -= (float)b.y;
    }
  }
}
// x as the sum of two fp16 terms (11 bits each).
__device__ __forceinline__ void terms_f16(const float (&x)[8], f16x8 (&u)[2]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // Pinned: where x is a product the compiler takes the first term once from
    // the rounded product and, for the difference, once from an fma that
    // rounds the exact product to fp16 (v_fma_mixlo_f16): next to the middle
    // between two fp16 numbers they are not the same.
    float y = x[e];
    asm("" : "+v"(y));
    u[0][e] = (_Float16)y;
    u[1][e] = (_Float16)(y - (float)u[0][e]);
  }
}

// The same in packed conversions: four operations for two values.  The difference
// is one fma of the fp16 half; x holds no product's result that is still exact.
__device__ __forceinline__ void terms_f16_packed(const float (&x)[8], f16x8 (&u)[2]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const f32x2 y = {x[e], x[e + 1]};
    const f16x2 a = __builtin_convertvector(y, f16x2);
    f32x2 r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r.x) : "v"(a), "v"(y.x));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r.y) : "v"(a), "v"(y.y));
    const f16x2 b = __builtin_convertvector(r, f16x2);
    u[0][e] = a.x;
    u[0][e + 1] = a.y;
    u[1][e] = b.x;
    u[1][e + 1] = b.y;
  }
}

// Eight int8 codes as fp16: code + 128 beside the bits of 1024 is 1152 + code,
// exactly, and the difference to 1152 is exact too.
__device__ __forceinline__ f16x8 codes_f16(uint32_t lo, uint32_t hi) {
  f16x8 r;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t u = (w ? hi : lo) ^ 0x80808080u;
    const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);   // bytes 0, 1
    const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);   // bytes 2, 3
    const f16x2 k = {(_Float16)1152.0f, (_Float16)1152.0f};
    const f16x2 x = __builtin_bit_cast(f16x2, a) - k, y = __builtin_bit_cast(f16x2, b) - k;
    r[4 * w] = x.x;
    r[4 * w + 1] = x.y;
    r[4 * w + 2] = y.x;
    r[4 * w + 3] = y.y;
  }
  return r;
}

// With 256 channels the sums of the products live in accumulation registers.
// The compiler puts no wait states between a product and a branch whose target
// reads them back (v_accvgpr_read), and the read then returns the old value:
// the waits are written here, with the registers passed through, so that every
// read comes after them.
template <int D, typename Sum, int N>
__device__ __forceinline__ void settle(Sum (&x)[N]) {
  if constexpr (D == 256) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+a"(x[i]));   // every product is issued
    asm volatile("s_nop 15\n\ts_nop 3");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+a"(x[i]));   // no read comes before
  }
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The power of two above x (x >= 0, below 2^126), at least 2^-100.
__device__ __forceinline__ float pow2_above(float x) {
  const uint32_t e = __builtin_bit_cast(uint32_t, x) & 0x7f800000u;
  const uint32_t lo = (127u - 100u) << 23;
  return __builtin_bit_cast(float, max(e + 0x00800000u, lo));
}
__device__ __forceinline__ float pow2_inverse(float p) {   // of a power of two
  return __builtin_bit_cast(float, (254u << 23) - __builtin_bit_cast(uint32_t, p));
}

}  // namespace bitnet
