// Device views and launchers of the paged key-value cache and of beam search.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bitnet_tm.h"

namespace bitnet {

// One layer of the cache, as the kernels see it (strides in elements).
struct KvView {
  void *k, *v;
  float *k_scale, *v_scale;
  int64_t page_stride, head_stride, token_stride;
  int32_t pages, kv_heads;
  int32_t page_shift;   // log2(page_size)
};

constexpr int kMaxRows = BITNET_MAX_ROWS;
constexpr int kMaxWidth = 32;   // beams of one group

// kv.hip
struct KvMapArgs {
  const int32_t *new_lens, *state_in;
  int32_t *state_out, *starts, *slots, *positions, *rows, *status;
  int32_t *tables, *owned, *free_pages;
  int32_t B, max_pages, pages, page_shift;
  int64_t T;
};
hipError_t launch_kv_map(const KvMapArgs &a, hipStream_t stream);

struct KvAppendArgs {
  KvView c;
  const float *q, *k, *v, *cos, *sin;
  float *q_out;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *slots, *positions;
  int32_t q_heads, max_pos;
  int64_t T;
};
hipError_t launch_kv_append(const KvAppendArgs &a, int dtype, int head_dim, hipStream_t stream);

struct ReorderArgs {
  KvView c;   // layer 0
  int64_t layer_stride;
  int32_t layers, head_dim, elem_bytes;
  int32_t B, W, max_pages;
  const int32_t *parents, *lens, *tables_in;
  int32_t *tables_out;
};
hipError_t launch_beam_reorder(const ReorderArgs &a, hipStream_t stream);

// attention.hip
struct AttendArgs {
  KvView c;
  const float *q;
  int64_t q_stride;
  const int32_t *tables, *rows, *lens;
  int32_t T, q_heads, table_rows, max_pages, max_len;
  float scale;
  float *out, *lse;
  uint8_t *ws;
};
size_t attend_workspace_bytes(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                              int64_t max_len);
hipError_t launch_attend(const AttendArgs &a, int dtype, int head_dim, hipStream_t stream);

// beam.hip
struct SelectArgs {
  const float *logits, *scores_in;
  const int32_t *finished_in;
  float *scores_out;
  int32_t *tokens, *parents, *finished_out;
  int64_t ld;
  int32_t B, W, V, eos;
  uint8_t *ws;
};
size_t select_workspace_bytes(int64_t B, int64_t W, int64_t V);
hipError_t launch_beam_select(const SelectArgs &a, hipStream_t stream);

// ---- reductions in registers ------------------------------------------------

// Over the four lanes 16 apart.  The exchanges put rows 0, 2 (halves 0) beside
// rows 1, 3 (halves 1).
__device__ __forceinline__ float across4(float v) {   // maximum
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t p0 = p[0], p1 = p[1];   // (a bit cast of an element itself reads element 0)
  const float m = fmaxf(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1));
  const uint32_t b = __builtin_bit_cast(uint32_t, m);
  const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t q0 = q[0], q1 = q[1];
  return fmaxf(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
}
__device__ __forceinline__ float sum4(float v) {
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t p0 = p[0], p1 = p[1];
  const float m = __builtin_bit_cast(float, p0) + __builtin_bit_cast(float, p1);
  const uint32_t b = __builtin_bit_cast(uint32_t, m);
  const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t q0 = q[0], q1 = q[1];
  return __builtin_bit_cast(float, q0) + __builtin_bit_cast(float, q1);
}
// Maximum or sum over the 16 lanes of a row: quads, then mirrored halves.
template <int CTRL, bool MAX>
__device__ __forceinline__ float row_step(float v) {
  const float o = __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
  return MAX ? fmaxf(v, o) : v + o;
}
template <bool MAX>
__device__ __forceinline__ float across16(float v) {
  v = row_step<0xB1, MAX>(v);    // quad_perm 1,0,3,2
  v = row_step<0x4E, MAX>(v);    // quad_perm 2,3,0,1
  v = row_step<0x141, MAX>(v);   // row_half_mirror
  return row_step<0x140, MAX>(v);   // row_mirror
}

// Sum over the wave, in every lane.
template <int CTRL>
__device__ __forceinline__ double row_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_total(double v) {
  v = row_add<0xB1>(v);
  v = row_add<0x4E>(v);
  v = row_add<0x141>(v);
  v = row_add<0x140>(v);
  uint64_t b = __builtin_bit_cast(uint64_t, v);
  const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
  const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  const uint64_t x0 = ((uint64_t)h[0] << 32) | l[0], x1 = ((uint64_t)h[1] << 32) | l[1];
  v = __builtin_bit_cast(double, x0) + __builtin_bit_cast(double, x1);
  b = __builtin_bit_cast(uint64_t, v);
  const auto m = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
  const auto n = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  const uint64_t y0 = ((uint64_t)n[0] << 32) | m[0], y1 = ((uint64_t)n[1] << 32) | m[1];
  return __builtin_bit_cast(double, y0) + __builtin_bit_cast(double, y1);
}

}  // namespace bitnet
