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

}  // namespace bitnet
