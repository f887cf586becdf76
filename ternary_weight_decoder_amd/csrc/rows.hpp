// Launchers of the calls between the projections, and of token log probabilities.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bitnet {

constexpr int kMaxRowWidth = 32768;   // of the norm and the gated activation

// rows.hip
struct NormArgs {
  const float *x, *residual, *weight;
  float *sum, *y;
  int8_t *xq;
  float *x_scale;
  int64_t x_stride, r_stride;
  int32_t M, K;
  float eps;
};
hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t stream);

struct GateArgs {
  const float *gate, *up;
  float *y;
  int8_t *xq;
  float *x_scale;
  int64_t g_stride, u_stride;
  int32_t M, K;
};
hipError_t launch_silu_mul(const GateArgs &a, hipStream_t stream);

// logprobs.hip
struct LogprobArgs {
  const float *logits;
  const int32_t *tokens;
  float *logprobs, *entropy, *top_logprobs;
  int32_t *top_tokens;
  int64_t ld;
  int32_t R, V, top;
  uint8_t *ws;
};
size_t logprobs_workspace_bytes(int64_t R, int64_t V, int64_t top);
hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t stream);

}  // namespace bitnet
