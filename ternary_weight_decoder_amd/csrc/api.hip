// C ABI of the ternary projection library: argument checks, workspace layout
// and dispatch to the gfx950 kernels.  Nothing is launched unless every check
// passes; no device memory is allocated here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>
#include <utility>

#include "bitnet_internal.hpp"
#include "bitnet_variants.hpp"
#include "kv.hpp"
#include "bitnet_tm.h"

using namespace bitnet;

// Built-in workspace of bitnet_ternary_matmul_noalloc, for callers that cannot
// allocate.  Every device the library runs on holds its own copy from module
// load until the process ends.  In host code `scratch` only names the symbol:
// its device address on the current device comes from hipGetSymbolAddress,
// looked up once per device (scratch_address) and passed to the kernels.
static __device__ __align__(256) uint8_t scratch[BITNET_SCRATCH_BYTES];

namespace {

constexpr int64_t kLimit = (int64_t)1 << 31;  // M*K, N*K, M*N must stay below this

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool shape_ok(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1) return false;
  if (K % 128 != 0) return false;  // 128 codes per packing unit
  if (M >= kLimit || N >= kLimit || K >= kLimit) return false;
  if (M * K >= kLimit || N * K >= kLimit || M * N >= kLimit) return false;
  // Byte offsets of the fp32 output, including a 128-row tile past M, stay 32-bit.
  if ((M + 128) * N * 4 >= kLimit) return false;
  return true;
}

// Per-device record of the architecture check: 0 unknown, 1 gfx950, 2 other.
constexpr int kMaxDevices = 64;
std::atomic<int> g_arch_ok[kMaxDevices];

bitnet_status device_check() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return BITNET_ERR_HIP;
  if (dev < 0 || dev >= kMaxDevices) return BITNET_ERR_DEVICE;
  int v = g_arch_ok[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return BITNET_ERR_HIP;
    v = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_arch_ok[dev].store(v, std::memory_order_relaxed);
  }
  return v == 1 ? BITNET_OK : BITNET_ERR_DEVICE;
}

bitnet_status from_hip(hipError_t e) { return e == hipSuccess ? BITNET_OK : BITNET_ERR_HIP; }

// Device address of `scratch` on each device (see its definition above).
constexpr size_t kScratchBytes = BITNET_SCRATCH_BYTES;
std::atomic<void *> g_scratch[kMaxDevices];
std::mutex g_scratch_mu;

bitnet_status scratch_address(void **out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return BITNET_ERR_HIP;
  if (dev < 0 || dev >= kMaxDevices) return BITNET_ERR_DEVICE;
  void *p = g_scratch[dev].load(std::memory_order_acquire);
  if (!p) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch[dev].load(std::memory_order_relaxed);
    if (!p) {
      if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return BITNET_ERR_HIP;
      if (!aligned(p, 256)) return BITNET_ERR_HIP;
      g_scratch[dev].store(p, std::memory_order_release);
    }
  }
  *out = p;
  return BITNET_OK;
}

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

bitnet_status check_problem(int64_t M, const bitnet_problem &p) {
  if (!p.x || !p.packed || !p.w_scale || !p.y) return BITNET_ERR_NULL;
  if (!shape_ok(M, p.N, p.K)) return BITNET_ERR_SHAPE;
  if (!aligned(p.x, 16) || !aligned(p.packed, 16) || !aligned(p.w_scale, 4) ||
      !aligned(p.y, 4))
    return BITNET_ERR_ALIGN;
  return BITNET_OK;
}

// owner[i]: the lowest index of the problems with the same x and K as
// problem i (i itself when there is none).  Such problems read the same rows,
// so they share one quantized copy: a decoder's q, k and v read one input, as
// do its gate and up.  count <= kMaxGroup.
void input_owners(const bitnet_problem *ph, int32_t count, int32_t *owner) {
  int32_t ix[kMaxGroup];
  for (int32_t i = 0; i < count; ++i) ix[i] = i;
  const auto key = [&](int32_t i) {
    return std::make_pair(reinterpret_cast<uintptr_t>(ph[i].x), ph[i].K);
  };
  std::sort(ix, ix + count, [&](int32_t a, int32_t b) {
    return key(a) != key(b) ? key(a) < key(b) : a < b;
  });
  for (int32_t r = 0; r < count;) {
    int32_t e = r;
    while (e < count && key(ix[e]) == key(ix[r])) owner[ix[e++]] = ix[r];
    r = e;
  }
}

// Workspace offsets (256-byte units) of each problem of a group; problems that
// share their input share its region.  count <= kMaxGroup.
size_t group_ws(int64_t M, const bitnet_problem *ph, int32_t count, uint32_t *off,
                int32_t *owner_out = nullptr) {
  int32_t owner_buf[kMaxGroup];
  int32_t *owner = owner_out ? owner_out : owner_buf;
  input_owners(ph, count, owner);
  uint32_t own[kMaxGroup];
  size_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (owner[i] == i) {
      own[i] = (uint32_t)(total / 256);
      total += align256(ws_layout(M, ph[i].K).total);
    } else {
      own[i] = own[owner[i]];
    }
    if (off) off[i] = own[i];
  }
  return total;
}

}  // namespace

extern "C" {

const char *bitnet_status_string(bitnet_status s) {
  switch (s) {
    case BITNET_OK: return "ok";
    case BITNET_ERR_NULL: return "required pointer is NULL";
    case BITNET_ERR_SHAPE: return "shape out of range (M,N,K >= 1, K % 128 == 0, products < 2^31)";
    case BITNET_ERR_ALIGN: return "pointer not aligned as required";
    case BITNET_ERR_WORKSPACE: return "workspace missing or too small";
    case BITNET_ERR_HIP: return "HIP runtime or launch error";
    case BITNET_ERR_DEVICE: return "current device is not a gfx950";
    case BITNET_ERR_ALIAS: return "outputs overlap each other or an input";
    case BITNET_ERR_SCRATCH:
      return "problem needs more workspace than the built-in scratch (bitnet_scratch_bytes())";
    default: return "unknown status";
  }
}

size_t bitnet_packed_bytes(int64_t N, int64_t K) {
  if (N < 1 || K < 1) return 0;
  return (size_t)(N * K / 4);
}

size_t bitnet_ternarize_workspace_bytes(int64_t N) {
  if (N < 1) return 0;
  return (size_t)N * sizeof(double);
}

bitnet_status bitnet_ternarize_pack(const float *W, int64_t N, int64_t K, uint8_t *packed,
                                    float *w_scale, void *workspace, size_t workspace_bytes,
                                    void *stream) {
  if (!W || !packed || !w_scale) return BITNET_ERR_NULL;
  if (!shape_ok(1, N, K)) return BITNET_ERR_SHAPE;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(w_scale, 4)) return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_ternarize_workspace_bytes(N))
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_ternarize_pack(W, (int)N, (int)K, packed, w_scale,
                                        reinterpret_cast<double *>(workspace),
                                        as_stream(stream)));
}

bitnet_status bitnet_quant_act(const float *x, int64_t M, int64_t K, int8_t *xq,
                               float *x_scale, void *stream) {
  if (!x || !xq || !x_scale) return BITNET_ERR_NULL;
  if (!shape_ok(M, 1, K)) return BITNET_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(x_scale, 4)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_quant_rows(x, (int)M, (int)K, xq, nullptr, x_scale, nullptr, nullptr,
                                    as_stream(stream)));
}

size_t bitnet_matmul_workspace_bytes(int64_t M, int64_t K) {
  if (M < 1 || K < 1) return 0;
  return ws_layout(M, K).total;
}

static bitnet_status matmul_from_ws(int64_t M, int64_t N, int64_t K, const uint8_t *packed,
                                    const float *w_scale, float *y, uint8_t *ws,
                                    int32_t *acc_out, hipStream_t s) {
  const WsLayout L = ws_layout(M, K);
  const int8_t *xqp = reinterpret_cast<const int8_t *>(ws + L.xq);
  const float *xs = reinterpret_cast<const float *>(ws + L.scale);
  const int32_t *rs = reinterpret_cast<const int32_t *>(ws + L.rowsum);
  if (M <= kGemvMaxM)
    return from_hip(launch_gemv((int)M, (int)N, (int)K, xqp, xs, rs, packed, w_scale, y,
                                acc_out, s));
  return from_hip(
      launch_gemm((int)M, (int)N, (int)K, xqp, xs, rs, packed, w_scale, y, acc_out, s));
}

// Argument checks of the single projection, apart from the workspace.
static bitnet_status matmul_args_ok(int64_t M, int64_t N, int64_t K, const float *x,
                                    const uint8_t *packed, const float *w_scale, float *y,
                                    int8_t *xq_out, float *x_scale_out, int32_t *acc_out) {
  if (!x || !packed || !w_scale || !y) return BITNET_ERR_NULL;
  if (!shape_ok(M, N, K)) return BITNET_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(w_scale, 4) || !aligned(y, 4) ||
      (xq_out && !aligned(xq_out, 16)) || (x_scale_out && !aligned(x_scale_out, 4)) ||
      (acc_out && !aligned(acc_out, 4)))
    return BITNET_ERR_ALIGN;
  return BITNET_OK;
}

// The single projection once its arguments are checked; `workspace` holds at
// least bitnet_matmul_workspace_bytes(M, K) bytes, 256-byte aligned.
static bitnet_status matmul_run(int64_t M, int64_t N, int64_t K, const float *x,
                                const uint8_t *packed, const float *w_scale, float *y,
                                void *workspace, int8_t *xq_out, float *x_scale_out,
                                int32_t *acc_out, hipStream_t s) {
  bitnet_status st;
  if (M <= kGemvMaxM && gemv_fusable(M, K))
    return from_hip(launch_gemv_fused((int)M, (int)N, (int)K, x, packed, w_scale, y, xq_out,
                                      x_scale_out, acc_out, s));
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  const WsLayout L = ws_layout(M, K);
  st = from_hip(launch_quant_rows(x, (int)M, (int)K, xq_out,
                                  reinterpret_cast<int8_t *>(ws + L.xq),
                                  reinterpret_cast<float *>(ws + L.scale), x_scale_out,
                                  reinterpret_cast<int32_t *>(ws + L.rowsum), s));
  if (st != BITNET_OK) return st;
  return matmul_from_ws(M, N, K, packed, w_scale, y, ws, acc_out, s);
}

bitnet_status bitnet_ternary_matmul(int64_t M, int64_t N, int64_t K, const float *x,
                                    const uint8_t *packed, const float *w_scale, float *y,
                                    void *workspace, size_t workspace_bytes, int8_t *xq_out,
                                    float *x_scale_out, int32_t *acc_out, void *stream) {
  bitnet_status st = matmul_args_ok(M, N, K, x, packed, w_scale, y, xq_out, x_scale_out, acc_out);
  if (st != BITNET_OK) return st;
  if (!workspace || workspace_bytes < bitnet_matmul_workspace_bytes(M, K))
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  st = device_check();
  if (st != BITNET_OK) return st;
  return matmul_run(M, N, K, x, packed, w_scale, y, workspace, xq_out, x_scale_out, acc_out,
                    as_stream(stream));
}

size_t bitnet_scratch_bytes(void) { return kScratchBytes; }

bitnet_status bitnet_ternary_matmul_noalloc(int64_t M, int64_t N, int64_t K, const float *x,
                                            const uint8_t *packed, const float *w_scale,
                                            float *y, int8_t *xq_out, float *x_scale_out,
                                            int32_t *acc_out, void *stream) {
  bitnet_status st = matmul_args_ok(M, N, K, x, packed, w_scale, y, xq_out, x_scale_out, acc_out);
  if (st != BITNET_OK) return st;
  if (bitnet_matmul_workspace_bytes(M, K) > kScratchBytes) return BITNET_ERR_SCRATCH;
  st = device_check();
  if (st != BITNET_OK) return st;
  void *ws = nullptr;
  st = scratch_address(&ws);
  if (st != BITNET_OK) return st;
  return matmul_run(M, N, K, x, packed, w_scale, y, ws, xq_out, x_scale_out, acc_out,
                    as_stream(stream));
}

bitnet_status bitnet_ternary_matmul_q8(int64_t M, int64_t N, int64_t K, const int8_t *xq,
                                       const float *x_scale, const uint8_t *packed,
                                       const float *w_scale, float *y, void *workspace,
                                       size_t workspace_bytes, int32_t *acc_out,
                                       void *stream) {
  if (!xq || !x_scale || !packed || !w_scale || !y) return BITNET_ERR_NULL;
  if (!shape_ok(M, N, K)) return BITNET_ERR_SHAPE;
  if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(packed, 16) ||
      !aligned(w_scale, 4) || !aligned(y, 4) || (acc_out && !aligned(acc_out, 4)))
    return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_matmul_workspace_bytes(M, K))
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  hipStream_t s = as_stream(stream);
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  const WsLayout L = ws_layout(M, K);
  st = from_hip(launch_permute_q8(xq, x_scale, (int)M, (int)K,
                                  reinterpret_cast<int8_t *>(ws + L.xq),
                                  reinterpret_cast<float *>(ws + L.scale),
                                  reinterpret_cast<int32_t *>(ws + L.rowsum), s));
  if (st != BITNET_OK) return st;
  return matmul_from_ws(M, N, K, packed, w_scale, y, ws, acc_out, s);
}

size_t bitnet_grouped_workspace_bytes(int64_t M, const bitnet_problem *problems_host,
                                      int32_t count) {
  if (M < 1 || !problems_host || count < 1 || count > kMaxGroup) return 0;
  return group_ws(M, problems_host, count, nullptr);
}

bitnet_status bitnet_ternary_matmul_grouped(int64_t M, const bitnet_problem *problems_dev,
                                            int32_t count, const bitnet_problem *problems_host,
                                            void *workspace, size_t workspace_bytes,
                                            void *stream) {
  if (!problems_dev || !problems_host) return BITNET_ERR_NULL;
  if (count < 1 || count > kMaxGroup) return BITNET_ERR_SHAPE;
  if (!aligned(problems_dev, 8)) return BITNET_ERR_ALIGN;
  for (int32_t i = 0; i < count; ++i) {
    bitnet_status st = check_problem(M, problems_host[i]);
    if (st != BITNET_OK) return st;
  }
  GroupTable tab;
  std::memset(&tab, 0, sizeof(tab));
  tab.count = count;
  tab.M = (int32_t)M;
  int32_t owner[kMaxGroup];
  const size_t need = group_ws(M, problems_host, count, tab.ws_off, owner);
  if (!workspace || workspace_bytes < need) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;

  // Dispatch order: longest K first, so the longest-running workgroups start
  // early and the tail of the launch is made of short ones.
  int32_t idx[kMaxGroup];
  for (int32_t i = 0; i < count; ++i) idx[i] = i;
  std::stable_sort(idx, idx + count, [&](int32_t a, int32_t b) {
    return problems_host[a].K > problems_host[b].K;
  });
  const bool gemv = M <= kGemvMaxM;
  int64_t kmax = 0;
  for (int32_t i = 0; i < count; ++i) kmax = std::max(kmax, problems_host[i].K);
  const bool fused = gemv && gemv_fusable(M, kmax);
  auto fill_blocks = [&](bool split) -> uint64_t {
    uint64_t total = 0;
    for (int32_t s = 0; s < count; ++s) {
      const bitnet_problem &p = problems_host[idx[s]];
      total += gemv ? (uint64_t)gemv_blocks(p.N, p.K, split) : (uint64_t)gemm_blocks(M, p.N);
      tab.blk_end[s] = (uint32_t)std::min<uint64_t>(total, UINT32_MAX);
      tab.order[s] = (uint16_t)idx[s];
    }
    return total;
  };
  uint64_t total = fill_blocks(false);
  if (total >= ((uint64_t)1 << 31)) return BITNET_ERR_SHAPE;
  // A single-row launch too small to fill the chip splits K across waves.
  if (fused && total < (uint64_t)kGemvSplitBelow) {
    tab.split = 1;
    total = fill_blocks(true);
  }
  hipStream_t hs = as_stream(stream);
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  // Workgroups of each dispatch slot, for the XCD schedule of the main launch.
  auto schedule = [&]() {
    uint32_t tiles[kMaxGroup];
    for (int32_t s = 0; s < count; ++s) {
      const bitnet_problem &p = problems_host[tab.order[s]];
      tiles[s] = gemv ? (uint32_t)gemv_blocks(p.N, p.K, tab.split != 0)
                      : (uint32_t)gemm_blocks(M, p.N);
    }
    xcd_schedule(tab, problems_host, tiles);
  };
  if (fused) {
    schedule();
    return from_hip(launch_gemv_grouped(problems_dev, tab, ws, true, kmax, hs));
  }
  QuantTable qt;
  std::memset(&qt, 0, sizeof(qt));
  qt.count = 0;
  qt.M = (int32_t)M;
  // One quantization per distinct input.
  uint64_t qtotal = 0;
  for (int32_t s = 0; s < count; ++s) {
    if (owner[idx[s]] != idx[s]) continue;
    qtotal += (uint64_t)quant_grouped_blocks(M, problems_host[idx[s]].K);
    if (qtotal >= ((uint64_t)1 << 31)) return BITNET_ERR_SHAPE;
    qt.wg_end[qt.count] = (uint32_t)qtotal;
    qt.order[qt.count] = (uint16_t)idx[s];
    ++qt.count;
  }
  std::memcpy(qt.ws_off, tab.ws_off, sizeof(qt.ws_off));
  st = from_hip(launch_quant_grouped(problems_dev, qt, ws, hs));
  if (st != BITNET_OK) return st;
  schedule();
  if (gemv) return from_hip(launch_gemv_grouped(problems_dev, tab, ws, false, kmax, hs));
  return from_hip(launch_gemm_grouped(problems_dev, tab, ws, hs));
}

// The prefill part of a grouped call over problems sub[0..n) (indices into
// the whole problem array, whose workspace offsets and input owners are
// given): the quantization launch of the inputs owned inside sub goes on qs,
// the GEMM launch on gs; with ev, gs waits for qs through it in between.
static bitnet_status prefill_chunk(int64_t M, const bitnet_problem *problems_dev,
                                   const bitnet_problem *ph, const int32_t *sub, int32_t n,
                                   const uint32_t *ws_off, const int32_t *owner, uint8_t *ws,
                                   hipStream_t qs, hipStream_t gs, hipEvent_t ev) {
  int32_t idx[kMaxGroup];
  std::copy(sub, sub + n, idx);
  std::stable_sort(idx, idx + n, [&](int32_t a, int32_t b) { return ph[a].K > ph[b].K; });
  GroupTable tab;
  std::memset(&tab, 0, sizeof(tab));
  tab.count = n;
  tab.M = (int32_t)M;
  std::memcpy(tab.ws_off, ws_off, sizeof(tab.ws_off));
  uint32_t tiles[kMaxGroup];
  uint64_t total = 0;
  for (int32_t s = 0; s < n; ++s) {
    tiles[s] = (uint32_t)gemm_blocks(M, ph[idx[s]].N);
    total += tiles[s];
    if (total >= ((uint64_t)1 << 31)) return BITNET_ERR_SHAPE;
    tab.blk_end[s] = (uint32_t)total;
    tab.order[s] = (uint16_t)idx[s];
  }
  QuantTable qt;
  std::memset(&qt, 0, sizeof(qt));
  qt.M = (int32_t)M;
  uint64_t qtotal = 0;
  for (int32_t s = 0; s < n; ++s) {
    if (owner[idx[s]] != idx[s]) continue;   // owned in this chunk or an earlier one
    qtotal += (uint64_t)quant_grouped_blocks(M, ph[idx[s]].K);
    if (qtotal >= ((uint64_t)1 << 31)) return BITNET_ERR_SHAPE;
    qt.wg_end[qt.count] = (uint32_t)qtotal;
    qt.order[qt.count] = (uint16_t)idx[s];
    ++qt.count;
  }
  std::memcpy(qt.ws_off, ws_off, sizeof(qt.ws_off));
  if (qt.count > 0) {
    bitnet_status st = from_hip(launch_quant_grouped(problems_dev, qt, ws, qs));
    if (st != BITNET_OK) return st;
  }
  if (ev) {
    if (hipEventRecord(ev, qs) != hipSuccess || hipStreamWaitEvent(gs, ev, 0) != hipSuccess)
      return BITNET_ERR_HIP;
  }
  xcd_schedule(tab, ph, tiles);
  return from_hip(launch_gemm_grouped(problems_dev, tab, ws, gs));
}

bitnet_status bitnet_ternary_matmul_grouped_overlap(int64_t M, const bitnet_problem *problems_dev,
                                                    int32_t count,
                                                    const bitnet_problem *problems_host,
                                                    int32_t nchunks, void *workspace,
                                                    size_t workspace_bytes, void *stream,
                                                    void *aux_stream) {
  if (M <= kGemvMaxM || nchunks <= 1 || aux_stream == stream)
    return bitnet_ternary_matmul_grouped(M, problems_dev, count, problems_host, workspace,
                                         workspace_bytes, stream);
  if (!problems_dev || !problems_host) return BITNET_ERR_NULL;
  if (count < 1 || count > kMaxGroup || nchunks > count || nchunks > BITNET_MAX_CHUNKS)
    return BITNET_ERR_SHAPE;
  if (!aligned(problems_dev, 8)) return BITNET_ERR_ALIGN;
  for (int32_t i = 0; i < count; ++i) {
    bitnet_status st = check_problem(M, problems_host[i]);
    if (st != BITNET_OK) return st;
  }
  uint32_t ws_off[kMaxGroup] = {0};
  int32_t owner[kMaxGroup];
  const size_t need = group_ws(M, problems_host, count, ws_off, owner);
  if (!workspace || workspace_bytes < need) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  // Chunks: contiguous runs of problems of about equal contraction work.
  uint64_t work_total = 0;
  for (int32_t i = 0; i < count; ++i)
    work_total += (uint64_t)problems_host[i].N * (uint64_t)problems_host[i].K;
  int32_t first[BITNET_MAX_CHUNKS + 1];
  int32_t c = 0;
  uint64_t acc = 0;
  first[0] = 0;
  for (int32_t i = 0; i < count && c + 1 < nchunks; ++i) {
    acc += (uint64_t)problems_host[i].N * (uint64_t)problems_host[i].K;
    if (acc * (uint64_t)nchunks >= work_total * (uint64_t)(c + 1) && i + 1 < count)
      first[++c] = i + 1;
  }
  const int32_t chunks = c + 1;
  first[chunks] = count;
  // Launch sizes over the whole call: every chunk's launches are smaller, so
  // no chunk can fail its own size check once some chunks are queued.
  uint64_t gemm_total = 0, quant_total = 0;
  for (int32_t i = 0; i < count; ++i) {
    gemm_total += (uint64_t)gemm_blocks(M, problems_host[i].N);
    if (owner[i] == i) quant_total += (uint64_t)quant_grouped_blocks(M, problems_host[i].K);
  }
  if (gemm_total >= ((uint64_t)1 << 31) || quant_total >= ((uint64_t)1 << 31))
    return BITNET_ERR_SHAPE;
  // Every event is created before the first launch, so a failure to create
  // one leaves nothing queued.  Events are released after use; HIP frees them
  // once their pending work completes.
  hipEvent_t ev[BITNET_MAX_CHUNKS + 1];
  int32_t made = 0;
  for (; made <= chunks; ++made)
    if (hipEventCreateWithFlags(&ev[made], hipEventDisableTiming) != hipSuccess) break;
  if (made <= chunks) {
    for (int32_t k = 0; k < made; ++k) hipEventDestroy(ev[k]);
    return BITNET_ERR_HIP;
  }
  hipStream_t gs = as_stream(stream), qs = as_stream(aux_stream);
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  // The auxiliary stream starts after everything already queued on the main
  // stream (the inputs, and an earlier call's contractions over the same
  // workspace).
  st = (hipEventRecord(ev[chunks], gs) == hipSuccess &&
        hipStreamWaitEvent(qs, ev[chunks], 0) == hipSuccess)
           ? BITNET_OK
           : BITNET_ERR_HIP;
  int32_t sub[kMaxGroup];
  for (int32_t k = 0; k < chunks && st == BITNET_OK; ++k) {
    const int32_t n = first[k + 1] - first[k];
    for (int32_t i = 0; i < n; ++i) sub[i] = first[k] + i;
    st = prefill_chunk(M, problems_dev, problems_host, sub, n, ws_off, owner, ws, qs, gs, ev[k]);
  }
  for (int32_t k = 0; k <= chunks; ++k) hipEventDestroy(ev[k]);
  return st;
}

// I8_S shapes: K a multiple of 64 (one GEMM step), the same size limits as the
// ternary path.
static bool i8_shape_ok(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 64 || K % 64 != 0) return false;
  if (M >= kLimit || N >= kLimit || K >= kLimit) return false;
  if (M * K >= kLimit || N * K >= kLimit || M * N >= kLimit) return false;
  if ((M + 128) * N * 4 >= kLimit) return false;
  return true;
}

size_t bitnet_i8_quant_workspace_bytes(void) { return 256; }

bitnet_status bitnet_i8_quant_weights(const float *W, int64_t N, int64_t K, int8_t *q,
                                      float *w_scale, void *workspace, size_t workspace_bytes,
                                      void *stream) {
  if (!W || !q || !w_scale) return BITNET_ERR_NULL;
  if (!i8_shape_ok(1, N, K)) return BITNET_ERR_SHAPE;
  if (!aligned(W, 16) || !aligned(q, 16) || !aligned(w_scale, 4)) return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_i8_quant_workspace_bytes())
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_i8_quant_weights(W, N, K, q, w_scale,
                                          reinterpret_cast<uint32_t *>(workspace),
                                          as_stream(stream)));
}

size_t bitnet_i8_linear_workspace_bytes(int64_t M, int64_t K) {
  if (M < 1 || K < 1) return 0;
  return align256((size_t)(M * K)) + align256((size_t)M * 4);
}

static bitnet_status i8_linear_common(int64_t M, int64_t N, int64_t K, const float *x,
                                      const int8_t *q, const float *w_scale, bool per_channel,
                                      const float *bias, int32_t relu, float *y, void *workspace,
                                      size_t workspace_bytes, int32_t *acc_out, void *stream) {
  if (!x || !q || !w_scale || !y) return BITNET_ERR_NULL;
  if (!i8_shape_ok(M, N, K)) return BITNET_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(w_scale, 4) || !aligned(y, 4) ||
      (bias && !aligned(bias, 4)) || (acc_out && !aligned(acc_out, 4)))
    return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_i8_linear_workspace_bytes(M, K))
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  hipStream_t s = as_stream(stream);
  uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
  int8_t *xq = reinterpret_cast<int8_t *>(ws);
  float *xs = reinterpret_cast<float *>(ws + align256((size_t)(M * K)));
  st = from_hip(launch_quant_rows(x, (int)M, (int)K, xq, nullptr, xs, nullptr, nullptr, s));
  if (st != BITNET_OK) return st;
  return from_hip(launch_i8_gemm((int)M, (int)N, (int)K, xq, xs, q, w_scale, per_channel, bias,
                                 relu != 0 ? 1 : 0, y, acc_out, s));
}

bitnet_status bitnet_i8_linear(int64_t M, int64_t N, int64_t K, const float *x, const int8_t *q,
                               const float *w_scale, const float *bias, int32_t relu, float *y,
                               void *workspace, size_t workspace_bytes, int32_t *acc_out,
                               void *stream) {
  return i8_linear_common(M, N, K, x, q, w_scale, false, bias, relu, y, workspace,
                          workspace_bytes, acc_out, stream);
}

bitnet_status bitnet_i8_linear_rows(int64_t M, int64_t N, int64_t K, const float *x,
                                    const int8_t *q, const float *w_scale, const float *bias,
                                    int32_t relu, float *y, void *workspace,
                                    size_t workspace_bytes, int32_t *acc_out, void *stream) {
  return i8_linear_common(M, N, K, x, q, w_scale, true, bias, relu, y, workspace,
                          workspace_bytes, acc_out, stream);
}

bitnet_status bitnet_i8_quant_weights_rows(const float *W, int64_t N, int64_t K, int8_t *q,
                                           float *w_scale, void *stream) {
  if (!W || !q || !w_scale) return BITNET_ERR_NULL;
  if (!i8_shape_ok(1, N, K)) return BITNET_ERR_SHAPE;
  if (!aligned(W, 16) || !aligned(q, 16) || !aligned(w_scale, 4)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_rowq_quant(W, N, K, q, w_scale, false, as_stream(stream)));
}

size_t bitnet_table_bytes(int64_t V, int64_t K) {
  if (!i8_shape_ok(1, V, K)) return 0;
  return table_bytes(V, K);
}

bitnet_status bitnet_table_quant(const float *W, int64_t V, int64_t K, int8_t *table,
                                 float *w_scale, void *stream) {
  if (!W || !table || !w_scale) return BITNET_ERR_NULL;
  if (!i8_shape_ok(1, V, K) || table_bytes(V, K) >= (size_t)kLimit) return BITNET_ERR_SHAPE;
  if (!aligned(W, 16) || !aligned(table, 16) || !aligned(w_scale, 4)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_rowq_quant(W, V, K, table, w_scale, true, as_stream(stream)));
}

bitnet_status bitnet_embed_lookup(const int32_t *ids, int64_t T, const int8_t *q,
                                  const float *w_scale, int64_t N, int64_t K, float *out,
                                  void *stream) {
  if (T == 0) return BITNET_OK;
  if (!ids || !q || !w_scale || !out) return BITNET_ERR_NULL;
  if (T < 0 || T >= kLimit || T * K >= kLimit || !i8_shape_ok(1, N, K) ||
      table_bytes(N, K) >= (size_t)kLimit)
    return BITNET_ERR_SHAPE;
  if (!aligned(ids, 4) || !aligned(q, 16) || !aligned(w_scale, 4) || !aligned(out, 16))
    return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_embed(ids, T, q, w_scale, N, K, out, as_stream(stream)));
}

bitnet_status bitnet_lm_head(int64_t M, int64_t N, int64_t K, const float *x, const int8_t *q,
                             const float *w_scale, float *y, int8_t *xq_out, float *x_scale_out,
                             int32_t *acc_out, void *stream) {
  if (!x || !q || !w_scale || !y) return BITNET_ERR_NULL;
  if (!i8_shape_ok(M, N, K) || M > kGemvMaxM || M * (K + 16) > kLmHeadMaxRows ||
      table_bytes(N, K) >= (size_t)kLimit)
    return BITNET_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(w_scale, 4) || !aligned(y, 4) ||
      (xq_out && !aligned(xq_out, 16)) || (x_scale_out && !aligned(x_scale_out, 4)) ||
      (acc_out && !aligned(acc_out, 4)))
    return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_lm_head((int)M, (int)N, (int)K, x, q, w_scale, y, xq_out, x_scale_out,
                                 acc_out, as_stream(stream)));
}

static bool dw_shape_ok(int64_t B, int64_t T, int64_t C, int64_t k) {
  if (B < 1 || T < 1 || C < 64 || C % 64 != 0 || k < 1 || k > kMaxDwTaps) return false;
  if (B > 65535 || C >= kLimit || T >= kLimit || B * T * C >= kLimit / 4) return false;
  return true;
}

bitnet_status bitnet_i8_dwconv_quant_weights(const float *W, int64_t C, int64_t k, int8_t *q,
                                             float *w_scale, void *stream) {
  if (!W || !q || !w_scale) return BITNET_ERR_NULL;
  if (!dw_shape_ok(1, 1, C, k)) return BITNET_ERR_SHAPE;
  if (!aligned(W, 4) || !aligned(w_scale, 4)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_dw_quant_weights(W, C, k, q, w_scale, as_stream(stream)));
}

size_t bitnet_i8_dwconv_workspace_bytes(int64_t B, int64_t T, int64_t C) {
  if (!dw_shape_ok(B, T, C, 1)) return 0;
  return (size_t)B * dw_chunks(T) * C * sizeof(float);
}

bitnet_status bitnet_i8_dwconv(int64_t B, int64_t T, int64_t C, int64_t k, const float *x,
                               const int8_t *q, const float *w_scale, const float *bias,
                               int32_t relu, float *y, void *workspace, size_t workspace_bytes,
                               int32_t *acc_out, float *x_scale_out, void *stream) {
  if (!x || !q || !w_scale || !y) return BITNET_ERR_NULL;
  if (!dw_shape_ok(B, T, C, k)) return BITNET_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(w_scale, 4) || !aligned(y, 16) ||
      (bias && !aligned(bias, 4)) || (acc_out && !aligned(acc_out, 16)) ||
      (x_scale_out && !aligned(x_scale_out, 4)))
    return BITNET_ERR_ALIGN;
  if (!workspace || workspace_bytes < bitnet_i8_dwconv_workspace_bytes(B, T, C))
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  return from_hip(launch_dwconv((int)B, (int)T, (int)C, (int)k, x, q, w_scale, bias,
                                relu != 0 ? 1 : 0, y, reinterpret_cast<float *>(workspace),
                                acc_out, x_scale_out, as_stream(stream)));
}

bitnet_status bitnet_ternary_matmul_lut_grouped(const bitnet_problem *problems_dev,
                                                int32_t count,
                                                const bitnet_problem *problems_host,
                                                void *stream) {
  if (!problems_dev || !problems_host) return BITNET_ERR_NULL;
  if (count < 1 || count > kMaxGroup) return BITNET_ERR_SHAPE;
  if (!aligned(problems_dev, 8)) return BITNET_ERR_ALIGN;
  for (int32_t i = 0; i < count; ++i) {
    bitnet_status st = check_problem(1, problems_host[i]);
    if (st != BITNET_OK) return st;
    if (problems_host[i].K > kLutMaxK) return BITNET_ERR_SHAPE;
  }
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  // Longest K first, as in the grouped call.
  int32_t idx[kMaxGroup];
  for (int32_t i = 0; i < count; ++i) idx[i] = i;
  std::stable_sort(idx, idx + count, [&](int32_t a, int32_t b) {
    return problems_host[a].K > problems_host[b].K;
  });
  GroupTable tab;
  std::memset(&tab, 0, sizeof(tab));
  tab.count = count;
  tab.M = 1;
  uint64_t total = 0;
  uint32_t tiles[kMaxGroup];
  for (int32_t s = 0; s < count; ++s) {
    tiles[s] = (uint32_t)lut_blocks(problems_host[idx[s]].N);
    total += tiles[s];
    if (total >= ((uint64_t)1 << 31)) return BITNET_ERR_SHAPE;
    tab.blk_end[s] = (uint32_t)total;
    tab.order[s] = (uint16_t)idx[s];
  }
  // Whole projections to the XCDs, as in the grouped call.
  xcd_schedule(tab, problems_host, tiles);
  return from_hip(launch_lut_grouped(problems_dev, tab, as_stream(stream)));
}

size_t bitnet_stages_workspace_bytes(int64_t M, const bitnet_problem *problems_host,
                                     int32_t count) {
  if (!problems_host || count < 1 || count > kMaxGroup || M < 1 || M > kGemvMaxM) return 0;
  for (int32_t i = 0; i < count; ++i)
    if (!shape_ok(M, problems_host[i].N, problems_host[i].K)) return 0;
  return stages_workspace_bytes(M, problems_host, count);
}

bitnet_status bitnet_ternary_matmul_stages(int64_t M, const bitnet_problem *problems_dev,
                                           int32_t count, const int32_t *stage_end,
                                           int32_t nstages, const bitnet_problem *problems_host,
                                           void *workspace, size_t workspace_bytes,
                                           void *stream) {
  if (!problems_dev || !problems_host || !stage_end) return BITNET_ERR_NULL;
  if (count < 1 || count > kMaxGroup || nstages < 1 || nstages > kMaxStages)
    return BITNET_ERR_SHAPE;
  if (M < 1 || M > kGemvMaxM) return BITNET_ERR_SHAPE;
  if (!aligned(problems_dev, 8)) return BITNET_ERR_ALIGN;
  for (int32_t i = 0; i < count; ++i) {
    bitnet_status st = check_problem(M, problems_host[i]);
    if (st != BITNET_OK) return st;
    if (!gemv_fusable(M, problems_host[i].K)) return BITNET_ERR_SHAPE;
  }
  int32_t prev = 0;
  int32_t stage_of[kMaxGroup];
  for (int32_t s = 0; s < nstages; ++s) {
    if (stage_end[s] <= prev || stage_end[s] > count) return BITNET_ERR_SHAPE;
    for (int32_t i = prev; i < stage_end[s]; ++i) stage_of[i] = s;
    prev = stage_end[s];
  }
  if (prev != count) return BITNET_ERR_SHAPE;
  // Producers: an x equal to the y of a problem of an earlier stage.  Every
  // other x is an input and must not overlap any y; y ranges are disjoint.
  int16_t src[kMaxGroup];
  auto y_lo = [&](int32_t j) { return reinterpret_cast<uintptr_t>(problems_host[j].y); };
  auto y_hi = [&](int32_t j) { return y_lo(j) + (uintptr_t)(M * problems_host[j].N) * 4; };
  for (int32_t i = 0; i < count; ++i) {
    src[i] = -1;
    for (int32_t j = 0; j < count; ++j)
      if (stage_of[j] < stage_of[i] && (const void *)problems_host[j].y == problems_host[i].x)
        src[i] = (int16_t)j;
    if (src[i] >= 0) {
      if (problems_host[src[i]].N != problems_host[i].K) return BITNET_ERR_SHAPE;
      continue;
    }
    const uintptr_t lo = reinterpret_cast<uintptr_t>(problems_host[i].x);
    const uintptr_t hi = lo + (uintptr_t)(M * problems_host[i].K) * 4;
    for (int32_t j = 0; j < count; ++j)
      if (lo < y_hi(j) && y_lo(j) < hi) return BITNET_ERR_ALIAS;
  }
  for (int32_t i = 0; i < count; ++i)
    for (int32_t j = i + 1; j < count; ++j)
      if (y_lo(i) < y_hi(j) && y_lo(j) < y_hi(i)) return BITNET_ERR_ALIAS;
  if (!workspace || workspace_bytes < stages_workspace_bytes(M, problems_host, count))
    return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;

  return from_hip(launch_stages(problems_dev, problems_host, count, stage_end, nstages, (int)M,
                                src, reinterpret_cast<uint8_t *>(workspace), as_stream(stream)));
}

// ---- the paged key-value cache and beam search -----------------------------

// An array of a call, for the overlap checks.
struct Range {
  const void *p;
  int64_t bytes;
};

static bool overlap(const Range &a, const Range &b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// The first `nout` ranges are written: none may overlap any other range.
static bool overlaps_any(const Range *r, int nout, int n) {
  for (int i = 0; i < nout; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(r[i], r[j])) return true;
  return false;
}

// One axis of the cache's rows: how many, and the bytes from one to the next.
struct Axis {
  int64_t n;
  __int128 stride;
};

// Whether bytes [lo, hi) meet the rows of `row` bytes along the n axes, which go from
// the widest stride down.  (Axes that run into each other count with what lies
// between their rows.)
static bool meets_rows(const Axis *x, int n, int64_t row, __int128 lo, __int128 hi) {
  __int128 span = row;   // of one step of the first axis
  for (int i = 1; i < n; ++i) span += (x[i].n - 1) * x[i].stride;
  if (n == 0 || x[0].stride < span)
    return hi > 0 && lo < span + (n ? (x[0].n - 1) * x[0].stride : 0);
  if (hi <= 0) return false;
  const __int128 s = x[0].stride;
  const __int128 first = lo < span ? 0 : (lo - span) / s + 1;
  const __int128 last = std::min<__int128>(x[0].n - 1, (hi - 1) / s);
  if (last - first >= 2) return true;   // those between the two lie inside
  for (__int128 i = first; i <= last; ++i)
    if (meets_rows(x + 1, n - 1, row, lo - i * s, hi - i * s)) return true;
  return false;
}

// Whether one of n arrays, of which the call writes the first `nout`, meets the
// cache's arrays of `layers` layers from `layer` on.  Outputs are held against all
// that lies between the first element and the last, inputs against the elements:
// they may lie between the rows of a strided cache.
static bool overlaps_cache(const bitnet_kv_cache *c, int32_t layer, int32_t layers,
                           const Range *r, int nout, int n) {
  const bool i8 = c->dtype == BITNET_KV_INT8;
  const int64_t es = i8 ? 1 : 2, ls = c->layers > 1 ? c->layer_stride : 0;
  const __int128 last = (__int128)(layers - 1) * ls + (__int128)(c->pages - 1) * c->page_stride +
                        (__int128)(c->kv_heads - 1) * c->head_stride +
                        (__int128)(c->page_size - 1) * c->token_stride + c->head_dim;
  const int64_t bytes = (int64_t)std::min<__int128>(last * es, (__int128)1 << 62);
  const int64_t scales = (int64_t)c->pages * c->kv_heads * c->page_size;
  const Range a[] = {{static_cast<uint8_t *>(c->k) + layer * ls * es, bytes},
                     {static_cast<uint8_t *>(c->v) + layer * ls * es, bytes},
                     {i8 ? c->k_scale + layer * scales : nullptr, layers * scales * 4},
                     {i8 ? c->v_scale + layer * scales : nullptr, layers * scales * 4}};
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < 4; ++j) {
      if (!overlap(r[i], a[j])) continue;
      if (i < nout || j >= 2) return true;
      Axis x[4];
      int axes = 0;
      const Axis all[] = {{layers, ls * es},
                          {c->pages, c->page_stride * es},
                          {c->kv_heads, c->head_stride * es},
                          {c->page_size, c->token_stride * es}};
      for (const Axis &y : all)
        if (y.n > 1) x[axes++] = y;
      std::sort(x, x + axes, [](const Axis &p, const Axis &q) { return p.stride > q.stride; });
      const __int128 lo = (__int128)(uintptr_t)r[i].p - (__int128)(uintptr_t)a[j].p;
      if (meets_rows(x, axes, c->head_dim * es, lo, lo + r[i].bytes)) return true;
    }
  return false;
}

static bool power_of_two(int64_t v) { return v >= 1 && (v & (v - 1)) == 0; }

static int shift_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << s) < v) ++s;
  return s;
}

constexpr int64_t kMaxLayerStride = (int64_t)1 << 40;   // of the cache, elements
constexpr int64_t kMaxTokens = kLimit / 256;       // rows of one call
constexpr int64_t kMaxVocab = kLimit / 2;

static bitnet_status check_cache(const bitnet_kv_cache *c, int32_t layer) {
  if (!c || !c->k || !c->v) return BITNET_ERR_NULL;
  const bool i8 = c->dtype == BITNET_KV_INT8;
  if (!i8 && c->dtype != BITNET_KV_BF16 && c->dtype != BITNET_KV_FP16) return BITNET_ERR_SHAPE;
  if (i8 && (!c->k_scale || !c->v_scale)) return BITNET_ERR_NULL;
  const int D = c->head_dim;
  if (D != 64 && D != 128 && D != 256) return BITNET_ERR_SHAPE;
  if (!power_of_two(c->page_size) || c->page_size > 1024) return BITNET_ERR_SHAPE;
  if (c->layers < 1 || c->layers > 1024 || layer < 0 || layer >= c->layers)
    return BITNET_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 256 || c->pages < 1 ||
      (int64_t)c->pages * c->page_size >= kLimit)
    return BITNET_ERR_SHAPE;
  if (i8 && (int64_t)c->pages * c->page_size * c->kv_heads >= 2 * kLimit) return BITNET_ERR_SHAPE;
  const int64_t per16 = i8 ? 16 : 8;   // elements in 16 bytes
  const int64_t ls = c->layers > 1 ? c->layer_stride : c->page_stride;
  for (const int64_t s : {c->page_stride, c->head_stride, c->token_stride})
    if (s < D || s >= kLimit) return BITNET_ERR_SHAPE;
  if (ls < D || ls >= kMaxLayerStride) return BITNET_ERR_SHAPE;
  if (c->page_stride % per16 || c->head_stride % per16 || c->token_stride % per16 || ls % per16)
    return BITNET_ERR_ALIGN;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return BITNET_ERR_ALIGN;
  if (i8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return BITNET_ERR_ALIGN;
  return BITNET_OK;
}

static KvView kv_view(const bitnet_kv_cache *c, int32_t layer) {
  const bool i8 = c->dtype == BITNET_KV_INT8;
  const int64_t off = layer ? layer * c->layer_stride * (i8 ? 1 : 2) : 0;
  const int64_t soff = (int64_t)layer * c->pages * c->kv_heads * c->page_size;
  KvView v;
  v.k = static_cast<uint8_t *>(c->k) + off;
  v.v = static_cast<uint8_t *>(c->v) + off;
  v.k_scale = i8 ? c->k_scale + soff : nullptr;
  v.v_scale = i8 ? c->v_scale + soff : nullptr;
  v.page_stride = c->page_stride;
  v.head_stride = c->head_stride;
  v.token_stride = c->token_stride;
  v.pages = c->pages;
  v.kv_heads = c->kv_heads;
  v.page_shift = shift_of(c->page_size);
  return v;
}

bitnet_status bitnet_kv_map(const bitnet_kv_pool *pool, int64_t T, const int32_t *new_lens,
                            const int32_t *state_in, int32_t *state_out, int32_t *starts,
                            int32_t *slots, int32_t *positions, int32_t *rows, int32_t *status,
                            void *stream) {
  if (!pool || !pool->tables || !pool->owned || !pool->free_pages || !new_lens || !state_in ||
      !state_out || !starts || !slots || !positions || !rows || !status)
    return BITNET_ERR_NULL;
  const int64_t B = pool->rows, mp = pool->max_pages, ps = pool->page_size;
  if (B < 1 || B > kMaxRows || mp < 1 || pool->pages < 1 || !power_of_two(ps) || ps > 1024 ||
      mp * ps >= kLimit || pool->pages * ps >= kLimit || T < 1 || T >= kLimit)
    return BITNET_ERR_SHAPE;
  const void *ptrs[] = {pool->tables, pool->owned, pool->free_pages, state_out, starts, slots,
                        positions, rows, status, new_lens, state_in};
  for (const void *p : ptrs)
    if (!aligned(p, 4)) return BITNET_ERR_ALIGN;
  const Range r[] = {{pool->tables, B * mp * 4}, {pool->owned, B * mp * 4},
                     {pool->free_pages, (int64_t)pool->pages * 4}, {state_out, (2 * B + 1) * 4},
                     {starts, (B + 1) * 4}, {slots, T * 4}, {positions, T * 4}, {rows, T * 4},
                     {status, B * 4}, {new_lens, B * 4},
                     {state_in == state_out ? nullptr : state_in, (2 * B + 1) * 4}};
  if (overlaps_any(r, 9, 11)) return BITNET_ERR_ALIAS;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  KvMapArgs a;
  a.new_lens = new_lens;
  a.state_in = state_in;
  a.state_out = state_out;
  a.starts = starts;
  a.slots = slots;
  a.positions = positions;
  a.rows = rows;
  a.status = status;
  a.tables = pool->tables;
  a.owned = pool->owned;
  a.free_pages = pool->free_pages;
  a.B = (int32_t)B;
  a.max_pages = pool->max_pages;
  a.pages = pool->pages;
  a.page_shift = shift_of(ps);
  a.T = T;
  return from_hip(launch_kv_map(a, as_stream(stream)));
}

bitnet_status bitnet_kv_append(const bitnet_kv_cache *cache, int32_t layer, int64_t T,
                               int64_t q_heads, const float *k, int64_t k_stride, const float *v,
                               int64_t v_stride, const int32_t *slots, const int32_t *positions,
                               const float *cos, const float *sin, int64_t max_pos,
                               const float *q, int64_t q_stride, float *q_out, void *stream) {
  bitnet_status st = check_cache(cache, layer);
  if (st != BITNET_OK) return st;
  if (T == 0) return BITNET_OK;
  if (!k || !v || !slots) return BITNET_ERR_NULL;
  const bool rotate = cos != nullptr;
  if (rotate != (sin != nullptr) || (rotate && !positions) || (q != nullptr) != (q_out != nullptr))
    return BITNET_ERR_NULL;
  if (q && !rotate) return BITNET_ERR_NULL;
  const int64_t D = cache->head_dim, kd = cache->kv_heads * D, qd = q ? q_heads * D : 0;
  if (T < 0 || T >= kMaxTokens || (q && (q_heads < 1 || q_heads >= kMaxTokens / D)) ||
      (rotate && (max_pos < 1 || max_pos >= kMaxTokens)))
    return BITNET_ERR_SHAPE;
  if (k_stride < kd || v_stride < kd || (q && q_stride < qd) || k_stride >= kLimit ||
      v_stride >= kLimit || (q && q_stride >= kLimit))
    return BITNET_ERR_SHAPE;
  if (k_stride % 4 || v_stride % 4 || (q && q_stride % 4) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(slots, 4) ||
      (rotate && (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(positions, 4))) ||
      (q && (!aligned(q, 16) || !aligned(q_out, 16))))
    return BITNET_ERR_ALIGN;
  const bool in_place = q_out == q && q_stride == qd;
  const Range r[] = {{q_out, T * qd * 4},
                     {in_place ? nullptr : q, q ? ((T - 1) * q_stride + qd) * 4 : 0},
                     {k, ((T - 1) * k_stride + kd) * 4},
                     {v, ((T - 1) * v_stride + kd) * 4},
                     {slots, T * 4},
                     {rotate ? positions : nullptr, T * 4},
                     {cos, rotate ? max_pos * D * 2 : 0},
                     {sin, rotate ? max_pos * D * 2 : 0}};
  if (overlaps_any(r, 1, 8) || overlaps_cache(cache, layer, 1, r, 1, 8)) return BITNET_ERR_ALIAS;
  st = device_check();
  if (st != BITNET_OK) return st;
  KvAppendArgs a;
  a.c = kv_view(cache, layer);
  a.q = q;
  a.k = k;
  a.v = v;
  a.cos = cos;
  a.sin = sin;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.positions = positions;
  a.q_heads = (int32_t)(q ? q_heads : 0);
  a.max_pos = (int32_t)max_pos;
  a.T = T;
  return from_hip(launch_kv_append(a, cache->dtype, cache->head_dim, as_stream(stream)));
}

// Shapes of an attention call, apart from the cache's own.
static bool attend_shape_ok(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                            int64_t max_len) {
  if (T < 1 || T >= kMaxTokens || kv_heads < 1 || kv_heads > 256 || q_heads < 1 ||
      q_heads % kv_heads != 0 || q_heads / kv_heads > 64)
    return false;
  if (T * kv_heads * ((q_heads / kv_heads + 15) / 16) >= kLimit) return false;
  return (D == 64 || D == 128 || D == 256) && max_len >= 1 && max_len < kLimit / 2;
}

size_t bitnet_paged_attention_workspace_bytes(int64_t T, int64_t q_heads, int64_t kv_heads,
                                              int64_t head_dim, int64_t max_len) {
  if (!attend_shape_ok(T, q_heads, kv_heads, head_dim, max_len)) return 0;
  return attend_workspace_bytes(T, q_heads, kv_heads, head_dim, max_len);
}

bitnet_status bitnet_paged_attention(const bitnet_kv_cache *cache, int32_t layer, int64_t T,
                                     int64_t q_heads, const float *q, int64_t q_stride,
                                     const int32_t *tables, int64_t table_rows,
                                     int64_t max_pages, const int32_t *rows, const int32_t *lens,
                                     int64_t max_len, float scale, float *out, float *lse,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  bitnet_status st = check_cache(cache, layer);
  if (st != BITNET_OK) return st;
  if (T == 0) return BITNET_OK;
  if (!q || !tables || !lens || !out) return BITNET_ERR_NULL;
  const int64_t D = cache->head_dim, qd = q_heads * D;
  if (!attend_shape_ok(T, q_heads, cache->kv_heads, D, max_len) || q_stride < qd ||
      q_stride >= kLimit || table_rows < 1 || table_rows >= kMaxTokens || max_pages < 1 ||
      max_pages >= kLimit || max_len > max_pages * cache->page_size ||
      (!rows && T > table_rows) || !std::isfinite(scale))
    return BITNET_ERR_SHAPE;
  if (q_stride % 4 || !aligned(q, 16) || !aligned(out, 16) || !aligned(tables, 4) ||
      !aligned(lens, 4) || (rows && !aligned(rows, 4)) || (lse && !aligned(lse, 4)))
    return BITNET_ERR_ALIGN;
  const size_t need = attend_workspace_bytes(T, q_heads, cache->kv_heads, D, max_len);
  if (!workspace || workspace_bytes < need) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  const Range r[] = {{out, T * qd * 4},
                     {lse, T * q_heads * 4},
                     {workspace, (int64_t)need},
                     {q, ((T - 1) * q_stride + qd) * 4},
                     {tables, table_rows * max_pages * 4},
                     {rows, T * 4},
                     {lens, T * 4}};
  if (overlaps_any(r, 3, 7) || overlaps_cache(cache, layer, 1, r, 3, 3)) return BITNET_ERR_ALIAS;
  st = device_check();
  if (st != BITNET_OK) return st;
  AttendArgs a;
  a.c = kv_view(cache, layer);
  a.q = q;
  a.q_stride = q_stride;
  a.tables = tables;
  a.rows = rows;
  a.lens = lens;
  a.T = (int32_t)T;
  a.q_heads = (int32_t)q_heads;
  a.table_rows = (int32_t)table_rows;
  a.max_pages = (int32_t)max_pages;
  a.max_len = (int32_t)max_len;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.ws = static_cast<uint8_t *>(workspace);
  return from_hip(launch_attend(a, cache->dtype, cache->head_dim, as_stream(stream)));
}

static bool beams_ok(int64_t B, int64_t W) {
  return B >= 1 && W >= 1 && W <= kMaxWidth && B <= kMaxRows && B * W <= kMaxRows;
}

size_t bitnet_beam_select_workspace_bytes(int64_t B, int64_t W, int64_t V) {
  if (!beams_ok(B, W) || V < W || V >= kMaxVocab) return 0;
  return select_workspace_bytes(B, W, V);
}

bitnet_status bitnet_beam_select(int64_t B, int64_t W, int64_t V, const float *logits, int64_t ld,
                                 const float *scores_in, const int32_t *finished_in, int32_t eos,
                                 float *scores_out, int32_t *tokens, int32_t *parents,
                                 int32_t *finished_out, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  if (!logits || !scores_in || !scores_out || !tokens || !parents ||
      (finished_in != nullptr) != (finished_out != nullptr))
    return BITNET_ERR_NULL;
  if (!beams_ok(B, W) || V < W || V >= kMaxVocab || ld < V || ld >= kLimit ||
      (finished_in && (eos < 0 || eos >= V)))
    return BITNET_ERR_SHAPE;
  const void *ptrs[] = {logits, scores_in, scores_out, tokens, parents, finished_in, finished_out};
  for (const void *p : ptrs)
    if (!aligned(p, 4)) return BITNET_ERR_ALIGN;
  const size_t need = select_workspace_bytes(B, W, V);
  if (!workspace || workspace_bytes < need) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_ALIGN;
  const int64_t n = B * W * 4;
  const Range r[] = {{scores_out, n}, {tokens, n}, {parents, n}, {finished_out, n},
                     {workspace, (int64_t)need},
                     {logits, ((B * W - 1) * ld + V) * 4},
                     {scores_in == scores_out ? nullptr : scores_in, n},
                     {finished_in == finished_out ? nullptr : finished_in, n}};
  if (overlaps_any(r, 5, 8)) return BITNET_ERR_ALIAS;
  bitnet_status st = device_check();
  if (st != BITNET_OK) return st;
  SelectArgs a;
  a.logits = logits;
  a.scores_in = scores_in;
  a.finished_in = finished_in;
  a.scores_out = scores_out;
  a.tokens = tokens;
  a.parents = parents;
  a.finished_out = finished_out;
  a.ld = ld;
  a.B = (int32_t)B;
  a.W = (int32_t)W;
  a.V = (int32_t)V;
  a.eos = eos;
  a.ws = static_cast<uint8_t *>(workspace);
  return from_hip(launch_beam_select(a, as_stream(stream)));
}

bitnet_status bitnet_beam_reorder(const bitnet_kv_cache *cache, int64_t B, int64_t W,
                                  const int32_t *parents, const int32_t *lens,
                                  const int32_t *tables_in, int32_t *tables_out,
                                  int64_t max_pages, void *stream) {
  bitnet_status st = check_cache(cache, 0);
  if (st != BITNET_OK) return st;
  if (!parents || !lens || !tables_in || !tables_out) return BITNET_ERR_NULL;
  if (!beams_ok(B, W) || max_pages < 1 || max_pages >= kLimit ||
      max_pages * cache->page_size >= kLimit)
    return BITNET_ERR_SHAPE;
  if (!aligned(parents, 4) || !aligned(lens, 4) || !aligned(tables_in, 4) ||
      !aligned(tables_out, 4))
    return BITNET_ERR_ALIGN;
  const int64_t n = B * W * 4;
  const Range r[] = {{tables_out, n * max_pages}, {tables_in, n * max_pages}, {parents, n},
                     {lens, n}};
  if (overlaps_any(r, 1, 4) || overlaps_cache(cache, 0, cache->layers, r, 1, 4))
    return BITNET_ERR_ALIAS;
  st = device_check();
  if (st != BITNET_OK) return st;
  ReorderArgs a;
  a.c = kv_view(cache, 0);
  a.layer_stride = cache->layers > 1 ? cache->layer_stride : 0;
  a.layers = cache->layers;
  a.head_dim = cache->head_dim;
  a.elem_bytes = cache->dtype == BITNET_KV_INT8 ? 1 : 2;
  a.B = (int32_t)B;
  a.W = (int32_t)W;
  a.max_pages = (int32_t)max_pages;
  a.parents = parents;
  a.lens = lens;
  a.tables_in = tables_in;
  a.tables_out = tables_out;
  return from_hip(launch_beam_reorder(a, as_stream(stream)));
}

}  // extern "C"
