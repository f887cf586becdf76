// The paged key-value cache: the page map of a step, the write of new tokens
// and the reordering of beams.  (The attention that reads the cache is in
// attention.hip.)
#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"

namespace bitnet {
namespace {

// ---------------------------------------------------------------------------
// Page map: lengths -> pages, slots, positions.
//
// Two running sums over the requests decide who is granted (pages needed and
// tokens added, over the requests that fit their tables), two more over the
// granted ones give each its first page and first token.  One workgroup does
// all of it, so that nothing but its own barriers orders the steps.
// ---------------------------------------------------------------------------

constexpr int kMapThreads = 1024;
constexpr int kMapWaves = kMapThreads / 64;

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  const int lo = __shfl_up((int)(uint32_t)v, d, 64);
  const int hi = __shfl_up((int)(v >> 32), d, 64);
  return ((int64_t)hi << 32) | (uint32_t)lo;
}

// Inclusive sum over the workgroup's threads, plus the total in *total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *wave_sums, int64_t *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = shfl_up64(v, d);
    if (lane >= d) v += u;
  }
  if (lane == 63) wave_sums[wave] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < kMapWaves; ++w) {
    const int64_t s = wave_sums[w];
    before += w < wave ? s : 0;
    all += s;
  }
  *total = all;
  __syncthreads();
  return v + before;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Token t of the step: its request by bisection of starts, its position from
// the request's length after the step, its slot from the table.
__device__ __forceinline__ void map_token(const KvMapArgs &a, const int32_t *starts,
                                          const int32_t *lens_after, int64_t t) {
  int slot = -1, pos = -1, row = -1;
  if (t < starts[a.B]) {
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {   // the last request that starts at or before t
      const int mid = (lo + hi + 1) >> 1;
      if (starts[mid] <= t) lo = mid; else hi = mid - 1;
    }
    row = lo;
    pos = lens_after[row] - (starts[row + 1] - (int)t);
    const int page = a.tables[(int64_t)row * a.max_pages + (pos >> a.page_shift)];
    if (page >= 0 && page < a.pages)
      slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  }
  a.slots[t] = slot;
  a.positions[t] = pos;
  a.rows[t] = row;
}

__global__ void __launch_bounds__(kMapThreads) kv_map_kernel(KvMapArgs a, int tokens_here) {
  __shared__ int64_t sums[kMapWaves];
  __shared__ int32_t starts[kMaxRows + 1];
  __shared__ int32_t lens_after[kMaxRows];
  const int tid = threadIdx.x;
  const int ps = 1 << a.page_shift;
  const int cap = a.max_pages << a.page_shift;   // tokens a table holds
  int64_t total;

  // Ended requests give their pages back.
  int64_t height = clampi(a.state_in[2 * a.B], 0, a.pages);
  for (int b0 = 0; b0 < a.B; b0 += kMapThreads) {
    const int r = b0 + tid;
    const bool ends = r < a.B && a.new_lens[r] < 0;
    const int held = ends ? clampi(a.state_in[a.B + r], 0, a.max_pages) : 0;
    const int64_t at = height + block_scan(held, sums, &total) - held;
    for (int i = 0; i < held; ++i)
      if (at + i < a.pages) a.free_pages[at + i] = a.owned[(int64_t)r * a.max_pages + i];
    height = min(height + total, (int64_t)a.pages);
  }
  __syncthreads();   // the stack is read below

  int64_t want_pages = 0, want_tokens = 0;   // of the requests before this chunk
  int64_t page0 = 0, token0 = 0;             // granted before this chunk
  for (int b0 = 0; b0 < a.B; b0 += kMapThreads) {
    const int r = b0 + tid;
    int len = 0, held = 0, add = 0;
    if (r < a.B) {
      const int n = a.new_lens[r];
      if (n >= 0) {
        len = clampi(a.state_in[r], 0, cap);
        held = clampi(a.state_in[a.B + r], 0, a.max_pages);
        add = n;
      }
    }
    const int first = (int)(((int64_t)len + ps - 1) >> a.page_shift);
    const int64_t after = (int64_t)len + add;
    const int64_t need64 = ((after + ps - 1) >> a.page_shift) - first;
    const bool fits = after <= cap && held + need64 <= a.max_pages;
    const int64_t need = fits ? need64 : 0;
    const int64_t upto_p = want_pages + block_scan(need, sums, &total);
    want_pages += total;
    const int64_t upto_t = want_tokens + block_scan(fits ? add : 0, sums, &total);
    want_tokens += total;
    const bool paged = need == 0 || upto_p <= height;
    const bool room = add == 0 || upto_t <= a.T;
    const bool ok = fits && paged && room;
    const int np = ok ? (int)need : 0, nt = ok ? add : 0;
    const int64_t p_at = page0 + block_scan(np, sums, &total) - np;
    page0 += total;
    const int64_t t_at = token0 + block_scan(nt, sums, &total) - nt;
    token0 += total;
    if (r < a.B) {
      for (int i = 0; i < np; ++i) {
        const int page = a.free_pages[height - 1 - p_at - i];
        a.tables[(int64_t)r * a.max_pages + first + i] = page;
        a.owned[(int64_t)r * a.max_pages + held + i] = page;
      }
      starts[r] = (int32_t)t_at;
      lens_after[r] = len + nt;
      a.starts[r] = (int32_t)t_at;
      a.status[r] = fits ? (paged ? (room ? 0 : 3) : 2) : 1;
      a.state_out[r] = len + nt;
      a.state_out[a.B + r] = held + np;
    }
  }
  if (tid == 0) {
    starts[a.B] = (int32_t)token0;
    a.starts[a.B] = (int32_t)token0;
    a.state_out[2 * a.B] = (int32_t)(height - page0);
  }
  __syncthreads();
  if (tokens_here)
    for (int64_t t = tid; t < a.T; t += kMapThreads) map_token(a, starts, lens_after, t);
}

__global__ void __launch_bounds__(256) kv_map_tokens_kernel(KvMapArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t < a.T) map_token(a, a.starts, a.state_out, t);
}

// Calls of up to this many tokens finish in the one workgroup.
constexpr int64_t kMapTokensHere = 8192;

// ---------------------------------------------------------------------------
// Append: rotate, convert, scatter.
//
// One workgroup per token; a thread holds four channels of each half of a
// head, so a rotation needs no exchange and an 8-bit row's maximum is a
// reduction over head_dim / 8 adjacent lanes.
// ---------------------------------------------------------------------------

template <int DT> struct KvElem;
template <> struct KvElem<BITNET_KV_BF16> { typedef __bf16 T; };
template <> struct KvElem<BITNET_KV_FP16> { typedef _Float16 T; };
template <> struct KvElem<BITNET_KV_INT8> { typedef int8_t T; };

// fl32(x*c - y*s) with the products exact and one rounding of their sum in fp64.
__device__ __forceinline__ float rot(float x, float c, float y, float s) {
  return (float)((double)x * (double)c - (double)y * (double)s);
}

__device__ __forceinline__ int8_t code8(float x, float s) {
  if (s == 0.0f) return 0;
  return (int8_t)fminf(fmaxf(__builtin_rintf(x / s), -127.0f), 127.0f);
}

template <int DT, int D>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendArgs a) {
  typedef typename KvElem<DT>::T E;
  typedef E E4 __attribute__((ext_vector_type(4)));
  constexpr int kPer = D / 8;   // threads per head
  const int64_t t = blockIdx.x;
  const int slot = a.slots[t];
  if (slot < 0 || (slot >> a.c.page_shift) >= a.c.pages) return;
  const bool rotate = a.cos != nullptr;
  int pos = 0;
  if (rotate) {
    pos = a.positions[t];
    if (pos < 0 || pos >= a.max_pos) return;
  }
  const int hq = a.q ? a.q_heads : 0;
  const int items = (hq + 2 * a.c.kv_heads) * kPer;
  const int64_t page = slot >> a.c.page_shift;
  const int tok = slot & ((1 << a.c.page_shift) - 1);
  for (int i0 = 0; i0 < items; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    if (i >= items) break;   // whole heads: a head's lanes leave together
    int h = i / kPer;
    const int c = (i % kPer) * 4;
    const bool is_q = h < hq;
    const bool is_v = h >= hq + a.c.kv_heads;
    const float *src;
    if (is_q) {
      src = a.q + t * a.q_stride + (int64_t)h * D;
    } else if (!is_v) {
      h -= hq;
      src = a.k + t * a.k_stride + (int64_t)h * D;
    } else {
      h -= hq + a.c.kv_heads;
      src = a.v + t * a.v_stride + (int64_t)h * D;
    }
    f32x4 x = ld_global<f32x4>(src + c), y = ld_global<f32x4>(src + c + D / 2);
    if (rotate && !is_v) {
      const f32x4 cs = ld_global<f32x4>(a.cos + (int64_t)pos * (D / 2) + c);
      const f32x4 sn = ld_global<f32x4>(a.sin + (int64_t)pos * (D / 2) + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = rot(x[j], cs[j], y[j], sn[j]);
        y[j] = rot(y[j], cs[j], x[j], -sn[j]);
        x[j] = p;
      }
    }
    if (is_q) {
      float *dst = a.q_out + (t * a.q_heads + h) * D;
      st_global<f32x4>(dst + c, x);
      st_global<f32x4>(dst + c + D / 2, y);
      continue;
    }
    E *dst = reinterpret_cast<E *>(is_v ? a.c.v : a.c.k) + page * a.c.page_stride +
             h * a.c.head_stride + tok * a.c.token_stride;
    E4 ex, ey;
    if constexpr (DT == BITNET_KV_INT8) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(x[j]), fabsf(y[j])));
#pragma unroll
      for (int d = kPer / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
      const float s = m / 127.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ex[j] = code8(x[j], s);
        ey[j] = code8(y[j], s);
      }
      if (c == 0)
        (is_v ? a.c.v_scale : a.c.k_scale)[((page * a.c.kv_heads + h) << a.c.page_shift) + tok] =
            s;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ex[j] = (E)x[j];
        ey[j] = (E)y[j];
      }
    }
    st_global<E4>(dst + c, ex);
    st_global<E4>(dst + c + D / 2, ey);
  }
}

// ---------------------------------------------------------------------------
// Beam reordering.
//
// The children of every beam are a bit mask per beam (lane p of a wave holds
// those of beam p), from which each wave finds for its row the parent and the
// beam whose last page it takes: no wave waits for another, and the pages
// read (last pages of beams with children) and written (of beams without)
// are disjoint, so one launch copies in place.
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(256) beam_reorder_kernel(ReorderArgs a) {
  const int row = blockIdx.x, layer = (int)blockIdx.y - 1;
  const int g0 = row / a.W * a.W, j = row - g0;
  const int lane = threadIdx.x & 63;
  int par = lane;
  if (lane < a.W) {
    const int p = a.parents[g0 + lane] - g0;
    if (p >= 0 && p < a.W) par = p;
  }
  uint64_t kids = 0;   // of beam `lane`
  for (int p = 0; p < a.W; ++p) {
    const uint64_t m = __ballot(lane < a.W && par == p);
    if (lane == p) kids = m;
  }
  const uint64_t none = __ballot(lane < a.W && kids == 0);
  const int first = kids ? __builtin_ctzll(kids) : -1;
  const uint64_t moves = __ballot(lane < a.W && __shfl(first, par, 64) != lane);
  const int parent = __shfl(par, j, 64);
  const bool move = (moves >> j) & 1;
  // The n-th mover takes the page of the n-th beam without a child.
  uint64_t left = none;
  for (int n = __builtin_popcountll(moves & ((1ull << j) - 1)); n > 0; --n) left &= left - 1;
  const int donor = move ? __builtin_ctzll(left) : parent;

  const int ps = 1 << a.c.page_shift;
  const int len = clampi(a.lens[g0], 0, a.max_pages << a.c.page_shift);
  const int tail = len & (ps - 1), last = len >> a.c.page_shift;
  const int32_t *from = a.tables_in + (int64_t)(g0 + parent) * a.max_pages;
  const int32_t *giver = a.tables_in + (int64_t)(g0 + donor) * a.max_pages;
  if (layer < 0) {
    const int32_t *self = a.tables_in + (int64_t)row * a.max_pages;
    int32_t *out = a.tables_out + (int64_t)row * a.max_pages;
    for (int i = threadIdx.x; i < a.max_pages; i += 256)
      out[i] = i < last ? from[i] : i == last && tail ? giver[i] : self[i];
    return;
  }
  if (!move || tail == 0) return;
  const int64_t src = from[last], dst = giver[last];
  if (src < 0 || src >= a.c.pages || dst < 0 || dst >= a.c.pages) return;
  const int vecs = a.head_dim * a.elem_bytes / 16;   // 16-byte pieces of a token's head
  const int n = a.c.kv_heads * tail * vecs;
  for (int side = 0; side < 2; ++side) {
    uint8_t *base = reinterpret_cast<uint8_t *>(side ? a.c.v : a.c.k) +
                    layer * a.layer_stride * a.elem_bytes;
    for (int i = threadIdx.x; i < n; i += 256) {
      const int piece = i % vecs, tok = i / vecs % tail, h = i / vecs / tail;
      const int64_t off =
          (h * a.c.head_stride + tok * a.c.token_stride) * a.elem_bytes + piece * 16;
      const int64_t pb = a.c.page_stride * a.elem_bytes;
      st_global<u32x4>(base + dst * pb + off, ld_global<u32x4>(base + src * pb + off));
    }
    float *sc = side ? a.c.v_scale : a.c.k_scale;
    if (sc != nullptr) {
      sc += (int64_t)layer * a.c.pages * a.c.kv_heads * ps;
      for (int i = threadIdx.x; i < a.c.kv_heads * tail; i += 256) {
        const int tok = i % tail, h = i / tail;
        sc[(dst * a.c.kv_heads + h) * ps + tok] = sc[(src * a.c.kv_heads + h) * ps + tok];
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_map(const KvMapArgs &a, hipStream_t stream) {
  const bool here = a.T <= kMapTokensHere;
  kv_map_kernel<<<1, kMapThreads, 0, stream>>>(a, here);
  if (!here) kv_map_tokens_kernel<<<(unsigned)((a.T + 255) / 256), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int DT>
static void append_dim(const KvAppendArgs &a, int D, hipStream_t stream) {
  const int items = ((a.q ? a.q_heads : 0) + 2 * a.c.kv_heads) * (D / 8);
  const int threads = items >= 256 ? 256 : (items + 63) / 64 * 64;
  if (D == 64)
    kv_append_kernel<DT, 64><<<(unsigned)a.T, threads, 0, stream>>>(a);
  else if (D == 128)
    kv_append_kernel<DT, 128><<<(unsigned)a.T, threads, 0, stream>>>(a);
  else
    kv_append_kernel<DT, 256><<<(unsigned)a.T, threads, 0, stream>>>(a);
}

hipError_t launch_kv_append(const KvAppendArgs &a, int dtype, int head_dim, hipStream_t stream) {
  if (dtype == BITNET_KV_BF16)
    append_dim<BITNET_KV_BF16>(a, head_dim, stream);
  else if (dtype == BITNET_KV_FP16)
    append_dim<BITNET_KV_FP16>(a, head_dim, stream);
  else
    append_dim<BITNET_KV_INT8>(a, head_dim, stream);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const ReorderArgs &a, hipStream_t stream) {
  beam_reorder_kernel<<<dim3((unsigned)(a.B * a.W), (unsigned)(a.layers + 1)), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace bitnet
