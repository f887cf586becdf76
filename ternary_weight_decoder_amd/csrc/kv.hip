// The paged key-value cache: the page map of a step, the write of new tokens
// and the reordering of beams.  (The attention that reads the cache is in
// attention.hip.)
#include <algorithm>

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
// all of it, so that nothing but its own barriers orders the steps; what bounds
// it is their latency.  So each pair of sums is one pass of saturating adds in
// registers and one barrier; pages given back and granted are moved a thread
// each, which finds its request by bisection of the sums; and the top of the
// stack is asked for at the start, for the calls in which no request ends.
// Steps of many tokens write their slots in a second kernel of many workgroups.
// (One step of 16 requests: 3.6 us, of which a launch is 1.8; with 64-bit sums
// through the lanes' exchange, two barriers each, and a thread moving all pages of
// its request it took 17.8.)
// ---------------------------------------------------------------------------

constexpr int kMapThreads = 1024;
constexpr int kMapWaves = kMapThreads / 64;

struct Pair {
  uint32_t p, t;   // pages, tokens
};
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
  return __builtin_elementwise_add_sat(a, b);
}
__device__ __forceinline__ Pair add_sat(Pair a, Pair b) {
  return {add_sat(a.p, b.p), add_sat(a.t, b.t)};
}
template <int CTRL, int ROWS>
__device__ __forceinline__ Pair scan_step(Pair v) {
  return add_sat(v, Pair{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)v.p, CTRL, ROWS, 0xF, false),
                         (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v.t, CTRL, ROWS, 0xF, false)});
}
// Inclusive sums over the rows of 16 lanes.
__device__ __forceinline__ Pair row_scan(Pair v) {
  v = scan_step<0x111, 0xF>(v);   // row_shr:1
  v = scan_step<0x112, 0xF>(v);
  v = scan_step<0x114, 0xF>(v);
  return scan_step<0x118, 0xF>(v);
}
__device__ __forceinline__ Pair lane_of(Pair v, int lane) {
  return {(uint32_t)__builtin_amdgcn_readlane((int)v.p, lane),
          (uint32_t)__builtin_amdgcn_readlane((int)v.t, lane)};
}

// Inclusive sums over the workgroup's threads, which saturate (and so stay above
// whatever they are compared with), and the total.  Calls in a row take different
// rows of `sums`: one barrier then orders them.
__device__ __forceinline__ Pair block_scan(Pair v, Pair *sums, Pair *total) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  v = row_scan(v);
  v = scan_step<0x142, 0xA>(v);   // row_bcast:15
  v = scan_step<0x143, 0xC>(v);   // row_bcast:31
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  Pair w = {0, 0};
  if (lane < (int)(blockDim.x >> 6)) w = sums[lane];
  w = row_scan(w);
  *total = lane_of(w, kMapWaves - 1);
  return wave ? add_sat(v, lane_of(w, wave - 1)) : v;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// The first i < n with ends[i] > k; the last of them is above k.
__device__ __forceinline__ int find(const uint32_t *ends, int n, uint32_t k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > k) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Tokens t0 + j * step of the step, j < N: the request by bisection of starts, the
// position from the request's length after the step, the slot from the table.
template <int N>
__device__ __forceinline__ void map_tokens(const KvMapArgs &a, const int32_t *starts,
                                           const int32_t *lens_after, int64_t t0, int step) {
  int lo[N], hi[N], pos[N], page[N];
  const int all = starts[a.B];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    lo[j] = 0;
    hi[j] = a.B - 1;
  }
  for (int n = a.B - 1; n > 0; n >>= 1)   // the last request that starts at or before t
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int mid = (lo[j] + hi[j] + 1) >> 1;
      const bool up = starts[mid] <= t0 + j * step;
      lo[j] = up ? mid : lo[j];
      hi[j] = up ? hi[j] : max(mid - 1, lo[j]);
    }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int64_t t = t0 + j * step;
    pos[j] = page[j] = -1;
    if (t < all) {
      pos[j] = lens_after[lo[j]] - (starts[lo[j] + 1] - (int)t);
      page[j] = a.tables[(int64_t)lo[j] * a.max_pages + (pos[j] >> a.page_shift)];
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int64_t t = t0 + j * step;
    if (t < a.T) {
      const bool there = page[j] >= 0 && page[j] < a.pages;
      a.slots[t] =
          there ? (page[j] << a.page_shift) + (pos[j] & ((1 << a.page_shift) - 1)) : -1;
      a.positions[t] = pos[j];
      a.rows[t] = t < all ? lo[j] : -1;
    }
  }
}

__global__ void __launch_bounds__(kMapThreads) kv_map_kernel(KvMapArgs a, int tokens_here) {
  __shared__ Pair sums[2][kMapWaves];
  __shared__ uint32_t ends[kMapThreads];
  __shared__ int32_t firsts[kMapThreads], helds[kMapThreads];
  __shared__ int32_t starts[kMaxRows + 1];
  __shared__ int32_t lens_after[kMaxRows];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int ps = 1 << a.page_shift;
  const int cap = a.max_pages << a.page_shift;   // tokens a table holds
  int flip = 0;
  Pair total;

  const int height0 = clampi(a.state_in[2 * a.B], 0, a.pages);
  const int top = tid < height0 ? a.free_pages[height0 - 1 - tid] : 0;

  // Ended requests give their pages back.
  int height = height0;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int r = b0 + tid, rows = min(threads, a.B - b0);
    const bool ends_here = r < a.B && a.new_lens[r] < 0;
    const int held = ends_here ? clampi(a.state_in[a.B + r], 0, a.max_pages) : 0;
    const Pair upto = block_scan({(uint32_t)held, 0}, sums[flip ^= 1], &total);
    if (total.p == 0) continue;   // the same for every thread
    ends[tid] = upto.p;
    __syncthreads();
    const uint32_t n = min(total.p, (uint32_t)(a.pages - height));
    for (uint32_t k0 = tid; k0 < n; k0 += 4 * threads) {
      int page[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t k = k0 + j * threads;
        if (k < n) {
          const int q = find(ends, rows, k);
          page[j] = a.owned[(int64_t)(b0 + q) * a.max_pages + (k - (q ? ends[q - 1] : 0))];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + j * threads < n) a.free_pages[height + k0 + j * threads] = page[j];
    }
    height += n;
  }
  const bool untouched = height == height0;   // else the stack is read below
  if (!untouched) __syncthreads();

  Pair want = {0, 0}, granted = {0, 0};   // of the requests before this chunk
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int r = b0 + tid, rows = min(threads, a.B - b0);
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
    const uint32_t need = fits ? (uint32_t)need64 : 0;
    const Pair upto = add_sat(
        want, block_scan({need, fits ? (uint32_t)add : 0}, sums[flip ^= 1], &total));
    want = add_sat(want, total);
    const bool paged = need == 0 || upto.p <= (uint32_t)height;
    const bool room = add == 0 || upto.t <= a.T;
    const bool ok = fits && paged && room;
    const uint32_t np = ok ? need : 0, nt = ok ? (uint32_t)add : 0;
    // (What is granted is at most the height and T: no sum saturates.)
    const Pair got = block_scan({np, nt}, sums[flip ^= 1], &total);
    ends[tid] = got.p;
    firsts[tid] = first;
    helds[tid] = held;
    if (r < a.B) {
      const int32_t at = (int32_t)(granted.t + got.t - nt);
      starts[r] = at;
      lens_after[r] = len + (int)nt;
      a.starts[r] = at;
      a.status[r] = fits ? (paged ? (room ? 0 : 3) : 2) : 1;
      a.state_out[r] = len + (int)nt;
      a.state_out[a.B + r] = held + (int)np;
    }
    __syncthreads();
    const int base = height - 1 - (int)granted.p;
    const bool have = untouched && granted.p == 0;
    for (uint32_t k0 = tid; k0 < total.p; k0 += 4 * threads) {
      int page[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + j * threads < total.p)
          page[j] = have && j == 0 && k0 == (uint32_t)tid
                        ? top
                        : a.free_pages[base - (int)(k0 + j * threads)];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t k = k0 + j * threads;
        if (k < total.p) {
          const int q = find(ends, rows, k);
          const int i = (int)(k - (q ? ends[q - 1] : 0));
          const int64_t row = (int64_t)(b0 + q) * a.max_pages;
          a.tables[row + firsts[q] + i] = page[j];
          a.owned[row + helds[q] + i] = page[j];
        }
      }
    }
    granted = add_sat(granted, total);
    __syncthreads();   // before the lists are written again, and the tables read
  }
  if (tid == 0) {
    starts[a.B] = (int32_t)granted.t;
    a.starts[a.B] = (int32_t)granted.t;
    a.state_out[2 * a.B] = height - (int32_t)granted.p;
  }
  if (!tokens_here) return;
  __syncthreads();
  for (int64_t t = tid; t < a.T; t += 4 * threads) {
    if (a.T <= threads)
      map_tokens<1>(a, starts, lens_after, t, threads);
    else
      map_tokens<4>(a, starts, lens_after, t, threads);
  }
}

// A token a thread: four, with fewer workgroups, took 1.7 us more (57,600 tokens
// of 256 requests).
constexpr int kTokenThreads = 256;

__global__ void __launch_bounds__(kTokenThreads) kv_map_tokens_kernel(KvMapArgs a) {
  __shared__ int32_t starts[kMaxRows + 1];
  for (int i = threadIdx.x; i <= a.B; i += kTokenThreads) starts[i] = a.starts[i];
  __syncthreads();
  const int64_t t = (int64_t)blockIdx.x * kTokenThreads + threadIdx.x;
  map_tokens<1>(a, starts, a.state_out, t, kTokenThreads);
}

// Calls of up to this many tokens finish in the one workgroup.
constexpr int64_t kMapTokensHere = 4096;

// ---------------------------------------------------------------------------
// Append: rotate, convert, scatter.
//
// One workgroup per token; a thread holds four channels of each half of a
// head, so a rotation needs no exchange and an 8-bit row's maximum is a
// reduction over head_dim / 8 adjacent lanes.  Bound by memory, short calls by the
// launch: 1800 tokens of 12 + 2 * 2 heads of 128 channels 8.8 us for 28.6 MB (9.3
// with the activations asked for after the slot), 16 tokens 2.5; 4096 tokens of
// 32 + 2 * 8 heads of 256 channels 72 us, 5.2 TB/s: the stream hides the fp64
// rotations.
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
  const int hq = a.q ? a.q_heads : 0;
  const int items = (hq + 2 * a.c.kv_heads) * kPer;
  // Everything that no other load decides is asked for at once.
  const int slot = a.slots[t];
  const bool rotate = a.cos != nullptr;
  const int pos = rotate ? a.positions[t] : 0;
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
    if (slot < 0 || page >= a.c.pages) return;
    if (rotate && (pos < 0 || pos >= a.max_pos)) return;
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
// are disjoint, so one launch copies in place.  A workgroup copies one side of
// one layer's page; the copies are the whole cost and are bound by memory.  128
// rows of 28 layers, up to 64 tokens of 2 heads of 128 channels in 16 bits: 31.5 us
// with eight pairs in flight and non-temporal stores, 40.9 with ordinary ones,
// 43.2 with a page's two sides in one workgroup.
// ---------------------------------------------------------------------------

constexpr int kEach = 8;   // (head, token) pairs of a thread in flight

__global__ void __launch_bounds__(256) beam_reorder_kernel(ReorderArgs a) {
  const int row = blockIdx.x;
  const int layer = (int)blockIdx.y - 1, side = blockIdx.z;
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
    if (side) return;
    const int32_t *self = a.tables_in + (int64_t)row * a.max_pages;
    int32_t *out = a.tables_out + (int64_t)row * a.max_pages;
    for (int i = threadIdx.x; i < a.max_pages; i += 256)
      out[i] = i < last ? from[i] : i == last && tail ? giver[i] : self[i];
    return;
  }
  if (!move || tail == 0) return;
  const int64_t src = from[last], dst = giver[last];
  if (src < 0 || src >= a.c.pages || dst < 0 || dst >= a.c.pages) return;
  // 16-byte pieces: a thread keeps its piece of a head and steps over (head,
  // token) pairs, several of them in flight.
  const int vec_shift = __builtin_ctz(a.head_dim * a.elem_bytes / 16);
  const int piece = threadIdx.x & ((1 << vec_shift) - 1);
  const int step = 256 >> vec_shift, n = a.c.kv_heads * tail;
  const float per_tail = __builtin_amdgcn_rcpf((float)tail);
  auto head_of = [&](int m) { return (int)(((float)m + 0.5f) * per_tail); };   // exact: m < 2^18
  const int64_t page_bytes = a.c.page_stride * a.elem_bytes;
  uint8_t *base = reinterpret_cast<uint8_t *>(side ? a.c.v : a.c.k) +
                  layer * a.layer_stride * a.elem_bytes + piece * 16;
  for (int m0 = threadIdx.x >> vec_shift; m0 < n; m0 += kEach * step) {
    u32x4 x[kEach];
    int64_t off[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int m = m0 + j * step;
      if (m < n) {
        const int h = head_of(m);
        off[j] = (h * a.c.head_stride + (m - h * tail) * a.c.token_stride) * a.elem_bytes;
        x[j] = ld_global<u32x4>(base + src * page_bytes + off[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (m0 + j * step < n)
        __builtin_nontemporal_store(
            x[j], (BITNET_GLOBAL u32x4 *)(base + dst * page_bytes + off[j]));
  }
  float *sc = side ? a.c.v_scale : a.c.k_scale;
  if (sc != nullptr) {
    sc += (int64_t)layer * a.c.pages * a.c.kv_heads * ps;
    for (int i = threadIdx.x; i < n; i += 256) {
      const int h = head_of(i), tok = i - h * tail;
      sc[(dst * a.c.kv_heads + h) * ps + tok] = sc[(src * a.c.kv_heads + h) * ps + tok];
    }
  }
}

}  // namespace

hipError_t launch_kv_map(const KvMapArgs &a, hipStream_t stream) {
  const bool here = a.T <= kMapTokensHere;
  // A thread for each request, or for four of the tokens or pages of a table; all
  // there can be for long steps, whose pages are many (256 requests, 57,600 tokens:
  // 9.8 us, 14.8 with 256 threads).
  const int64_t want = std::max<int64_t>(
      {a.B, here ? a.T / 4 : kMapThreads, a.max_pages / 4, here && a.T <= 256 ? a.T : 0});
  const int threads = (int)std::min<int64_t>((want + 63) / 64 * 64, kMapThreads);
  kv_map_kernel<<<1, threads, 0, stream>>>(a, here);
  if (!here) {
    kv_map_tokens_kernel<<<(unsigned)((a.T + kTokenThreads - 1) / kTokenThreads), kTokenThreads, 0,
                           stream>>>(a);
  }
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
  beam_reorder_kernel<<<dim3((unsigned)(a.B * a.W), (unsigned)(a.layers + 1), 2), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace bitnet
