// Attention of the new tokens of several requests over the paged key-value
// cache: prompts, pieces of prompts, guessed tokens.
//
//   token i of the n new ones of a request of len tokens sees L = len - n + i + 1:
//   s_j = scale * q . k_j,   p_j = exp(s_j - max s),   out = sum_j<L p_j v_j / sum p_j
//
// A key/value row serves all new tokens of its request and all query heads of
// its group, so the rows of the product are (token, head) pairs, 128 of them to
// an item, a wave each 32; tiles of 32 tokens of keys and values go through LDS
// once for the item.  The work is bound by the matrix cores.
//
// Tile.  Keys are the row operand of v_mfma_f32_32x32x16 and queries the column
// operand, so the scores arrive transposed: lane (c, h) holds column c, tokens
// 8 a + 4 h + e (a, e < 4).  That is how the second product takes its
// probabilities, once its contraction steps are numbered to match: step k = 8 h
// + j of 16-token half s is token 16 s + 4 h + j, or 16 s + 8 + 4 h + j - 4 from
// j = 4 on.  The values come in that order by the transposing LDS reads, four
// tokens of a channel at a time.  Nothing crosses lanes but the two halves'
// maximum.
//
// Precision.  As in the attention of single tokens: queries and probabilities
// enter as sums of 16-bit terms that carry fp32's precision together, three of
// bf16 against bf16 values, two of fp16 against fp16 values and 8-bit codes,
// scaled by powers of two into fp16's range.
//
// Work.  The items of a call, each as long as its last row sees, lie on one
// line, which is cut into equal stretches, a workgroup each, from the lengths
// on the device.  A tile of an item costs what its last row sees, counted in
// rows: a linear function of the tile's number, so every place on the line has
// a closed form and no list of items is made.  A stretch may hold the end of an
// item, whole ones and the beginning of another; the parts of an item are joined
// by the workgroup that finishes last.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"
#include "terms.hpp"

namespace bitnet {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCols = 32;                 // rows (token, head) of a wave
constexpr int kRows = kCols * kWaves;     // of an item
constexpr int kTile = 32;                 // tokens of a step
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

constexpr int kGrid = 512;                // workgroups: two a compute unit
constexpr int kHeaderBytes = 4 * kGrid;   // a counter for each
constexpr int kLeast = 1;                 // tiles of a stretch, at least

struct ChunkPlan {
  int groups;
  size_t outs, stats, total;   // workspace offsets
};

ChunkPlan chunk_plan(int64_t T, int64_t R, int64_t q_heads, int64_t kv_heads, int64_t D,
                     int64_t max_len) {
  const int64_t items = kv_heads * (T * (q_heads / kv_heads) / kRows + R);
  const int64_t tiles = (max_len + kTile - 1) / kTile;
  ChunkPlan p;
  p.groups = (int)std::min<int64_t>(D == 256 ? kGrid / 2 : kGrid, items * tiles);
  // Two places a workgroup: for the item at its beginning and the one at its end.
  const size_t rows = 2 * (size_t)p.groups * kRows;
  p.outs = kHeaderBytes;
  p.stats = p.outs + rows * D * 4;
  p.total = p.stats + rows * 8;
  return p;
}

template <int DT> struct Operand;
template <> struct Operand<BITNET_KV_BF16> {
  typedef bf16x8 V;
  static constexpr int kBytes = 2, kTerms = 3;
  static constexpr bool kHalf = false;
  static __device__ __forceinline__ f32x16 mfma(V a, V b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ void split(const float (&x)[8], V (&t)[3]) {
    terms_bf16(x, t);
  }
};
struct OperandF16 {
  typedef f16x8 V;
  static constexpr int kTerms = 2;
  static constexpr bool kHalf = true;
  static __device__ __forceinline__ f32x16 mfma(V a, V b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ void split(const float (&x)[8], V (&t)[2]) {
    terms_f16(x, t);
  }
};
template <> struct Operand<BITNET_KV_FP16> : OperandF16 { static constexpr int kBytes = 2; };
template <> struct Operand<BITNET_KV_INT8> : OperandF16 { static constexpr int kBytes = 1; };

// Maximum and sum over the two halves of a wave.
__device__ __forceinline__ float max2(float v) {
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const uint32_t p0 = p[0], p1 = p[1];
  return fmaxf(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1));
}
__device__ __forceinline__ float sum2(float v) {
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const uint32_t p0 = p[0], p1 = p[1];
  return __builtin_bit_cast(float, p0) + __builtin_bit_cast(float, p1);
}

// Inclusive sum and maximum over the wave.  Places on the line are whole numbers
// below 2^53, held in fp64, whose division and square root are short.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double scan_sum(double v) {
  v = add_from<0x111, 0xF>(v);   // row_shr:1
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);   // row_bcast:15
  return add_from<0x143, 0xC>(v);   // row_bcast:31
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int max_from(int v) {   // v >= 0
  return max(v, __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ int scan_max(int v) {
  v = max_from<0x111, 0xF>(v);
  v = max_from<0x112, 0xF>(v);
  v = max_from<0x114, 0xF>(v);
  v = max_from<0x118, 0xF>(v);
  v = max_from<0x142, 0xA>(v);
  return max_from<0x143, 0xC>(v);
}
// floor(x / d) of whole numbers below 2^53.
__device__ __forceinline__ double quotient(double x, double d) {
  const double q = floor(x / d);
  return q * d > x ? q - 1.0 : q;
}
__device__ __forceinline__ double uniform(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int DT, int D>
struct ChunkShape {
  static constexpr int kBytes = Operand<DT>::kBytes;
  static constexpr int kPieces = D * kBytes / 16;             // of a cached row
  static constexpr int kPass = kThreads / kPieces < kTile ? kThreads / kPieces : kTile;   // tokens
  static constexpr int kLoads = kTile / kPass;                // of a thread, keys and values each
  static constexpr int kRow = 2 * D + 16;                     // bytes of a row in LDS
};

template <int DT, int D>
struct ChunkShared {
  typedef ChunkShape<DT, D> S;
  __attribute__((aligned(16))) uint8_t k[2][kTile * S::kRow], v[2][kTile * S::kRow];
  float scales[kWaves][2][kTile];   // 8-bit caches: the tile's key and value scales
  double first[kThreads];           // places before each thread's requests
  int top[kThreads];                // largest start before them
  double wave_sum[kWaves];
  int wave_top[kWaves];
  uint32_t last;
};

struct ChunkGrid {
  int64_t outs_off, stats_off;
  int32_t groups, per;   // workgroups; query heads per key/value head
};

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
chunk_kernel(ChunkArgs a, ChunkGrid g) {
  typedef Operand<DT> F;
  typedef typename F::V V;
  typedef ChunkShape<DT, D> S;
  constexpr bool kI8 = DT == BITNET_KV_INT8;
  constexpr int kSteps = D / 16;       // contraction steps of the scores
  constexpr int kBlocks = D / 32;      // channel blocks of the outputs
  constexpr int kTerms = F::kTerms;
  constexpr float kUp = F::kHalf ? 14.0f : 0.0f;   // probabilities are scaled by 2^kUp
  __shared__ ChunkShared<DT, D> sh;

  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = g.per, kv_heads = a.c.kv_heads;

  // A request's new tokens [from, to), the largest start so far being `top`
  // (starts are taken in ascending order whatever they hold), and what it adds
  // to the line for each key/value head.
  struct Request {
    int from, n, old, tiles;   // old: tokens before the new ones (may be negative)
    double rows, lead, line;   // n * per; rows that lie before an item's own; places
  };
  auto request = [&](int r, int &top) {
    top = max(top, ld_global<int>(a.starts + r));
    Request q;
    q.from = min(top, a.T);
    const int to = min(max(top, ld_global<int>(a.starts + r + 1)), a.T);
    q.n = to - q.from;
    q.old = min(max(ld_global<int>(a.lens + r), 0), a.max_len) - q.n;
    const int rows = q.n * per;
    q.tiles = (rows + kRows - 1) / kRows;
    q.rows = rows;
    q.lead = (double)max(q.old, 0) * per;
    q.line = q.tiles == 0 ? 0.0
                          : q.tiles * q.lead + (double)(kRows / 2) * q.tiles * (q.tiles - 1) + q.rows;
    return q;
  };

  const int each = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(tid * each, a.R), r1 = min(r0 + each, a.R);
  double total;
  {
    int top = 0;
    for (int r = r0; r < r1; ++r) top = max(top, ld_global<int>(a.starts + r));
    const int upto = scan_max(top);
    if (lane == 63) sh.wave_top[wave] = upto;
    sh.top[tid] = upto;
    __syncthreads();
    int before = tid % 64 ? sh.top[tid - 1] : 0;
    for (int w = 0; w < wave; ++w) before = max(before, sh.wave_top[w]);
    __syncthreads();
    sh.top[tid] = top = before;
    double sum = 0.0;
    for (int r = r0; r < r1; ++r) sum += request(r, top).line * kv_heads;
    const double all = scan_sum(sum);
    if (lane == 63) sh.wave_sum[wave] = all;
    __syncthreads();
    double from = all - sum;
    total = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      from += w < wave ? sh.wave_sum[w] : 0.0;
      total += sh.wave_sum[w];
    }
    sh.first[tid] = from;
    __syncthreads();
    total = uniform(total);
  }
  const double unit = (double)per * kTile;   // of a tile of tokens
  const double stretch = uniform(fmax(quotient(total + g.groups - 1, g.groups), kLeast * unit));
  const int w = blockIdx.x;
  const double begin = w * stretch, stop = fmin(begin + stretch, total);
  double pos = begin;
  int buf = 0;

  while (pos < stop) {
    // The item at pos.
    Request q;
    int r, kvh, tile0;   // tile0: the item's number among the request's of this head
    double item0, item_end;
    {
      int at = 0;
#pragma unroll
      for (int i = 0; i < kThreads; i += 64) at += __builtin_popcountll(__ballot(sh.first[i + lane] <= pos));
      at -= 1;
      int top = sh.top[at];
      double from = sh.first[at];
      r = at * each;
      for (;;) {
        q = request(r, top);
        const double next = from + q.line * kv_heads;
        if (pos < next || r + 1 >= min(at * each + each, a.R)) break;
        from = next;
        ++r;
      }
      kvh = min((int)quotient(pos - from, q.line), kv_heads - 1);
      from += kvh * q.line;
      const double o = pos - from, b = q.lead + kRows / 2;
      auto before = [&](int j) { return j * q.lead + (double)(kRows / 2) * j * (j + 1.0); };
      int j = (int)((sqrt(b * b + 2.0 * kRows * o) - b) / kRows);
      j = max(min(j, q.tiles - 1), 0);
      while (j > 0 && before(j) > o) --j;
      while (j + 1 < q.tiles && before(j + 1) <= o) ++j;
      tile0 = j;
      item0 = from + before(j);
      item_end = item0 + q.lead + fmin((j + 1.0) * kRows, q.rows);
    }
    r = __builtin_amdgcn_readfirstlane(r);
    kvh = __builtin_amdgcn_readfirstlane(kvh);
    tile0 = __builtin_amdgcn_readfirstlane(tile0);
    item0 = uniform(item0);
    item_end = uniform(item_end);
    const int from = __builtin_amdgcn_readfirstlane(q.from), old = __builtin_amdgcn_readfirstlane(q.old);
    const int m0 = tile0 * kRows;
    const int count = min(kRows, __builtin_amdgcn_readfirstlane(q.n) * per - m0);
    const int len = min(max(old + (m0 + count - 1) / per + 1, 0), a.max_len);   // that the last row sees
    const int tiles = (len + kTile - 1) / kTile;
    // Tiles [first, end) of the item are this stretch's.
    auto cut = [&](double at) {
      return at <= item0 ? 0 : (int)fmin(quotient(at - item0, unit), (double)tiles);
    };
    const int first = __builtin_amdgcn_readfirstlane(cut(begin));
    const int end = __builtin_amdgcn_readfirstlane(item_end <= stop ? tiles : cut(stop));
    const bool whole = first == 0 && end == tiles;
    const double here = pos;
    pos = fmax(fmin(item_end, stop), here + 1.0);   // (item_end > here: the loop ends in any case)
    if (first == end && !(tiles == 0 && here == item0)) continue;

    // This lane's row.
    const int in = wave * kCols + c, m = m0 + min(in, count - 1);
    const bool live = in < count, active = wave * kCols < count;
    const int i = m / per, head = kvh * per + (m - i * per);
    const int limit = min(max(old + i + 1, 0), a.max_len);
    // What the wave's first and last rows see.
    const int limit_lo = __builtin_amdgcn_readlane(limit, 0);
    const int limit_hi = active ? __builtin_amdgcn_readlane(limit, 31) : 0;
    const int item_lo = min(max(old + m0 / per + 1, 0), a.max_len);
    const int64_t out_row = (int64_t)(from + i) * a.q_heads + head;

    const int64_t head_off = (int64_t)kvh * a.c.head_stride * S::kBytes;
    const uint8_t *kbase = reinterpret_cast<const uint8_t *>(a.c.k) + head_off;
    const uint8_t *vbase = reinterpret_cast<const uint8_t *>(a.c.v) + head_off;
    const int32_t *table = a.tables + (int64_t)r * a.max_pages;
    const uint64_t page_bytes = (uint64_t)a.c.page_stride * S::kBytes;
    const uint32_t tok_bytes = (uint32_t)(a.c.token_stride * S::kBytes);
    const int tok_mask = (1 << a.c.page_shift) - 1;
    // Staging: this thread's 16-byte piece of tokens st0, st0 + kPass, ...
    const int piece = tid % S::kPieces, st0 = tid / S::kPieces;
    const bool stages = st0 < kTile;

    int pg = 0;                      // page of token c of the tile after the loaded one
    u32x4 kr[S::kLoads], vr[S::kLoads];
    uint32_t mask_next = 0;          // tokens of the loaded tile that are there
    float ksc = 0.0f, vsc = 0.0f;
    auto load_page = [&](int tile) {
      const int j = min(tile * kTile + c, len - 1);
      pg = ld_global<int>(table + (j >> a.c.page_shift));
    };
    auto load_rows = [&](int tile) {
      const int j = tile * kTile + c;
      const bool ok = j < len && (uint32_t)pg < (uint32_t)a.c.pages;
      mask_next = (uint32_t)__ballot(ok);
      const uint32_t page = ok ? pg : 0, tok = ok ? j & tok_mask : 0;
      if constexpr (kI8) {
        const uint32_t at = ((page * (uint32_t)kv_heads + kvh) << a.c.page_shift) + tok;
        ksc = ld_global<float>(a.c.k_scale + at);
        vsc = ld_global<float>(a.c.v_scale + at);
      }
#pragma unroll
      for (int l = 0; l < S::kLoads; ++l) {
        const int t = (st0 + l * S::kPass) & (kTile - 1);
        const uint64_t off = (uint64_t)(uint32_t)__shfl((int)page, t) * page_bytes +
                             (uint64_t)(uint32_t)__shfl((int)tok, t) * tok_bytes + 16 * piece;
        if (stages) {
          kr[l] = ld_global<u32x4>(kbase + off);
          vr[l] = ld_global<u32x4>(vbase + off);
        }
      }
    };

    if (first < end) load_page(first);
    // Queries as terms.
    V qt[kSteps][kTerms];
    float unscale = 1.0f;   // of the scores
    {
      const float *src = a.q + (int64_t)(from + i) * a.q_stride + (int64_t)head * D;
      f32x4 x[kSteps][2];
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        x[f][0] = ld_global<f32x4>(src + 16 * f + 8 * h);
        x[f][1] = ld_global<f32x4>(src + 16 * f + 8 * h + 4);
      }
      if (first < end) {
        load_rows(first);
        load_page(first + 1);
      }
      float big = 0.0f;
#pragma unroll
      for (int f = 0; f < kSteps; ++f)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[f][e >> 2][e & 3] *= a.scale * kLog2e;
          big = fmaxf(big, fabsf(x[f][e >> 2][e & 3]));
        }
      float up = 1.0f;
      if constexpr (F::kHalf) {
        const float p2 = pow2_above(max2(big));
        unscale = p2 * 0x1p-14f;
        up = pow2_inverse(p2) * 0x1p14f;
      }
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[f][e >> 2][e & 3] * up;
        F::split(y, qt[f]);
      }
    }

    float mx = -INFINITY, l = 0.0f;   // mx in units of 1 / unscale
    f32x16 o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[b][e] = 0.0f;
    float vmax = pow2_above(0.0f);    // 8-bit caches: o is in units of this

    for (int tile = first; tile < end; ++tile) {
      const uint32_t mask = mask_next;
      const bool edge = (tile + 1) * kTile > item_lo;   // not every row sees all of the tile
      // The tile into LDS.  Tokens that are not there get values of zero; where
      // not every row sees every token, values that are not finite do too, so
      // that they reach no row that must not see them.
      if (stages) {
#pragma unroll
        for (int n = 0; n < S::kLoads; ++n) {
          const int t = st0 + n * S::kPass;
          u32x4 v = vr[n];
          if (mask != 0xffffffffu && !((mask >> t) & 1)) v = u32x4{0u, 0u, 0u, 0u};
          if (!kI8 && edge)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              constexpr uint32_t kInf = DT == BITNET_KV_BF16 ? 0x7f80u : 0x7c00u;
              if ((v[e] & kInf) == kInf) v[e] &= 0xffff0000u;
              if ((v[e] >> 16 & kInf) == kInf) v[e] &= 0xffffu;
            }
          if constexpr (kI8) {
            uint8_t *kd = sh.k[buf] + t * S::kRow + 32 * piece, *vd = sh.v[buf] + t * S::kRow + 32 * piece;
            *reinterpret_cast<f16x8 *>(kd) = codes_f16(kr[n].x, kr[n].y);
            *reinterpret_cast<f16x8 *>(kd + 16) = codes_f16(kr[n].z, kr[n].w);
            *reinterpret_cast<f16x8 *>(vd) = codes_f16(v.x, v.y);
            *reinterpret_cast<f16x8 *>(vd + 16) = codes_f16(v.z, v.w);
          } else {
            *reinterpret_cast<u32x4 *>(sh.k[buf] + t * S::kRow + 16 * piece) = kr[n];
            *reinterpret_cast<u32x4 *>(sh.v[buf] + t * S::kRow + 16 * piece) = v;
          }
        }
      }
      const float ks_now = ksc, vs_now = vsc;
      if (tile + 1 < end) {
        load_rows(tile + 1);
        load_page(tile + 2);
      }
      __syncthreads();
      const uint8_t *krows = sh.k[buf], *vrows = sh.v[buf];
      buf ^= 1;
      if (tile * kTile >= limit_hi) continue;   // the wave sees none of it

      const bool all = mask == 0xffffffffu && (tile + 1) * kTile <= limit_lo;
      float ks[16], vs[16], vkeep = 1.0f;
      if constexpr (kI8) {
        const bool ok = (mask >> c) & 1;
        if (h == 0) {
          sh.scales[wave][0][c] = ok ? ks_now : 0.0f;
          sh.scales[wave][1][c] = ok && fabsf(vs_now) < INFINITY ? vs_now : 0.0f;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 ks4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][0][8 * b + 4 * h]);
          const f32x4 vs4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][1][8 * b + 4 * h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ks[4 * b + e] = ks4[e];
            vs[4 * b + e] = vs4[e];
          }
        }
        __builtin_amdgcn_wave_barrier();
        // Relative to the power of two above the largest that the row has seen.
        float big = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (!all && tile * kTile + 8 * (e >> 2) + 4 * h + (e & 3) >= limit) vs[e] = 0.0f;
          big = fmaxf(big, vs[e]);
        }
        const float v_new = fmaxf(vmax, pow2_above(max2(big)));
        const float inv = pow2_inverse(v_new);
        vkeep = vmax * inv;
        vmax = v_new;
#pragma unroll
        for (int e = 0; e < 16; ++e) vs[e] *= inv;
      }

      f32x16 s[1];
#pragma unroll
      for (int e = 0; e < 16; ++e) s[0][e] = 0.0f;
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        const V k = *reinterpret_cast<const V *>(krows + c * S::kRow + 32 * f + 16 * h);
#pragma unroll
        for (int p = kTerms - 1; p >= 0; --p) s[0] = F::mfma(k, qt[f][p], s[0]);
      }
      settle<D>(s);
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = kI8 ? s[0][e] * ks[e] : s[0][e];
      if (!all)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int t = 8 * (e >> 2) + 4 * h + (e & 3);
          if (!((mask >> t) & 1) || tile * kTile + t >= limit) x[e] = -INFINITY;
        }
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
      const float m_new = fmaxf(mx, max2(top));
      const float base = m_new == -INFINITY ? 0.0f : m_new;
      const float lkeep = exp2_fast((mx - base) * unscale);
      const float keep = lkeep * vkeep;
      mx = m_new;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = exp2_fast(__builtin_fmaf(x[e] - base, unscale, kUp));
        sum += x[e];
      }
      l = l * lkeep + sum;   // not in units of vmax
      if constexpr (kI8)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= vs[e];
      if (__any(keep != 1.0f))
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[b] *= keep;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[8 * half + e];
        V p[kTerms];
        F::split(y, p);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const int cc = lane & 15;
          const uint8_t *at = vrows + (16 * half + 4 * h + (cc >> 2)) * S::kRow + 64 * b +
                              32 * (lane >> 4 & 1) + 8 * (cc & 3);
          s16x4 t[2];
          t[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((BITNET_LDS s16x4 *)at);
          t[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((BITNET_LDS s16x4 *)(at + 8 * S::kRow));
          const V v = __builtin_bit_cast(V, t);
#pragma unroll
          for (int n = kTerms - 1; n >= 0; --n) o[b] = F::mfma(v, p[n], o[b]);
        }
      }
      settle<D>(o);
    }
    mx *= unscale;
    l = sum2(l);
    if constexpr (kI8)
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) o[b] *= vmax;

    auto finish = [&]() {
      if (!live) return;
      float *out = a.out + out_row * D;
      const float over = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x4 y = {o[b][4 * e], o[b][4 * e + 1], o[b][4 * e + 2], o[b][4 * e + 3]};
          st_global<f32x4>(out + 32 * b + 8 * e + 4 * h,
                           l > 0.0f ? y * over : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        }
      if (a.lse && h == 0) a.lse[out_row] = l > 0.0f ? (mx - kUp + __log2f(l)) * kLn2 : -INFINITY;
    };
    if (whole) {
      finish();
      continue;
    }

    // The stretches that hold the item: of them w_first is the first with a tile.
    const int w_end = (int)quotient(item_end - 1.0, stretch);
    const int w_first = min((int)quotient(item0 + unit - 1.0, stretch), w_end);
    const int w_last = min((int)quotient(item0 + tiles * unit - 1.0, stretch), w_end);
    const int parts = __builtin_amdgcn_readfirstlane(w_last - w_first + 1);
    const int w0 = __builtin_amdgcn_readfirstlane(w_first);
    auto place_of = [&](int ww) { return 2 * ww + (item0 > ww * stretch ? 1 : 0); };
    constexpr uint32_t kPartBytes = kRows * D * 4;
    const __amdgpu_buffer_rsrc_t outs = make_rsrc(a.ws + g.outs_off, 2 * g.groups * kPartBytes);
    uint64_t *stats = reinterpret_cast<uint64_t *>(a.ws + g.stats_off);
    const uint32_t mine = (wave * kBlocks * 4 * 64 + lane) * 16;
    if (active) {
      const uint32_t at = place_of(w) * kPartBytes + mine;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_device(outs, at + (b * 4 + e) * 1024,
                     f32x4{o[b][4 * e], o[b][4 * e + 1], o[b][4 * e + 2], o[b][4 * e + 3]});
      if (h == 0)
        __hip_atomic_store((BITNET_GLOBAL uint64_t *)&stats[place_of(w) * kRows + in],
                           __builtin_bit_cast(uint64_t, f32x2{mx, l}), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    // Each wave's stores have been acknowledged before the counter moves.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    uint32_t *ticket = reinterpret_cast<uint32_t *>(a.ws) + w0;
    if (tid == 0) {
      const uint32_t n = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sh.last = n == (uint32_t)parts - 1;
      if (sh.last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!sh.last || !active) continue;
    auto stat = [&](int p) {
      return __builtin_bit_cast(
          f32x2, (uint64_t)__hip_atomic_load((const BITNET_GLOBAL uint64_t *)&stats[place_of(w0 + p) * kRows + in],
                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    };
    float tm = -INFINITY;
    for (int p = 0; p < parts; ++p) tm = fmaxf(tm, stat(p).x);
    const float base = tm == -INFINITY ? 0.0f : tm;
    l = 0.0f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[b][e] = 0.0f;
    for (int p = 0; p < parts; ++p) {
      const f32x2 st = stat(p);
      const uint32_t at = place_of(w0 + p) * kPartBytes + mine;
      f32x4 y[kBlocks][4];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[b][e] = ld_device(outs, at + (b * 4 + e) * 1024);
      const float f = exp2_fast(st.x - base);
      l += st.y * f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[b][e] += y[b][e >> 2][e & 3] * f;
    }
    mx = tm;
    finish();
  }
}

template <int DT>
void chunk_type(const ChunkArgs &a, int D, hipStream_t stream) {
  const ChunkPlan p = chunk_plan(a.T, a.R, a.q_heads, a.c.kv_heads, D, a.max_len);
  ChunkGrid g;
  g.outs_off = (int64_t)p.outs;
  g.stats_off = (int64_t)p.stats;
  g.groups = p.groups;
  g.per = a.q_heads / a.c.kv_heads;
  if (D == 64)
    chunk_kernel<DT, 64><<<p.groups, kThreads, 0, stream>>>(a, g);
  else if (D == 128)
    chunk_kernel<DT, 128><<<p.groups, kThreads, 0, stream>>>(a, g);
  else
    chunk_kernel<DT, 256><<<p.groups, kThreads, 0, stream>>>(a, g);
}

}  // namespace

size_t chunk_workspace_bytes(int64_t T, int64_t R, int64_t q_heads, int64_t kv_heads,
                             int64_t head_dim, int64_t max_len) {
  return chunk_plan(T, R, q_heads, kv_heads, head_dim, max_len).total;
}

hipError_t launch_chunk(const ChunkArgs &a, int dtype, int head_dim, hipStream_t stream) {
  if (dtype == BITNET_KV_BF16)
    chunk_type<BITNET_KV_BF16>(a, head_dim, stream);
  else if (dtype == BITNET_KV_FP16)
    chunk_type<BITNET_KV_FP16>(a, head_dim, stream);
  else
    chunk_type<BITNET_KV_INT8>(a, head_dim, stream);
  return hipGetLastError();
}

}  // namespace bitnet
