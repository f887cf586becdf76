// Attention of one new token per row over the paged key-value cache.
//
//   s_j = scale * q . k_j,   p_j = exp(s_j - max s),   out = sum p_j v_j / sum p_j
//
// The cache is read once and everything else is small, so the kernel is a
// stream of key and value rows.  A workgroup takes one row t, one key/value
// head with up to 16 of its query heads, and a part of the row's length; its
// waves walk 32-token tiles, each with its own running maximum, sum and
// outputs, and join them in LDS at the end.  Parts of a long row are joined by
// the workgroup that finishes last.
//
// Tile.  Lane L = c + 16h loads, for tokens c and c + 16, the 16-byte pieces
// h, h + 4, ... of the key row and of the value row: keys and values lie at
// equal offsets, so a tile costs two addresses per lane.  The keys are, as
// loaded, the token operand of v_mfma_f32_16x16x32 (row c, eight channels);
// with the queries as the other operand the scores arrive transposed, lane
// (c, h) holding head c and tokens 4h..4h+3 (+ 16).  That is the layout in
// which the second product takes its probabilities, once its 32 contraction
// steps are numbered to match: steps 8h..8h+3 are tokens 4h.. and steps
// 8h+4.. tokens 16+4h...  The values need the same order with channels in
// rows: they go through LDS and come back by the transposing reads, four
// tokens of one channel per lane.  Nothing else crosses lanes but the tile's
// maximum (two exchanges).
//
// Precision.  The matrix cores multiply 16-bit terms, exactly, into fp32 sums,
// so queries and probabilities enter as sums of terms: three of bf16 (8 bits
// each) against bf16 values, two of fp16 (11 bits each) against fp16 values
// and against 8-bit codes, which are exact in fp16.  fp16's range is made to
// do by powers of two: queries by their head's largest channel, probabilities
// by 2^14, and with 8-bit values by the largest value scale so far.
//
// While a tile is worked on, the next one's rows are in flight: its keys are
// asked for once the scores are done with the registers, its values once
// they are in LDS, its pages a tile earlier.  All loads are unconditional, so
// that the waits count exactly: a token that is not there (behind the length,
// or on a page out of range) reads row 0 of page 0 instead; its score becomes
// -inf and its value zero, whatever memory holds.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"

namespace bitnet {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

#define BITNET_LDS __attribute__((address_space(3)))

#ifndef BITNET_ATTEND_WAVES
#define BITNET_ATTEND_WAVES 4
#endif
constexpr int kWaves = BITNET_ATTEND_WAVES;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32;         // tokens of a wave's step
constexpr int kHeads = 16;        // query heads of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Tickets of the parts' joins: one counter per (row, head) pair that is split.
constexpr int kTickets = 4096;
constexpr int kHeaderBytes = 4 * kTickets;

// How a call is cut: items = rows x key/value heads x groups of 16 query
// heads, each in up to `parts` parts of at least kMinTiles tiles.
#ifndef BITNET_ATTEND_MIN_TILES
#define BITNET_ATTEND_MIN_TILES 16
#endif
#ifndef BITNET_ATTEND_GROUPS
#define BITNET_ATTEND_GROUPS 2048
#endif
constexpr int kMinTiles = BITNET_ATTEND_MIN_TILES;
constexpr int kTargetGroups = BITNET_ATTEND_GROUPS;
constexpr int kMaxParts = 64;

// Partial results cross the chip through device-coherent accesses (cache
// policy sc1), so that no workgroup has to write back or invalidate a cache,
// as a fence of device scope does.
constexpr int kDeviceAux = 16;
__device__ __forceinline__ void st_device(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, off, 0, kDeviceAux);
}
__device__ __forceinline__ f32x4 ld_device(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
  return __builtin_bit_cast(f32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, kDeviceAux));
}

struct AttendSplit {
  int64_t items;
  int parts;
  size_t stats, total;   // workspace offsets: partial outputs at kHeaderBytes, then (max, sum)
};

AttendSplit attend_split(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_len) {
  const int64_t per = q_heads / kv_heads;
  AttendSplit s;
  s.items = T * kv_heads * ((per + kHeads - 1) / kHeads);
  const int64_t tiles = (max_len + kTile - 1) / kTile;
  int64_t parts = 1;
  if (s.items <= kTickets)
    parts = std::min<int64_t>((kTargetGroups + s.items - 1) / s.items,
                              (tiles + kMinTiles - 1) / kMinTiles);
  s.parts = (int)std::max<int64_t>(1, std::min<int64_t>(parts, kMaxParts));
  const int64_t n = s.parts > 1 ? s.items * s.parts * kHeads : 0;
  s.stats = kHeaderBytes + (size_t)n * D * 4;
  s.total = s.stats + (size_t)n * 8;
  return s;
}

// The operands of a type: products of 16 x 32 by 32 x 16, and fp32 values as
// terms.  Folded (up to 8 heads), the 16 columns of an operand hold two terms
// of 8 heads, the first in columns 0-7 and the second in columns 8-15: two
// terms take one product, three take two.
template <int DT> struct Frag;
template <> struct Frag<BITNET_KV_BF16> {
  typedef bf16x8 V;
  static constexpr int kBytes = 2;
  static constexpr bool kHalf = false;
  static constexpr int products(bool fold) { return fold ? 2 : 3; }
  static __device__ __forceinline__ f32x4 mfma(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  template <bool FOLD>
  static __device__ __forceinline__ void split(const float (&x)[8], bool second,
                                               V (&t)[FOLD ? 2 : 3]) {
    bf16x8 u[3];
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
    if constexpr (FOLD) {
      t[0] = second ? u[1] : u[0];
      t[1] = second ? bf16x8{} : u[2];
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i] = u[i];
    }
  }
};
struct FragF16 {
  typedef f16x8 V;
  static constexpr bool kHalf = true;
  static constexpr int products(bool fold) { return fold ? 1 : 2; }
  static __device__ __forceinline__ f32x4 mfma(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  template <bool FOLD>
  static __device__ __forceinline__ void split(const float (&x)[8], bool second,
                                               V (&t)[FOLD ? 1 : 2]) {
    f16x8 u[2];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u[0][e] = (_Float16)x[e];
      u[1][e] = (_Float16)(x[e] - (float)u[0][e]);
    }
    if constexpr (FOLD) {
      t[0] = second ? u[1] : u[0];
    } else {
      t[0] = u[0];
      t[1] = u[1];
    }
  }
};
template <> struct Frag<BITNET_KV_FP16> : FragF16 { static constexpr int kBytes = 2; };
template <> struct Frag<BITNET_KV_INT8> : FragF16 { static constexpr int kBytes = 1; };

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

// The lanes of one column are 16 apart.  The exchanges put rows 0, 2 (halves
// 0) beside rows 1, 3 (halves 1), without leaving the registers.
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
// x plus x of the column eight further (row_ror:8).
__device__ __forceinline__ float fold8(float x) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xF, 0xF, false);
  return x + __builtin_bit_cast(float, o);
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

template <int DT, int D>
struct Shape {
  static constexpr int kBytes = Frag<DT>::kBytes;
  static constexpr int kPieces = D * kBytes / 64;          // 16-byte pieces per lane and token
  static constexpr int kRow = D * kBytes + 16;             // value row in LDS
  static constexpr int kWaveLds = kTile * kRow > kHeads * D * 4 ? kTile * kRow : kHeads * D * 4;
};

template <int DT, int D>
struct AttendShared {
  __attribute__((aligned(16))) uint8_t tile[kWaves][Shape<DT, D>::kWaveLds];
  float scales[kWaves][2][kTile];      // 8-bit caches: the tile's key and value scales
  float m[kWaves][kHeads], l[kWaves][kHeads], unit[kWaves];
  float weight[kHeads][kMaxParts];     // of the joined parts
  uint32_t last;
};

template <int DT, int D, bool FOLD>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
attend_kernel(AttendArgs a, int parts, int64_t stats_off) {
  typedef Frag<DT> F;
  typedef typename F::V V;
  typedef Shape<DT, D> S;
  constexpr bool kI8 = DT == BITNET_KV_INT8;
  constexpr int kSteps = D / 32;       // contraction steps of the scores
  constexpr int kBlocks = D / 16;      // channel blocks of the outputs
  constexpr int kProducts = F::products(FOLD);
  constexpr float kUp = F::kHalf ? 14.0f : 0.0f;   // probabilities are scaled by 2^kUp
  __shared__ AttendShared<DT, D> sh;

  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool second = FOLD && c >= 8;
  const int col = FOLD ? c & 7 : c;    // this lane's head
  const int per = a.q_heads / a.c.kv_heads;
  const int groups = (per + kHeads - 1) / kHeads;
  const int part = parts > 1 ? blockIdx.x : 0;
  const int item = parts > 1 ? blockIdx.y : blockIdx.x;
  const int t = item / (a.c.kv_heads * groups);
  const int kvh = item / groups % a.c.kv_heads;
  const int head0 = kvh * per + item % groups * kHeads;   // first query head
  const int nh = min(kHeads, per - item % groups * kHeads);

  // The queries: asked for first, used once the first rows are on their way.
  f32x4 qx[kSteps][2];
  {
    const float *src = a.q + t * a.q_stride + (int64_t)(head0 + min(col, nh - 1)) * D;
#pragma unroll
    for (int f = 0; f < kSteps; ++f) {
      const int d = kI8 ? (f >> 1) * 64 + 16 * h + (f & 1) * 8 : f * 32 + 8 * h;
      qx[f][0] = ld_global<f32x4>(src + d);
      qx[f][1] = ld_global<f32x4>(src + d + 4);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  const int r = a.rows ? a.rows[t] : t;
  const int len = r >= 0 && r < a.table_rows ? min(max(a.lens[t], 0), a.max_len) : 0;
  const int tiles = (len + kTile - 1) / kTile;
  const int share = max((tiles + parts - 1) / parts, kMinTiles);
  const int used = max((tiles + share - 1) / share, 1);   // parts with work
  if (part >= used) return;
  const int first = part * share, end = min(first + share, tiles);

  // Rows of the cache.
  const int64_t head_off = (int64_t)kvh * a.c.head_stride * S::kBytes + 16 * h;
  const uint8_t *kbase = reinterpret_cast<const uint8_t *>(a.c.k) + head_off;
  const uint8_t *vbase = reinterpret_cast<const uint8_t *>(a.c.v) + head_off;
  const int32_t *table = a.tables + (int64_t)max(min(r, a.table_rows - 1), 0) * a.max_pages;
  const uint32_t page_bytes = (uint32_t)(a.c.page_stride * S::kBytes);
  const uint32_t tok_bytes = (uint32_t)(a.c.token_stride * S::kBytes);
  const int tok_mask = (1 << a.c.page_shift) - 1;

  int pg[2];                       // pages of tokens c, c + 16 of the tile after the loaded one
  u32x4 kr[2][S::kPieces], vr[2][S::kPieces];
  float ksc[2], vsc[2];
  uint32_t mask_next;              // tokens of the loaded tile that are there
  uint64_t off[2];

  auto load_pages = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = min(tile * kTile + c + 16 * i, len - 1);
      pg[i] = ld_global<int>(table + (j >> a.c.page_shift));
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto place = [&](int tile) {   // from pg: row offsets and mask of this tile
    uint32_t m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = tile * kTile + c + 16 * i;
      const bool ok = tile < end && j < len && (uint32_t)pg[i] < (uint32_t)a.c.pages;
      const uint32_t page = ok ? pg[i] : 0, tok = ok ? j & tok_mask : 0;
      off[i] = (uint64_t)page * page_bytes + (uint64_t)tok * tok_bytes;
      if constexpr (kI8) {
        const uint32_t at = ((page * (uint32_t)a.c.kv_heads + kvh) << a.c.page_shift) + tok;
        const float ks = ld_global<float>(a.c.k_scale + at), vs = ld_global<float>(a.c.v_scale + at);
        ksc[i] = ok ? ks : 0.0f;
        vsc[i] = ok ? vs : 0.0f;
      }
      m[i] = (uint32_t)__ballot(ok) & 0xffffu;
    }
    mask_next = m[0] | (m[1] << 16);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_rows = [&](const uint8_t *base, u32x4 (&x)[2][S::kPieces]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < S::kPieces; ++p) x[i][p] = ld_global<u32x4>(base + off[i] + 64 * p);
    // Waits count loads in order of issue, so the groups stay in order.
    __builtin_amdgcn_sched_barrier(0);
  };

  float m = -INFINITY, l = 0.0f;
  f32x4 o[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) o[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float vmax = pow2_above(0.0f);   // 8-bit caches: o is in units of this

  int tile = first + wave;
  if (tile < end) {
    load_pages(tile);
    place(tile);
    load_pages(tile + kWaves);
    load_rows(vbase, vr);
    load_rows(kbase, kr);

    // Queries as terms.
    V q[kSteps][kProducts];
    float unscale = 1.0f;
    {
      float x[kSteps][8];
      float big = 0.0f;
#pragma unroll
      for (int f = 0; f < kSteps; ++f)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[f][e] = qx[f][e >> 2][e & 3] * (a.scale * kLog2e);
          big = fmaxf(big, fabsf(x[f][e]));
        }
      float up = 1.0f;
      if constexpr (F::kHalf) {
        const float p2 = pow2_above(across4(big));
        unscale = p2 * 0x1p-14f;
        up = pow2_inverse(p2) * 0x1p14f;
      }
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[f][e] *= up;
        F::template split<FOLD>(x[f], second, q[f]);
      }
    }

    uint8_t *rows = sh.tile[wave];
    for (; tile < end; tile += kWaves) {
      const uint32_t mask = mask_next;
      const bool all = mask == 0xffffffffu;
      // Values into LDS, as rows; scales too.
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool here = all || ((mask >> (c + 16 * i)) & 1);
#pragma unroll
        for (int pc = 0; pc < S::kPieces; ++pc) {
          u32x4 v = vr[i][pc];
          if (!here) v = u32x4{0u, 0u, 0u, 0u};
          *reinterpret_cast<u32x4 *>(rows + (c + 16 * i) * S::kRow + 64 * pc + 16 * h) = v;
        }
      }
      float ks[8], vs[8];
      if constexpr (kI8) {
        if (h == 0) {
          sh.scales[wave][0][c] = ksc[0];
          sh.scales[wave][0][c + 16] = ksc[1];
          sh.scales[wave][1][c] = vsc[0];
          sh.scales[wave][1][c + 16] = vsc[1];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 ks4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][0][16 * i + 4 * h]);
          const f32x4 vs4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][1][16 * i + 4 * h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ks[4 * i + e] = ks4[e] * unscale;
            vs[4 * i + e] = vs4[e];
          }
        }
      }
      // The next tile's values.
      place(tile + kWaves);
      load_pages(tile + 2 * kWaves);
      load_rows(vbase, vr);

      // Scores of tokens 16 i + 4 h + e for this column.
      f32x4 s[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) s[i][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int f = 0; f < kSteps; ++f)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          V k;
          if constexpr (kI8)
            k = f & 1 ? codes_f16(kr[i][f >> 1].z, kr[i][f >> 1].w)
                      : codes_f16(kr[i][f >> 1].x, kr[i][f >> 1].y);
          else
            k = __builtin_bit_cast(V, kr[i][f]);
#pragma unroll
          for (int p = kProducts - 1; p >= 0; --p) s[i][f & 1] = F::mfma(k, q[f][p], s[i][f & 1]);
        }
      // The next tile's keys.
      __builtin_amdgcn_sched_barrier(0);
      load_rows(kbase, kr);

      float x[8];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = s[i][0][e] + s[i][1][e];
          if constexpr (FOLD) y = fold8(y);
          y *= kI8 ? ks[4 * i + e] : unscale;
          x[4 * i + e] = y;
        }
      if (!all)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((mask >> (16 * i + 4 * h + e)) & 1)) x[4 * i + e] = -INFINITY;
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
      const float m_new = fmaxf(m, across4(top));
      const float base = m_new == -INFINITY ? 0.0f : m_new;
      const float lkeep = exp2_fast(m - base);
      float keep = lkeep;
      float inv = 1.0f;
      if constexpr (kI8) {
        float vt = vs[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) vt = fmaxf(vt, vs[e]);
        const float v_new = fmaxf(vmax, pow2_above(across4(vt)));
        inv = pow2_inverse(v_new);
        keep *= vmax * inv;
        vmax = v_new;
      }
      m = m_new;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = exp2_fast(x[e] - (base - kUp));
        sum += x[e];
      }
      l = l * lkeep + sum;   // not in units of vmax
      if constexpr (kI8)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= vs[e] * inv;
      if (__any(keep != 1.0f))
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[b] *= keep;
      V p[kProducts];
      F::template split<FOLD>(x, second, p);

      // Values back from LDS, four tokens of a channel at a time.
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        V v;
        if constexpr (kI8) {
          const int row = 4 * h + (c >> 1 & 3) + 16 * (c >> 3);
          typedef int v2i __attribute__((ext_vector_type(2)));
          const v2i w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (BITNET_LDS v2i *)(rows + row * S::kRow + 16 * b + 8 * (c & 1)));
          v = codes_f16((uint32_t)w.x, (uint32_t)w.y);
        } else {
          const uint8_t *at = rows + (4 * h + (c >> 2)) * S::kRow + 32 * b + 8 * (c & 3);
          s16x4 w[2];
          w[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((BITNET_LDS s16x4 *)at);
          w[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((BITNET_LDS s16x4 *)(at + 16 * S::kRow));
          v = __builtin_bit_cast(V, w);
        }
#pragma unroll
        for (int i = kProducts - 1; i >= 0; --i) o[b] = F::mfma(v, p[i], o[b]);
      }
      __builtin_amdgcn_wave_barrier();
    }
    if constexpr (FOLD)
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][e] = fold8(o[b][e]);
  }

  // Join the waves: outputs 16 b + 4 h + e of head c, each wave's relative to
  // its own maximum (folded: columns 8-15 repeat heads 0-7 and are left out).
  l = sum4(l);
  if (h == 0) {
    sh.m[wave][c] = m;
    sh.l[wave][c] = l;
  }
  if (lane == 0) sh.unit[wave] = vmax;
  f32x4 *mine = reinterpret_cast<f32x4 *>(sh.tile[wave]);
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (!second) mine[c * (D / 4) + 4 * b + h] = o[b];
  __syncthreads();
  constexpr int kQuads = D / 4;        // of a head
  const int n4 = nh * kQuads;
  // Workspace of this item: outputs [parts][kHeads][D], (max, sum) [parts][kHeads].
  const uint32_t part_bytes = kHeads * D * 4;
  const __amdgpu_buffer_rsrc_t outs =
      make_rsrc(a.ws + kHeaderBytes + (int64_t)item * parts * part_bytes, parts * part_bytes);
  f32x2 *stats = reinterpret_cast<f32x2 *>(a.ws + stats_off) + (int64_t)item * parts * kHeads;
  f32x4 *out = reinterpret_cast<f32x4 *>(a.out + ((int64_t)t * a.q_heads + head0) * D);
  auto finish = [&](int i, int head, f32x4 sum, float tm, float tl) {
    st_global<f32x4>(out + i, tl > 0.0f ? sum / tl : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
    if (a.lse && i % kQuads == 0)
      a.lse[(int64_t)t * a.q_heads + head0 + head] =
          tl > 0.0f ? (tm - kUp + __log2f(tl)) * kLn2 : -INFINITY;
  };
  for (int i = threadIdx.x; i < n4; i += kThreads) {
    const int head = i / kQuads;
    float tm = sh.m[0][head];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) tm = fmaxf(tm, sh.m[w][head]);
    const float base = tm == -INFINITY ? 0.0f : tm;
    float tl = 0.0f;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = exp2_fast(sh.m[w][head] - base);
      tl += sh.l[w][head] * f;
      sum += reinterpret_cast<const f32x4 *>(sh.tile[w])[i] * (kI8 ? f * sh.unit[w] : f);
    }
    if (used == 1) {
      finish(i, head, sum, tm, tl);
    } else {
      st_device(outs, part * part_bytes + 16 * i, sum);
      if (i % kQuads == 0)
        __hip_atomic_store((BITNET_GLOBAL uint64_t *)&stats[part * kHeads + head],
                           __builtin_bit_cast(uint64_t, f32x2{tm, tl}), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (used == 1) return;

  // The last part to arrive joins them all; it leaves the counter at zero.
  // Each wave's stores have been acknowledged before the counter moves.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t *ticket = reinterpret_cast<uint32_t *>(a.ws) + item;
    const uint32_t n =
        __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sh.last = n == (uint32_t)used - 1;
    if (sh.last) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!sh.last) return;
  // Wave w adds up parts w, w + kWaves, ..., a lane per four channels in each
  // of kWide stretches of the outputs; the loads of kJoin parts go out at once,
  // the first ones before the weights are known.
  constexpr int kWide = (FOLD ? 8 : kHeads) * kQuads / 64;
  constexpr int kJoin = kWide >= 8 ? 2 : 16 / kWide;
  f32x4 x[kJoin][kWide], sum[kWide];
  auto load_parts = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kJoin; ++u)
#pragma unroll
      for (int b = 0; b < kWide; ++b)
        x[u][b] = ld_device(outs, min(p0 + u * kWaves, used - 1) * part_bytes +
                                      16 * min(64 * b + lane, n4 - 1));
  };
  load_parts(wave);
  // A wave per head turns the parts' maxima and sums into weights.
  for (int head = wave; head < nh; head += kWaves) {
    f32x2 st = {-INFINITY, 0.0f};
    if (lane < used)
      st = __builtin_bit_cast(f32x2, (uint64_t)__hip_atomic_load(
                                         (const BITNET_GLOBAL uint64_t *)&stats[lane * kHeads + head],
                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    const float tm = across16<true>(across4(st.x));
    const float f = exp2_fast(st.x - (tm == -INFINITY ? 0.0f : tm));
    const float tl = across16<false>(sum4(st.y * f));
    if (lane < used) sh.weight[head][lane] = f;
    if (lane == 0) {
      sh.m[0][head] = tm;
      sh.l[0][head] = tl;
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kWide; ++b) sum[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int p0 = wave; p0 < used; p0 += kJoin * kWaves) {
    if (p0 != wave) load_parts(p0);
#pragma unroll
    for (int u = 0; u < kJoin; ++u)
      if (p0 + u * kWaves < used)
#pragma unroll
        for (int b = 0; b < kWide; ++b)
          sum[b] += x[u][b] * sh.weight[min(64 * b + lane, n4 - 1) / kQuads][p0 + u * kWaves];
  }
#pragma unroll
  for (int b = 0; b < kWide; ++b)
    if (64 * b + lane < n4) mine[64 * b + lane] = sum[b];
  __syncthreads();
  for (int i = threadIdx.x; i < n4; i += kThreads) {
    f32x4 sum = reinterpret_cast<const f32x4 *>(sh.tile[0])[i];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += reinterpret_cast<const f32x4 *>(sh.tile[w])[i];
    finish(i, i / kQuads, sum, sh.m[0][i / kQuads], sh.l[0][i / kQuads]);
  }
}

template <int DT, bool FOLD>
void attend_dim(const AttendArgs &a, int D, hipStream_t stream) {
  const AttendSplit s = attend_split(a.T, a.q_heads, a.c.kv_heads, D, a.max_len);
  const dim3 grid = s.parts > 1 ? dim3(s.parts, s.items) : dim3(s.items);
  if (D == 64)
    attend_kernel<DT, 64, FOLD><<<grid, kThreads, 0, stream>>>(a, s.parts, s.stats);
  else if (D == 128)
    attend_kernel<DT, 128, FOLD><<<grid, kThreads, 0, stream>>>(a, s.parts, s.stats);
  else
    attend_kernel<DT, 256, FOLD><<<grid, kThreads, 0, stream>>>(a, s.parts, s.stats);
}

template <int DT>
void attend_type(const AttendArgs &a, int D, hipStream_t stream) {
  if (a.q_heads <= 8 * a.c.kv_heads)
    attend_dim<DT, true>(a, D, stream);
  else
    attend_dim<DT, false>(a, D, stream);
}

}  // namespace

size_t attend_workspace_bytes(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                              int64_t max_len) {
  return attend_split(T, q_heads, kv_heads, head_dim, max_len).total;
}

hipError_t launch_attend(const AttendArgs &a, int dtype, int head_dim, hipStream_t stream) {
  if (dtype == BITNET_KV_BF16)
    attend_type<BITNET_KV_BF16>(a, head_dim, stream);
  else if (dtype == BITNET_KV_FP16)
    attend_type<BITNET_KV_FP16>(a, head_dim, stream);
  else
    attend_type<BITNET_KV_INT8>(a, head_dim, stream);
  return hipGetLastError();
}

}  // namespace bitnet
