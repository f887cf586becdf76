// Attention of one new token per row over the paged key-value cache.
//
//   s_j = scale * q . k_j,   p_j = exp(s_j - max s),   out = sum p_j v_j / sum p_j
//
// The cache is read once and everything else is small, so the kernel is a
// stream of key and value rows.  A workgroup takes one row t, one key/value
// head with up to 16 of its query heads, and a part of the row's length; its
// waves walk 32-token tiles, each with its own running maximum, sum and
// outputs, and join them in LDS at the end.  Parts of a row are joined by the
// workgroup that finishes last.
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
// While a tile's softmax and outputs are worked on, the next one's rows are in
// flight: asked for once the scores are done with the keys' registers and the
// values are in LDS, their pages a tile earlier.  A token that is not there
// (behind the length, or on a page out of range) reads row 0 of page 0
// instead; its score becomes -inf and its value zero, whatever memory holds.
//
// Measured (2 key/value heads of 128 channels, 12 query heads, inputs rotating,
// a launch in a graph): 64 bf16 rows of 1800-32,768 tokens, 1066 MB, 178-203 us
// from one device to the next, 5.3-6.0 TB/s, reads within 0.5% of the cache's
// bytes, waves waiting 26% of their time; one fp16 row of 32,767 tokens 17.2-17.5
// us; 16 int8 rows of 225-1801 tokens 11.4; one row of 257 tokens 9.4-9.6, a chain
// of fetches that a launch (1.8 us) begins.  The same with 64 channels and 4
// key/value heads: 64 rows of 16,384 tokens 192 us in 16 bits, 5.6 TB/s, 112 in 8
// bits, 5.1.
#include <algorithm>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"
#include "terms.hpp"

namespace bitnet {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32;         // tokens of a wave's step
constexpr int kHeads = 16;        // query heads of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Work.  An item is one row, one key/value head and one group of up to 16 of
// its query heads.  Its tiles follow each other, and the items each other, in
// one line, which is cut into equal stretches, a workgroup each, from the
// lengths on the device.
//   - Much work: stretches of total / grid tiles, so that ragged rows keep no
//     workgroup waiting; a stretch may hold the end of one item, several whole
//     ones and the beginning of another.
//   - Little work (up to kShort tiles a stretch): every item starts a stretch
//     of its own, so that none begins inside one and short ones need no join.
// The grid is one round of workgroups, two a compute unit (one with 256
// channels); with many items it is larger, so that small rows can have a
// workgroup each.  (64 bf16 rows of 1800-32768 tokens: 183 us with 512
// stretches, 187 with 1024, 190 with 2048, 195 with each item in 16 equal
// parts.)
constexpr int kGrid = 512, kGridMany = 2048;
constexpr int kFill = 256;         // stretches wanted before they grow beyond a tile a wave
constexpr int kShort = 16;
constexpr int kSingle = 3 * kWaves;   // items up to this are not cut: a join costs three tiles' time
constexpr int kLine = 8;           // tiles of a stretch that is shared by items, at least
// Parts that are joined at once: the loads of 16 are in flight together.  (One
// row of 32,767 fp16 tokens: 17.3 us; 21.5 with its 86 parts in one join, of
// which the join took 8, and longer stretches to keep the parts few.)
constexpr int kJoined = 16;
constexpr int kMaxParts = kJoined * kJoined;   // stretches that one item may lie in
constexpr int kLineRows = 1024;    // rows whose lengths a workgroup sums up itself
// A grid's first axis holds fewer than 2^32 threads: a workgroup per item takes
// as many rows of workgroups as it needs.
constexpr int64_t kGridAxis = (int64_t)1 << 23;
constexpr int kHeaderBytes = 16384;
static_assert(8 * kGridMany <= kHeaderBytes, "two counters per stretch");

// A call's grid and workspace: with `line`, `groups` stretches, each of which
// has room for the outputs [kHeads][D] and (max, sum) [kHeads] of two items it
// holds in part; else a workgroup per item and nothing in parts.
struct AttendPlan {
  bool line;
  int64_t groups;
  size_t stats, total;   // workspace offsets: outputs from kHeaderBytes, then (max, sum)
};

AttendPlan attend_plan(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_len) {
  const int64_t per = q_heads / kv_heads;
  const int64_t items = T * kv_heads * ((per + kHeads - 1) / kHeads);
  const int64_t tiles = (max_len + kTile - 1) / kTile;
  AttendPlan p;
  p.line = T <= kLineRows && items * tiles < ((int64_t)1 << 30);
  p.groups = items;
  p.stats = p.total = kHeaderBytes;
  if (p.line) {
    const int64_t grid = 2 * items > kGrid ? kGridMany : D == 256 ? kGrid / 2 : kGrid;
    p.groups = std::min<int64_t>(grid, items * (tiles / kWaves + 2));
    const size_t slots = 2 * (size_t)p.groups * kHeads;
    p.stats = kHeaderBytes + slots * D * 4;
    p.total = p.stats + slots * 8;
  }
  return p;
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
    terms_bf16(x, u);
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
    terms_f16(x, u);
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

// Inclusive sum over the wave (rows of 16, then the rows' last lanes onward).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return v;
}
// x plus x of the column eight further (row_ror:8).
__device__ __forceinline__ float fold8(float x) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xF, 0xF, false);
  return x + __builtin_bit_cast(float, o);
}

template <int DT, int D, bool FOLD>
struct Shape {
  static constexpr int kBytes = Frag<DT>::kBytes;
  static constexpr int kCols = FOLD ? 8 : kHeads;          // query heads of a product
  static constexpr int kPieces = D * kBytes / 64;          // 16-byte pieces per lane and token
  static constexpr int kRow = D * kBytes + 16;             // value row in LDS
  static constexpr int kWaveLds = kTile * kRow > kCols * D * 4 ? kTile * kRow : kCols * D * 4;
};

template <int DT, int D, bool FOLD, bool FEW>
struct AttendShared {
  typedef Shape<DT, D, FOLD> S;
  __attribute__((aligned(16))) uint8_t tile[kWaves][S::kWaveLds];   // values, then outputs
  float scales[kWaves][2][kTile];      // 8-bit caches: the tile's key and value scales
  float m[kWaves][kHeads], l[kWaves][kHeads], unit[kWaves];
  float weight[S::kCols][kJoined];   // of the joined parts
  int32_t start[FEW ? 1 : kLineRows + 1];   // tiles before each row
  int32_t wave_sum[kWaves], wave_max[kWaves];
  uint32_t last;
};

// An item's tiles [first, end) in a stretch.
struct Segment {
  int t, len, table_row;   // row, its tokens, its row of the table
  int in_row;              // which of the row's items
  int first, end, tiles;
  int item0, next;         // places in the line: of the item, behind the segment
};

// What the host works out once: query heads per key/value head, groups of
// heads, items per row.
struct AttendGrid {
  int64_t stats_off;
  int32_t line, per, groups, row_items;
  int32_t grid;   // workgroups of the first axis
};

// FEW: up to 64 rows, whose lengths every wave holds a lane each.  (A kernel of
// its own, because a small call's time is a chain of first fetches, of
// instructions too: branches around the other cases' code cost it 1-2 us.)
template <int DT, int D, bool FOLD, bool FEW>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
attend_kernel(AttendArgs a, AttendGrid g0) {
  typedef Frag<DT> F;
  typedef typename F::V V;
  typedef Shape<DT, D, FOLD> S;
  constexpr bool kI8 = DT == BITNET_KV_INT8;
  constexpr int kSteps = D / 32;       // contraction steps of the scores
  constexpr int kBlocks = D / 16;      // channel blocks of the outputs
  constexpr int kProducts = F::products(FOLD);
  constexpr float kUp = F::kHalf ? 14.0f : 0.0f;   // probabilities are scaled by 2^kUp
  __shared__ AttendShared<DT, D, FOLD, FEW> sh;

  const int lane = threadIdx.x & 63, c = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool second = FOLD && c >= 8;
  const int col = FOLD ? c & 7 : c;    // this lane's head
  // The arguments take several cache lines: asked for together here, not one
  // after the other where they are used.
  asm volatile("" ::"s"(a.q), "s"(a.tables), "s"(a.c.k), "s"(a.c.v), "s"(a.c.page_stride),
               "s"(a.c.pages), "s"(a.out), "s"(a.ws), "s"(a.scale), "s"(a.lens), "s"(a.rows),
               "s"(g0.grid), "s"(g0.line), "s"(a.lse));
  const bool line = FEW || g0.line != 0;
  const int per = g0.per, row_items = g0.row_items;
  const int groups = FOLD ? 1 : g0.groups;

  auto table_row = [&](int t) { return a.rows ? a.rows[t] : t; };
  auto length = [&](int t, int r) {
    return r >= 0 && r < a.table_rows ? min(max(a.lens[t], 0), a.max_len) : 0;
  };
  auto tiles_of = [](int n) { return (n + kTile - 1) / kTile; };

  // This workgroup's stretch [pos, stop) of the line.
  int my_row = 0, my_len = 0, my_start = 0;
  const uint32_t item = blockIdx.y * (uint32_t)g0.grid + blockIdx.x;   // without a line
  int pos = 0, stop = item < (uint32_t)(a.T * row_items) ? 1 : 0, stretch = 1;
  bool apart = false;                  // every item starts a stretch
  // (Exact: the quotients are below 2^13, so half a unit outweighs the error of
  // the reciprocal.)
  auto padded = [&](int tiles) {
    if (!apart) return tiles;
    return (int)(((float)(tiles + stretch - 1) + 0.5f) * __builtin_amdgcn_rcpf((float)stretch)) *
           stretch;
  };
  if (line) {
    const int each = (a.T + kThreads - 1) / kThreads;
    const int t0 = threadIdx.x * each, t1 = min(t0 + each, a.T);
    int raw, most;
    if constexpr (FEW) {
      if (lane < a.T) {
        my_row = table_row(lane);
        my_len = length(lane, my_row);
      }
      raw = __builtin_amdgcn_readlane(wave_scan(tiles_of(my_len)), 63);
      most = tiles_of((int)across16<true>(across4((float)my_len)));
    } else {
      int sum = 0, top = 0;
      for (int t = t0; t < t1; ++t) {
        const int n = tiles_of(length(t, table_row(t)));
        sum += n;
        top = max(top, n);
      }
      sum = wave_scan(sum);
      top = (int)across16<true>(across4((float)top));
      if (lane == 63) {
        sh.wave_sum[wave] = sum;
        sh.wave_max[wave] = top;
      }
      __syncthreads();
      raw = most = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        raw += sh.wave_sum[w];
        most = max(most, sh.wave_max[w]);
      }
      __syncthreads();
    }
    // (A length's rounding to fp32 is far below the slack of kMaxParts.)
    raw = __builtin_amdgcn_readfirstlane(raw) * row_items;
    most = __builtin_amdgcn_readfirstlane(most);
    const int grid = g0.grid;
    const int least = most / (kMaxParts - 2) + 1;
    auto whole_rounds = [](int n) { return (n + kWaves - 1) & ~(kWaves - 1); };
    stretch = whole_rounds(max(max((raw + kFill - 1) / kFill, most <= kSingle ? kSingle : 1), least));
    apart = stretch <= kShort && a.T * row_items * stretch + raw <= grid * stretch;
    if (!apart)
      stretch = whole_rounds(max(max((int)(((uint32_t)raw + grid - 1) / (uint32_t)grid), kLine),
                                 least));
    int total;
    if constexpr (FEW) {
      const int n = padded(tiles_of(my_len)), upto = wave_scan(n);
      my_start = upto - n;
      total = __builtin_amdgcn_readlane(upto, 63);
    } else {
      int sum = 0;
      for (int t = t0; t < t1; ++t) sum += padded(tiles_of(length(t, table_row(t))));
      const int upto = wave_scan(sum);
      if (lane == 63) sh.wave_sum[wave] = upto;
      __syncthreads();
      int before = upto - sum;
      total = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        before += w < wave ? sh.wave_sum[w] : 0;
        total += sh.wave_sum[w];
      }
      for (int t = t0; t < t1; ++t) {
        sh.start[t] = before;
        before += padded(tiles_of(length(t, table_row(t))));
      }
      if (threadIdx.x == 0) sh.start[a.T] = total;
      __syncthreads();
    }
    total = __builtin_amdgcn_readfirstlane(total) * row_items;
    pos = (int)min((int64_t)blockIdx.x * stretch, (int64_t)total);
    stop = min(pos + stretch, total);
    // Rows without tokens lie in no stretch.
    for (int t = blockIdx.x; t < a.T; t += grid) {
      if (FEW ? __builtin_amdgcn_readlane(my_len, t) != 0 : sh.start[t] != sh.start[t + 1])
        continue;
      for (int i = threadIdx.x; i < a.q_heads * (D / 4); i += kThreads)
        st_global<f32x4>(a.out + (int64_t)t * a.q_heads * D + 4 * i, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      if (a.lse)
        for (int i = threadIdx.x; i < a.q_heads; i += kThreads)
          a.lse[(int64_t)t * a.q_heads + i] = -INFINITY;
    }
  }
  const int begin = pos;

  auto locate = [&]() {
    Segment g;
    if (!line) {   // a workgroup per item
      g.t = item / (uint32_t)row_items;
      g.in_row = item - (uint32_t)(g.t * row_items);
      g.table_row = table_row(g.t);
      g.len = length(g.t, g.table_row);
      g.tiles = g.end = tiles_of(g.len);
      g.first = g.item0 = 0;
      g.next = stop;
      return g;
    }
    int row0;   // the last row that starts at or before pos
    if constexpr (FEW) {
      g.t = __builtin_popcountll(__ballot(lane < a.T && my_start * row_items <= pos)) - 1;
      g.len = __builtin_amdgcn_readlane(my_len, g.t);
      g.table_row = __builtin_amdgcn_readlane(my_row, g.t);
      row0 = __builtin_amdgcn_readlane(my_start, g.t) * row_items;
    } else {
      int lo = 0, hi = a.T - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sh.start[mid] * row_items <= pos) lo = mid; else hi = mid - 1;
      }
      g.t = __builtin_amdgcn_readfirstlane(lo);
      g.table_row = table_row(g.t);
      g.len = length(g.t, g.table_row);
      row0 = __builtin_amdgcn_readfirstlane(sh.start[g.t]) * row_items;
    }
    g.tiles = tiles_of(g.len);
    const int space = padded(g.tiles);
    g.in_row = row_items <= 64 ? __builtin_popcountll(
                                     __ballot(lane < row_items && lane * space <= pos - row0)) - 1
                               : (int)((uint32_t)(pos - row0) / (uint32_t)space);
    g.item0 = row0 + g.in_row * space;
    g.first = pos - g.item0;
    g.end = min(g.tiles, stop - g.item0);
    g.next = min(g.item0 + space, stop);
    return g;
  };

  while (pos < stop) {
    const Segment g = locate();
    const int kvh = FOLD ? g.in_row : g.in_row / groups;
    const int head0 = kvh * per + (g.in_row - kvh * groups) * kHeads;   // first query head
    const int nh = min(kHeads, per - (g.in_row - kvh * groups) * kHeads);
    const bool whole = g.first == 0 && g.end == g.tiles;

    // Rows of the cache.
    const int64_t head_off = (int64_t)kvh * a.c.head_stride * S::kBytes + 16 * h;
    const uint8_t *kbase = reinterpret_cast<const uint8_t *>(a.c.k) + head_off;
    const uint8_t *vbase = reinterpret_cast<const uint8_t *>(a.c.v) + head_off;
    const int32_t *table = a.tables + (int64_t)max(min(g.table_row, a.table_rows - 1), 0) * a.max_pages;
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
        const int j = min(tile * kTile + c + 16 * i, g.len - 1);
        pg[i] = ld_global<int>(table + (j >> a.c.page_shift));
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto place = [&](int tile) {   // from pg: row offsets and mask of this tile
      uint32_t m[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = tile * kTile + c + 16 * i;
        const bool ok = j < g.len && (uint32_t)pg[i] < (uint32_t)a.c.pages;
        const uint32_t page = ok ? pg[i] : 0, tok = ok ? j & tok_mask : 0;
        off[i] = (uint64_t)page * page_bytes + (uint64_t)tok * tok_bytes;
        if constexpr (kI8) {
          const uint32_t at = ((page * (uint32_t)a.c.kv_heads + kvh) << a.c.page_shift) + tok;
          // (Looked at only with the rows: a select here waits for them, 10% of the time.)
          ksc[i] = ld_global<float>(a.c.k_scale + at);
          vsc[i] = ld_global<float>(a.c.v_scale + at);
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

    int tile = g.first + wave;
    if (tile < g.end) load_pages(tile);
    // The queries: asked for early, used once the first rows are on their way.
    f32x4 qx[kSteps][2];
    {
      const float *src = a.q + g.t * a.q_stride + (int64_t)(head0 + min(col, nh - 1)) * D;
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        const int d = kI8 ? (f >> 1) * 64 + 16 * h + (f & 1) * 8 : f * 32 + 8 * h;
        qx[f][0] = ld_global<f32x4>(src + d);
        qx[f][1] = ld_global<f32x4>(src + d + 4);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (tile < g.end) {
      place(tile);
      load_rows(kbase, kr);
      load_rows(vbase, vr);
      load_pages(tile + kWaves);
    }

    // The stretches that hold the item: `used` of them from w0 on.
    int w0 = 0, used = 1;
    if (!whole) {
      w0 = (uint32_t)g.item0 / (uint32_t)stretch;
      used = (uint32_t)(g.item0 + g.tiles - 1) / (uint32_t)stretch - w0 + 1;
    }

    // Queries as terms.
    V q[kSteps][kProducts];
    float unscale = 1.0f;   // of the scores
    {
      float big = 0.0f;
#pragma unroll
      for (int f = 0; f < kSteps; ++f)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          qx[f][e >> 2][e & 3] *= a.scale * kLog2e;
          big = fmaxf(big, fabsf(qx[f][e >> 2][e & 3]));
        }
      float up = 1.0f;
      if constexpr (F::kHalf) {
        const float p2 = pow2_above(across4(big));
        unscale = p2 * 0x1p-14f;
        up = pow2_inverse(p2) * 0x1p14f;
      }
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = qx[f][e >> 2][e & 3] * up;
        F::template split<FOLD>(x, second, q[f]);
      }
    }

    float m = -INFINITY, l = 0.0f;   // m in units of 1 / unscale
    f32x4 o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) o[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float vmax = pow2_above(0.0f);   // 8-bit caches: o is in units of this
    uint8_t *rows = sh.tile[wave];

    for (; tile < g.end; tile += kWaves) {
      const uint32_t mask = mask_next;
      const bool all = mask == 0xffffffffu;
      // Scales, from a lane per token to the scores' layout; the values' relative
      // to the power of two above the largest so far.
      float ks[8], vs[8], vkeep = 1.0f;
      if constexpr (kI8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool ok = (mask >> (c + 16 * i)) & 1;
          ksc[i] = ok ? ksc[i] : 0.0f;
          vsc[i] = ok ? vsc[i] : 0.0f;
        }
        const float v_new = fmaxf(vmax, pow2_above(across16<true>(fmaxf(vsc[0], vsc[1]))));
        const float inv = pow2_inverse(v_new);
        vkeep = vmax * inv;
        vmax = v_new;
        if (h == 0) {
          sh.scales[wave][0][c] = ksc[0];
          sh.scales[wave][0][c + 16] = ksc[1];
          sh.scales[wave][1][c] = vsc[0] * inv;
          sh.scales[wave][1][c + 16] = vsc[1] * inv;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 ks4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][0][16 * i + 4 * h]);
          const f32x4 vs4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][1][16 * i + 4 * h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ks[4 * i + e] = ks4[e];
            vs[4 * i + e] = vs4[e];
          }
        }
      }
      // Scores of tokens 16 i + 4 h + e for this column.
      f32x4 s[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        V k[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (kI8)
            k[i] = f & 1 ? codes_f16(kr[i][f >> 1].z, kr[i][f >> 1].w)
                         : codes_f16(kr[i][f >> 1].x, kr[i][f >> 1].y);
          else
            k[i] = __builtin_bit_cast(V, kr[i][f]);
        }
#pragma unroll
        for (int p = kProducts - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < 2; ++i) s[i] = F::mfma(k[i], q[f][p], s[i]);
      }
      settle<D>(s);
      // Values into LDS, as rows.
      if (!all)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (!((mask >> (c + 16 * i)) & 1))
#pragma unroll
            for (int pc = 0; pc < S::kPieces; ++pc) vr[i][pc] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int pc = 0; pc < S::kPieces; ++pc)
          *reinterpret_cast<u32x4 *>(rows + (c + 16 * i) * S::kRow + 64 * pc + 16 * h) = vr[i][pc];
      // The next tile.
      __builtin_amdgcn_sched_barrier(0);
      if (tile + kWaves < g.end) {
        place(tile + kWaves);
        load_rows(kbase, kr);
        load_rows(vbase, vr);
        load_pages(tile + 2 * kWaves);
      }

      float x[8];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = s[i][e];
          if constexpr (FOLD) y = fold8(y);
          if constexpr (kI8) y *= ks[4 * i + e];
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
      const float lkeep = exp2_fast((m - base) * unscale);
      const float keep = lkeep * vkeep;
      m = m_new;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = exp2_fast(__builtin_fmaf(x[e] - base, unscale, kUp));
        sum += x[e];
      }
      l = l * lkeep + sum;   // not in units of vmax
      if constexpr (kI8)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= vs[e];
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
      settle<D>(o);
      __builtin_amdgcn_wave_barrier();
    }
    m *= unscale;
    if constexpr (FOLD)
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][e] = fold8(o[b][e]);

    // Join the waves: outputs 16 b + 4 h + e of head c, each wave's relative to
    // its own maximum (folded: columns 8-15 repeat heads 0-7 and are left out).
    l = sum4(l);
    if (h == 0) {
      sh.m[wave][c] = m;
      sh.l[wave][c] = l;
    }
    if (lane == 0) sh.unit[wave] = vmax;
    constexpr int kQuads = D / 4;        // of a head
    f32x4 *mine = reinterpret_cast<f32x4 *>(sh.tile[wave]);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      if (!second) mine[c * kQuads + 4 * b + h] = o[b];
    __syncthreads();
    const int n4 = nh * kQuads;
    // This stretch's two places in the workspace: for the item at its beginning
    // and for one that begins inside it and goes on behind it.
    constexpr uint32_t kPartBytes = kHeads * D * 4;
    const int my_place = 2 * blockIdx.x + (pos == begin ? 0 : 1);
    const __amdgpu_buffer_rsrc_t outs =
        make_rsrc(a.ws + kHeaderBytes, line ? 2 * g0.grid * kPartBytes : 0);
    f32x2 *stats = reinterpret_cast<f32x2 *>(a.ws + g0.stats_off);
    f32x4 *out = reinterpret_cast<f32x4 *>(a.out + ((int64_t)g.t * a.q_heads + head0) * D);
    auto finish = [&](int i, int head, f32x4 sum, float tm, float tl) {
      st_global<f32x4>(out + i, tl > 0.0f ? sum / tl : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      if (a.lse && i % kQuads == 0)
        a.lse[(int64_t)g.t * a.q_heads + head0 + head] =
            tl > 0.0f ? (tm - kUp + __log2f(tl)) * kLn2 : -INFINITY;
    };
    auto keep_part = [&](int place, int i, int head, f32x4 sum, float tm, float tl) {
      st_device(outs, place * kPartBytes + 16 * i, sum);
      if (i % kQuads == 0)
        __hip_atomic_store((BITNET_GLOBAL uint64_t *)&stats[place * kHeads + head],
                           __builtin_bit_cast(uint64_t, f32x2{tm, tl}), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
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
      if (whole) {
        finish(i, head, sum, tm, tl);
      } else {
        keep_part(my_place, i, head, sum, tm, tl);
      }
    }

    if (!whole) {
      // The last stretch of the item to arrive joins its parts; with more than
      // kJoined of them, the last of each group of kJoined joins the group into
      // its first part's place, and the last of the groups joins those.  Each
      // leaves its counter at zero: the group's first stretch's (of a group of
      // two or more, so that no other item begins there), and for the groups the
      // item's first stretch's among the second counters.  Each wave's stores have
      // been acknowledged before a counter moves.
      const int inside = g.item0 != w0 * stretch ? 1 : 0;   // begins inside its first stretch
      auto place_of = [&](int p) { return 2 * (w0 + p) + (p == 0 ? inside : 0); };
      uint32_t *counters = reinterpret_cast<uint32_t *>(a.ws) + w0;
      bool final = used <= kJoined;
      int first = final ? 0 : ((int)blockIdx.x - w0) & -kJoined;
      int step = 1, parts = min(kJoined, used - first);
      uint32_t *ticket = counters + first;
      for (;;) {
        if (parts > 1) {
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          __syncthreads();
          if (threadIdx.x == 0) {
            const uint32_t n =
                __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            sh.last = n == (uint32_t)parts - 1;
            if (sh.last)
              __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          }
          __syncthreads();
          if (!sh.last) break;
          // Wave w adds up parts w, w + kWaves, ..., a lane per four channels in
          // each of kWide blocks of the outputs; the loads of kJoin parts go out
          // at once, the first ones before the weights are known.
          constexpr int kWide = S::kCols * kQuads / 64;
          constexpr int kJoin = kWide >= 8 ? 2 : 16 / kWide;
          f32x4 x[kJoin][kWide], sum[kWide];
          auto load_parts = [&](int p0) {
#pragma unroll
            for (int u = 0; u < kJoin; ++u)
#pragma unroll
              for (int b = 0; b < kWide; ++b)
                x[u][b] = ld_device(
                    outs, place_of(first + step * min(p0 + u * kWaves, parts - 1)) * kPartBytes +
                              16 * min(64 * b + lane, n4 - 1));
          };
          load_parts(wave);
          // The parts' maxima and sums become weights: four heads a wave, a lane
          // per part.
          {
            const int head = 4 * wave + h;
            f32x2 st = {-INFINITY, 0.0f};
            if (c < parts && head < nh)
              st = __builtin_bit_cast(
                  f32x2, (uint64_t)__hip_atomic_load(
                             (const BITNET_GLOBAL uint64_t *)&stats[place_of(first + step * c) *
                                                                        kHeads + head],
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
            const float tm = across16<true>(st.x);
            const float f = exp2_fast(st.x - (tm == -INFINITY ? 0.0f : tm));
            const float tl = across16<false>(st.y * f);
            if (head < nh) {
              sh.weight[head][c] = f;
              if (c == 0) {
                sh.m[0][head] = tm;
                sh.l[0][head] = tl;
              }
            }
          }
          __syncthreads();
#pragma unroll
          for (int b = 0; b < kWide; ++b) sum[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          for (int p0 = wave; p0 < parts; p0 += kJoin * kWaves) {
            if (p0 != wave) load_parts(p0);
#pragma unroll
            for (int u = 0; u < kJoin; ++u)
              if (p0 + u * kWaves < parts)
#pragma unroll
                for (int b = 0; b < kWide; ++b)
                  sum[b] += x[u][b] *
                            sh.weight[min(64 * b + lane, n4 - 1) / kQuads][p0 + u * kWaves];
          }
#pragma unroll
          for (int b = 0; b < kWide; ++b)
            if (64 * b + lane < n4) mine[64 * b + lane] = sum[b];
          __syncthreads();
          for (int i = threadIdx.x; i < n4; i += kThreads) {
            const int head = i / kQuads;
            f32x4 all = reinterpret_cast<const f32x4 *>(sh.tile[0])[i];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) all += reinterpret_cast<const f32x4 *>(sh.tile[w])[i];
            if (final)
              finish(i, head, all, sh.m[0][head], sh.l[0][head]);
            else
              keep_part(place_of(first), i, head, all, sh.m[0][head], sh.l[0][head]);
          }
        }
        if (final) break;
        final = true;
        parts = (used + kJoined - 1) / kJoined;
        step = kJoined;
        first = 0;
        ticket = counters + kGridMany;
      }
    }
    pos = g.next;
    if (pos < stop) __syncthreads();   // the next segment writes where this one reads
  }
}

template <int DT, int D, bool FOLD>
void attend_rows(const AttendArgs &a, const AttendGrid &g, const dim3 &grid, hipStream_t stream) {
  if (a.T <= 64 && g.line)
    attend_kernel<DT, D, FOLD, true><<<grid, kThreads, 0, stream>>>(a, g);
  else
    attend_kernel<DT, D, FOLD, false><<<grid, kThreads, 0, stream>>>(a, g);
}

template <int DT, bool FOLD>
void attend_dim(const AttendArgs &a, int D, hipStream_t stream) {
  const AttendPlan p = attend_plan(a.T, a.q_heads, a.c.kv_heads, D, a.max_len);
  AttendGrid g;
  g.stats_off = (int64_t)p.stats;
  g.line = p.line;
  g.per = a.q_heads / a.c.kv_heads;
  g.groups = (g.per + kHeads - 1) / kHeads;
  g.row_items = a.c.kv_heads * g.groups;
  const int64_t axes = (p.groups + kGridAxis - 1) / kGridAxis;
  g.grid = (int32_t)((p.groups + axes - 1) / axes);
  const dim3 grid((unsigned)g.grid, (unsigned)axes);
  if (D == 64)
    attend_rows<DT, 64, FOLD>(a, g, grid, stream);
  else if (D == 128)
    attend_rows<DT, 128, FOLD>(a, g, grid, stream);
  else
    attend_rows<DT, 256, FOLD>(a, g, grid, stream);
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
  return attend_plan(T, q_heads, kv_heads, head_dim, max_len).total;
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
