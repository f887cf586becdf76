// Attention of the new tokens of several requests over the paged key-value
// cache: prompts, pieces of prompts, guessed tokens.
//
//   token i of the n new ones of a request of len tokens sees L = len - n + i + 1:
//   s_j = scale * q . k_j,   p_j = exp(s_j - max s),   out = sum_j<L p_j v_j / sum p_j
//
// A key/value row serves all new tokens of its request and all query heads of
// its group, so the rows of the product are (token, head) pairs, 128 of them to
// an item, 32 to a wave.  The work is bound by the matrix cores where it is long,
// and by what each item has to wait for where it is short.
//
// Groups.  An item has two groups of four waves (a SIMD's two waves are one of
// each), a block of 32 tokens of the 64-token tile each, in LDS of its own.  They
// take turns: one has its products on the matrix cores (the values of its block,
// then the keys of its next one) while the other goes from scores to
// probabilities and stages what was loaded; a barrier lies between the turns.
// (Eight waves that each do both by themselves: 1800 fp16 tokens 60 us, in turns 46.)
// In the end the groups join in LDS.  With 256 channels a wave's outputs and
// queries fill the registers of its SIMD alone, and there is one group.
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
// a closed form and no list of items is made.  What an item's beginning and end
// cost (queries as terms, the first tiles' way from memory, the joining) counts as
// 256 tokens, 160 with 256 channels.  A stretch may hold the end of an item, whole ones and the
// beginning of another; the parts of items that are cut go to the workspace, and a
// second launch joins them.  (Its launch takes 2 us and what it reads and writes 2
// of a tail of 4 tokens, 6 of a prompt of 1800, near HBM's rate.)
//
// Measured, 12 heads over 2 of 128 channels, on the same inputs again and in turn over
// several: 1800 fp16 tokens 44 and 46 us (20 GFLOP of terms' products: 18 us at a large
// product's rate; then 2 us of start, 3 of plan and place, 6 of first tiles and queries
// for each of an item's parts, 8 of parts and join); 16 requests of 1..256 tokens behind
// up to 1800 in 8 bits 62 and 66 us; 450 bf16 tokens behind 32,317 231 to 242 us by the
// card (270 GFLOP: 1.12 to 1.17 PFLOP/s, a large product's rate); 4 tokens behind 253
// 14.1 to 14.6 us.
#include <algorithm>
#include <type_traits>

#include "bitnet_device.hpp"
#include "bitnet_internal.hpp"
#include "kv.hpp"
#include "terms.hpp"

namespace bitnet {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kCols = 32;                 // rows (token, head) of a wave
constexpr int kRowWaves = 4;
constexpr int kRows = kCols * kRowWaves;  // of an item
constexpr int kBlock = 32;                // tokens of a wave's step
// Two groups of waves take the blocks of a tile, and join in LDS at the end; with
// 256 channels a wave fills its SIMD's registers, and there is one group.
constexpr int split_of(int D) { return D == 256 ? 1 : 2; }
constexpr int threads_of(int D) { return 64 * kRowWaves * split_of(D); }
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Workgroups, one a compute unit (512: the prompt of 1800 tokens 58 us, 48 with 256).
constexpr int kGrid = 256;
// Tokens that an item's beginning and end cost as much as (128 channels: 96, 192, 256,
// 384: that prompt 58, 49.6, 46.4, 45.1 us, 16 ragged requests 75, 63.4, 63.7, 65.3; 64
// channels: 256, 320, 384, 512: 36, 37, 38, 37 and 54, 52.5, 53, 58; 256 channels, whose
// tokens take longer: 64, 128, 160, 256: 113, 94, 94.6, 101, and 22 requests of some 220
// fp16 tokens 58, 56, 53.7, 51).
constexpr int fixed_of(int D) { return D == 256 ? 160 : 256; }
// 8-bit caches: exponent of the outputs' unit before there is a value.
constexpr float kNoUnit = -126.0f;
// Tiles of a stretch, at least (1, 2, 4: a tail of 4 tokens 15.1, 14.6, 17.0 us).
constexpr int kLeast = 2;

struct ChunkPlan {
  int groups;
  size_t outs, stats, units, total;   // workspace offsets; records first
};
// Of a place in the workspace, of which a workgroup has two: the item of which it holds
// a part (parts: 0 for none).  The parts' places are `place`, then every second one from
// 2 (w + 1) on.
struct Record {
  int32_t parts, w, place, from, m0, count, kvh, pad;
};

ChunkPlan chunk_plan(int64_t T, int64_t R, int64_t q_heads, int64_t kv_heads, int64_t D,
                     int64_t max_len) {
  const int64_t items = kv_heads * (T * (q_heads / kv_heads) / kRows + R);
  const int64_t tile = kBlock * split_of((int)D), tiles = (max_len + tile - 1) / tile;
  ChunkPlan p;
  p.groups = (int)std::min<int64_t>(kGrid, items * (tiles + fixed_of((int)D) / tile));
  // Two places a workgroup: for the item at its beginning and the one at its end.
  const size_t rows = 2 * (size_t)p.groups * kRows;
  p.outs = 2 * kGrid * sizeof(Record);
  p.stats = p.outs + rows * D * 4;
  p.units = p.stats + rows * 8;
  p.total = p.units + rows * 4;
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
    terms_f16_packed(x, t);
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

// Maximum over the 32 lanes of a half that hold the same in both.
__device__ __forceinline__ float across32(float v) {
  v = across16<true>(v);
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t p0 = p[0], p1 = p[1];
  return fmaxf(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1));
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
__device__ __forceinline__ double read_lane(double v, int i) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, i);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), i);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// floor(x / d) of whole numbers, x below 2^53, the quotient below 2^30, inv = 1 / d
// within 2^-40 (a division is thirty instructions, which a short call waits for).
__device__ __forceinline__ double inverse(double d) {
  const double r = __builtin_amdgcn_rcp(d);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
__device__ __forceinline__ double quotient(double x, double d, double inv) {
  const double q = floor(x * inv), r = __builtin_fma(-q, d, x);
  return r < 0.0 ? q - 1.0 : r >= d ? q + 1.0 : q;
}
__device__ __forceinline__ double uniform(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int DT, int D>
struct ChunkShape {
  static constexpr int kSplit = split_of(D), kTile = kBlock * kSplit;   // tokens of a step
  static constexpr int kWaves = kRowWaves * kSplit, kThreads = threads_of(D);
  static constexpr int kBytes = Operand<DT>::kBytes;
  static constexpr int kPieces = D * kBytes / 16;             // of a cached row
  static constexpr int kPass = 256 / kPieces < kBlock ? 256 / kPieces : kBlock;   // tokens
  static constexpr int kLoads = kBlock / kPass;               // of a thread, keys and values each
  static constexpr int kWaveTokens = 64 / kPieces;            // of a wave's load
  // Bytes of a row in LDS: eight rows' pieces of keys, and the four rows that a
  // transposing read takes of values, lie on banks of their own.
  static constexpr int kKeyRow = 2 * D + 16, kValueRow = 2 * D + 32;
  static constexpr int kMine = D / 32 / kSplit;               // channel blocks a wave ends up with
  // Of three terms of the queries the smallest stays in LDS: registers are short.
  static constexpr int kTerms = Operand<DT>::kTerms;
  static constexpr int kKept = kTerms == 3 && D >= 128 ? 2 : kTerms;
};

// A request's new tokens: rows [from, from + n) of q; `old` tokens lie before them
// (may be negative).  Its rows (token, head) make `tiles` items for each key/value
// head, on `line` places of the line.  An item has `lead` of them for the tokens
// before the new ones and what its beginning and end cost.
struct Request {
  int from, n, old, tiles;
  double lead, line;
};
template <int DT, int D, bool FEW>
struct ChunkShared {
  typedef ChunkShape<DT, D> S;
  // Of each group a block of keys, then one of values; in the end what the groups
  // exchange.
  static constexpr int kKeyBytes = kBlock * S::kKeyRow, kValueBytes = kBlock * S::kValueRow;
  static constexpr int kBytes = std::max(S::kSplit * (kKeyBytes + kValueBytes),
                                         (S::kSplit - 1) * S::kWaves * S::kMine * 4096);
  __attribute__((aligned(16))) uint8_t kv[kBytes];
  __attribute__((aligned(16))) uint8_t q[S::kKept < S::kTerms ? S::kWaves * 64 * D : 16];
  float stats[S::kWaves][DT == BITNET_KV_INT8 ? 3 : 2][kCols];   // and their bases, sums, units
  int pages[S::kWaves][64];
  float scales[S::kWaves][2][2][kBlock];   // 8-bit caches: two blocks' key and value scales
  double first[FEW ? 64 : S::kThreads];    // places before each request, or each thread's
  Request request[FEW ? 64 : 1];
  int top[FEW ? 1 : S::kThreads];          // largest start before them
  double wave_sum[S::kWaves];
  int wave_top[S::kWaves];
};

struct ChunkGrid {
  int64_t outs_off, stats_off, units_off;   // in the workspace
  double over_groups, over_unit;   // 1 / workgroups, 1 / (a tile of tokens' places)
  int32_t groups, per;   // workgroups; query heads per key/value head
};

// From the largest start up to this request's, which is the next one's at least.
template <int D>
__device__ __forceinline__ Request request_of(const ChunkArgs &a, int per, int start, int next,
                                              int len) {
  Request q;
  q.from = min(start, a.T);
  q.n = min(max(start, next), a.T) - q.from;
  q.old = min(max(len, 0), a.max_len) - q.n;
  const int rows = q.n * per;
  q.tiles = (rows + kRows - 1) / kRows;
  q.lead = (double)(max(q.old, 0) + fixed_of(D)) * per;
  q.line = q.tiles == 0 ? 0.0
                        : q.tiles * q.lead + (double)(kRows / 2) * q.tiles * (q.tiles - 1) + rows;
  return q;
}

// What a row has summed up, times the reciprocal of its probabilities' sum, and of 8-bit
// caches times its unit, 2^unit.  (Not the sums times the unit: those pass the largest
// value by up to 2^15 a token.)
template <bool I8>
__device__ __forceinline__ f32x4 mean_of(f32x4 y, float over, float unit) {
  y *= over;
  if constexpr (I8) y *= exp2_fast(unit);
  return y;
}
// Exponent of the power of two above x >= 0, at least -100.
__device__ __forceinline__ float exponent_above(float x) {
  return (float)((int)(__builtin_bit_cast(uint32_t, pow2_above(x)) >> 23) - 127);
}
__device__ __forceinline__ float row_lse(float base, float sum) {
  return sum > 0.0f ? (base + __log2f(sum)) * kLn2 : -INFINITY;
}

// FEW: up to 64 requests, which every wave holds a lane each (through LDS instead, as
// for more: a prompt 1 us more, 450 tokens at 32,767 6 us).
// HALVES: 16 tokens in a row always lie on one page, at 32-bit offsets (a page a token
// instead: a prompt 2 us more, 8-bit requests the same).
template <int DT, int D, bool FEW, bool HALVES>
__global__ void __launch_bounds__(threads_of(D)) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
chunk_kernel(ChunkArgs a, ChunkGrid g) {
  typedef Operand<DT> F;
  typedef typename F::V V;
  typedef ChunkShape<DT, D> S;
  constexpr bool kI8 = DT == BITNET_KV_INT8;
  constexpr int kSteps = D / 16;       // contraction steps of the scores
  constexpr int kBlocks = D / 32;      // channel blocks of the outputs
  constexpr int kTerms = F::kTerms;
  constexpr int kTile = S::kTile, kWaves = S::kWaves, kThreads = S::kThreads, kSplit = S::kSplit;
  // Probabilities are relative to 2^-kUp of a base that the running maximum
  // exceeds by up to 2^kSlack, so that it need not follow every new maximum.  With
  // 8-bit values the products take bare codes, and probabilities times scales, relative
  // to 2^v_base above the largest scale so far.
  constexpr float kSlack = 6.0f, kUp = F::kHalf ? 15.0f - kSlack : 0.0f;
  typedef ChunkShared<DT, D, FEW> Sh;
  __shared__ Sh sh;

  const int tid = threadIdx.x, lane = tid & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = wave % kRowWaves, part = wave / kRowWaves;   // 32 rows of an item; block of a tile
  const int per = g.per, kv_heads = a.c.kv_heads;

  const int each = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(tid * each, a.R), r1 = min(r0 + each, a.R);
  double total;
  if constexpr (FEW) {
    const int r = min(lane, a.R - 1);
    const int start = ld_global<int>(a.starts + r), next = ld_global<int>(a.starts + r + 1);
    const int len = ld_global<int>(a.lens + r);
    Request mine = request_of<D>(a, per, scan_max(max(start, 0)), next, len);
    if (lane >= a.R) mine.line = 0.0;
    const double upto = scan_sum(mine.line * kv_heads);
    total = read_lane(upto, 63);
    if (wave == 0) {
      sh.request[lane] = mine;
      sh.first[lane] = lane < a.R ? upto - mine.line * kv_heads : total + 1.0;
    }
    __syncthreads();
  } else {
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
    for (int r = r0; r < r1; ++r) {
      top = max(top, ld_global<int>(a.starts + r));
      sum += request_of<D>(a, per, top, ld_global<int>(a.starts + r + 1), ld_global<int>(a.lens + r)).line *
             kv_heads;
    }
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
  const double stretch =
      uniform(fmax(quotient(total + g.groups - 1, g.groups, g.over_groups), kLeast * unit));
  const double over_stretch = inverse(stretch);
  // Workgroups go round the eight dies in turn: neighbours on the line, which read the
  // same keys and values, to one of them (a prompt fetches 18 MB instead of 38 and takes
  // 0.5 us less, 16 ragged requests 28 MB instead of 74).
  const int w = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
  const double begin = w * stretch, stop = fmin(begin + stretch, total);
  double pos = begin;
  Record *records = reinterpret_cast<Record *>(a.ws);
  if (tid < 2) records[2 * w + tid].parts = 0;

  while (pos < stop) {
    // The item at pos: request r, key/value head kvh, the tile0-th of those.
    Request q;
    int r;
    double from;   // the request's first place
    if constexpr (FEW) {
      r = __builtin_popcountll(__ballot(sh.first[lane] <= pos)) - 1;
      q = sh.request[r];
      from = sh.first[r];
    } else {
      int at = 0;
#pragma unroll
      for (int i = 0; i < kThreads; i += 64) at += __builtin_popcountll(__ballot(sh.first[i + lane] <= pos));
      at -= 1;
      int top = sh.top[at];
      from = sh.first[at];
      r = at * each;
      for (;;) {
        top = max(top, ld_global<int>(a.starts + r));
        q = request_of<D>(a, per, top, ld_global<int>(a.starts + r + 1), ld_global<int>(a.lens + r));
        const double next = from + q.line * kv_heads;
        if (pos < next || r + 1 >= min(at * each + each, a.R)) break;
        from = next;
        ++r;
      }
      r = __builtin_amdgcn_readfirstlane(r);
    }
    q.from = __builtin_amdgcn_readfirstlane(q.from);
    q.n = __builtin_amdgcn_readfirstlane(q.n);
    q.old = __builtin_amdgcn_readfirstlane(q.old);
    const int rows = q.n * per;
    int kvh = min((int)quotient(pos - from, q.line, inverse(q.line)), kv_heads - 1), tile0;
    double item0, item_end;
    {
      from += kvh * q.line;
      const double o = pos - from, b = q.lead + kRows / 2;
      auto before = [&](int j) { return j * q.lead + (double)(kRows / 2) * j * (j + 1.0); };
      // (Nearly: the loops behind it find the tile.)
      int j = (int)((__builtin_amdgcn_sqrtf((float)(b * b + 2.0 * kRows * o)) - (float)b) * (1.0f / kRows));
      j = max(min(j, q.tiles - 1), 0);
      while (j > 0 && before(j) > o) --j;
      while (j + 1 < q.tiles && before(j + 1) <= o) ++j;
      tile0 = __builtin_amdgcn_readfirstlane(j);
      item0 = uniform(from + before(j));
      item_end = uniform(item0 + q.lead + min((j + 1) * kRows, rows));
    }
    kvh = __builtin_amdgcn_readfirstlane(kvh);
    const int old = q.old;
    const int m0 = tile0 * kRows, count = min(kRows, rows - m0);
    const int len = min(max(old + (m0 + count - 1) / per + 1, 0), a.max_len);   // that the last row sees
    const int tiles = (len + kTile - 1) / kTile;
    // Tiles [first, end) of the item are this stretch's.
    const double tile_at = item0 + (double)fixed_of(D) * per;   // the place of the first
    auto cut = [&](double at) {
      return at <= tile_at ? 0 : (int)fmin(quotient(at - tile_at, unit, g.over_unit), (double)tiles);
    };
    const int first = __builtin_amdgcn_readfirstlane(cut(begin));
    const int end = __builtin_amdgcn_readfirstlane(item_end <= stop ? tiles : cut(stop));
    const bool whole = first == 0 && end == tiles;
    const double here = pos;
    pos = fmax(fmin(item_end, stop), here + 1.0);   // (item_end > here: the loop ends in any case)
    if (first == end && !(tiles == 0 && here == item0)) continue;

    const int64_t head_off = (int64_t)kvh * a.c.head_stride * S::kBytes;
    const uint8_t *kbase = reinterpret_cast<const uint8_t *>(a.c.k) + head_off;
    const uint8_t *vbase = reinterpret_cast<const uint8_t *>(a.c.v) + head_off;
    const int32_t *table = a.tables + (int64_t)r * a.max_pages;
    const uint32_t page_bytes = (uint32_t)(a.c.page_stride * S::kBytes);
    const uint32_t tok_bytes = (uint32_t)(a.c.token_stride * S::kBytes);
    const int tok_mask = (1 << a.c.page_shift) - 1;
    const uint32_t lane_off = (lane / S::kPieces) * tok_bytes + 16 * (lane % S::kPieces);
    // Staging: the 16-byte piece of tokens st0, st0 + kPass, ... of its group's block.
    const int gt = tid & 255, piece = gt % S::kPieces, st0 = gt / S::kPieces;
    const bool stages = S::kPieces >= 8 || st0 < kBlock;
    uint8_t *const kd = sh.kv + part * (Sh::kKeyBytes + Sh::kValueBytes);
    uint8_t *const vd = kd + Sh::kKeyBytes;

    // Pages: of 16 tokens each, for a batch of tiles; or (small pages) of token c of
    // the group's next block.
    constexpr int kSixteens = kTile / 16, kBatch = 64 / kSixteens;
    int pg_lo = 0, pg_hi = 0;
    u32x4 kr[S::kLoads], vr[S::kLoads];   // the keys of the block after the values'
    uint64_t off[S::kLoads];         // of the block whose keys are loaded
    uint32_t scale_at = 0;
    float v_exp0 = 0.0f, v_exp1 = 0.0f;   // 8-bit caches: exponent above the largest value scale
    uint32_t mask0 = 0, mask1 = 0, mask2 = 0;   // tokens that are there: of the block worked
                                                // on, the next one, the one loaded last
    float ks_next = 0.0f, vs_next = 0.0f;   // of the block whose keys are loaded
    auto page_at = [&](int token) { return ld_global<int>(table + (min(token, len - 1) >> a.c.page_shift)); };
    // The first ones, asked for ahead of the queries.
    int asked = 0;
    if (first < end) asked = page_at(first * kTile + (HALVES ? 16 * lane : part * kBlock + c));
    auto load_pages = [&](int tile) {   // of the tile, and of those behind it
      int lo, hi = 0;
      if constexpr (HALVES) {   // (in LDS: a register for them is one too many)
        if ((tile - first) % kBatch == 0)
          sh.pages[wave][lane] = tile == first ? asked : page_at(tile * kTile + 16 * lane);
        __builtin_amdgcn_wave_barrier();
        const int n = kSixteens * ((tile - first) % kBatch) + 2 * part;
        lo = sh.pages[wave][n];
        hi = sh.pages[wave][n + 1];
      } else {
        lo = tile == first ? asked : page_at(tile * kTile + part * kBlock + c);
      }
      pg_lo = lo;
      pg_hi = hi;
    };
    // The rows of the keys of a tile: where they are, and which are there.
    auto load_keys = [&](int tile) {
      const int j0 = tile * kTile + part * kBlock;
      if constexpr (HALVES) {
        uint32_t page[2];
        mask2 = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t p = __builtin_amdgcn_readfirstlane(i ? pg_hi : pg_lo);
          const bool ok = p < (uint32_t)a.c.pages;
          page[i] = ok ? p : 0;
          mask2 |= ok ? 0xffffu << (16 * i) : 0;
        }
        const int left = len - j0;
        if (left < kBlock) mask2 &= left <= 0 ? 0u : (1u << left) - 1;
        if constexpr (kI8)
          scale_at = (((c < 16 ? page[0] : page[1]) * (uint32_t)kv_heads + kvh) << a.c.page_shift) +
                     ((j0 + c) & tok_mask);
#pragma unroll
        for (int l = 0; l < S::kLoads; ++l) {
          const int t = rw * S::kWaveTokens + l * S::kPass;   // the wave's first
          off[l] = (uint64_t)page[(t >> 4) & 1] * page_bytes +
                   (uint64_t)(uint32_t)((j0 + t) & tok_mask) * tok_bytes + lane_off;
        }
      } else {
        const bool ok = j0 + c < len && (uint32_t)pg_lo < (uint32_t)a.c.pages;
        mask2 = (uint32_t)__ballot(ok);
        const uint32_t page = ok ? pg_lo : 0, tok = ok ? (j0 + c) & tok_mask : 0;
        if constexpr (kI8)
          scale_at = ((page * (uint32_t)kv_heads + kvh) << a.c.page_shift) + tok;
#pragma unroll
        for (int l = 0; l < S::kLoads; ++l) {
          const int t = (st0 + l * S::kPass) & (kBlock - 1);
          off[l] = (uint64_t)(uint32_t)__shfl((int)page, t) * page_bytes +
                   (uint64_t)(uint32_t)__shfl((int)tok, t) * tok_bytes + 16 * piece;
        }
      }
      if (stages)
#pragma unroll
        for (int l = 0; l < S::kLoads; ++l) kr[l] = ld_global<u32x4>(kbase + off[l]);
      if constexpr (kI8) {
        ks_next = ld_global<float>(a.c.k_scale + scale_at);
        vs_next = ld_global<float>(a.c.v_scale + scale_at);
      }
    };
    auto load_values = [&]() {   // of the block whose keys were loaded last
      if (stages)
#pragma unroll
        for (int l = 0; l < S::kLoads; ++l) vr[l] = ld_global<u32x4>(vbase + off[l]);
    };
    // 8-bit caches: the scales of the block whose keys are loaded.
    auto stage_scales = [&](int tile, uint32_t mask) {
      if constexpr (kI8) {
        const bool ok = (mask >> c) & 1;
        const float ks = ok ? ks_next : 0.0f, vs = ok && fabsf(vs_next) < INFINITY ? vs_next : 0.0f;
        v_exp1 = exponent_above(across32(vs));
        if (h == 0) {
          sh.scales[wave][tile & 1][0][c] = ks;
          sh.scales[wave][tile & 1][1][c] = vs;
        }
      }
    };
    auto stage_keys = [&](int n) {   // the n-th of this thread's pieces
      const int t = st0 + n * S::kPass;
      uint8_t *at = kd + t * S::kKeyRow + (kI8 ? 32 : 16) * piece;
      if (!stages) return;
      if constexpr (kI8) {
        *reinterpret_cast<f16x8 *>(at) = codes_f16(kr[n].x, kr[n].y);
        *reinterpret_cast<f16x8 *>(at + 16) = codes_f16(kr[n].z, kr[n].w);
      } else {
        *reinterpret_cast<u32x4 *>(at) = kr[n];
      }
    };
    // Tokens that are not there get values of zero, and values that are not finite
    // become finite: a row that must not see them has probabilities of zero for them.
    auto stage_values = [&](uint32_t mask, int n) {
      const int t = st0 + n * S::kPass;
      uint8_t *at = vd + t * S::kValueRow + (kI8 ? 32 : 16) * piece;
      if (!stages) return;
      const bool ok = (mask >> t) & 1;
      u32x4 v = vr[n];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (!kI8) {
          typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
          constexpr unsigned short kMost = DT == BITNET_KV_BF16 ? 0x7f7f : 0x7bff;
          const u16x2 m = __builtin_elementwise_min(
              __builtin_bit_cast(u16x2, v[e] & 0x7fff7fffu), u16x2{kMost, kMost});
          v[e] = __builtin_bit_cast(uint32_t, m) | (v[e] & 0x80008000u);
        }
        v[e] = ok ? v[e] : 0u;
      }
      if constexpr (kI8) {
        *reinterpret_cast<f16x8 *>(at) = codes_f16(v.x, v.y);
        *reinterpret_cast<f16x8 *>(at + 16) = codes_f16(v.z, v.w);
      } else {
        *reinterpret_cast<u32x4 *>(at) = v;
      }
    };
    // The values of `tile` and the keys of the next one into LDS, and their
    // successors' loads.  (Behind the last tile it is that once more, and not looked
    // at.)
    auto staging = [&](int tile) {
#pragma unroll
      for (int n = 0; n < S::kLoads; ++n) stage_values(mask0, n);
      load_values();
#pragma unroll
      for (int n = 0; n < S::kLoads; ++n) stage_keys(n);
      stage_scales(tile + 1, mask1);
      load_keys(min(tile + 2, end - 1));
      load_pages(min(tile + 3, end - 1));
    };


    // This lane's row.
    const int in = rw * kCols + c, m = m0 + min(in, count - 1);
    const bool live = in < count, active = rw * kCols < count;
    const int i = m / per, head = kvh * per + (m - i * per);
    const int limit = min(max(old + i + 1, 0), a.max_len);
    // What the wave's first and last rows see.
    const int limit_lo = __builtin_amdgcn_readlane(limit, 0);
    const int limit_hi = active ? __builtin_amdgcn_readlane(limit, 31) : 0;
    // Queries as terms.
    constexpr int kKept = S::kKept;
    V qt[kSteps][kKept];
    uint8_t *qlds = sh.q + wave * 64 * D + 16 * lane;   // of the last term, 1 KB a step
    float unscale = 1.0f;   // of the scores
    {
      const float *src = a.q + (int64_t)(q.from + i) * a.q_stride + (int64_t)head * D;
      f32x4 x[kSteps][2];
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        x[f][0] = ld_global<f32x4>(src + 16 * f + 8 * h);
        x[f][1] = ld_global<f32x4>(src + 16 * f + 8 * h + 4);
      }
      if (first < end) {
        load_pages(first);
        load_keys(first);
        load_pages(min(first + 1, end - 1));
        load_values();
      }
      float up = a.scale * kLog2e;
      if constexpr (F::kHalf) {
        float big = 0.0f;
#pragma unroll
        for (int f = 0; f < kSteps; ++f)
#pragma unroll
          for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[f][e >> 2][e & 3]));
        const float p2 = pow2_above(max2(big) * fabsf(up));
        unscale = p2 * 0x1p-14f;
        const float to_half = pow2_inverse(p2) * 0x1p14f;
        // Both in one factor, which is exact, unless tiny queries meet so large a scale
        // that it is infinite: those are below 2^-113 and raised first.
        const bool tiny = fabsf(up * to_half) == INFINITY;
        if (__any(tiny)) {
#pragma unroll
          for (int f = 0; f < kSteps; ++f)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[f][e >> 2][e & 3] *= tiny ? 0x1p120f : 1.0f;
        }
        up = (tiny ? up * 0x1p-120f : up) * to_half;
      }
#pragma unroll
      for (int f = 0; f < kSteps; ++f) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = x[f][e >> 2][e & 3] * up;
          asm("" : "+v"(y[e]));
        }
        V t[kTerms];
        F::split(y, t);
#pragma unroll
        for (int p = 0; p < kKept; ++p) qt[f][p] = t[p];
        if constexpr (kKept < kTerms) *reinterpret_cast<V *>(qlds + 1024 * f) = t[kKept];
      }
    }

    float base = -INFINITY, l = 0.0f;   // of the exponents, without kUp
    float v_base = kNoUnit;             // 8-bit caches: exponent of the outputs' unit
    f32x16 o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[b][e] = 0.0f;
    f32x16 s[1];                      // scores
    V p[2][kTerms];                   // probabilities

    // The products of a turn: the outputs' with the block's values, then the scores'
    // with the next one's keys; the LDS reads stay kAhead operands in front.
    constexpr int kValues = 2 * kBlocks, kAhead = kKept < kTerms ? 2 : 3;
    V ring[kAhead + 1], qring[kKept < kTerms ? kAhead + 1 : 1];
    auto fetch = [&](int n) {   // operand n: values, then keys
      if (n < kValues) {
        const int cc = lane & 15;
        const uint8_t *at = vd + (4 * h + (cc >> 2)) * S::kValueRow + 32 * (lane >> 4 & 1) + 8 * (cc & 3) +
                            16 * (n / kBlocks) * S::kValueRow + 64 * (n % kBlocks);
        s16x4 t[2];
        t[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((BITNET_LDS s16x4 *)at);
        t[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((BITNET_LDS s16x4 *)(at + 8 * S::kValueRow));
        ring[n % (kAhead + 1)] = __builtin_bit_cast(V, t);
      } else if (n < kValues + kSteps) {
        const int f = n - kValues;
        ring[n % (kAhead + 1)] = *reinterpret_cast<const V *>(kd + c * S::kKeyRow + 32 * f + 16 * h);
        if constexpr (kKept < kTerms)
          qring[n % (kAhead + 1)] = *reinterpret_cast<const V *>(qlds + 1024 * f);
      }
    };
    auto product = [&](int n) {
      const V &x = ring[n % (kAhead + 1)];
      if (n < kValues) {
        f32x16 &y = o[n % kBlocks];
#pragma unroll
        for (int t = kTerms - 1; t >= 0; --t) y = F::mfma(x, p[n / kBlocks][t], y);
      } else {
        const int f = n - kValues;
        if constexpr (kKept < kTerms) s[0] = F::mfma(x, qring[n % (kAhead + 1)], s[0]);
#pragma unroll
        for (int t = kKept - 1; t >= 0; --t) s[0] = F::mfma(x, qt[f][t], s[0]);
      }
    };
    // Operands [FROM, TO).
    auto turn = [&](auto from_, auto to_) {
      constexpr int kFrom = decltype(from_)::value, kTo = decltype(to_)::value;
      if constexpr (kTo > kValues)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[0][e] = 0.0f;
#pragma unroll
      for (int n = kFrom; n < kFrom + kAhead; ++n) fetch(n);
#pragma unroll
      for (int n = kFrom; n < kTo; ++n) {
        __builtin_amdgcn_sched_barrier(0);
        if (n + kAhead < kTo) fetch(n + kAhead);
        __builtin_amdgcn_sched_barrier(0);
        product(n);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 0> kBegin{};
    constexpr std::integral_constant<int, kValues> kBetween{};
    constexpr std::integral_constant<int, kValues + kSteps> kEnd{};
    // From the scores of a tile to its probabilities.
    auto probabilities = [&](int tile, uint32_t mask) {
      const int t0 = tile * kTile + part * kBlock;   // the wave's first token
      const bool all = mask == 0xffffffffu && t0 + kBlock <= limit_lo;
      // Those of this lane's tokens that its row sees: bit 8 a + e for token 8 a + 4 h + e.
      const int left = limit - t0;
      const uint32_t seen = (mask & (left >= kBlock ? ~0u : left <= 0 ? 0u : (1u << left) - 1)) >> 4 * h;
      // The scales of this lane's 16 tokens.
      auto scales = [&](int which, float (&y)[16]) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 y4 = *reinterpret_cast<const f32x4 *>(&sh.scales[wave][tile & 1][which][8 * b + 4 * h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[4 * b + e] = y4[e];
        }
      };
      // Exponent above the largest of the values' scales that the row sees.
      float v_exp = kNoUnit;
      if constexpr (kI8) {
        v_exp = v_exp0;
        if (!all) {
          float big = 0.0f, vs[16];
          scales(1, vs);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            big = fmaxf(big, seen >> (8 * (e >> 2) + (e & 3)) & 1 ? vs[e] : 0.0f);
          v_exp = exponent_above(max2(big));
        }
      }
      f32x16 &x = s[0];
      if constexpr (kI8) {
        float ks[16];
        scales(0, ks);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= ks[e];
      }
      if (!all) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (!(seen >> (8 * (e >> 2) + (e & 3)) & 1)) x[e] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
      top = max2(top) * unscale;
      if (__any(top > base + kSlack || (kI8 && v_exp > v_base))) {
        const float b_new = fmaxf(base, top);
        float keep = base == -INFINITY ? 0.0f : exp2_fast(base - b_new);
        base = b_new;
        l *= keep;
        if constexpr (kI8) {
          const float v_new = fmaxf(v_base, v_exp);
          keep *= exp2_fast(v_base - v_new);
          v_base = v_new;
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[b] *= keep;
      }
      // (What rounds off the base is the same factor for all that a row sums up.)
      const float shift = kUp - (base == -INFINITY ? 0.0f : base);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = exp2_fast(__builtin_fmaf(x[e], unscale, shift));
        sum += x[e];
      }
      l += sum;
      if constexpr (kI8) {
        float vs[16];
        __builtin_amdgcn_sched_barrier(0);   // (asked for earlier they take registers too many)
        scales(1, vs);
        // (A scale above that of all that the row sees goes with a probability of zero,
        // which comes first, so that the product is zero.)
        const float over = exp2_fast(-v_base);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * over * vs[e];
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = x[8 * half + e];
          if constexpr (kI8) asm("" : "+v"(y[e]));   // one rounding of the product for both terms
        }
        F::split(y, p[half]);
      }
    };

    // The groups of waves take turns: while one has its products on the matrix
    // cores, the other works out its probabilities; a barrier between the turns
    // keeps them apart.
    if (first < end) {
      mask0 = mask2;
      stage_scales(first, mask0);
      v_exp0 = v_exp1;
#pragma unroll
      for (int n = 0; n < S::kLoads; ++n) stage_keys(n);
      load_keys(min(first + 1, end - 1));
      load_pages(min(first + 2, end - 1));
      mask1 = mask2;
      __syncthreads();
      if (kSplit == 2 && part == 1) __syncthreads();
      auto next_masks = [&]() {
        mask0 = mask1;
        mask1 = mask2;
        v_exp0 = v_exp1;
      };
      if (first * kTile + part * kBlock < limit_hi) {
        turn(kBetween, kEnd);
        settle<D>(s);
        int tile = first;
        for (; tile + 1 < end; ++tile) {
          __syncthreads();
          staging(tile);
          probabilities(tile, mask0);
          next_masks();
          __syncthreads();
          turn(kBegin, kEnd);
          settle<D>(s);
          settle<D>(o);
        }
        __syncthreads();
        staging(tile);
        probabilities(tile, mask0);
        __syncthreads();
        turn(kBegin, kBetween);
        settle<D>(o);
      } else {   // rows that see nothing of it: the staging alone
        for (int tile = first; tile < end; ++tile) {
          __syncthreads();
          staging(tile);
          next_masks();
          __syncthreads();
        }
      }
      if (kSplit == 2 && part == 0) __syncthreads();
    }
    l = sum2(l);
    // The groups of waves join: of a pair each wave keeps half of the channels.
    constexpr int kMine = S::kMine;   // channel blocks, from b0 on
    const int b0 = part * kMine;
    f32x16 y[kMine];
    __syncthreads();   // all are done with the tiles
    if constexpr (kSplit == 2) {
      uint8_t *mine_x = sh.kv + wave * (kMine * 4096) + 16 * lane;
      const uint8_t *other_x = sh.kv + (wave ^ kRowWaves) * (kMine * 4096) + 16 * lane;
#pragma unroll
      for (int b = 0; b < kMine; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x16 &z = part ? o[b] : o[kMine + b];
          *reinterpret_cast<f32x4 *>(mine_x + (4 * b + e) * 1024) =
              f32x4{z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]};
        }
      if (h == 0) {
        sh.stats[wave][0][c] = base;
        sh.stats[wave][1][c] = l;
        if constexpr (kI8) sh.stats[wave][2][c] = v_base;
      }
      __syncthreads();
      const float base2 = sh.stats[wave ^ kRowWaves][0][c], l2 = sh.stats[wave ^ kRowWaves][1][c];
      const float top = fmaxf(base, base2), zero = top == -INFINITY ? 0.0f : top;
      float f1 = exp2_fast(base - zero), f2 = exp2_fast(base2 - zero);
      base = top;
      l = l * f1 + l2 * f2;
      if constexpr (kI8) {
        const float v2 = sh.stats[wave ^ kRowWaves][2][c], v_top = fmaxf(v_base, v2);
        f1 *= exp2_fast(v_base - v_top);
        f2 *= exp2_fast(v2 - v_top);
        v_base = v_top;
      }
#pragma unroll
      for (int b = 0; b < kMine; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x4 z = *reinterpret_cast<const f32x4 *>(other_x + (4 * b + e) * 1024);
#pragma unroll
          for (int d = 0; d < 4; ++d)
            y[b][4 * e + d] = (part ? o[kMine + b] : o[b])[4 * e + d] * f1 + z[d] * f2;
        }
      // (The next item's first tile goes where this was.)
      if (pos < stop) __syncthreads();
    } else {
#pragma unroll
      for (int b = 0; b < kMine; ++b) y[b] = o[b];
    }

    if (whole) {
      if (live) {
        // (Without a token the sums are zeros.)
        const int64_t row = (int64_t)(q.from + i) * a.q_heads + head;
        const float over = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int b = 0; b < kMine; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e)   // 16 of a row's 32 channels of a block
            st_global<f32x4>(a.out + row * D + 32 * (b0 + b) + 4 * h + 8 * e,
                             mean_of<kI8>(f32x4{y[b][4 * e], y[b][4 * e + 1], y[b][4 * e + 2], y[b][4 * e + 3]},
                                          over, v_base));
        if (a.lse && h == 0 && part == 0) a.lse[row] = row_lse(base - kUp, l);
      }
      continue;
    }
    // A part of an item: into the workspace, for the join.
    const int place = 2 * w + (item0 > begin ? 1 : 0);
    if (active) {
      float *part_out = reinterpret_cast<float *>(a.ws + g.outs_off) + (int64_t)place * kRows * D +
                        (rw * kBlocks + b0) * 1024 + 4 * lane;
#pragma unroll
      for (int b = 0; b < kMine; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_global<f32x4>(part_out + (4 * b + e) * 256,
                           f32x4{y[b][4 * e], y[b][4 * e + 1], y[b][4 * e + 2], y[b][4 * e + 3]});
      if (h == 0 && part == 0) {
        st_global<f32x2>(a.ws + g.stats_off + ((int64_t)place * kRows + in) * 8, f32x2{base - kUp, l});
        if constexpr (kI8) st_global<float>(a.ws + g.units_off + ((int64_t)place * kRows + in) * 4, v_base);
      }
    }
    if (tid == (place & 1)) {   // (which cleared it)
      // The first and the last stretch that hold a tile of the item.
      const int w0 = (int)quotient(tile_at + unit - 1.0, stretch, over_stretch);
      const int w_end = (int)quotient(item_end - 1.0, stretch, over_stretch);
      const int w_last = min((int)quotient(tile_at + tiles * unit - 1.0, stretch, over_stretch), w_end);
      records[place] = Record{w_last - w0 + 1, w0, 2 * w0 + (item0 > w0 * stretch ? 1 : 0),
                              q.from, m0, count, kvh, 0};
    }
  }
}

// Joins the parts of the items that are cut.  The workgroups of an item's n parts share
// the work, kHelpers for each: blocks of 32 rows and 32 channels, a wave each; from
// kMany parts on a quarter of the channels each, and a quarter of the parts to a wave.
// (A workgroup for each item and 32 rows of it: 8 tokens at 12,324 of 8 bits take 37.5
// us, 19.5 so, 64 at 32,064 63 and 21.7, a prompt of 512 23.4 and 24.1; kHelpers 1 and 4
// and kMany 8 and 6 leave that prompt at 25 to 26.)
constexpr int kHelpers = 2, kMany = 16;

template <int D, bool I8>
__global__ void __launch_bounds__(256) join_kernel(ChunkArgs a, ChunkGrid g) {
  constexpr int kBlocks = D / 32;
  __shared__ f32x4 sh_z[4][64];
  __shared__ f32x2 sh_st[4][64];
  __shared__ float sh_unit[4][I8 ? 64 : 1];
  const Record in = reinterpret_cast<const Record *>(a.ws)[blockIdx.x];
  if (in.parts == 0) return;
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int helper = ((int)(blockIdx.x >> 1) - in.w) * kHelpers + blockIdx.y, helpers = in.parts * kHelpers;
  const int blocks = (in.count + kCols - 1) / kCols * kBlocks;
  const float *outs = reinterpret_cast<const float *>(a.ws + g.outs_off) + 4 * lane;
  const float *stats = reinterpret_cast<const float *>(a.ws + g.stats_off) + 2 * c;
  const float *units = reinterpret_cast<const float *>(a.ws + g.units_off) + c;
  // Adds up to J parts first, first + step, ... of block `at`, E quads of a lane from e0 on.
  auto add = [&](auto J_, int at, int e0, int first, int step, float &top, float &sum, float &unit, auto &z) {
    constexpr int J = decltype(J_)::value, E = sizeof(z) / sizeof(z[0]);
    f32x2 st[J];
    float un[J];
    f32x4 x[J][E];
#pragma unroll
    for (int u = 0; u < J; ++u) {
      const int p = first + u * step;
      st[u] = f32x2{-INFINITY, 0.0f};
      un[u] = kNoUnit;
#pragma unroll
      for (int e = 0; e < E; ++e) x[u][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (p < in.parts) {
        const int64_t place = p == 0 ? in.place : 2 * (in.w + p);
        st[u] = ld_global<f32x2>(stats + (place * kRows + at / kBlocks * kCols) * 2);
        if constexpr (I8) un[u] = ld_global<float>(units + place * kRows + at / kBlocks * kCols);
#pragma unroll
        for (int e = 0; e < E; ++e)
          x[u][e] = ld_global<f32x4>(outs + place * kRows * D + at * 1024 + (e0 + e) * 256);
      }
    }
    float t = top;
#pragma unroll
    for (int u = 0; u < J; ++u) t = fmaxf(t, st[u].x);
    const float zero = t == -INFINITY ? 0.0f : t;
    float keep = exp2_fast(top - zero);
    top = t;
    sum *= keep;
    if constexpr (I8) {
      float w = unit;
#pragma unroll
      for (int u = 0; u < J; ++u) w = fmaxf(w, un[u]);
      keep *= exp2_fast(unit - w);
      unit = w;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] *= keep;
#pragma unroll
    for (int u = 0; u < J; ++u) {
      float f = exp2_fast(st[u].x - zero);
      sum += st[u].y * f;
      if constexpr (I8) f *= exp2_fast(un[u] - unit);
#pragma unroll
      for (int e = 0; e < E; ++e) z[e] += x[u][e] * f;
    }
  };
  auto store = [&](int at, int e0, float top, float sum, float unit, const auto &z) {
    const int group = at / kBlocks, b = at % kBlocks, at_row = group * kCols + c;
    if (at_row >= in.count) return;
    const int m = in.m0 + at_row, i = m / g.per;
    const int64_t row = (int64_t)(in.from + i) * a.q_heads + in.kvh * g.per + (m - i * g.per);
    const float over = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int e = 0; e < (int)(sizeof(z) / sizeof(z[0])); ++e)
      st_global<f32x4>(a.out + row * D + 32 * b + 8 * (e0 + e) + 4 * h, mean_of<I8>(z[e], over, unit));
    if (a.lse && b == 0 && e0 == 0 && h == 0) a.lse[row] = row_lse(top, sum);
  };
  constexpr f32x4 kZero = {0.0f, 0.0f, 0.0f, 0.0f};
  if (in.parts < kMany) {
    for (int at = 4 * helper + wave; at < blocks; at += 4 * helpers) {
      float top = -INFINITY, sum = 0.0f, unit = kNoUnit;
      f32x4 z[4] = {kZero, kZero, kZero, kZero};
      for (int p = 0; p < in.parts; p += 8)
        add(std::integral_constant<int, 8>{}, at, 0, p, 1, top, sum, unit, z);
      store(at, 0, top, sum, unit, z);
    }
    return;
  }
  for (int n = helper; n < 4 * blocks; n += helpers) {
    const int at = n >> 2, e = n & 3;
    float top = -INFINITY, sum = 0.0f, unit = kNoUnit;
    f32x4 z[1] = {kZero};
    for (int p = wave; p < in.parts; p += 4 * 16)
      add(std::integral_constant<int, 16>{}, at, e, p, 4, top, sum, unit, z);
    sh_z[wave][lane] = z[0];
    sh_st[wave][lane] = f32x2{top, sum};
    if constexpr (I8) sh_unit[wave][lane] = unit;
    __syncthreads();
    if (wave == 0) {
      float all = -INFINITY;
#pragma unroll
      for (int s = 0; s < 4; ++s) all = fmaxf(all, sh_st[s][lane].x);
      const float zero = all == -INFINITY ? 0.0f : all;
      if constexpr (I8)
#pragma unroll
        for (int s = 0; s < 4; ++s) unit = fmaxf(unit, sh_unit[s][lane]);
      sum = 0.0f;
      z[0] = kZero;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float f = exp2_fast(sh_st[s][lane].x - zero);
        sum += sh_st[s][lane].y * f;
        if constexpr (I8) f *= exp2_fast(sh_unit[s][lane] - unit);
        z[0] += sh_z[s][lane] * f;
      }
      store(at, e, all, sum, unit, z);
    }
    __syncthreads();
  }
}

template <int DT, int D>
void chunk_requests(const ChunkArgs &a, const ChunkGrid &g, hipStream_t stream) {
  const bool halves =
      a.c.page_shift >= 4 && a.c.token_stride * Operand<DT>::kBytes < ((int64_t)1 << 27);
  if (a.R <= 64 && halves)
    chunk_kernel<DT, D, true, true><<<g.groups, threads_of(D), 0, stream>>>(a, g);
  else if (halves)
    chunk_kernel<DT, D, false, true><<<g.groups, threads_of(D), 0, stream>>>(a, g);
  else
    chunk_kernel<DT, D, false, false><<<g.groups, threads_of(D), 0, stream>>>(a, g);
  if (g.groups > 1)   // (else nothing is cut)
    join_kernel<D, DT == BITNET_KV_INT8><<<dim3(2 * g.groups, kHelpers), 256, 0, stream>>>(a, g);
}

template <int DT>
void chunk_type(const ChunkArgs &a, int D, hipStream_t stream) {
  const ChunkPlan p = chunk_plan(a.T, a.R, a.q_heads, a.c.kv_heads, D, a.max_len);
  ChunkGrid g;
  g.outs_off = (int64_t)p.outs;
  g.stats_off = (int64_t)p.stats;
  g.units_off = (int64_t)p.units;
  g.groups = p.groups;
  g.per = a.q_heads / a.c.kv_heads;
  g.over_groups = 1.0 / g.groups;
  g.over_unit = 1.0 / ((double)g.per * kBlock * split_of(D));
  if (D == 64)
    chunk_requests<DT, 64>(a, g, stream);
  else if (D == 128)
    chunk_requests<DT, 128>(a, g, stream);
  else
    chunk_requests<DT, 256>(a, g, stream);
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
