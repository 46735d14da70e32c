// quantize_dispatch.cu - the MXFP8 operands of the experts' GEMMs straight from the tokens' rows.
//
// Segment row r holds token entry_of[r] / top_k's row, times that entry's weight if there are
// weights (an FP32 product, rounded to BF16), or zeros where there is no entry. Its row-wise copy
// (blocks of 32 along the columns) and its column-wise copy (blocks of 32 along the rows,
// transposed) are the bytes of the grouped quantizer on the dispatched BF16 rows, which are never
// written: that saves a write of 2 bytes and a read of 2 for each element. Format and layouts as
// in quantize.cu.
//
// The row copy goes by tokens, because what a token's row becomes row-wise does not depend on the
// expert: a warp reads a part of a row, converts it once and sends the codes to all of the token's
// rows. The column copy's blocks mix the tokens of a segment, so it goes by half tiles of the
// segments, whose rows come out of L2 for all but a token's first expert. Both copies together go
// so, side by side or in turn. CTAs are persistent and derive the segments from the offsets once.
//
// 8192 tokens of 2048 columns, 8 of 128 experts each (69504 rows): row copy 32 us, column copy 45,
// both 75 (with weights 56, 60 and 111; that instance spills 80 bytes at its 64 registers, which
// the row and the column copy share). What bounds them: the row copy the rate at which an SM
// sends bulk copies away (22 bytes a clock) and the scattered scale words (6 us); the column copy
// 268 MB read from L2 (27 us of it), the ALU pipe and the L1 path, each busy half of the time, and
// two barriers a tile. What counted most: results leave by lines that L2 evicts first, so that the
// tokens' rows stay in it (column copy 58 us without, 50 with), and loads in flight need the L1 cache, so
// that tables are sized by the experts and a CTA holds one stage buffer (87 us with two buffers of
// 52 KB a CTA). One read of a tile for both copies, as the grouped quantizer makes them, took 105
// us.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "convert.cuh"
#include "device.cuh"
#include "internal.h"
#include "mxfp8.h"
#include "segments.cuh"

namespace mxfp8 {
namespace {

constexpr int kTile = 128;
constexpr int kHalf = 64;   // columns that a CTA takes at a time for the column copy
constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kCtasPerSm = 8;
constexpr int kPiece = 512;   // columns a warp converts at once, 16 a lane
constexpr int kZeros = 512;   // bytes of zeros that padding rows are copied from
constexpr unsigned kFull = 0xFFFFFFFFu;

struct Params {
  const uint16_t* src;       // [tokens][cols]
  const float* weights;      // [tokens][k], or nullptr
  const int32_t* row_of;     // [tokens][k]
  const int32_t* entry_of;   // [rows]
  const int32_t* offsets;
  int64_t tokens, entries, rows, cols;
  uint32_t k;
  int E;
  uint8_t* row_codes;
  uint8_t* row_scales;
  uint8_t* col_codes;
  uint8_t* col_scales;
  int64_t col_tiles, row_tiles;     // 128 x 128 tiles; row_tiles: the most that segments have
  uint32_t parts, part_cols;        // of a token's row: how many, and their columns
  uint32_t token_units;             // tokens * parts
  uint32_t pad_cols, pad_units;     // of a padding unit, and how many units
  uint32_t col_ctas;                // that make the column copy
  int* status;
};

struct RowStage {   // of a warp
  __align__(16) uint8_t codes[4 * kPiece];
  uint32_t words[4 * kPiece / kTile];
};

struct RowShared {
  RowStage row[kWarps];
  __align__(16) uint8_t zeros[kZeros];
};

struct TileShared {
  __align__(16) uint8_t stage[kHalf * kTile];   // transposed codes of a half tile
  __align__(16) uint8_t scales[256];             // and its half of the scale tile
};

constexpr size_t kBuffers =
    sizeof(RowShared) > sizeof(TileShared) ? sizeof(RowShared) : sizeof(TileShared);

__device__ __forceinline__ uint32_t block_max(const uint32_t (&w)[8]) {
  return max_abs_bf16x2(
      max_abs_bf16x2(max_abs_bf16x2(w[0], w[1]), max_abs_bf16x2(w[2], w[3])),
      max_abs_bf16x2(max_abs_bf16x2(w[4], w[5]), max_abs_bf16x2(w[6], w[7])));
}

// Two BF16 values times a weight, each product rounded to FP32 and then to BF16.
__device__ __forceinline__ uint32_t weigh(uint32_t x, float w) {
  return cvt_bf16x2(__fmul_rn(__uint_as_float(x & 0xFFFF0000u), w),
                    __fmul_rn(__uint_as_float(x << 16), w));
}

// The scale bytes of the four blocks of a lane's eight lanes in one word, from each lane's own (zero
// past the columns).
__device__ __forceinline__ uint32_t scale_word_of(uint32_t s, bool valid) {
  uint32_t word = valid ? s << (8 * ((threadIdx.x >> 1) & 3)) : 0u;
  word |= __shfl_xor_sync(kFull, word, 2);
  return word | __shfl_xor_sync(kFull, word, 4);
}

// Magnitude of the largest of a block's values, two lanes' 16 each, as BF16 bits.
__device__ __forceinline__ uint32_t row_block_max(const uint32_t (&w)[8]) {
  uint32_t m2 = block_max(w);
  m2 = max_abs_bf16x2(m2, __shfl_xor_sync(kFull, m2, 1)) & kAbs2;
  return max(m2 & 0xFFFFu, m2 >> 16);
}

// 16 columns a lane of a block with scale byte s: the lane's codes.
__device__ __forceinline__ uint4 convert_piece(const uint32_t (&w)[8], uint32_t s) {
  if (__builtin_expect(s != 0xFFu, 1)) {
    const uint32_t mul2 = inv_scale_bf16(s) * 0x10001u;
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) scale_bf16x2(w[i], mul2, f[2 * i], f[2 * i + 1]);
    return make_uint4(e4m3x4_f32(f[0], f[1], f[2], f[3]), e4m3x4_f32(f[4], f[5], f[6], f[7]),
                      e4m3x4_f32(f[8], f[9], f[10], f[11]),
                      e4m3x4_f32(f[12], f[13], f[14], f[15]));
  }
  return make_uint4(nan4(w[0], w[1]), nan4(w[2], w[3]), nan4(w[4], w[5]), nan4(w[6], w[7]));
}

// The same of a block times a weight. Rounding is monotone, so the products' largest magnitude is
// that of x, `amax`, times the weight's, rounded like them: it is found once for all weights.
// The power of two of the block's scale goes into the weight: products and their roundings to FP32
// and BF16 are the same times that power, as long as neither the scaled weight nor a product that a
// code other than 0 comes from leaves the normal numbers. Codes of 2^-10 and more of the scale are
// normal BF16 products from scale byte 11 on, and the scaled weight is about 2^8 / amax, finite
// where amax has an exponent field of 10 or more. Found anew for each weight, maximum and scale
// included, the row copy takes 7% longer.
__device__ __forceinline__ uint4 weigh_piece(const uint32_t (&x)[8], uint32_t amax, float w,
                                             uint32_t& s) {
  const uint32_t top = cvt_bf16x2(0.f, __fmul_rn(__uint_as_float(amax << 16), fabsf(w)));
  s = scale_byte(top & 0x7FFFu, MXFP8_RULE_FLOOR);
  uint32_t y[8];
  if (__builtin_expect(s >= 12 && s != 0xFFu && amax >= 10u << 7, 1)) {
    const float sw = __fmul_rn(w, inv_scale(s));
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = weigh(x[2 * i], sw), b = weigh(x[2 * i + 1], sw);
      o[i] = e4m3x4_f32(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u),
                        __uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = weigh(x[i], w);
  return convert_piece(y, s);
}

// Row copy. A warp takes a part of a token's row: it converts it once (once for each weight, with
// weights) into shared memory, from where one bulk copy a segment row takes the codes away; the
// lane that has the row issues it and writes the row's scale words. Without weights a part is
// up to 2048 columns, in one buffer; with them up to 1024, in two buffers in turn.
template <bool kWeighted>
__device__ __forceinline__ void token_unit(const Params& p, const SegmentView& seg, RowStage& st,
                                           uint32_t u, int& buf) {
  constexpr int kPieces = kWeighted ? 2 : 4;
  constexpr int kPart = kPieces * kPiece;
  const int lane = threadIdx.x & 31;
  const uint32_t t = u / p.parts;
  const int64_t c0 = static_cast<int64_t>(u - t * p.parts) * p.part_cols;
  const int cols = static_cast<int>(p.cols - c0 < p.part_cols ? p.cols - c0 : p.part_cols);
  const uint16_t* x = p.src + t * p.cols + c0 + 16 * lane;
  uint32_t v[kPieces][8];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (kPiece * i + 16 * lane < cols) {   // cols % 32 == 0
      const uint4 a = ld_nc_v4(x + kPiece * i), b = ld_nc_v4(x + kPiece * i + 8);
      v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
      v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
    } else {
#pragma unroll
      for (int h = 0; h < 8; ++h) v[i][h] = 0;
    }
  }
  uint32_t amax[kPieces];
  if constexpr (kWeighted) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) amax[i] = row_block_max(v[i]);
  }
  const auto convert = [&](float w, uint32_t* scales_to) {
    if (kWeighted) {
      buf ^= 1;
      bulk_wait_read_but_one();
    } else {
      bulk_wait_read_all();
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (kPiece * i >= cols) break;
      const int c = kPiece * i + 16 * lane;
      uint32_t scale;
      uint4 o;
      if constexpr (kWeighted) {
        o = weigh_piece(v[i], amax[i], w, scale);
      } else {
        scale = scale_byte(row_block_max(v[i]), MXFP8_RULE_FLOOR);
        o = convert_piece(v[i], scale);
      }
      const uint32_t word = scale_word_of(scale, c < cols);
      if (c < cols) *reinterpret_cast<uint4*>(st.codes + buf * kPart + c) = o;
      if constexpr (kWeighted) {
        if ((lane & 7) == 0 && c < cols) scales_to[c] = word;
      } else {
        if ((lane & 7) == 0) st.words[c / kTile] = word;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
  };
  const auto store = [&](int32_t row) {
    bulk_store(p.row_codes + row * p.cols + c0, st.codes + buf * kPart,
               static_cast<uint32_t>(cols), evict_first_policy());
  };
  uint32_t* scale_words = reinterpret_cast<uint32_t*>(p.row_scales) + c0;  // 128 a tile
  if (!kWeighted) convert(1.f, nullptr);
  for (uint32_t j0 = 0; j0 < p.k; j0 += 32) {
    int32_t row = -1;
    float w = 1.f;
    int64_t scales = 0;   // the row's first scale word
    if (lane < p.k - j0) {
      const int64_t entry = static_cast<int64_t>(t) * p.k + j0 + lane;
      row = p.row_of[entry];
      if (row >= p.rows) {   // a plan of other sizes
        latch_error(p.status, MXFP8_ERR_BAD_OFFSETS);
        row = -1;
      }
      if (row >= 0) {
        if (kWeighted) w = p.weights[entry];
        int lo = 0, hi = p.E - 1;   // the last expert that starts at or before the row
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (seg.off[mid] <= row) lo = mid; else hi = mid - 1;
        }
        const int local = row - seg.off[lo];
        scales = (seg.tile_base[lo] + (local >> 7)) * p.col_tiles * kTile + (local & 31) * 4 +
                 ((local & 127) >> 5);
      }
    }
    if constexpr (kWeighted) {
      for (unsigned live = __ballot_sync(kFull, row >= 0); live; live &= live - 1) {
        const int j = __ffs(live) - 1;
        convert(__shfl_sync(kFull, w, j), scale_words + __shfl_sync(kFull, scales, j));
        if (lane == j) store(row);
        bulk_commit_group();
      }
    } else {
      if (row >= 0) {
        store(row);
        for (int c = 0; c < cols; c += kTile) scale_words[scales + c] = st.words[c / kTile];
      }
    }
  }
  if (!kWeighted) bulk_commit_group();
}

// The place of global tile row `tile_row` in the segments.
struct TileRow {
  int64_t row0;        // its first row
  int rows;            // of the segment in it
  int64_t index, seg_tiles, seg_base;
};

__device__ __forceinline__ TileRow tile_row_of(const SegmentView& seg, int E, int tile_row) {
  const int e = find_expert(seg, E, tile_row);
  TileRow q;
  q.seg_base = seg.tile_base[e];
  q.index = tile_row - q.seg_base;
  const int64_t count = seg.off[e + 1] - seg.off[e];
  q.row0 = seg.off[e] + q.index * kTile;
  const int64_t left = count - q.index * kTile;
  q.rows = static_cast<int>(left < kTile ? left : kTile);
  q.seg_tiles = (count + kTile - 1) / kTile;
  return q;
}

// Row copy of rows without an entry: zero codes, and zero bytes in the scale tiles, past the
// segments' ends too. A warp takes a part of 32 rows of a tile row; the lane of a row issues its
// copies from a block of zeros.
__device__ __forceinline__ void pad_unit(const Params& p, const SegmentView& seg,
                                         const uint8_t* zeros, uint32_t u) {
  const int lane = threadIdx.x & 31;
  const uint32_t quarters = static_cast<uint32_t>(p.row_tiles) * 4, part = u / quarters;
  u -= part * quarters;
  const int64_t c0 = static_cast<int64_t>(part) * p.pad_cols;
  const int64_t c1 = c0 + p.pad_cols < p.cols ? c0 + p.pad_cols : p.cols;
  const int64_t tiles = (c1 - c0 + kTile - 1) / kTile;
  const int tile_row = static_cast<int>(u >> 2), r = 32 * (u & 3) + lane;
  uint8_t* scales = p.row_scales + (tile_row * p.col_tiles + c0 / kTile) * 512;
  if (tile_row >= seg.tile_base[p.E]) {   // no segment's: a quarter of its tiles
    uint4* quarter = reinterpret_cast<uint4*>(scales) + (u & 3) * tiles * 8;
    for (int64_t i = lane; i < tiles * 8; i += 32) quarter[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const TileRow q = tile_row_of(seg, p.E, tile_row);
  const int64_t row = q.row0 + r;
  if (r < q.rows && p.entry_of[row] >= 0) return;
  uint32_t* word = reinterpret_cast<uint32_t*>(scales) + (r & 31) * 4 + (r >> 5);
  for (int64_t i = 0; i < tiles; ++i) word[i * kTile] = 0;
  if (r >= q.rows) return;
  for (int64_t c = c0; c < c1; c += kZeros)
    bulk_store(p.row_codes + row * p.cols + c, zeros,
               static_cast<uint32_t>(c1 - c < kZeros ? c1 - c : kZeros), evict_first_policy());
}

// Column copy of a run of half tiles, 128 rows x 64 columns, beside one another: with half a tile and
// four warps between two barriers it takes 45 us, with a whole one and eight 50. A thread holds 8 consecutive rows
// of 8 columns; the four lanes that hold a block's 32 rows share its maximum. The conversion takes
// two values at once, here from two rows, which leaves a column's 8 codes in 8 consecutive bytes.
// They pass through shared memory (8-byte units, their index XORed with twice the column's
// eighth, so that both the writes and the reads of 16 bytes are free of bank conflicts) and leave
// as rows of 128 bytes; the next tile's loads are in flight meanwhile. A warp that keeps 16 rows of
// 4 columns a thread needs neither the stage nor a barrier, but its stores of 32 bytes took 77 us.
struct Patch {
  uint32_t x[8][4];
};

// A thread's rows: their places in x in units of 8 values (tokens * cols is below 2^35), and
// which of them there are.
struct PatchRows {
  uint32_t at[8];
  uint32_t there;
  bool all;      // of the warp's rows
};

__device__ __forceinline__ void load_patch(const Params& p, const PatchRows& rows, int64_t col,
                                           Patch& t) {
  const uint16_t* x = p.src + col;
  if (rows.all && col < p.cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = ld_nc_v4(x + static_cast<uint64_t>(rows.at[i]) * 8);
      t.x[i][0] = v.x;
      t.x[i][1] = v.y;
      t.x[i][2] = v.z;
      t.x[i][3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = (rows.there >> i & 1) && col < p.cols
                          ? ld_nc_v4(x + static_cast<uint64_t>(rows.at[i]) * 8)
                          : make_uint4(0, 0, 0, 0);
      t.x[i][0] = v.x;
      t.x[i][1] = v.y;
      t.x[i][2] = v.z;
      t.x[i][3] = v.w;
    }
  }
}

// Eight codes of each of two columns (low and high halves) of eight rows, scaled by mul's halves.
__device__ __forceinline__ void convert_pair(const Patch& t, int h, uint32_t mul, uint2& o0,
                                             uint2& o1) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = mul_bf16x2(t.x[i][h], mul);
  const auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  const auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  o0.x = e4m3x4_f32(lo(b[0]), lo(b[1]), lo(b[2]), lo(b[3]));
  o0.y = e4m3x4_f32(lo(b[4]), lo(b[5]), lo(b[6]), lo(b[7]));
  o1.x = e4m3x4_f32(hi(b[0]), hi(b[1]), hi(b[2]), hi(b[3]));
  o1.y = e4m3x4_f32(hi(b[4]), hi(b[5]), hi(b[6]), hi(b[7]));
}

// The same where a block of the two columns holds a NaN or an infinity (scale byte 0xFF).
__device__ __forceinline__ void convert_pair_nan(const Patch& t, int h, uint32_t s0,
                                                 uint32_t s1, uint2& o0, uint2& o1) {
  const float mul0 = inv_scale(s0), mul1 = inv_scale(s1);
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = __byte_perm(t.x[2 * i][h], t.x[2 * i + 1][h], 0x5410);
    hi[i] = __byte_perm(t.x[2 * i][h], t.x[2 * i + 1][h], 0x7632);
  }
  o0.x = s0 == 0xFFu ? nan4(lo[0], lo[1]) : e4m3x4(lo[0], lo[1], mul0);
  o0.y = s0 == 0xFFu ? nan4(lo[2], lo[3]) : e4m3x4(lo[2], lo[3], mul0);
  o1.x = s1 == 0xFFu ? nan4(hi[0], hi[1]) : e4m3x4(hi[0], hi[1], mul1);
  o1.y = s1 == 0xFFu ? nan4(hi[2], hi[3]) : e4m3x4(hi[2], hi[3], mul1);
}

template <bool kWeighted>
__device__ __forceinline__ void tile_run(const Params& p, const SegmentView& seg, TileShared& sh,
                                         int tile_row, int64_t bx0, int64_t bx1) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int block = warp, sub = lane >> 3, vec = lane & 7;
  const int c = 8 * vec;   // the thread's first column of a half tile
  const TileRow q = tile_row_of(seg, p.E, tile_row);
  const bool rows_ok = 32 * block < q.rows;  // segments are multiples of 32 rows
  uint32_t token = 0;
  float weight = 0.f;
  int32_t entry = rows_ok ? p.entry_of[q.row0 + 32 * block + lane] : -1;
  if (entry >= p.entries) {   // a plan of other sizes
    latch_error(p.status, MXFP8_ERR_BAD_OFFSETS);
    entry = -1;
  }
  if (entry >= 0) {
    token = static_cast<uint32_t>(entry) / p.k;
    if (kWeighted) weight = p.weights[entry];
  }
  PatchRows rows;
  const uint32_t row_units = static_cast<uint32_t>(p.cols / 8);
  const unsigned there = __ballot_sync(kFull, entry >= 0);
  rows.all = there == kFull;
  rows.there = (there >> (8 * sub)) & 0xFFu;
#pragma unroll
  for (int i = 0; i < 8; ++i) rows.at[i] = __shfl_sync(kFull, token, 8 * sub + i) * row_units;

  Patch t;
  if (rows_ok) load_patch(p, rows, bx0 * kHalf + c, t);
  const int out_row = tid >> 3, chunk = tid & 7;   // a column of the tile, 16 rows of it
  uint8_t* out = p.col_codes + (bx0 * kHalf + out_row) * p.rows + q.row0 + 16 * chunk;
  const int64_t tile0 = p.col_tiles * q.seg_base + q.index, rows16 = 16 * p.rows;
  for (int64_t bx = bx0; bx < bx1; ++bx) {
    const int64_t col0 = bx * kHalf;   // may pass the last column: half of a tile's scales
    const int cols = static_cast<int>(p.cols - col0 < kHalf ? p.cols - col0 : kHalf);
    if (kWeighted && rows_ok) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = __shfl_sync(kFull, weight, 8 * sub + i);
#pragma unroll
        for (int h = 0; h < 4; ++h) t.x[i][h] = weigh(t.x[i][h], w);
      }
    }
    uint32_t exps[4], worst = 0;
    if (rows_ok) {
      // Of two columns at once: the exponent fields of the block maxima, and from them the scale
      // bytes max(E - 8, 0) and the BF16 factors 2^(127 - byte), in place at bit 7 of each half.
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t m2 = max_abs_bf16x2(
            max_abs_bf16x2(max_abs_bf16x2(t.x[0][h], t.x[1][h]),
                           max_abs_bf16x2(t.x[2][h], t.x[3][h])),
            max_abs_bf16x2(max_abs_bf16x2(t.x[4][h], t.x[5][h]),
                           max_abs_bf16x2(t.x[6][h], t.x[7][h])));
        m2 = max_abs_bf16x2(m2, __shfl_xor_sync(kFull, m2, 8));
        m2 = max_abs_bf16x2(m2, __shfl_xor_sync(kFull, m2, 16));
        exps[h] = max_u16x2(m2 & 0x7F807F80u, 0x04000400u);
        worst = max_u16x2(worst, exps[h]);
      }
    }
    __syncthreads();   // the tile before has left the stage
    const int a = c + 2 * sub;   // each of the four lanes writes the scale bytes of a column pair
    uint8_t* scale_to = sh.scales + (a & 31) * 8 + (a >> 5) * 4 + block;
    if (rows_ok) {
      const bool finite = worst < 0x7F800000u && (worst & 0xFFFFu) < 0x7F80u;
      uint8_t* stage = sh.stage + c * kTile + 8 * ((4 * block + sub) ^ (2 * vec));
      // columns past the last are zeros, whose scale byte is 0 as it should be, unless a weight that
      // is no number has made them NaN
      uint32_t e = (sub & 2 ? (sub & 1 ? exps[3] : exps[2]) : (sub & 1 ? exps[1] : exps[0])) -
                   0x04000400u;
      if (kWeighted && c >= cols) e = 0;
      if (__builtin_expect(finite, 1)) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {   // columns c + 2h (low halves) and c + 2h + 1
          uint2 o0, o1;
          convert_pair(t, h, 0x83008300u - exps[h], o0, o1);
          *reinterpret_cast<uint2*>(stage + 2 * h * kTile) = o0;
          *reinterpret_cast<uint2*>(stage + (2 * h + 1) * kTile) = o1;
        }
        scale_to[0] = static_cast<uint8_t>(e >> 7);
        scale_to[8] = static_cast<uint8_t>(e >> 23);
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t e0 = (exps[h] >> 7) & 0xFFu, e1 = exps[h] >> 23;
          uint2 o0, o1;
          convert_pair_nan(t, h, e0 == 0xFFu ? 0xFFu : e0 - 8, e1 == 0xFFu ? 0xFFu : e1 - 8, o0,
                           o1);
          *reinterpret_cast<uint2*>(stage + 2 * h * kTile) = o0;
          *reinterpret_cast<uint2*>(stage + (2 * h + 1) * kTile) = o1;
        }
        scale_to[0] = static_cast<uint8_t>((e >> 7 & 0xFFu) == 0xF7u ? 0xFFu : e >> 7);
        scale_to[8] = static_cast<uint8_t>(e >> 23 == 0xF7u ? 0xFFu : e >> 23);
      }
    } else {
      scale_to[0] = scale_to[8] = 0;
    }
    if (rows_ok && bx + 1 < bx1) load_patch(p, rows, col0 + kHalf + c, t);
    __syncthreads();
    if (16 * chunk < q.rows) {
      const uint8_t* from = sh.stage + out_row * kTile;
      uint8_t* to = out;
#pragma unroll
      for (int i = 0; i < 4; ++i, to += rows16) {
        if (out_row + 16 * i < cols)
          __stcs(reinterpret_cast<uint4*>(to),   // 50 us, 58 with stores that stay in L2
                 *reinterpret_cast<const uint4*>(
                     from + 16 * i * kTile + 16 * (chunk ^ (((out_row >> 3) + 2 * i) & 7))));
      }
    }
    out += 4 * rows16;
    if (tid < 32)
      *reinterpret_cast<uint2*>(p.col_scales + (tile0 + (bx >> 1) * q.seg_tiles) * 512 + 16 * tid +
                                8 * (bx & 1)) = reinterpret_cast<const uint2*>(sh.scales)[tid];
  }
}

// The first col_ctas CTAs make the column copy, the others the row copy: either alone, or both side
// by side, as the row copy waits for its writes and the column copy for its reads.
template <bool kWeighted>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) quantize_dispatch_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  SegmentView seg(reinterpret_cast<int32_t*>(dyn + kBuffers), p.E);
  grid_dependency_wait();
  grid_launch_dependents();
  load_segments<kThreads>(seg, p.offsets, p.E, p.rows, p.status);   // ends in a barrier
  if (!seg.ok) return;
  if (blockIdx.x < p.col_ctas) {
    TileShared& sh = *reinterpret_cast<TileShared*>(dyn);
    // Items of up to 8 half tiles beside one another, all rows of a part of the columns before the
    // next part, so that the CTAs read the same columns of the tokens at a time and find them in
    // L2 (with whole tiles and 16384 tokens of 7168 columns: 342 us, 564 with a contiguous share a
    // CTA). What does not fill a last round of the CTAs is cut into as many pieces as do.
    const uint32_t ctas = p.col_ctas, rows = seg.tile_base[p.E];
    const uint32_t halves = 2 * static_cast<uint32_t>(p.col_tiles), all = rows * halves;
    uint32_t run = all / ctas;   // at half of it 37 x 8 x 2048: 14 us, 12.8 so
    run = run < 1 ? 1 : run > 8 ? 8 : run;
    const uint32_t parts = (halves + run - 1) / run;
    run = (halves + parts - 1) / parts;
    const uint32_t items = rows * parts;
    const uint32_t rest = items % ctas, whole = items - rest;
    uint32_t pieces = rest ? ctas / rest : 1;
    if (pieces > run) pieces = run;
    const uint32_t step = (run + pieces - 1) / pieces;
    for (uint32_t i = blockIdx.x; i < whole + rest * pieces; i += ctas) {
      uint32_t item = i, from = 0, to = run;
      if (i >= whole) {
        const uint32_t piece = (i - whole) / rest;
        item = i - piece * rest;
        from = piece * step;
        to = from + step < run ? from + step : run;
      }
      const uint32_t part = item / rows;
      from += part * run;
      to += part * run;
      if (to > halves) to = halves;
      if (from < to) tile_run<kWeighted>(p, seg, sh, item - part * rows, from, to);
    }
    // the scales past the segments' tiles
    uint4* tail = reinterpret_cast<uint4*>(p.col_scales) + int64_t{all} * 16;
    const uint64_t n = (p.row_tiles * p.col_tiles * 2 - all) * 16;
    for (uint64_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += p.col_ctas * kThreads)
      tail[i] = make_uint4(0, 0, 0, 0);
  } else {
    RowShared& sh = *reinterpret_cast<RowShared*>(dyn);
    static_assert(kZeros == 4 * kThreads, "one store a thread");
    reinterpret_cast<uint32_t*>(sh.zeros)[threadIdx.x] = 0;
    fence_proxy_async_smem();
    __syncthreads();
    // Neighbouring units go to different SMs: the padding that the last segment takes is one run,
    // and an SM sends copies away at 22 bytes a clock at most.
    const int warp = threadIdx.x >> 5;
    const uint32_t ctas = gridDim.x - p.col_ctas;
    const uint32_t units = p.token_units + p.pad_units;   // each below 2^31
    int buf = 0;
    for (uint32_t u = warp * ctas + blockIdx.x - p.col_ctas; u < units; u += ctas * kWarps) {
      if (u < p.token_units) {
        token_unit<kWeighted>(p, seg, sh.row[warp], u, buf);
      } else {
        pad_unit(p, seg, sh.zeros, u - p.token_units);
        __syncwarp();
        bulk_commit_group();
      }
    }
    bulk_wait_read_all();
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

static_assert(kBuffers + sizeof(int32_t) * SegmentView::words(kMaxExperts) <= 48 * 1024,
              "no leave needed for the shared memory");

cudaError_t launch(void (*k)(const Params), int64_t wanted, size_t dyn, const Params& p,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(wanted), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = dyn;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  cfg.numAttrs = pdl_attr(&attr[0]);
  return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace

cudaError_t launch_quantize_dispatch(const QuantizeDispatchArgs& a, cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return cudaSuccess;
  Params p{};
  p.src = static_cast<const uint16_t*>(a.src);
  p.weights = a.weights;
  p.row_of = a.row_of;
  p.entry_of = a.entry_of;
  p.offsets = a.offsets;
  p.tokens = a.tokens;
  p.entries = a.tokens * a.top_k;
  p.rows = a.rows;
  p.cols = a.cols;
  p.k = static_cast<uint32_t>(a.top_k);
  p.E = a.num_experts;
  p.row_codes = static_cast<uint8_t*>(a.row_out);
  p.row_scales = static_cast<uint8_t*>(a.row_scales);
  p.col_codes = static_cast<uint8_t*>(a.col_out);
  p.col_scales = static_cast<uint8_t*>(a.col_scales);
  p.col_tiles = cdiv(a.cols, kTile);
  p.row_tiles = cdiv(a.rows, kTile) + a.num_experts;
  p.status = a.status;
  const int64_t most = int64_t{kCtasPerSm} * num_sms();   // CTAs
  const size_t table = sizeof(int32_t) * SegmentView::words(p.E);
  auto k = a.weights ? quantize_dispatch_kernel<true> : quantize_dispatch_kernel<false>;
  int64_t row_ctas = 0, col_ctas = 0;
  if (a.row_out) {
    // parts of a row as long as the buffers take, while each warp keeps a unit
    p.part_cols = (a.weights ? 2 : 4) * kPiece;
    while (p.part_cols > kPiece && a.tokens * cdiv(a.cols, p.part_cols) < most * kWarps)
      p.part_cols /= 2;
    const int64_t parts = cdiv(a.cols, p.part_cols), units = a.tokens * parts;
    // The same of padding, whose rows wait for nothing: 8 tokens of 4096 columns, 2 of 8 experts
    // each, 10.3 to 3.9 us (37 of 2048 columns, 8 of 128: 7.4 to 5.8; 8192: 33.5 to 32.0).
    p.pad_cols = 4 * kPiece;
    while (p.pad_cols > kPiece && 4 * p.row_tiles * cdiv(a.cols, p.pad_cols) < most * kWarps)
      p.pad_cols /= 2;
    const int64_t pads = 4 * p.row_tiles * cdiv(a.cols, p.pad_cols);
    if (units > 0x7FFFFFFF || pads > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.parts = static_cast<uint32_t>(parts);
    p.token_units = static_cast<uint32_t>(units);
    p.pad_units = static_cast<uint32_t>(pads);
    row_ctas = std::min(most, cdiv(units + pads, kWarps));
  }
  if (a.col_out) {
    if (p.row_tiles * p.col_tiles * 2 > 0x7FFFFFFF) return cudaErrorInvalidValue;
    col_ctas = std::min(most, p.row_tiles * p.col_tiles * 2);
  }
  const size_t dyn = kBuffers + table;
  // Both copies side by side, in shares of the CTAs after what each copy costs: ns for 1024
  // values, fitted to each alone (a token converts once, with weights once an expert, and goes out
  // once an expert; a segment's last tile costs as much as a full one). Shares go by eighths, so
  // that the SMs hold like mixtures: a share of 28% in place of 25 or 37 costs up to 7%. Where
  // there is much to do, the copies go in turn: the second launch counts for little there, and each
  // copy has L2 to itself. The rule goes by the values to be written; the size of the tokens' rows,
  // which is what L2 holds, does not tell the better way either (1024 tokens of 64 experts). Times, us,
  // side by side and in turn (tokens x experts of each x columns): 37 x 8 x 2048: 12, 18; 4096 x 8 x
  // 2048: 44, 48; 8192 x 8 x 2048: 76, 82; 16384 x 2 x 7168: 197, 196; 16384 x 1 x 8192: 149, 155;
  // 16384 x 8 x 2048: 157, 156; 16384 x 4 x 4096: 166, 171; 16384 x 1 x 16352: 326, 330; 1024 x 64 x
  // 4096: 132, 144; 1024 x 64 x 8192: 303, 290; 32768 x 1 x 8192: 304, 294; 16384 x 8 x 7168: 740, 607.
  // With weights 4096 x 8 x 2048: 64, 66; 8192 x 8 x 2048: 112, 116; 16384 x 1 x 8192: 205, 196; 16384
  // x 4 x 4096: 233, 229. Over 48 such sizes the rule's way is the slower one by 9% at most.
  if (a.row_out && a.col_out) {
    if (p.entries * a.cols < int64_t{1} << 28) {
      const double x = static_cast<double>(a.tokens);
      const double y = static_cast<double>(std::min(p.entries, a.rows));
      const double pad = static_cast<double>(a.rows) - y;
      const double row = (a.weights ? 0.58 * x + 0.38 * y : 0.37 * x + 0.21 * y) + 0.12 * pad;
      const double col = 0.32 * x + (a.weights ? 0.33 : 0.25) * (a.rows + 0.5 * kTile * p.E);
      const int64_t eighths = std::clamp<int64_t>(std::llround(8 * row / (row + col)), 2, 6);
      row_ctas = std::min(row_ctas, most * eighths / 8);
      col_ctas = std::min(col_ctas, most - row_ctas);
    } else {
      const cudaError_t e = launch(k, row_ctas, dyn, p, stream);
      if (e != cudaSuccess) return e;
      row_ctas = 0;
    }
  }
  p.col_ctas = static_cast<uint32_t>(col_ctas);
  return launch(k, col_ctas + row_ctas, dyn, p, stream);
}

}  // namespace mxfp8
