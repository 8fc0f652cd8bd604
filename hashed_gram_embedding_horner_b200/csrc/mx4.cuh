// Microscaled 4-bit floating point (MXFP4 of the OCP Microscaling Formats specification,
// v1.0): quantisation, the row gather of the layer's 4-bit sub-tables, and the product.
//
// A row of C elements (C % 32 == 0) is C / 2 bytes of E2M1 codes (element 2j in the low half
// of byte j; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit) and C / 32 bytes of E8M0
// scales (2^(e - 127); 255 is NaN), one for each block of 32 elements. Scales lie either by
// rows ([R x C / 32], the layout of a table whose rows are gathered) or in tiles, the layout
// the tensor cores take them in: 512 bytes for 128 rows x 4 blocks, the byte of row r and
// block b at (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4 of tile (r / 128, b / 4), tiles
// row-block by row-block, the blocks of one row block next to one another.
#pragma once

#include "common.cuh"
#include "hash.cuh"

namespace ngram {

constexpr int kMxBlock = 32;       // elements under one scale
constexpr int kMxTileBytes = 512;  // 128 rows x 4 scales

// Bytes of the tile of scale (row r, block b), with kt = ceil(C / 128) tiles a row block.
__device__ __forceinline__ size_t mx4_tile_at(int64_t r, int b, int kt) {
  return (static_cast<size_t>(r >> 7) * kt + (b >> 2)) * kMxTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// q = x / d for x < 2^32 by one 64-bit multiplication: m = ceil(2^(32 + s) / d), s = ceil(log2 d)
// (Granlund and Montgomery, PLDI 1994: exact for every 32-bit x; m takes 33 bits, its top bit
// is the added x).
struct FastDiv {
  uint32_t d, m, s;
  __host__ void set(uint32_t div) {
    d = div;
    s = 0;
    while ((uint64_t(1) << s) < div) ++s;
    m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << s) - div)) / div + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t x) const {
    const uint64_t t = static_cast<uint64_t>(__umulhi(x, m)) + x;
    return static_cast<uint32_t>(t >> s);
  }
};

// ------------------------------------------------------------------ work on rows of vectors
//
// How the row-wise kernels (quantisation, lookup) spread rows of `per_row` vectors of eight
// elements over warps: a warp takes U vectors a lane along the columns of R = 4 / U rows (or
// groups of rows where a row is narrower than a warp: 2^lg lanes a row), so the division that
// finds its rows, the row addresses and the ids are paid once for four vectors a lane, and all
// of a lane's loads are in flight together.
struct RowMap {
  uint32_t rows, per_row;  // vectors of eight elements a row
  uint32_t lg;             // log2 of the lanes a row
  FastDiv by_segs;         // column segments of a row: 2^lg * U vectors each
  uint32_t items;          // warps
  __host__ void set(uint32_t r, uint32_t vecs, int U) {
    rows = r;
    per_row = vecs;
    lg = 0;
    while (lg < 5 && (1u << lg) < vecs) ++lg;
    const uint32_t segs = (vecs + (static_cast<uint32_t>(U) << lg) - 1) / (static_cast<uint32_t>(U) << lg);
    by_segs.set(segs);
    const uint32_t group = (32u >> lg) * static_cast<uint32_t>(4 / U);  // rows a warp
    items = (r + group - 1) / group * segs;
  }
  // Columns a lane: as many as rows of this width fill.
  __host__ static int unroll(uint32_t vecs) { return vecs >= 128 ? 4 : (vecs >= 64 ? 2 : 1); }
};

// A lane's part of its warp's item: rows row0 + r * row_step, r < 4 / U, and vectors vec + u *
// stride of each; either may lie past the last.
template <int U>
struct RowPart {
  static constexpr int R = 4 / U;
  uint32_t row0, row_step, vec, stride;
  bool live;  // the warp has work
  __device__ __forceinline__ explicit RowPart(const RowMap& m) {
    const uint32_t item = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    live = item < m.items;
    const uint32_t rg = m.by_segs.div(item), seg = item - rg * m.by_segs.d;
    row_step = 32u >> m.lg;
    row0 = rg * row_step * R + (lane >> m.lg);
    stride = 1u << m.lg;
    vec = seg * (stride * U) + (lane & (stride - 1));
  }
};

// ------------------------------------------------------------------ quantisation

// Two floats to one byte of E2M1 codes: round to nearest, ties to even, saturating at 6;
// the first in the low half.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

struct Mx4QuantParams {
  RowMap map;
  const void* src;     // [rows x cols], row stride src_stride elements
  int64_t src_stride;
  int64_t row0;        // first row of this launch (tiles)
  int cols, kt;        // kt = ceil(cols / 128)
  uint8_t* codes;      // of row 0 of this launch
  uint8_t* scales;     // rows: of row 0 of this launch; tiles: of row 0 of the array
  int tiles;           // 1: scales in tiles
};

// Eight elements of a row, as they lie; VEC: 16-byte loads.
template <typename T, bool VEC>
__device__ __forceinline__ void mx4_load8(const T* src, uint32_t (&w)[2 * sizeof(T)]) {
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) {
      const uint4 v = ld_stream_v4(reinterpret_cast<const uint8_t*>(src) + 16 * h);
      w[4 * h] = v.x;
      w[4 * h + 1] = v.y;
      w[4 * h + 2] = v.z;
      w[4 * h + 3] = v.w;
    }
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int h = 0; h < 4; ++h) w[h] = src[2 * h] | (static_cast<uint32_t>(src[2 * h + 1]) << 16);
  } else {
#pragma unroll
    for (int h = 0; h < 8; ++h) w[h] = __float_as_uint(src[h]);
  }
}

// The bits of the largest magnitude of eight elements, as fp32 (they order as the magnitudes
// do, infinities and NaN above every number).
template <typename T>
__device__ __forceinline__ uint32_t mx4_amax8(const uint32_t (&w)[2 * sizeof(T)]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h) m = __vmaxu2(m, w[h] & 0x7FFF7FFFu);
    return max(m << 16, m & 0xFFFF0000u);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 8; ++h) m = max(m, w[h] & 0x7FFFFFFFu);
    return m;
  }
}

// A block's scale byte: two below the exponent of its largest magnitude (the exponent of
// E2M1's largest power of two is 2), clamped to 2^-127; 0 for a block of zeros, 255 (NaN)
// for a block that holds an infinity or a NaN. `amax` as from mx4_amax8.
__device__ __forceinline__ int mx4_scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255;
  const int e = static_cast<int>(amax >> 23) - 2;  // subnormal magnitudes: below 2^-126, clamped
  return e < 0 ? 0 : e;
}
// 2^(127 - e), the factor that undoes scale byte e <= 252.
__device__ __forceinline__ float mx4_inverse(int e) { return __uint_as_float(static_cast<uint32_t>(254 - e) << 23); }

// Four lanes hold the 32 elements of a block, 8 each: the maximum by two shuffles, then one
// conversion instruction for two elements; every lane's 16- or 32-byte load and 4-byte store
// are part of a warp-wide contiguous access. One pass: 2 or 4 bytes read and 17/32 written an
// element, bound by HBM.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const __grid_constant__ Mx4QuantParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const RowPart<U> part(p.map);
  if (!part.live) return;
  constexpr int R = RowPart<U>::R;
  uint32_t w[R][U][2 * sizeof(T)];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t row = part.row0 + r * part.row_step;
    const T* src = static_cast<const T*>(p.src) + static_cast<int64_t>(row) * p.src_stride + part.vec * 8;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row < p.map.rows && part.vec + u * part.stride < p.map.per_row) {
        mx4_load8<T, VEC>(src + u * part.stride * 8, w[r][u]);
      } else {
#pragma unroll
        for (int h = 0; h < static_cast<int>(2 * sizeof(T)); ++h) w[r][u][h] = 0;
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t row = part.row0 + r * part.row_step;
    const int64_t at = static_cast<int64_t>(row) * p.map.per_row + part.vec;  // in vectors
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t vec = part.vec + u * part.stride;
      uint32_t amax = mx4_amax8<T>(w[r][u]);
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (row >= p.map.rows || vec >= p.map.per_row) continue;
      const int e = mx4_scale_byte(amax);
      uint32_t codes = 0;
      if (e != 255) {
        const float inv = mx4_inverse(e);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          if constexpr (sizeof(T) == 2) {
            lo = bf16_bits_to_float(w[r][u][j] & 0xFFFFu);
            hi = __uint_as_float(w[r][u][j] & 0xFFFF0000u);
          } else {
            lo = __uint_as_float(w[r][u][2 * j]);
            hi = __uint_as_float(w[r][u][2 * j + 1]);
          }
          c[j] = e2m1x2(lo * inv, hi * inv);
        }
        codes = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
      }
      reinterpret_cast<uint32_t*>(p.codes)[at + u * part.stride] = codes;
      if ((vec & 3u) == 0) {
        if (!p.tiles) {
          p.scales[(at + u * part.stride) >> 2] = static_cast<uint8_t>(e);
        } else {
          const int b = static_cast<int>(vec >> 2);
          uint8_t* to = p.scales + mx4_tile_at(p.row0 + row, b, p.kt);
          *to = static_cast<uint8_t>(e);
          // the row's blocks end inside a tile: the rest of the tile's row is read as scales of
          // zero codes, and must not be NaN
          if (b == p.cols / kMxBlock - 1)
            for (int k = 1; ((b + k) & 3) != 0; ++k) to[k] = 0;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ row gather

struct Mx4Rows {
  const uint8_t* codes;   // [V x d / 2]
  const uint8_t* scales;  // [V x d / 32]
};

struct Mx4GatherParams {
  Mx4Rows E[kMaxS];
  const int32_t* idx;     // [T x S], nullptr: Eq. 2 from h
  HashParams h;           // tokens, T, V0, S, the moduli V and status in any case
  int row_blocks;         // d / 32, blocks of one sub-row
  FastDiv by_row, by_sub; // ceil(D / 128) * 4 blocks of a padded row; row_blocks
  int blocks;             // D / 32
  int kt;
  int tokens;             // a block takes, at most kMx4GatherThreads / S and kMx4GatherMaxTokens
  uint8_t* G;             // [T x D / 2] codes
  uint8_t* Gs;            // scales, in tiles
};

constexpr int kMx4GatherThreads = 256;
constexpr int kMx4GatherMaxTokens = 32;  // of a block
constexpr int kMx4GatherUnroll = 4;
constexpr int kMx4GatherOffsets = 1024;  // offsets staged in shared memory when B + 1 fits

// The given index of token i in sub-table s, checked; for s = 0 its token too, by which the
// product's epilogue reads E_0.
__device__ __forceinline__ uint32_t mx4_given_row(const Mx4GatherParams& p, int64_t i, int s) {
  const HashParams& h = p.h;
  const uint32_t row = static_cast<uint32_t>(p.idx[i * h.S + s]);
  if (row >= h.V[s] || (s == 0 && static_cast<uint32_t>(h.tokens[i]) >= h.V0)) set_status(h.status, NGRAM_STATUS_BAD_TOKEN);
  return row < h.V[s] ? row : 0;
}

// Blocks base, base + THREADS, ... (UNROLL of them) of the `total` blocks of the padded rows of
// tokens i0, i0 + 1, ... whose table rows are s_row[token * S + s]: one 16-byte code block and
// one scale byte each, all loads in flight together; four neighbouring lanes' scale bytes leave
// as one word.
template <int THREADS, int UNROLL>
__device__ __forceinline__ void mx4_copy_blocks(const Mx4GatherParams& p, int64_t i0, const uint32_t* s_row, uint32_t base,
                                                uint32_t total) {
  uint4 code[UNROLL];
  uint32_t scale[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t v = base + u * THREADS;
    scale[u] = 0;
    if (v < total) {
      const uint32_t k = p.by_row.div(v), b = v - k * p.by_row.d;
      if (b < static_cast<uint32_t>(p.blocks)) {
        const uint32_t s = p.by_sub.div(b), c = b - s * p.row_blocks;
        const size_t at = static_cast<size_t>(s_row[k * p.h.S + s]) * p.row_blocks + c;
        code[u] = ld_stream_v4(p.E[s].codes + at * 16);
        scale[u] = __ldg(p.E[s].scales + at);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t v = base + u * THREADS;
    if (v >= total) continue;  // a padded row is a multiple of 4 blocks: four neighbours alike
    const uint32_t quad = 0xFu << (threadIdx.x & 28);
    uint32_t w = scale[u] << ((threadIdx.x & 3) * 8);
    w |= __shfl_xor_sync(quad, w, 1);
    w |= __shfl_xor_sync(quad, w, 2);
    const uint32_t k = p.by_row.div(v), b = v - k * p.by_row.d;
    if (b < static_cast<uint32_t>(p.blocks))
      *reinterpret_cast<uint4*>(p.G + (static_cast<size_t>(i0 + k) * p.blocks + b) * 16) = code[u];
    if ((threadIdx.x & 3) == 0)
      *reinterpret_cast<uint32_t*>(p.Gs + mx4_tile_at(i0 + k, static_cast<int>(b), p.kt)) = w;
  }
}

// G[i] = the concatenated 4-bit sub-rows of token i, its scales in tiles. A block takes a few
// tokens: their places in their sequences, a thread each; their row indices (Eq. 2, or idx), a
// thread each; then their rows. Hashing in the launch that gathers takes 8.6 us at a decode step
// of 1280 tokens, D = 4096, where two launches took 6.7 and 5.6. 17/32 bytes an element each way,
// random rows from HBM: 71 us at 65536 tokens of D = 4096, which move 302 MB with the sectors of
// the scales read whole.
//
// Running it beside the product (as resident blocks that the product waits for 256 rows at a
// time, or in the product's idle warps) was slower, 522 and 765 us for the two against 503 one
// after the other: the product keeps the L2 busy, and the gather's loads queue behind its.
__global__ void __launch_bounds__(kMx4GatherThreads) mx4_gather_kernel(const __grid_constant__ Mx4GatherParams p) {
  __shared__ int32_t s_off[kMx4GatherOffsets];
  __shared__ TokenPlace s_place[kMx4GatherMaxTokens];
  __shared__ uint32_t s_row[kMx4GatherThreads];
  pdl_launch_dependents();
  pdl_wait();
  const HashParams& h = p.h;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int n = h.T - i0 < p.tokens ? static_cast<int>(h.T - i0) : p.tokens;
  if (!p.idx) {
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; k <= h.num_seqs;
         k += static_cast<int64_t>(gridDim.x) * blockDim.x)
      check_offset(h, k);
    const bool staged = h.num_seqs + 1 <= kMx4GatherOffsets;
    if (staged)
      for (int k = threadIdx.x; k <= h.num_seqs; k += blockDim.x) s_off[k] = h.offsets[k];
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < n) s_place[threadIdx.x] = token_place(h, i0 + threadIdx.x, staged ? s_off : h.offsets);
    __syncthreads();
  }
  if (static_cast<int>(threadIdx.x) < n * h.S) {
    const int k = threadIdx.x / h.S, s = threadIdx.x - k * h.S;
    const TokenPlace t = s_place[k];
    s_row[threadIdx.x] = p.idx ? mx4_given_row(p, i0 + k, s)
                               : hash_sub(h, i0 + k, t.start, t.slot, t.hist_len, t.hist_from, s);
  }
  __syncthreads();
  const uint32_t total = static_cast<uint32_t>(n) * p.by_row.d;
  for (uint32_t base = threadIdx.x; base < total; base += kMx4GatherThreads * kMx4GatherUnroll)
    mx4_copy_blocks<kMx4GatherThreads, kMx4GatherUnroll>(p, i0, s_row, base, total);
}

// ------------------------------------------------------------------ product
//
// out[m][n] = (sum_k A[m][k] B[n][k] (+ E_0[tokens[m]][n])) * scale, A and B in mx4, on
// tcgen05.mma.kind::mxf4: K = 64 elements an instruction, the block scales read from TMEM,
// fp32 accumulators in TMEM, rounded once at the end.
//
// A stage holds 256 elements of K: 128 rows of A and BN of B, one 128-byte swizzle row each
// (codes of 256 elements), and their scale tiles. The scale tiles are copied into TMEM by
// tcgen05.cp (32 lanes x 16 bytes, repeated for the four lane quarters), issued by the MMA
// thread in front of the stage's MMAs; the tensor pipe keeps their order.
struct Mx4Maps {
  CUtensorMap A;   // [M x K / 2] bytes, box 128 x 128 rows
  CUtensorMap B;   // [N x K / 2] bytes, box 128 x the rows of a CTA's first part of B
  CUtensorMap B1;  // of its second part
  CUtensorMap At;  // boxes of the rows that the last box of A or B holds, to a multiple of 8:
  CUtensorMap Bt;  // a box with many rows past the array's end takes far longer to fill
  CUtensorMap SA;  // scale tiles as [row blocks x kt * 128] words, box 256 words (two tiles) x 1
  CUtensorMap SB;  // the same of B, box 256 words x the tile's row blocks
};

// Rows of a box of `box` rows from `row` on that are loaded, of an array of `rows`: all of it,
// the tail's, or none.
__device__ __forceinline__ int mx4_box_rows(int rows, int row, int box) {
  const int left = rows - row;
  return left >= box ? box : (left <= 0 ? 0 : (left + 7) & ~7);
}

struct Mx4GemmParams {
  int M, N, K;
  int num_m_blocks, num_n_blocks, num_k_blocks;  // k-blocks of 256
  float scale;
  const int32_t* tokens;  // E_0 rows to add (nullptr: none)
  const void* E0;         // [V0 x N], element type of out
  uint32_t V0;
  void* out;
  int64_t ldo;            // elements
  int vec16, vec32;       // out and E_0 rows admit 16-byte, 32-byte accesses
  int* status;
};

constexpr int kMxEpiWarps = 8;
constexpr int kMxStageWords = 32 * 9;  // of shared memory an epilogue warp: 32 bytes of 32 rows, padded
constexpr int kMxThreads = 128 + 32 * kMxEpiWarps;  // warp 0 loads, warp 1 MMA and TMEM, warps 4-11 epilogue

// PAIR: CTA pairs, 256 x BN tiles; each CTA holds its 128 rows of A with their scales, half of
// B's rows, and the scales of all of B's rows. Tiles wider than an instruction (256 columns) are
// computed in parts side by side, of which each CTA of a pair holds half.
template <int BN, int STAGES, bool PAIR = false>
struct Mx4Smem {
  static constexpr int kABytes = 128 * 128;
  static constexpr int kParts = BN > 256 ? 2 : 1;
  __host__ __device__ static constexpr int part_n(int part) {
    const int n0 = BN > 256 ? (BN / 2 + 63) / 64 * 64 : BN;
    return part ? BN - n0 : n0;
  }
  // scale_vec::2X takes scales from an even column on, of 32 rows each
  static_assert(BN % 64 == 0 && part_n(0) <= 256, "parts begin at an even column of scales");
  __host__ __device__ static constexpr int part_rows(int part) { return PAIR ? part_n(part) / 2 : part_n(part); }  // in a CTA
  // first row of CTA `rank`'s part of a tile's rows of B
  __host__ __device__ static constexpr int part_row(int part, int rank) { return part * part_n(0) + rank * part_rows(part); }
  static constexpr int kPartOffset = part_rows(0) * 128;  // of part 1
  static constexpr int kBBytes = (PAIR ? BN / 2 : BN) * 128;
  static constexpr int kSfbRows = (BN + 127) / 128;  // row blocks of B's scales a tile touches
  static constexpr int kSfaOffset = kABytes + kBBytes;
  static constexpr int kSfbOffset = kSfaOffset + 2 * kMxTileBytes;
  static constexpr int kStageBytes = kSfbOffset + kSfbRows * 2 * kMxTileBytes;
  static constexpr int kBarOffset = STAGES * kStageBytes;
  static constexpr int kNumBars = 2 * STAGES + 5;
  static constexpr int kStgOffset = (kBarOffset + kNumBars * 8 + 16 + 15) / 16 * 16;
  static constexpr int kBytes = kStgOffset + kMxEpiWarps * kMxStageWords * 4;
  static constexpr int kLaunchBytes = kBytes + 1024;
  static_assert(kStageBytes % 1024 == 0 && kPartOffset % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
  // TMEM: two accumulators and the stage's scales. At BN = 256 the accumulators share 32
  // columns ([224, 256)), which leaves 32 for the scales: the epilogue drains the shared
  // columns first and hands them over, so the next tile's MMAs still overlap the drain. Wider
  // tiles have one accumulator.
  static constexpr bool kOverlap = BN == 256;
  static constexpr int kAccs = BN > 256 ? 1 : 2;
  static constexpr int kAccStride = kAccs == 1 ? 0 : (kOverlap ? 224 : BN);
  static constexpr int kSfaCol = kAccStride + BN;
  static constexpr int kSfbCol = kSfaCol + 8;
  static constexpr int kTmemCols = kSfbCol + kSfbRows * 8 <= 256 ? 256 : 512;
  static_assert(kSfbCol + kSfbRows * 8 <= 512, "accumulators and scales exceed TMEM");
};

// Instruction descriptor, kind::mxf4: E2M1 A and B (K-major), E8M0 scales, fp32 D, M x N;
// `id` selects the scale bytes of a column word: 0 its low half, 2 its high half.
__host__ __device__ constexpr uint32_t umma_idesc_mx4(int M, int N, uint32_t id) {
  return (id << 4)                                // B scale data id
         | (1u << 7)                              // A format: E2M1
         | (1u << 10)                             // B format: E2M1
         | (static_cast<uint32_t>(N >> 3) << 17)  // N / 8
         | (1u << 23)                             // scale format: E8M0
         | (static_cast<uint32_t>(M >> 4) << 24)  // M / 16
         | (id << 29);                            // A scale data id
}

__device__ __forceinline__ void umma_mx4(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Scale tile (32 rows of 16 bytes) from shared memory to four TMEM columns, for all four lane
// quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Pair forms: operands, scales and accumulators of both CTAs at the same addresses.
__device__ __forceinline__ void umma_mx4_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}

// Descriptor of a scale tile: unswizzled, 8 rows of 16 bytes 128 bytes apart.
__device__ __forceinline__ uint64_t scale_tile_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu)
         | (static_cast<uint64_t>(128 >> 4) << 32)  // stride byte offset: next 8 rows
         | (static_cast<uint64_t>(1) << 46);        // descriptor version for sm_100
}

// 32-byte global accesses (sm_100: eight registers an instruction), 32-byte aligned.
__device__ __forceinline__ void ld_global_v8(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 columns of a row of E_0, as they lie, in 32-byte accesses: two (bf16) or four (f32).
template <typename OutT>
struct Mx4E0 {
  static constexpr int kAcc = sizeof(OutT);
  static constexpr int kCols = 32 / kAcc;
  uint32_t v[kAcc][8];
  // e0 at the first of the columns, nullptr: zeros
  __device__ __forceinline__ void load(const OutT* e0, bool vec32) {
#pragma unroll
    for (int h = 0; h < kAcc; ++h) {
      if (e0 && vec32) {
        ld_global_v8(e0 + h * kCols, v[h]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 x = e0 ? __ldg(reinterpret_cast<const uint4*>(e0 + h * kCols) + k) : make_uint4(0, 0, 0, 0);
          v[h][4 * k] = x.x;
          v[h][4 * k + 1] = x.y;
          v[h][4 * k + 2] = x.z;
          v[h][4 * k + 3] = x.w;
        }
      }
    }
  }
};

// The row of E_0 that output row `row` adds, or nullptr.
template <typename OutT>
__device__ __forceinline__ const OutT* mx4_e0_row(const Mx4GemmParams& p, int row) {
  if (!p.tokens || row >= p.M) return nullptr;
  uint32_t t = static_cast<uint32_t>(__ldg(p.tokens + row));
  if (t >= p.V0) t = 0;
  return static_cast<const OutT*>(p.E0) + static_cast<int64_t>(t) * p.N;
}

// 32 columns of 32 output rows (a row a lane) from col: (acc + E_0) * scale, rounded once. A lane
// stores its own row, 32 bytes (a whole sector) an access, 16 where rows are less aligned.
// Rows that admit neither, and the columns at a row's end, go through `stg` (kMxStageWords words
// of the warp's own), a piece of 32 bytes a row at a time, so that neighbouring lanes store
// neighbouring columns (a lane storing element by element took five times as long: 25 us for
// 128 x 4090 at K = 4096, against 9 for 128 x 4096).
template <typename OutT>
__device__ __forceinline__ void mx4_store_rows(const Mx4GemmParams& p, int row0, int lane, int col, const uint32_t (&v)[32],
                                               const Mx4E0<OutT>& e, uint32_t* stg) {
  if (col >= p.N) return;
  constexpr int kAcc = Mx4E0<OutT>::kAcc, kCols = Mx4E0<OutT>::kCols;
  const int row = row0 + lane;
  OutT* dst = static_cast<OutT*>(p.out) + static_cast<int64_t>(row) * p.ldo + col;
#pragma unroll
  for (int h = 0; h < kAcc; ++h) {
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (sizeof(OutT) == 2)
        o[j] = pack_bf16x2((__uint_as_float(v[h * 16 + 2 * j]) + bf16_bits_to_float(e.v[h][j] & 0xFFFFu)) * p.scale,
                           (__uint_as_float(v[h * 16 + 2 * j + 1]) + __uint_as_float(e.v[h][j] & 0xFFFF0000u)) * p.scale);
      else
        o[j] = __float_as_uint((__uint_as_float(v[h * 8 + j]) + __uint_as_float(e.v[h][j])) * p.scale);
    }
    const int left = p.N - col - h * kCols;  // columns inside the row
    if (p.vec16 && left >= kCols) {
      if (row >= p.M) continue;
      if (p.vec32) {
        st_global_v8(dst + h * kCols, o);
      } else {
        *reinterpret_cast<uint4*>(dst + h * kCols) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + h * kCols + kCols / 2) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) stg[lane * 9 + j] = o[j];
      __syncwarp();
      const OutT* in = reinterpret_cast<const OutT*>(stg);
      constexpr int kPitch = 36 / static_cast<int>(sizeof(OutT));
      const int c = lane % kCols;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int r = i * (32 / kCols) + lane / kCols;
        if (row0 + r < p.M && c < left)
          static_cast<OutT*>(p.out)[static_cast<int64_t>(row0 + r) * p.ldo + col + h * kCols + c] = in[r * kPitch + c];
      }
      __syncwarp();
    }
  }
}

// One tile's epilogue for one of the eight warps: TMEM lanes q * 32 .. + 31 (a row a lane), the
// tile's column half g, 32 columns at a time: accumulators from TMEM, the row's E_0 added,
// scaled, rounded and stored by the lane that holds them, 32 bytes (a whole sector) an access.
// (Through shared memory, with whole rows in by cp.async and out by TMA stores, a tile takes as
// long: the epilogue then waits for the accumulator a third of the time.) E_0
// rows are random reads: the columns of all four chunks (bf16; two of them f32) are asked for
// before the accumulator is ready.
// `ready` waits for the accumulator (false: abort); `release` hands it back.
template <typename L, int BN, typename OutT, typename Ready, typename Release>
__device__ __forceinline__ bool mx4_epilogue(const Mx4GemmParams& p, uint32_t* stg, uint32_t tmem_base, int q, int g, int lane,
                                             int row0, int col0, int acc, Ready ready, Release release) {
  constexpr int kChunks = BN / 64;
  // The columns shared with the other accumulator go first: the last chunk of accumulator 0
  // (of the half g = 1) or the first of accumulator 1 (g = 0). The other half has nothing to
  // hand over and says so at once. Both only after this tile's accumulator is ready: an arrival
  // before that could stand in for a slower warp's of the tile before.
  const bool shares = L::kOverlap && g == (acc ^ 1);
  const int rot = shares && g == 1 ? kChunks - 1 : 0;
  const int row = row0 + lane;
  auto chunk_col = [&](int cc) { return g * (BN / 2) + (L::kOverlap ? (cc + rot) & (kChunks - 1) : cc) * 32; };
  constexpr int kInFlight = 8 / static_cast<int>(sizeof(OutT));
  constexpr int kDepth = kChunks < kInFlight ? kChunks : kInFlight;  // chunks of E_0 in flight
  Mx4E0<OutT> e[kDepth];
  const OutT* e0 = mx4_e0_row<OutT>(p, row);
  // N is a multiple of 32 where there is an E_0
  auto load_e = [&](int slot, int col) { e[slot].load(e0 && col < p.N ? e0 + col : nullptr, p.vec32 != 0); };
#pragma unroll
  for (int cc = 0; cc < kDepth; ++cc) load_e(cc, col0 + chunk_col(cc));
  if (!ready()) return false;
  if (L::kOverlap && !shares) {
    tc_fence_before();  // this warp's reads of the tile before
    release();
  }
  const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * L::kAccStride);
#pragma unroll
  for (int cc = 0; cc < kChunks; ++cc) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(taddr + chunk_col(cc), v);
    tmem_wait_ld();
    if (L::kOverlap ? (cc == 0 && shares) : cc + 1 == kChunks) {
      tc_fence_before();
      release();
    }
    mx4_store_rows<OutT>(p, row0, lane, col0 + chunk_col(cc), v, e[cc % kDepth], stg);
    if (cc + kDepth < kChunks) load_e(cc % kDepth, col0 + chunk_col(cc + kDepth));
  }
  return true;
}

// A stage's scale copies and MMAs (issued by one lane): K elements `left` from the stage's start
// to the row's end (256 a stage), `first`: the sum starts here. col0: the tile's first column.
template <typename L, int BN, bool PAIR>
__device__ __forceinline__ void mx4_issue_stage(uint32_t at, uint32_t tmem_base, int col0, uint32_t d_tmem, int left,
                                                bool first) {
  const uint64_t adesc = sw128_kmajor_desc(at), bdesc = sw128_kmajor_desc(at + L::kABytes);
  const uint64_t da = scale_tile_desc(at + L::kSfaOffset), db = scale_tile_desc(at + L::kSfbOffset);
  const uint32_t sfa = tmem_base + L::kSfaCol;
  // a tile that is not whole row blocks of scales may start inside a block's four columns
  const uint32_t sfb = tmem_base + L::kSfbCol + (BN % 128 ? static_cast<uint32_t>((col0 & 127) >> 5) : 0u);
  // scales of 128 elements of K, then their MMAs of 64
  auto half = [&](int h, bool both) {
    if (PAIR) tmem_cp_scales_pair(sfa + h * 4, da + h * (kMxTileBytes >> 4));
    else tmem_cp_scales(sfa + h * 4, da + h * (kMxTileBytes >> 4));
#pragma unroll
    for (int r = 0; r < L::kSfbRows; ++r) {
      const uint32_t to = tmem_base + L::kSfbCol + (h * L::kSfbRows + r) * 4;
      if (PAIR) tmem_cp_scales_pair(to, db + (r * 2 + h) * (kMxTileBytes >> 4));
      else tmem_cp_scales(to, db + (r * 2 + h) * (kMxTileBytes >> 4));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !both) break;
      const uint32_t more = !first || h != 0 || k != 0 ? 1u : 0u;
      const uint64_t ka = adesc + 2u * (2 * h + k);
#pragma unroll
      for (int part = 0; part < L::kParts; ++part) {
        const uint32_t idesc = umma_idesc_mx4(PAIR ? 256 : 128, L::part_n(part), 2 * k);
        const uint32_t d = d_tmem + part * L::part_n(0), fb = sfb + h * L::kSfbRows * 4 + part * (L::part_n(0) / 32);
        const uint64_t kbd = bdesc + 2u * (2 * h + k) + part * (L::kPartOffset >> 4);
        if (PAIR) umma_mx4_pair(d, ka, kbd, idesc, sfa + h * 4, fb, more);
        else umma_mx4(d, ka, kbd, idesc, sfa + h * 4, fb, more);
      }
    }
  };
  if (left >= 256) {
    half(0, true);
    half(1, true);
  } else {  // the last stage of a row may hold less
    half(0, left > 64);
    if (left > 128) half(1, left > 192);
  }
}

// The kernel: one CTA a 128 x BN tile, or (PAIR) a cluster of two a 256 x BN tile. In a pair
// every load signals CTA 0's stage barrier (.cta_group::2 loads, no multicast), one thread of
// CTA 0 issues the copies of the scales and the MMAs for both, and its commits arrive in both.
template <int BN, int STAGES, typename OutT, bool PAIR>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ Mx4Maps maps, const __grid_constant__ Mx4GemmParams p) {
  using L = Mx4Smem<BN, STAGES, PAIR>;
  constexpr int kRanks = PAIR ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::kBarOffset;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBarOffset + L::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto stage_at = [&](int s) { return sbase + s * L::kStageBytes; };
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  auto wait = [&](uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
    return PAIR ? mbar_wait_cluster(bar, parity, abort_flag, p.status, limit_ns)
                : mbar_wait(bar, parity, abort_flag, p.status, limit_ns);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1u);   // CTA 0's producer's byte count
      mbar_init(empty_bar(s), 1u);  // one tcgen05.commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1u);
      mbar_init(tempty_bar(a), 32u * kMxEpiWarps + (PAIR ? kMxEpiWarps : 0));  // and CTA 1's warps, one arrival each
    }
    mbar_init(drain_bar, 1u);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.A);
    tma_prefetch_desc(&maps.B);
    if (L::kParts > 1) tma_prefetch_desc(&maps.B1);
    tma_prefetch_desc(&maps.At);
    tma_prefetch_desc(&maps.Bt);
    tma_prefetch_desc(&maps.SA);
    tma_prefetch_desc(&maps.SB);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), L::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // nothing above touches global memory

  const int num_tiles = p.num_m_blocks * p.num_n_blocks;
  const int KB = p.num_k_blocks;
  const int worker = blockIdx.x / kRanks, workers = gridDim.x / kRanks;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      // B (a weight that every row block reads) stays in L2 before the rest: 95.7 -> 91.9 us for the
      // layer at D = 2048, 32768 tokens
      const uint64_t pol = l2_policy_evict_normal(), pol_b = l2_policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = worker; tile < num_tiles && ok; tile += workers) {
        const int m_blk = (tile / p.num_n_blocks) * kRanks + static_cast<int>(rank), n_blk = tile % p.num_n_blocks;
        const int a_rows = mx4_box_rows(p.M, m_blk * 128, 128);
        const void* map_a = a_rows == 128 ? &maps.A : &maps.At;
        uint32_t tx = kRanks * (L::kStageBytes - L::kABytes - L::kBBytes) + a_rows * 128;
        if (PAIR) tx += mx4_box_rows(p.M, m_blk * 128 + 128, 128) * 128;  // rank 0 posts the bytes of both
        int brow[L::kParts], b_rows[L::kParts];
#pragma unroll
        for (int part = 0; part < L::kParts; ++part) {
          const int kRows = L::part_rows(part);
          brow[part] = n_blk * BN + L::part_row(part, static_cast<int>(rank));
          b_rows[part] = mx4_box_rows(p.N, brow[part], kRows);
          tx += b_rows[part] * 128;
          if (PAIR) tx += mx4_box_rows(p.N, brow[part] + kRows, kRows) * 128;
        }
        auto map_b = [&](int part) -> const void* {
          return b_rows[part] != L::part_rows(part) ? &maps.Bt : (part ? &maps.B1 : &maps.B);
        };
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait(empty_bar(stage), phase ^ 1u)) { ok = false; break; }
          const uint32_t at = stage_at(stage);
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), tx);
          // bytes and scale tiles past the end of an array count and are filled with zeros
          if (PAIR) {
            const uint32_t bar = map_to_cta(full_bar(stage), 0);
            if (a_rows) tma_load_2d_pair(at, map_a, kb * 128, m_blk * 128, bar, pol);
#pragma unroll
            for (int part = 0; part < L::kParts; ++part)
              if (b_rows[part])
                tma_load_2d_pair(at + L::kABytes + part * L::kPartOffset, map_b(part), kb * 128, brow[part], bar, pol_b);
            tma_load_2d_pair(at + L::kSfaOffset, &maps.SA, kb * 256, m_blk, bar, pol);
            tma_load_2d_pair(at + L::kSfbOffset, &maps.SB, kb * 256, n_blk * BN >> 7, bar, pol_b);
          } else {
            const uint32_t bar = full_bar(stage);
            tma_load_2d(at, map_a, kb * 128, m_blk * 128, bar, pol);
            static_assert(PAIR || L::kParts == 1, "one CTA's B is one part");
            tma_load_2d(at + L::kABytes, map_b(0), kb * 128, brow[0], bar, pol_b);
            tma_load_2d(at + L::kSfaOffset, &maps.SA, kb * 256, m_blk, bar, pol);
            tma_load_2d(at + L::kSfbOffset, &maps.SB, kb * 256, n_blk * BN >> 7, bar, pol_b);
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // an abort: the copies in flight land before the block ends
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000ull * 1000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales to TMEM, MMA (CTA 0)
    // One elected lane. (Chosen by `lane == 0`, whose values the compiler does not take for
    // warp-uniform, the loop needed about 1000 cycles a k-block to issue, whatever its MMAs took.)
    if (rank == 0 && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int local = 0;
      for (int tile = worker; tile < num_tiles && ok; tile += workers, ++local) {
        const int n_blk = tile % p.num_n_blocks;
        const int acc = L::kAccs == 1 ? 0 : local & 1;
        if (L::kOverlap || L::kAccs == 1) {  // the columns that the previous tile held too have been drained
          if (local > 0 && !wait(tempty_bar(0), (local - 1) & 1u)) { ok = false; break; }
        } else {
          if (!wait(tempty_bar(acc), ((local >> 1) & 1u) ^ 1u)) { ok = false; break; }
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * L::kAccStride);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait(full_bar(stage), phase)) { ok = false; break; }
          tc_fence_after();
          {
            mx4_issue_stage<L, BN, PAIR>(stage_at(stage), tmem_base, n_blk * BN, d_tmem, p.K - kb * 256, kb == 0);
            if (PAIR) umma_commit_pair_both(empty_bar(stage));
            else umma_commit(empty_bar(stage));
            if (kb + 1 == KB) {
              if (PAIR) umma_commit_pair_both(tfull_bar(acc));
              else umma_commit(tfull_bar(acc));
            }
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (PAIR) umma_commit_pair_both(drain_bar);
      else umma_commit(drain_bar);
    }
    __syncwarp();
    // the last commit: every MMA is done
    if (rank == 0) mbar_wait_drain(drain_bar, 0, kWaitLimitNs);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (own 128 rows)
    const int q = warp & 3, g = (warp - 4) >> 2;
    uint32_t* stg = reinterpret_cast<uint32_t*>(smem + L::kStgOffset) + (warp - 4) * kMxStageWords;
    int local = 0;
    for (int tile = worker; tile < num_tiles; tile += workers, ++local) {
      const int m_blk = (tile / p.num_n_blocks) * kRanks + static_cast<int>(rank), n_blk = tile % p.num_n_blocks;
      const int acc = L::kAccs == 1 ? 0 : local & 1;
      auto ready = [&] {
        bool got = false;
        // a whole tile's k-blocks, ten times what they were measured at (one tile of K = 2^31 takes
        // 2.36 s)
        if (lane == 0)
          got = wait(tfull_bar(acc), (L::kAccs == 1 ? local : local >> 1) & 1u,
                     kWaitLimitNs + static_cast<uint64_t>(KB) * 4096);
        if (!__shfl_sync(0xffffffffu, got, 0)) return false;
        tc_fence_after();
        return true;
      };
      auto release = [&] {
        const uint32_t bar = tempty_bar(L::kOverlap ? 0 : acc);
        if (rank == 0) {
          mbar_arrive_relaxed(bar);
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(map_to_cta(bar, 0));
        }
      };
      if (!mx4_epilogue<L, BN, OutT>(p, stg, tmem_base, q, g, lane, m_blk * 128 + q * 32, n_blk * BN, acc, ready, release))
        break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) {
    // CTA 1: the last commit's arrival has landed, and so have all earlier ones. Waited for from
    // the end of its epilogue on: from the kernel's start the limit would cover the whole product.
    if (rank == 1 && warp == 1) mbar_wait_drain(drain_bar, 0, kWaitLimitNs);
    __syncthreads();
    cluster_sync();  // no remote arrival or pair MMA is outstanding past this point
  }
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, L::kTmemCols);
    else tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

// ------------------------------------------------------------------ product of few rows
//
// The same product for at most R <= 4 rows of A, where a tile's 128 rows would be idle: a warp
// takes one column n, its lanes the blocks of the row B[n], read once. Twice an E2M1 value is an
// integer of magnitude at most 12, so a block's sum of 32 products is an exact integer by dp4a,
// scaled by a power of two and added in fp32. A's rows are decoded to int8 in shared memory once
// a block of eight warps. One token's 4096 x 4096 takes 4.6 us in a graph (7.2 on tiles), 8.9 MB
// that L2 holds, and 6.8 (9.4) with B from HBM and the quantisation in front: the launch and one
// round of loads, an instruction a clock. Large products are bound by its instructions, about 60
// a block of B and 12 more a row. Asking L2 for B's rows before the wait for the
// quantisation gained nothing.

constexpr int kMxFewWarps = 8;
constexpr int kMxFewUnroll = 4;                     // blocks of B in flight a lane
constexpr int kMxFewBlocks = 32 * kMxFewUnroll;     // of a row, at a time

struct Mx4FewParams {
  Mx4GemmParams g;
  const uint8_t *A, *SA, *B, *SB;  // codes and scale tiles
};

// Eight E2M1 codes to int8 of twice their values, in order. (Bytes of the magnitudes and of
// their negatives by permutation, chosen by each code's sign spread over its byte.)
__device__ __forceinline__ void e2m1x8_twice(uint32_t codes, uint32_t (&x)[2]) {
  const uint32_t up = codes << 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sel = (codes >> (16 * h)) & 0x7777u;
    uint32_t neg;  // the intrinsic has no sign mode
    asm("prmt.b32 %0, %1, 0, 0xBA98;" : "=r"(neg) : "r"(__byte_perm(up, codes, h ? 0x7362 : 0x5140)));
    const uint32_t pos_v = __byte_perm(0x03020100u, 0x0C080604u, sel), neg_v = __byte_perm(0xFDFEFF00u, 0xF4F8FAFCu, sel);
    x[h] = (pos_v & ~neg) | (neg_v & neg);
  }
}

// x * 2^e for a sum x of twice-values of two blocks with scale bytes ea and eb: 2^e in two
// halves, which are normal where the result is not zero.
__device__ __forceinline__ float mx4_scale_pair(int x, uint32_t ea, uint32_t eb) {
  int e = static_cast<int>(ea + eb) - 256;  // 2 * 127, and twice two
  e = max(e, -252);
  const int h = e >> 1;
  const float s1 = __uint_as_float(static_cast<uint32_t>(h + 127) << 23), s2 = __uint_as_float(static_cast<uint32_t>(e - h + 127) << 23);
  const float v = static_cast<float>(x) * s1 * s2;
  return ea == 255 || eb == 255 ? __uint_as_float(0x7FC00000u) : v;
}

template <int R, typename OutT>
__global__ void __launch_bounds__(32 * kMxFewWarps) mx4_few_kernel(const __grid_constant__ Mx4FewParams p) {
  __shared__ uint4 s_a[R][2][kMxFewBlocks];  // first and second halves of blocks: no bank conflicts
  __shared__ uint8_t s_e[R][kMxFewBlocks];
  pdl_wait();
  const Mx4GemmParams& g = p.g;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int blocks = g.K / kMxBlock, kt = (g.K + 127) / 128;
  // a block's columns share the 32-byte sectors of the scales' tiles: two neighbours in each quarter
  const int n = (blockIdx.x >> 4) * 128 + (blockIdx.x & 15) * 2 + (w & 1) + (w >> 1) * 32;
  const bool on = n < g.N;
  const uint4* row = reinterpret_cast<const uint4*>(p.B) + static_cast<int64_t>(on ? n : 0) * blocks;
  float acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = 0.f;
  for (int b0 = 0; b0 < blocks; b0 += kMxFewBlocks) {
    uint4 code[kMxFewUnroll];
    uint32_t eb[kMxFewUnroll];
#pragma unroll
    for (int u = 0; u < kMxFewUnroll; ++u) {
      const int b = b0 + u * 32 + lane;
      code[u] = make_uint4(0, 0, 0, 0);
      eb[u] = 0;
      if (on && b < blocks) {
        code[u] = ld_stream_v4(row + b);
        eb[u] = __ldg(p.SB + mx4_tile_at(n, b, kt));
      }
    }
    if (b0) __syncthreads();
    for (int i = threadIdx.x; i < R * kMxFewBlocks; i += 32 * kMxFewWarps) {
      const int r = i / kMxFewBlocks, k = i % kMxFewBlocks, b = b0 + k;
      uint4 c = make_uint4(0, 0, 0, 0);
      uint32_t e = 0;
      if (r < g.M && b < blocks) {
        c = __ldg(reinterpret_cast<const uint4*>(p.A) + static_cast<int64_t>(r) * blocks + b);
        e = __ldg(p.SA + mx4_tile_at(r, b, kt));
      }
      uint32_t x[4][2];
      e2m1x8_twice(c.x, x[0]);
      e2m1x8_twice(c.y, x[1]);
      e2m1x8_twice(c.z, x[2]);
      e2m1x8_twice(c.w, x[3]);
      s_a[r][0][k] = make_uint4(x[0][0], x[0][1], x[1][0], x[1][1]);
      s_a[r][1][k] = make_uint4(x[2][0], x[2][1], x[3][0], x[3][1]);
      s_e[r][k] = static_cast<uint8_t>(e);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMxFewUnroll; ++u) {
      const int k = u * 32 + lane;
      if (b0 + u * 32 >= blocks) break;
      uint32_t y[4][2];
      e2m1x8_twice(code[u].x, y[0]);
      e2m1x8_twice(code[u].y, y[1]);
      e2m1x8_twice(code[u].z, y[2]);
      e2m1x8_twice(code[u].w, y[3]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 lo = s_a[r][0][k], hi = s_a[r][1][k];
        const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        int d = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) d = __dp4a(static_cast<int>(x[j]), static_cast<int>(y[j >> 1][j & 1]), d);
        acc[r] += mx4_scale_pair(d, s_e[r][k], eb[u]);
      }
    }
  }
  float mine = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v = acc[r];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == r) mine = v;
  }
  if (!on || lane >= R || lane >= g.M) return;
  const OutT* e0 = mx4_e0_row<OutT>(g, lane);
  OutT* out = static_cast<OutT*>(g.out) + static_cast<int64_t>(lane) * g.ldo + n;
  if constexpr (sizeof(OutT) == 2)
    *out = static_cast<uint16_t>(pack_bf16x2((mine + (e0 ? bf16_bits_to_float(e0[n]) : 0.f)) * g.scale, 0.f));
  else
    *out = (mine + (e0 ? e0[n] : 0.f)) * g.scale;
}

}  // namespace ngram
