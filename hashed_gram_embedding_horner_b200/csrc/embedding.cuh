// One table's lookup, out[i] = scale * table[ids[i]], and its gradient by sorted ids.
//
// Lookup: the table in bf16, f32 or mx4 (by rows, see mx4.cuh), a vector of eight elements at a
// time (RowMap in mx4.cuh). Bound by HBM where its instructions leave it: an mx4 vector costs
// about 60, most of them the decoding.
//
// Gradient: dTable[v] = scale * sum_{i : ids[i] = v} g_i. The positions are sorted by id with
// a stable radix sort; runs of equal ids are summed in fp32 by whoever owns them, without
// atomics, so the sum's order, and its bits, depend on the ids alone:
//   - the sorted positions are cut into pieces (of 128, 32 or 8: the longest that fill the GPU);
//     a warp sums the rows of a piece for 256 columns, in ascending position order;
//   - a run inside one piece is written out by that warp; a run that crosses a piece's border
//     leaves one partial sum in each piece it touches, which a second kernel adds in piece
//     order.
#pragma once

#include "common.cuh"
#include "mx4.cuh"

namespace ngram {

// ------------------------------------------------------------------ lookup

enum TableType : int { kTableBf16 = 0, kTableF32 = 1, kTableMx4 = 2 };

struct LookupParams {
  RowMap map;             // positions of this launch x D / 8 vectors
  const void* table;      // bf16 / f32 rows, or mx4 codes
  const uint8_t* scales;  // mx4 scales by rows
  const int32_t* ids;     // [n], nullptr: row i
  uint32_t V;
  int64_t pad_id;         // positions with this id get a row of zeros (negative: none)
  float scale;
  void* out;              // of position 0 of this launch, row stride out_stride elements
  int64_t out_stride;
  int64_t row0;           // first row of this launch when ids is nullptr
  uint32_t pad_pos;       // position of this launch whose row is pad_id then (2^32 - 1: none)
  int* status;
};

// Eight E2M1 codes (low halves first) to floats. The upper half of a code's fp32 is a function
// of its four bits: byte permutations look up four magnitudes at once (high bytes
// 00 3F 3F 3F 40 40 40 40, low bytes 00 00 80 C0 00 40 80 C0) and collect their signs. The
// conversion instructions (E2M1 to f16, then f16 to f32) run at an eighth of that rate.
__device__ __forceinline__ void e2m1x8(uint32_t codes, float (&x)[8]) {
  const uint32_t up = codes << 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sel = (codes >> (16 * h)) & 0x7777u;
    const uint32_t sign = __byte_perm(up, codes, h ? 0x7362 : 0x5140) & 0x80808080u;  // of codes 0 .. 3, in their bytes
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel) | sign, lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    const uint32_t m0 = __byte_perm(lo, hi, 0x5140), m1 = __byte_perm(lo, hi, 0x7362);  // codes 0, 1 and 2, 3
    x[4 * h] = __uint_as_float(m0 << 16);
    x[4 * h + 1] = __uint_as_float(m0 & 0xFFFF0000u);
    x[4 * h + 2] = __uint_as_float(m1 << 16);
    x[4 * h + 3] = __uint_as_float(m1 & 0xFFFF0000u);
  }
}

// E8M0 byte to 2^(e - 127) as the product of two powers of two of half the exponent (NaN for
// 255): neither is subnormal, and a code times the first is exact.
__device__ __forceinline__ void e8m0_halves(uint32_t e, float& s1, float& s2) {
  const int k = static_cast<int>(e) - 127, h = k >> 1;
  s1 = __uint_as_float(static_cast<uint32_t>(h + 127) << 23);
  s2 = e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(k - h + 127) << 23);
}

template <typename OutT>
__device__ __forceinline__ void store8(OutT* dst, const float (&x)[8]) {
  if constexpr (sizeof(OutT) == 2) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(dst) + 1) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <int TABLE, typename OutT, int U>
__global__ void __launch_bounds__(256) lookup_kernel(const __grid_constant__ LookupParams p) {
  pdl_wait();
  const RowPart<U> part(p.map);
  if (!part.live) return;
  constexpr int R = RowPart<U>::R;
  uint4 raw[R][U][TABLE == kTableF32 ? 2 : 1];
  uint32_t e[R][U];
  bool zero[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t pos = part.row0 + r * part.row_step;
    int64_t row = p.row0 + pos;
    zero[r] = pos >= p.map.rows || pos == p.pad_pos;
    if (p.ids && !zero[r]) {
      const int32_t id = __ldg(p.ids + pos);
      zero[r] = p.pad_id >= 0 && id == p.pad_id;
      row = id;
      if (static_cast<uint32_t>(id) >= p.V && !zero[r]) {
        set_status(p.status, NGRAM_STATUS_BAD_TOKEN);
        row = 0;
      }
    }
    const int64_t at = row * p.map.per_row + part.vec;  // in vectors of eight elements
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (zero[r] || part.vec + u * part.stride >= p.map.per_row) continue;
      const int64_t v = at + u * part.stride;
      if constexpr (TABLE == kTableBf16) {
        raw[r][u][0] = ld_stream_v4(static_cast<const uint16_t*>(p.table) + v * 8);
      } else if constexpr (TABLE == kTableF32) {
        raw[r][u][0] = ld_stream_v4(static_cast<const float*>(p.table) + v * 8);
        raw[r][u][1] = ld_stream_v4(static_cast<const float*>(p.table) + v * 8 + 4);
      } else {
        raw[r][u][0].x = __ldg(static_cast<const uint32_t*>(p.table) + v);
        e[r][u] = __ldg(p.scales + (v >> 2));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t pos = part.row0 + r * part.row_step;
    if (pos >= p.map.rows) continue;
    OutT* out = static_cast<OutT*>(p.out) + static_cast<int64_t>(pos) * p.out_stride + part.vec * 8;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (part.vec + u * part.stride >= p.map.per_row) continue;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (!zero[r]) {
        const uint4 a = raw[r][u][0];
        if constexpr (TABLE == kTableBf16) {
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            x[2 * h] = bf16_bits_to_float(w[h] & 0xFFFFu) * p.scale;
            x[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u) * p.scale;
          }
        } else if constexpr (TABLE == kTableF32) {
          const uint4 b = raw[r][u][1];
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]) * p.scale;
        } else {
          float s1, s2;
          e8m0_halves(e[r][u], s1, s2);
          e2m1x8(a.x, x);
          const float f = s1 * p.scale * s2, m = fabsf(f);
          if (m >= 0x1p-124f && m <= 0x1p124f) {  // scale * 2^k is exact: one rounding, at its product
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= f;
          } else {
            // a scale, a power of two or results near fp32's ends: the product is exact in 64 bits
            // (24 + 2 bits, exponents of at most 300), so it is rounded once, and overflows or
            // vanishes only if the result does
            const double w = static_cast<double>(s1) * static_cast<double>(p.scale) * static_cast<double>(s2);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(static_cast<double>(x[j]) * w);
          }
        }
      }
      store8<OutT>(out + u * part.stride * 8, x);
    }
  }
}

// ------------------------------------------------------------------ stable radix sort of ids
//
// Least significant digit first, `bits` bits a pass, three launches a pass: digit counts of
// each tile of kSortTile positions, an exclusive scan of every digit's counts over the tiles,
// and the scatter, which ranks a tile's positions digit by digit in their order (a warp's
// equal digits by __match_any_sync, the warps by a scan of their counts).

constexpr int kSortThreads = 256;
constexpr int kSortItems = 4;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kSortMaxBits = 8;

struct SortParams {
  const int32_t* ids;   // first pass: the ids themselves
  uint32_t V;
  int64_t pad_id;
  uint32_t n;
  const uint32_t* key_in;  // later passes
  const int32_t* pos_in;
  uint32_t* key_out;
  int32_t* pos_out;
  int shift, bits;
  uint32_t tiles;
  uint32_t* counts;     // [2^bits x tiles]
  uint32_t* totals;     // [2^bits]
  int* status;
};

// The sort key of position i: its id, or V (behind every id) for a padded position.
__device__ __forceinline__ uint32_t sort_key(const SortParams& p, uint32_t i, bool report) {
  if (p.key_in) return p.key_in[i];
  const int32_t id = p.ids[i];
  if (p.pad_id >= 0 && id == p.pad_id) return p.V;
  if (static_cast<uint32_t>(id) >= p.V) {
    if (report) set_status(p.status, NGRAM_STATUS_BAD_TOKEN);
    return 0;
  }
  return static_cast<uint32_t>(id);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortParams p) {
  __shared__ uint32_t hist[1 << kSortMaxBits];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  const uint32_t i0 = blockIdx.x * kSortTile + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = i0 + j * kSortThreads;
    if (i < p.n) atomicAdd(hist + ((sort_key(p, i, true) >> p.shift) & (bins - 1)), 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) p.counts[static_cast<size_t>(b) * p.tiles + blockIdx.x] = hist[b];
}

// Exclusive scan of one value a thread over the block (kSortThreads threads).
__device__ __forceinline__ uint32_t sort_block_scan(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < kSortThreads / 32; ++k) {
    if (k < w) before += warp_sums[k];
    total += warp_sums[k];
  }
  __syncthreads();
  return before + s - x;
}

// One block a digit: its counts over the tiles become exclusive sums, its total is kept.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(const __grid_constant__ SortParams p) {
  __shared__ uint32_t warp_sums[kSortThreads / 32];
  uint32_t* c = p.counts + static_cast<size_t>(blockIdx.x) * p.tiles;
  uint32_t carry = 0;
  for (uint32_t t0 = 0; t0 < p.tiles; t0 += kSortThreads) {
    const uint32_t t = t0 + threadIdx.x;
    const uint32_t x = t < p.tiles ? c[t] : 0u;
    uint32_t total;
    const uint32_t e = sort_block_scan(x, warp_sums, total);
    if (t < p.tiles) c[t] = carry + e;
    carry += total;
  }
  if (threadIdx.x == 0) p.totals[blockIdx.x] = carry;
}

__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const __grid_constant__ SortParams p) {
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t cnt[kWarps][1 << kSortMaxBits];
  __shared__ uint32_t start[1 << kSortMaxBits];
  __shared__ uint32_t warp_sums[kWarps];
  const int bins = 1 << p.bits;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int b = threadIdx.x; b < kWarps * (1 << kSortMaxBits); b += kSortThreads) (&cnt[0][0])[b] = 0;
  // a digit's first slot for this tile: all smaller digits, then its earlier tiles
  uint32_t ignored;
  const uint32_t tot = static_cast<int>(threadIdx.x) < bins ? p.totals[threadIdx.x] : 0u;
  const uint32_t before = sort_block_scan(tot, warp_sums, ignored);
  if (static_cast<int>(threadIdx.x) < bins)
    start[threadIdx.x] = before + p.counts[static_cast<size_t>(threadIdx.x) * p.tiles + blockIdx.x];
  __syncthreads();
  // warp w ranks positions [w * 32 * kSortItems, ...) of the tile, 32 at a time
  const uint32_t i0 = blockIdx.x * kSortTile + w * (32 * kSortItems) + lane;
  uint32_t key[kSortItems], rank[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = i0 + j * 32;
    key[j] = i < p.n ? sort_key(p, i, false) : 0u;
  }
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = i0 + j * 32;
    const uint32_t dg = i < p.n ? (key[j] >> p.shift) & (bins - 1) : 0xFFFFFFFFu;
    const uint32_t peers = __match_any_sync(0xffffffffu, dg);
    const int leader = __ffs(peers) - 1;
    uint32_t at = 0;
    if (i < p.n && lane == leader) {
      at = cnt[w][dg];
      cnt[w][dg] = at + __popc(peers);
    }
    at = __shfl_sync(0xffffffffu, at, leader);
    rank[j] = at + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t run = start[b];
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const uint32_t x = cnt[k][b];
      cnt[k][b] = run;
      run += x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = i0 + j * 32;
    if (i >= p.n) continue;
    const uint32_t at = cnt[w][(key[j] >> p.shift) & (bins - 1)] + rank[j];
    p.key_out[at] = key[j];
    p.pos_out[at] = p.pos_in ? p.pos_in[i] : static_cast<int32_t>(i);
  }
}

// ------------------------------------------------------------------ sums over sorted runs

struct GradParams {
  const uint32_t* key;    // [n] sorted; padded positions (key V) last
  const int32_t* pos;     // [n]
  uint32_t n;
  uint32_t V;
  uint32_t tiles;         // of kSortTile sorted positions
  uint32_t* tile_heads;   // [tiles]: first positions of runs in each tile
  uint32_t piece;         // positions a piece
  int32_t* piece_run;     // [ceil(n / piece)]: the run (unique id) a piece begins in
  int32_t* rows_out;      // compact form: the unique ids
  int32_t* count_out;
  const void* g;          // [n x D], row stride g_stride elements
  int64_t g_stride;
  int D, chunks;          // chunks = ceil(D / 256)
  float scale;
  float* partial;         // [pieces x 2 x D]: 0 the run a piece begins in, 1 the one it ends in
  int32_t* crossing;      // [2]: runs that cross pieces: of few pieces, of more than kJoinShort more
  int32_t* lists;         // [2 x pieces]: the pieces that they begin in, in no order
  uint32_t pieces;
  float* out;             // compact: [unique x D]; dense: [V x D], added to
  int dense;
};

__device__ __forceinline__ bool run_head(const GradParams& p, uint32_t i) {
  return i < p.n && p.key[i] < p.V && (i == 0 || p.key[i - 1] != p.key[i]);
}

__global__ void __launch_bounds__(kSortThreads) grad_heads_kernel(const __grid_constant__ GradParams p) {
  __shared__ uint32_t warp_sums[kSortThreads / 32];
  uint32_t mine = 0, total;
#pragma unroll
  for (int j = 0; j < kSortItems; ++j)
    mine += run_head(p, blockIdx.x * kSortTile + threadIdx.x * kSortItems + j) ? 1u : 0u;
  sort_block_scan(mine, warp_sums, total);
  if (threadIdx.x == 0) p.tile_heads[blockIdx.x] = total;
}

// Runs numbered in order: the id of each (compact form), the run every piece begins in, and
// their count.
__global__ void __launch_bounds__(kSortThreads) grad_number_kernel(const __grid_constant__ GradParams p) {
  __shared__ uint32_t warp_sums[kSortThreads / 32];
  uint32_t before = 0, total;
  for (uint32_t t = threadIdx.x; t < blockIdx.x; t += kSortThreads) before += p.tile_heads[t];
  sort_block_scan(before, warp_sums, total);
  const uint32_t base = total;  // heads of all earlier tiles
  const uint32_t i0 = blockIdx.x * kSortTile + threadIdx.x * kSortItems;
  uint32_t mine = 0;
  bool head[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    head[j] = run_head(p, i0 + j);
    mine += head[j] ? 1u : 0u;
  }
  uint32_t run = base + sort_block_scan(mine, warp_sums, total);  // heads before i0
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = i0 + j;
    if (head[j]) {
      if (p.rows_out) p.rows_out[run] = static_cast<int32_t>(p.key[i]);
      ++run;
    }
    if (i < p.n && i % p.piece == 0) p.piece_run[i / p.piece] = static_cast<int32_t>(run) - 1;
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) p.crossing[threadIdx.x] = 0;
  if (p.count_out && blockIdx.x + 1 == p.tiles && threadIdx.x == 0) *p.count_out = static_cast<int32_t>(base + total);
}

template <typename T>
__device__ __forceinline__ void grad_load8(const T* src, uint4 (&r)[sizeof(T) / 2]) {
  r[0] = ld_stream_v4(src);
  if constexpr (sizeof(T) == 4) r[1] = ld_stream_v4(src + 4);
}

template <typename T>
__device__ __forceinline__ void grad_add8(const uint4 (&r)[sizeof(T) / 2], float (&acc)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      acc[2 * h] += bf16_bits_to_float(w[h] & 0xFFFFu);
      acc[2 * h + 1] += bf16_bits_to_float(w[h] >> 16);
    }
  } else {
    const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += __uint_as_float(w[j]);
  }
}

// The finished sum of run `run` (id `key`) at column c: scaled, and stored or added.
__device__ __forceinline__ void grad_finish(const GradParams& p, int32_t run, uint32_t key, int c, const float (&acc)[8]) {
  float4* dst = reinterpret_cast<float4*>(p.out + static_cast<int64_t>(p.dense ? static_cast<int64_t>(key) : run) * p.D + c);
  float4 a = make_float4(acc[0] * p.scale, acc[1] * p.scale, acc[2] * p.scale, acc[3] * p.scale);
  float4 b = make_float4(acc[4] * p.scale, acc[5] * p.scale, acc[6] * p.scale, acc[7] * p.scale);
  if (p.dense) {
    const float4 x = dst[0], y = dst[1];
    a = make_float4(x.x + a.x, x.y + a.y, x.z + a.z, x.w + a.w);
    b = make_float4(y.x + b.x, y.y + b.y, y.z + b.z, y.w + b.w);
  }
  dst[0] = a;
  dst[1] = b;
}

__device__ __forceinline__ float4* grad_partial(const GradParams& p, uint32_t piece, int which, int c) {
  return reinterpret_cast<float4*>(p.partial + (static_cast<size_t>(piece) * 2 + which) * p.D + c);
}

constexpr int kJoinShort = 16;  // pieces after its first that a warp alone joins a run of

// One warp a (piece, 256 columns), eight columns a lane, kGradLoads rows in flight.
constexpr int kGradLoads = 8;

template <typename T, int PIECE>
__global__ void __launch_bounds__(256) grad_reduce_kernel(const __grid_constant__ GradParams p) {
  constexpr int kLanes = PIECE < 32 ? PIECE : 32;  // sorted positions a lane holds one of at a time
  pdl_launch_dependents();
  pdl_wait();
  const uint64_t item = static_cast<uint64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t piece = static_cast<uint32_t>(item / p.chunks);
  const int c = static_cast<int>(item - static_cast<uint64_t>(piece) * p.chunks) * 256 + lane * 8;
  const uint32_t begin = piece * PIECE;
  if (begin >= p.n || p.key[begin] >= p.V) return;  // padded positions are last
  const bool on = c < p.D;  // lanes past the last column only carry their position
  int32_t run = p.piece_run[piece];
  uint32_t cur = p.key[begin];
  bool open = begin > 0 && p.key[begin - 1] == cur;  // the current run began in an earlier piece
  const T* g = static_cast<const T*>(p.g) + c;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto finish = [&](uint32_t id) {
    if (on) grad_finish(p, run, id, c, acc);
  };
  auto leave = [&](int which) {
    if (!on) return;
    float4* dst = grad_partial(p, piece, which, c);
    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  };
  int len = kLanes;
#pragma unroll 1
  for (int part = 0; part < PIECE / kLanes && len == kLanes; ++part) {
    const uint32_t i = begin + part * kLanes + lane;
    const bool mine = lane < kLanes && i < p.n;
    const uint32_t key = mine ? p.key[i] : p.V;
    const int32_t pos = mine ? p.pos[i] : 0;
    len = __popc(__ballot_sync(0xffffffffu, key < p.V));
#pragma unroll 1
    for (int r0 = 0; r0 < len; r0 += kGradLoads) {
      uint4 rows[kGradLoads][sizeof(T) / 2];
#pragma unroll
      for (int r = 0; r < kGradLoads; ++r) {
        const int32_t at = __shfl_sync(0xffffffffu, pos, (r0 + r) & 31);
        if (on && r0 + r < len) grad_load8<T>(g + static_cast<int64_t>(at) * p.g_stride, rows[r]);
      }
#pragma unroll
      for (int r = 0; r < kGradLoads; ++r) {
        const uint32_t kr = __shfl_sync(0xffffffffu, key, (r0 + r) & 31);
        if (r0 + r >= len) continue;
        if (kr != cur) {
          if (open) leave(0); else finish(cur);
          open = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = 0.f;
          cur = kr;
          ++run;
        }
        grad_add8<T>(rows[r], acc);
      }
    }
  }
  const uint64_t end = static_cast<uint64_t>(begin) + PIECE;
  if (end < p.n && p.key[end] == cur) {  // it goes on in the next piece
    leave(open ? 0 : 1);
    if (!open && c == 0) {  // it begins here: for the join (one lane of the piece's warps)
      const uint64_t far = end + static_cast<uint64_t>(kJoinShort) * PIECE;
      const int which = far < p.n && p.key[far] == cur ? 1 : 0;
      p.lists[static_cast<size_t>(which) * p.pieces + atomicAdd(p.crossing + which, 1)] = static_cast<int32_t>(piece);
    }
  } else if (open) {
    leave(0);
  } else {
    finish(cur);
  }
}

// The runs that cross pieces: their partial sums are added in piece order, kJoinLoads of them in
// flight, 128 columns at a time: a run of few pieces by a warp; a long one, of a frequent id, by a
// block, whose warps add an eighth of the pieces each and whose first warp adds those. The runs
// come from the lists that the sums left, so few blocks suffice and none looks for work (a warp
// for every piece, joining whatever its run's length: 92 us of 130 for 65536 Zipf ids of 256
// columns).
constexpr int kJoinLoads = 8;
constexpr int kJoinBlocksPerSm = 4;

__global__ void __launch_bounds__(256, kJoinBlocksPerSm) grad_join_kernel(const __grid_constant__ GradParams p) {
  __shared__ float4 s_part[8][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t chunks = static_cast<uint32_t>((p.D + 127) / 128);
  auto partial = [&](uint32_t q, int which, int c) {
    return reinterpret_cast<const float4*>(p.partial + (static_cast<size_t>(q) * 2 + which) * p.D + c);
  };
  auto add = [](float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  };
  // pieces [q0, q1) of a run that began earlier, onto acc
  auto sum = [&](float4& acc, uint32_t q0, uint32_t q1, int c) {
    for (uint32_t q = q0; q < q1; q += kJoinLoads) {
      float4 x[kJoinLoads];
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k)
        if (q + k < q1) x[k] = __ldcg(partial(q + k, 0, c));
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k)
        if (q + k < q1) add(acc, x[k]);
    }
  };
  // the finished sum of the run that begins in `piece` (its number: that of the next piece's
  // beginning, which lies in it)
  auto finish = [&](uint32_t piece, uint32_t key, int c, const float4& acc) {
    const int64_t row = p.dense ? static_cast<int64_t>(key) : p.piece_run[piece + 1];
    float4* dst = reinterpret_cast<float4*>(p.out + row * p.D + c);
    float4 y = make_float4(acc.x * p.scale, acc.y * p.scale, acc.z * p.scale, acc.w * p.scale);
    if (p.dense) add(y, *dst);
    *dst = y;
  };
  auto key_of = [&](uint32_t piece) { return p.key[static_cast<uint64_t>(piece + 1) * p.piece - 1]; };
  // pieces after `piece` that begin with its last id: the lanes look 32 steps ahead at once, of
  // 1024 pieces each (a long run), then of 32, then of one
  auto pieces_after = [&](uint32_t piece, uint32_t key, uint32_t stride) {
    uint64_t m = 0;
    for (; stride; stride >>= 5) {
      for (bool more = true; more;) {
        const uint64_t at = (piece + m + static_cast<uint64_t>(lane + 1) * stride) * p.piece;
        const unsigned in = __ballot_sync(0xffffffffu, at < p.n && p.key[at] == key);
        more = in == 0xffffffffu;
        m += static_cast<uint64_t>(more ? 32 : __ffs(~in) - 1) * stride;
      }
    }
    return static_cast<uint32_t>(m);
  };
  const uint64_t long_items = static_cast<uint64_t>(p.crossing[1]) * chunks;
  for (uint64_t item = blockIdx.x; item < long_items; item += gridDim.x) {
    const uint32_t piece = static_cast<uint32_t>(p.lists[p.pieces + item / chunks]);
    const int c = static_cast<int>(item % chunks) * 128 + lane * 4;
    const uint32_t key = key_of(piece), m = pieces_after(piece, key, 1024);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.D) {
      if (w == 0) acc = __ldcg(partial(piece, 1, c));
      sum(acc, piece + 1 + static_cast<uint32_t>(static_cast<uint64_t>(m) * w / 8),
          piece + 1 + static_cast<uint32_t>(static_cast<uint64_t>(m) * (w + 1) / 8), c);
    }
    s_part[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < p.D) {
#pragma unroll
      for (int k = 1; k < 8; ++k) add(acc, s_part[k][lane]);
      finish(piece, key, c, acc);
    }
    __syncthreads();
  }
  const uint64_t short_items = static_cast<uint64_t>(p.crossing[0]) * chunks;
  for (uint64_t item = static_cast<uint64_t>(blockIdx.x) * 8 + w; item < short_items; item += static_cast<uint64_t>(gridDim.x) * 8) {
    const uint32_t piece = static_cast<uint32_t>(p.lists[item / chunks]);
    const int c = static_cast<int>(item % chunks) * 128 + lane * 4;
    const uint32_t key = key_of(piece), m = pieces_after(piece, key, 1);
    if (c >= p.D) continue;
    float4 acc = __ldcg(partial(piece, 1, c));
    sum(acc, piece + 1, piece + 1 + m, c);
    finish(piece, key, c, acc);
  }
}

// ------------------------------------------------------------------ sort in one cluster
//
// Up to kClusterMax positions are sorted and their runs numbered in one launch, by a cluster of
// CTAs that hold all of them in shared memory: each CTA ranks its positions by digit, the CTAs
// exchange their digit counts, and every position is stored straight into its place in the
// shared memory of the CTA that the place belongs to. Positions past n carry the largest key,
// so they stay last. The gradient of 1000 / 32768 / 65536 rows of eight columns
// takes 14 / 32 / 42 us in a graph, against 28 / 45 / 49 with the tiled sort and the numbering
// kernels, which are ten launches more (15 / 32 / 42 against 45 / 67 / 71 one call after another).
// Devices that place no cluster of the size take the tiled sort too (cluster_limit).

constexpr int kClusterThreads = 1024;
constexpr int kClusterMaxItems = 4;  // positions a thread: 1, 2 or 4, as few as hold n
constexpr int kClusterCtas = 16;
constexpr int kClusterMax = kClusterThreads * kClusterMaxItems * kClusterCtas;
constexpr int kClusterMaxBits = 9;

template <int ITEMS>
struct ClusterSmem {
  uint2 item[kClusterThreads * ITEMS];  // key, position
  uint16_t warp_count[kClusterThreads / 32][1 << kClusterMaxBits];
  uint32_t count[kClusterCtas][1 << kClusterMaxBits];  // of every CTA, pushed by it
  uint32_t start[1 << kClusterMaxBits];
  uint32_t heads[kClusterCtas];
  uint32_t warp_sums[32];
};

struct ClusterSortParams {
  SortParams s;    // ids, V, pad_id, n, bits; key_out and pos_out of the sorted positions
  int passes;
  GradParams r;    // rows_out, count_out, piece_run
};

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Lanes whose digit equals this lane's: a vote a bit. (__match_any_sync does it in one
// instruction, at about 2 us an item and pass for the 32 warps of a block.)
__device__ __forceinline__ uint32_t match_digit(uint32_t dg, int bits) {
  uint32_t same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const bool on = (dg >> b) & 1u;
    const uint32_t votes = __ballot_sync(0xffffffffu, on);
    same &= on ? votes : ~votes;
  }
  return same;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Every thread of the cluster. The block's own barrier comes first: it brings each warp together
// again after the divergent code in front of it, which the aligned cluster barrier requires.
__device__ __forceinline__ void cluster_barrier(uint32_t ctas) {
  __syncthreads();
  if (ctas > 1) cluster_sync();
}

// Exclusive scan of one value a thread over 1024 threads.
__device__ __forceinline__ uint32_t cluster_block_scan(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();  // warp_sums may still be read from the scan before
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  const uint32_t ws = warp_sums[lane];
  uint32_t p = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += y;
  }
  total = __shfl_sync(0xffffffffu, p, 31);
  return __shfl_sync(0xffffffffu, p - ws, w) + s - x;
}

template <int ITEMS>
__global__ void __launch_bounds__(kClusterThreads, 1) sort_cluster_kernel(const __grid_constant__ ClusterSortParams a) {
  constexpr uint32_t kItems = kClusterThreads * ITEMS;  // of one CTA
  constexpr int kWarpItems = 32 * ITEMS;
  extern __shared__ __align__(16) uint8_t cluster_raw[];
  auto& m = *reinterpret_cast<ClusterSmem<ITEMS>*>(cluster_raw);
  pdl_wait();
  pdl_launch_dependents();
  const SortParams& p = a.s;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  const int bins = 1 << p.bits;
  const uint32_t base = rank * kItems;
  constexpr uint32_t kLast = 0xFFFFFFFFu;
  uint32_t key[ITEMS];
  int32_t pos[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const uint32_t i = base + w * kWarpItems + j * 32 + lane;
    key[j] = i < p.n ? sort_key(p, i, true) : kLast;
    pos[j] = static_cast<int32_t>(i);
  }
  cluster_barrier(ctas);  // every CTA runs before its shared memory is written
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * p.bits;
    uint32_t rk[ITEMS];
    for (int b = lane; b < bins; b += 32) m.warp_count[w][b] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint32_t dg = (key[j] >> shift) & (bins - 1);
      const uint32_t peers = match_digit(dg, p.bits);
      const uint32_t before = m.warp_count[w][dg];
      __syncwarp();
      rk[j] = before + __popc(peers & ((1u << lane) - 1u));
      if (lane == __ffs(peers) - 1) m.warp_count[w][dg] = static_cast<uint16_t>(before + __popc(peers));
      __syncwarp();
    }
    __syncthreads();
    if (tid < bins) {  // the digit's ranks over the CTA's warps; its count to every CTA
      uint32_t run = 0;
#pragma unroll 8
      for (int k = 0; k < kClusterThreads / 32; ++k) {
        const uint32_t x = m.warp_count[k][tid];
        m.warp_count[k][tid] = static_cast<uint16_t>(run);
        run += x;
      }
      const uint32_t to = smem_u32(&m.count[rank][tid]);
      for (uint32_t r = 0; r < ctas; ++r) st_cluster_u32(map_to_cta(to, r), run);
    }
    cluster_barrier(ctas);
    uint32_t all = 0, lower = 0, ignored;
    if (tid < bins)
      for (uint32_t r = 0; r < ctas; ++r) {
        const uint32_t x = m.count[r][tid];
        if (r < rank) lower += x;
        all += x;
      }
    const uint32_t smaller = cluster_block_scan(all, m.warp_sums, ignored);
    if (tid < bins) m.start[tid] = smaller + lower;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint32_t dg = (key[j] >> shift) & (bins - 1);
      const uint32_t at = m.start[dg] + m.warp_count[w][dg] + rk[j];
      const uint32_t cta = at / kItems, in = at % kItems;
      st_cluster_v2(map_to_cta(smem_u32(&m.item[in]), cta), key[j], static_cast<uint32_t>(pos[j]));
    }
    cluster_barrier(ctas);
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const uint2 x = m.item[w * kWarpItems + j * 32 + lane];
      key[j] = x.x;
      pos[j] = static_cast<int32_t>(x.y);
    }
  }
  // sorted: out, and the runs numbered, ITEMS neighbouring positions a thread
  const uint32_t l0 = tid * ITEMS;
  uint32_t prev = l0 > 0 ? m.item[l0 - 1].x : kLast;
  const bool first = rank == 0 && tid == 0;
  if (tid == 0 && rank > 0) prev = ld_cluster_u32(map_to_cta(smem_u32(&m.item[kItems - 1].x), rank - 1));
  bool head[ITEMS];
  uint32_t mine = 0, k4[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const uint2 x = m.item[l0 + j];
    k4[j] = x.x;
    head[j] = base + l0 + j < p.n && k4[j] < p.V && ((first && j == 0) || k4[j] != prev);
    prev = k4[j];
    mine += head[j] ? 1u : 0u;
    if (base + l0 + j < p.n) {
      p.key_out[base + l0 + j] = k4[j];
      p.pos_out[base + l0 + j] = static_cast<int32_t>(x.y);
    }
  }
  uint32_t total;
  uint32_t run = cluster_block_scan(mine, m.warp_sums, total);
  if (tid < static_cast<int>(ctas)) st_cluster_u32(map_to_cta(smem_u32(&m.heads[rank]), tid), total);
  cluster_barrier(ctas);
  uint32_t all = 0;
  for (uint32_t r = 0; r < ctas; ++r) {
    if (r < rank) run += m.heads[r];
    all += m.heads[r];
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const uint32_t i = base + l0 + j;
    if (head[j]) {
      if (a.r.rows_out) a.r.rows_out[run] = static_cast<int32_t>(k4[j]);
      ++run;
    }
    if (i < p.n && i % a.r.piece == 0) a.r.piece_run[i / a.r.piece] = static_cast<int32_t>(run) - 1;
  }
  if (rank == 0 && tid < 2) a.r.crossing[tid] = 0;
  if (a.r.count_out && first) *a.r.count_out = static_cast<int32_t>(all);
}

}  // namespace ngram
