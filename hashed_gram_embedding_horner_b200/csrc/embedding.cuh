// One table's lookup, out[i] = scale * table[ids[i]], and its gradient by sorted ids.
//
// Lookup: the table in bf16, f32 or mx4 (by rows, see mx4.cuh); eight elements a thread, the
// next positions' loads in flight beside them.
//
// Gradient: dTable[v] = scale * sum_{i : ids[i] = v} g_i. The positions are sorted by id with
// a stable radix sort; runs of equal ids are summed in fp32 by whoever owns them, without
// atomics, so the sum's order, and its bits, depend on the ids alone:
//   - the sorted positions are cut into pieces of kGradPiece; a warp sums the rows of a piece
//     for 256 columns, in ascending position order;
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
  const void* table;      // bf16 / f32 rows, or mx4 codes
  const uint8_t* scales;  // mx4 scales by rows
  const int32_t* ids;     // [n], nullptr: row i
  uint32_t V;
  int64_t pad_id;         // positions with this id get a row of zeros (negative: none)
  FastDiv per_row;        // D / 8
  uint32_t vecs;          // n * D / 8 of this launch
  float scale;
  void* out;              // of position 0 of this launch, row stride out_stride elements
  int64_t out_stride;
  int64_t row0;           // first row of this launch when ids is nullptr
  int* status;
};

constexpr int kLookupUnroll = 4;

// Eight E2M1 codes (low halves first) to floats.
__device__ __forceinline__ void e2m1x8(uint32_t codes, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t f16;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(f16) : "r"(codes >> (8 * h)));
    float lo, hi;
    asm("{\n\t.reg .b16 a, c;\n\tmov.b32 {a, c}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, c;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(f16));
    x[2 * h] = lo;
    x[2 * h + 1] = hi;
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

template <int TABLE, typename OutT>
__global__ void __launch_bounds__(256) lookup_kernel(const __grid_constant__ LookupParams p) {
  const uint32_t base = blockIdx.x * (256u * kLookupUnroll) + threadIdx.x;
  const uint32_t per_row = p.per_row.d;
  int64_t row[kLookupUnroll];  // -1: zeros
  uint32_t c[kLookupUnroll], pos[kLookupUnroll];
#pragma unroll
  for (int u = 0; u < kLookupUnroll; ++u) {
    const uint32_t v = base + u * 256u;
    row[u] = -1;
    if (v >= p.vecs) continue;
    pos[u] = p.per_row.div(v);
    c[u] = v - pos[u] * per_row;
    if (!p.ids) {
      row[u] = p.row0 + pos[u];
      continue;
    }
    const int32_t id = __ldg(p.ids + pos[u]);
    if (p.pad_id >= 0 && id == p.pad_id) continue;
    row[u] = id;
    if (static_cast<uint32_t>(id) >= p.V) {
      set_status(p.status, NGRAM_STATUS_BAD_TOKEN);
      row[u] = 0;
    }
  }
  uint4 raw[kLookupUnroll][TABLE == kTableF32 ? 2 : 1];
  uint32_t e[kLookupUnroll];
#pragma unroll
  for (int u = 0; u < kLookupUnroll; ++u) {
    if (row[u] < 0) continue;
    const size_t at = static_cast<size_t>(row[u]) * per_row + c[u];  // in units of eight elements
    if constexpr (TABLE == kTableBf16) {
      raw[u][0] = ld_stream_v4(static_cast<const uint16_t*>(p.table) + at * 8);
    } else if constexpr (TABLE == kTableF32) {
      raw[u][0] = ld_stream_v4(static_cast<const float*>(p.table) + at * 8);
      raw[u][1] = ld_stream_v4(static_cast<const float*>(p.table) + at * 8 + 4);
    } else {
      raw[u][0].x = __ldg(static_cast<const uint32_t*>(p.table) + at);
      e[u] = __ldg(p.scales + (at >> 2));
    }
  }
#pragma unroll
  for (int u = 0; u < kLookupUnroll; ++u) {
    const uint32_t v = base + u * 256u;
    if (v >= p.vecs) continue;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row[u] >= 0) {
      if constexpr (TABLE == kTableBf16) {
        const uint32_t w[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          x[2 * h] = bf16_bits_to_float(w[h] & 0xFFFFu) * p.scale;
          x[2 * h + 1] = bf16_bits_to_float(w[h] >> 16) * p.scale;
        }
      } else if constexpr (TABLE == kTableF32) {
        const uint32_t w[8] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w,
                               raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]) * p.scale;
      } else {
        // 2^k in two halves around the user's scale: each product by one is exact, so a value
        // is rounded once, at the scale, and overflows only if the result does
        float s1, s2;
        e8m0_halves(e[u], s1, s2);
        e2m1x8(raw[u][0].x, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * s1 * p.scale * s2;
      }
    }
    store8<OutT>(static_cast<OutT*>(p.out) + static_cast<int64_t>(pos[u]) * p.out_stride + c[u] * 8, x);
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

constexpr int kGradPiece = 32;

struct GradParams {
  const uint32_t* key;    // [n] sorted; padded positions (key V) last
  const int32_t* pos;     // [n]
  uint32_t n;
  uint32_t V;
  uint32_t tiles;         // of kSortTile sorted positions
  uint32_t* tile_heads;   // [tiles]: first positions of runs in each tile
  int32_t* piece_run;     // [ceil(n / kGradPiece)]: the run (unique id) a piece begins in
  int32_t* rows_out;      // compact form: the unique ids
  int32_t* count_out;
  const void* g;          // [n x D], row stride g_stride elements
  int64_t g_stride;
  int D, chunks;          // chunks = ceil(D / 256)
  float scale;
  float* partial;         // [pieces x 2 x D]: 0 the run a piece begins in, 1 the one it ends in
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
    if (i < p.n && i % kGradPiece == 0) p.piece_run[i / kGradPiece] = static_cast<int32_t>(run) - 1;
  }
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

// One warp a (piece, 256 columns), eight columns a lane, kGradLoads rows in flight.
constexpr int kGradLoads = 8;

template <typename T>
__global__ void __launch_bounds__(256) grad_reduce_kernel(const __grid_constant__ GradParams p) {
  const uint64_t item = static_cast<uint64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t piece = static_cast<uint32_t>(item / p.chunks);
  const int c = static_cast<int>(item - static_cast<uint64_t>(piece) * p.chunks) * 256 + lane * 8;
  const uint32_t k0 = piece * kGradPiece;
  if (k0 >= p.n) return;
  // this lane's sorted position of the piece
  const uint32_t i = k0 + lane;
  const uint32_t key = i < p.n ? p.key[i] : p.V;
  const int32_t pos = i < p.n ? p.pos[i] : 0;
  const int len = __popc(__ballot_sync(0xffffffffu, key < p.V));  // padded positions are last
  if (len == 0) return;
  const bool on = c < p.D;  // lanes past the last column only carry their position
  const uint32_t first = __shfl_sync(0xffffffffu, key, 0), last = __shfl_sync(0xffffffffu, key, len - 1);
  const bool from_before = k0 > 0 && p.key[k0 - 1] == first;
  const bool to_after = len == kGradPiece && k0 + kGradPiece < p.n && p.key[k0 + kGradPiece] == last;
  int32_t run = p.piece_run[piece];
  const T* g = static_cast<const T*>(p.g) + c;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool open = from_before;  // the current run began in an earlier piece
  auto finish = [&](uint32_t id) {
    if (on) grad_finish(p, run, id, c, acc);
  };
  auto leave = [&](int which) {
    if (!on) return;
    float4* dst = grad_partial(p, piece, which, c);
    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  };
  uint32_t cur = first;
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
  if (to_after) leave(open ? 0 : 1);
  else if (open) leave(0);
  else finish(cur);
}

// The runs that cross pieces: one warp a (piece whose last run begins in it and goes on, 256
// columns) adds the partial sums in piece order.
__global__ void __launch_bounds__(256) grad_join_kernel(const __grid_constant__ GradParams p) {
  const uint64_t item = static_cast<uint64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t piece = static_cast<uint32_t>(item / p.chunks);
  const int c = static_cast<int>(item - static_cast<uint64_t>(piece) * p.chunks) * 256 + lane * 8;
  const uint64_t k0 = static_cast<uint64_t>(piece) * kGradPiece, k1 = k0 + kGradPiece;
  if (k1 >= p.n) return;
  const uint32_t key = p.key[k1 - 1];
  if (key >= p.V || p.key[k1] != key) return;
  if (p.key[k0] == key && k0 > 0 && p.key[k0 - 1] == key) return;  // it began earlier
  if (c >= p.D) return;
  // the run's last position: pieces up to the one that holds it
  uint32_t lo = static_cast<uint32_t>(k1), hi = p.n;  // key[lo] == key, key[hi] beyond
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (p.key[mid] == key) lo = mid; else hi = mid;
  }
  const uint32_t last = lo / kGradPiece;
  float acc[8];
  {
    const float4* s = grad_partial(p, piece, 1, c);
    const float4 a = __ldcg(s), b = __ldcg(s + 1);
    acc[0] = a.x; acc[1] = a.y; acc[2] = a.z; acc[3] = a.w;
    acc[4] = b.x; acc[5] = b.y; acc[6] = b.z; acc[7] = b.w;
  }
#pragma unroll 4
  for (uint32_t q = piece + 1; q <= last; ++q) {
    const float4* s = grad_partial(p, q, 0, c);
    const float4 a = __ldcg(s), b = __ldcg(s + 1);
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
  }
  // the run's number: that of the next piece's beginning, which lies in it
  grad_finish(p, p.piece_run[piece + 1], key, c, acc);
}

}  // namespace ngram
