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

// ------------------------------------------------------------------ quantisation

// Two floats to one byte of E2M1 codes: round to nearest, ties to even, saturating at 6;
// the first in the low half.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

struct Mx4QuantParams {
  const void* src;     // [rows x cols], row stride src_stride elements
  int64_t src_stride;
  uint32_t vecs;       // rows * cols / 8 of this launch
  FastDiv per_row;     // cols / 8
  int64_t row0;        // first row of this launch (tiles)
  int cols, kt;        // kt = ceil(cols / 128)
  uint8_t* codes;      // of row 0 of this launch
  uint8_t* scales;     // rows: of row 0 of this launch; tiles: of row 0 of the array
  int tiles;           // 1: scales in tiles
};

constexpr int kMx4QuantUnroll = 4;

// Eight elements of a row as floats; VEC: 16-byte loads.
template <typename T, bool VEC>
__device__ __forceinline__ void mx4_load8(const T* src, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
    if constexpr (VEC) {
      const uint4 v = ld_stream_v4(src);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h] = src[2 * h] | (static_cast<uint32_t>(src[2 * h + 1]) << 16);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      x[2 * h] = bf16_bits_to_float(w[h] & 0xFFFFu);
      x[2 * h + 1] = bf16_bits_to_float(w[h] >> 16);
    }
  } else {
    if constexpr (VEC) {
      const uint4 a = ld_stream_v4(src), b = ld_stream_v4(src + 4);
      x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
      x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
      for (int h = 0; h < 8; ++h) x[h] = src[h];
    }
  }
}

// A block's scale byte: two below the exponent of its largest magnitude (the exponent of
// E2M1's largest power of two is 2), clamped to 2^-127; 0 for a block of zeros, 255 (NaN)
// for a block that holds an infinity or a NaN. `amax` is the bits of the largest magnitude:
// they order as the magnitudes do, infinities and NaN above every number.
__device__ __forceinline__ int mx4_scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255;
  const int e = static_cast<int>(amax >> 23) - 2;  // subnormal magnitudes: below 2^-126, clamped
  return e < 0 ? 0 : e;
}
// 2^(127 - e), the factor that undoes scale byte e <= 252.
__device__ __forceinline__ float mx4_inverse(int e) { return __uint_as_float(static_cast<uint32_t>(254 - e) << 23); }

// Four lanes hold the 32 elements of a block, 8 each: the maximum by two shuffles, then one
// conversion instruction for two elements; every lane's 16- or 32-byte load and 4-byte store
// are part of a warp-wide contiguous access, and each thread has kMx4QuantUnroll of them in
// flight. One pass: 2 or 4 bytes read and 17/32 written an element, bound by HBM.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const __grid_constant__ Mx4QuantParams p) {
  const T* src = static_cast<const T*>(p.src);
  const uint32_t base = blockIdx.x * (256u * kMx4QuantUnroll) + threadIdx.x;
  float x[kMx4QuantUnroll][8];
#pragma unroll
  for (int u = 0; u < kMx4QuantUnroll; ++u) {
    const uint32_t v = base + u * 256u;
    if (v < p.vecs) {
      const uint32_t r = p.per_row.div(v), c = (v - r * p.per_row.d) * 8;
      mx4_load8<T, VEC>(src + static_cast<int64_t>(r) * p.src_stride + c, x[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kMx4QuantUnroll; ++u) {
    const uint32_t v = base + u * 256u;
    uint32_t amax = 0;
    if (v < p.vecs) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = __float_as_uint(x[u][j]) & 0x7FFFFFFFu;
        amax = m > amax ? m : amax;
      }
    }
    uint32_t other = __shfl_xor_sync(0xffffffffu, amax, 1);
    amax = other > amax ? other : amax;
    other = __shfl_xor_sync(0xffffffffu, amax, 2);
    amax = other > amax ? other : amax;
    if (v >= p.vecs) continue;
    const int e = mx4_scale_byte(amax);
    uint32_t codes = 0;
    if (e != 255) {
      const float inv = mx4_inverse(e);
#pragma unroll
      for (int j = 0; j < 4; ++j) codes |= e2m1x2(x[u][2 * j] * inv, x[u][2 * j + 1] * inv) << (8 * j);
    }
    reinterpret_cast<uint32_t*>(p.codes)[v] = codes;
    if ((v & 3u) == 0) {
      if (!p.tiles) {
        p.scales[v >> 2] = static_cast<uint8_t>(e);
      } else {
        const uint32_t r = p.per_row.div(v);
        const int b = static_cast<int>(v - r * p.per_row.d) >> 2;
        uint8_t* at = p.scales + mx4_tile_at(p.row0 + r, b, p.kt);
        *at = static_cast<uint8_t>(e);
        // the row's blocks end inside a tile: the rest of the tile's row is read as scales of
        // zero codes, and must not be NaN
        if (b == p.cols / kMxBlock - 1)
          for (int k = 1; ((b + k) & 3) != 0; ++k) at[k] = 0;
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
  uint32_t Vs[kMaxS];
  const int32_t* idx;     // [T x S]
  const int32_t* tokens;  // [T]: only checked (the projection's epilogue reads E_0 by them)
  uint32_t V0;
  uint32_t T;
  int S, row_blocks;      // row_blocks = d / 32, blocks of one sub-row
  FastDiv by_row, by_sub; // ceil(D / 128) * 4 blocks of a padded row; row_blocks
  int blocks;             // D / 32
  int kt;
  uint8_t* G;             // [T x D / 2] codes
  uint8_t* Gs;            // scales, in tiles
  int* status;
};

constexpr int kMx4GatherUnroll = 4;

// G[i] = the concatenated 4-bit sub-rows of token i, its scales in tiles: one 16-byte code
// block and one scale byte a thread, kMx4GatherUnroll of each in flight; four neighbouring
// threads' scale bytes leave as one word. 17/32 bytes an element each way: bound by HBM's
// random rows at first sight of a row, and by L2 after (G is read back from there).
__global__ void __launch_bounds__(256) mx4_gather_kernel(const __grid_constant__ Mx4GatherParams p) {
  const uint32_t total = p.T * p.by_row.d;
  const uint32_t base = blockIdx.x * (256u * kMx4GatherUnroll) + threadIdx.x;
  uint4 code[kMx4GatherUnroll];
  uint32_t scale[kMx4GatherUnroll];
#pragma unroll
  for (int u = 0; u < kMx4GatherUnroll; ++u) {
    const uint32_t v = base + u * 256u;
    scale[u] = 0;
    if (v < total) {
      const uint32_t i = p.by_row.div(v), b = v - i * p.by_row.d;
      if (b == 0 && p.tokens && static_cast<uint32_t>(p.tokens[i]) >= p.V0) set_status(p.status, NGRAM_STATUS_BAD_TOKEN);
      if (b < static_cast<uint32_t>(p.blocks)) {
        const uint32_t s = p.by_sub.div(b), c = b - s * p.row_blocks;
        uint32_t row = static_cast<uint32_t>(p.idx[static_cast<int64_t>(i) * p.S + s]);
        if (row >= p.Vs[s]) {
          set_status(p.status, NGRAM_STATUS_BAD_TOKEN);
          row = 0;
        }
        const size_t at = static_cast<size_t>(row) * p.row_blocks + c;
        code[u] = ld_stream_v4(p.E[s].codes + at * 16);
        scale[u] = __ldg(p.E[s].scales + at);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kMx4GatherUnroll; ++u) {
    const uint32_t v = base + u * 256u;
    uint32_t w = scale[u] << ((threadIdx.x & 3) * 8);
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    if (v >= total) continue;
    const uint32_t i = p.by_row.div(v), b = v - i * p.by_row.d;
    if (b < static_cast<uint32_t>(p.blocks))
      *reinterpret_cast<uint4*>(p.G + (static_cast<size_t>(i) * p.blocks + b) * 16) = code[u];
    if ((threadIdx.x & 3) == 0)
      *reinterpret_cast<uint32_t*>(p.Gs + mx4_tile_at(i, static_cast<int>(b), p.kt)) = w;
  }
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
  CUtensorMap A;  // [M x K / 2] bytes, box 128 x 128 rows
  CUtensorMap B;  // [N x K / 2] bytes, box 128 x BN rows
};

struct Mx4GemmParams {
  const uint8_t* sa;  // scale tiles
  const uint8_t* sb;
  int M, N, K;
  int kt;             // ceil(K / 128): scale tiles of a row block
  int num_m_blocks, num_n_blocks, num_k_blocks;  // k-blocks of 256
  float scale;
  const int32_t* tokens;  // E_0 rows to add (nullptr: none)
  const void* E0;         // [V0 x N], element type of out
  uint32_t V0;
  void* out;
  int64_t ldo;            // elements
  int vec;                // out rows admit 16-byte stores
  int* status;
};

constexpr int kMxThreads = 256;  // warp 0 loads, warp 1 MMA and TMEM, warps 4-7 epilogue

template <int BN, int STAGES>
struct Mx4Smem {
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = BN * 128;
  static constexpr int kSfbRows = BN > 128 ? BN / 128 : 1;  // row blocks of B's scales a tile touches
  static constexpr int kSfaOffset = kABytes + kBBytes;
  static constexpr int kSfbOffset = kSfaOffset + 2 * kMxTileBytes;
  static constexpr int kStageBytes = kSfbOffset + kSfbRows * 2 * kMxTileBytes;
  static constexpr int kBarOffset = STAGES * kStageBytes;
  static constexpr int kNumBars = 2 * STAGES + 5;
  static constexpr int kEpiOffset = (kBarOffset + kNumBars * 8 + 16 + 127) / 128 * 128;
  static constexpr int kBytes = kEpiOffset + 4 * 32 * 32 * 4;
  static constexpr int kLaunchBytes = kBytes + 1024;
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
  // TMEM: two accumulators and the stage's scales. At BN = 256 the accumulators share 32
  // columns ([224, 256)), which leaves 32 for the scales: the epilogue drains the shared
  // columns first and hands them over, so the next tile's MMAs still overlap the drain.
  static constexpr bool kOverlap = BN == 256;
  static constexpr int kAccStride = kOverlap ? 224 : BN;
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

// Descriptor of a scale tile: unswizzled, 8 rows of 16 bytes 128 bytes apart.
__device__ __forceinline__ uint64_t scale_tile_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu)
         | (static_cast<uint64_t>(128 >> 4) << 32)  // stride byte offset: next 8 rows
         | (static_cast<uint64_t>(1) << 46);        // descriptor version for sm_100
}

// Eight columns of an output row: x[j] (+ e0[j]) times scale, `n` of them inside the row.
template <typename OutT>
__device__ __forceinline__ void mx4_store8(OutT* dst, const float (&x)[8], const OutT* e0, float scale, int n, bool vec) {
  if (vec && n >= 8) {
    if constexpr (sizeof(OutT) == 2) {
      uint32_t ew[4] = {0, 0, 0, 0};
      if (e0) {
        const uint4 e = __ldg(reinterpret_cast<const uint4*>(e0));
        ew[0] = e.x; ew[1] = e.y; ew[2] = e.z; ew[3] = e.w;
      }
      uint32_t o[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        o[h] = pack_bf16x2((x[2 * h] + bf16_bits_to_float(ew[h] & 0xFFFFu)) * scale,
                           (x[2 * h + 1] + bf16_bits_to_float(ew[h] >> 16)) * scale);
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e0) e = __ldg(reinterpret_cast<const float4*>(e0) + h);
        *(reinterpret_cast<float4*>(dst) + h) = make_float4((x[4 * h] + e.x) * scale, (x[4 * h + 1] + e.y) * scale,
                                                             (x[4 * h + 2] + e.z) * scale, (x[4 * h + 3] + e.w) * scale);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= n) break;
      if constexpr (sizeof(OutT) == 2) {
        const float e = e0 ? bf16_bits_to_float(e0[j]) : 0.f;
        dst[j] = static_cast<uint16_t>(pack_bf16x2((x[j] + e) * scale, 0.f));
      } else {
        dst[j] = (x[j] + (e0 ? e0[j] : 0.f)) * scale;
      }
    }
  }
}

template <int BN, int STAGES, typename OutT>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ Mx4Maps maps, const __grid_constant__ Mx4GemmParams p) {
  using L = Mx4Smem<BN, STAGES>;
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

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1u);   // the producer's byte count
      mbar_init(empty_bar(s), 1u);  // one tcgen05.commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1u);
      mbar_init(tempty_bar(a), 128u);
    }
    mbar_init(drain_bar, 1u);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.A);
    tma_prefetch_desc(&maps.B);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_tiles = p.num_m_blocks * p.num_n_blocks;
  const int KB = p.num_k_blocks;
  const int n_row_blocks = (p.N + 127) >> 7;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
        const int m_blk = tile / p.num_n_blocks, n_blk = tile % p.num_n_blocks;
        const int rb0 = n_blk * BN >> 7;  // first row block of B's scales
        const int rbs = n_row_blocks - rb0 < L::kSfbRows ? n_row_blocks - rb0 : L::kSfbRows;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          const uint32_t at = stage_at(stage);
          // the last k-block may hold one scale tile of a row block instead of two
          const uint32_t sbytes = (p.kt - 2 * kb >= 2 ? 2u : 1u) * kMxTileBytes;
          mbar_arrive_expect_tx(full_bar(stage), L::kABytes + L::kBBytes + (1 + rbs) * sbytes);
          tma_load_2d(at, &maps.A, kb * 128, m_blk * 128, full_bar(stage), pol);
          tma_load_2d(at + L::kABytes, &maps.B, kb * 128, n_blk * BN, full_bar(stage), pol);
          bulk_load_g2s(at + L::kSfaOffset, p.sa + (static_cast<size_t>(m_blk) * p.kt + 2 * kb) * kMxTileBytes, sbytes,
                        full_bar(stage));
          for (int r = 0; r < rbs; ++r)
            bulk_load_g2s(at + L::kSfbOffset + r * 2 * kMxTileBytes,
                          p.sb + (static_cast<size_t>(rb0 + r) * p.kt + 2 * kb) * kMxTileBytes, sbytes, full_bar(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // an abort: the copies in flight land before the block ends
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000ull * 1000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales to TMEM, MMA
    if (lane == 0) {
      const uint32_t idesc[2] = {umma_idesc_mx4(128, BN, 0), umma_idesc_mx4(128, BN, 2)};
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int local = 0;
      for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x, ++local) {
        const int n_blk = tile % p.num_n_blocks;
        const int acc = local & 1;
        if (L::kOverlap) {  // the previous tile's shared columns have been drained
          if (local > 0 && !mbar_wait(tempty_bar(0), (local - 1) & 1u, abort_flag, p.status)) { ok = false; break; }
        } else {
          if (!mbar_wait(tempty_bar(acc), ((local >> 1) & 1u) ^ 1u, abort_flag, p.status)) { ok = false; break; }
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * L::kAccStride);
        const uint32_t sfa = tmem_base + L::kSfaCol;
        const uint32_t sfb = tmem_base + L::kSfbCol;
        // a tile narrower than a row block of scales starts inside its four columns
        const uint32_t sfb_in = BN < 128 ? static_cast<uint32_t>((n_blk * BN & 127) >> 5) : 0u;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t at = stage_at(stage);
          const int left = p.K - kb * 256;
          const int steps = left >= 256 ? 4 : (left + 63) >> 6;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (2 * h >= steps) break;
            tmem_cp_scales(sfa + h * 4, scale_tile_desc(at + L::kSfaOffset + h * kMxTileBytes));
#pragma unroll
            for (int r = 0; r < L::kSfbRows; ++r)
              tmem_cp_scales(sfb + (h * L::kSfbRows + r) * 4,
                             scale_tile_desc(at + L::kSfbOffset + (r * 2 + h) * kMxTileBytes));
          }
          const uint64_t adesc = sw128_kmajor_desc(at);
          const uint64_t bdesc = sw128_kmajor_desc(at + L::kABytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= steps) break;
            umma_mx4(d_tmem, adesc + 2u * k, bdesc + 2u * k, idesc[k & 1], sfa + (k >> 1) * 4,
                     sfb + sfb_in + (k >> 1) * L::kSfbRows * 4, (kb | k) != 0 ? 1u : 0u);
          }
          umma_commit(empty_bar(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok) umma_commit(tfull_bar(acc));
      }
      umma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, 100ull * 1000 * 1000);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    // Per 32-column chunk: a row a lane from TMEM into the warp's staging area, then four
    // lanes a row read it back, 8 columns each, so that every access to E_0 and out covers
    // 8 rows x 64 (bf16) or 128 (f32) contiguous bytes. Staging: row r at r * 128 bytes,
    // 16-byte unit w at (w ^ (r & 7)) * 16: no bank conflicts either way.
    const int q = warp & 3;
    const uint32_t stg = sbase + L::kEpiOffset + static_cast<uint32_t>(q) * 4096u;
    const int rsub = lane >> 2, u2 = lane & 3;
    const uint32_t row_w = stg + static_cast<uint32_t>(lane) * 128u;
    const uint32_t rd_lo = stg + static_cast<uint32_t>(rsub) * 128u + (static_cast<uint32_t>((2 * u2) ^ rsub) << 4);
    const uint32_t rd_hi = stg + static_cast<uint32_t>(rsub) * 128u + (static_cast<uint32_t>((2 * u2 + 1) ^ rsub) << 4);
    int local = 0;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++local) {
      const int m_blk = tile / p.num_n_blocks, n_blk = tile % p.num_n_blocks;
      const int acc = local & 1;
      const int row0 = m_blk * 128 + q * 32;
      const OutT* e0[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e0[i] = nullptr;
        const int gr = row0 + i * 8 + rsub;
        if (p.tokens && gr < p.M) {
          uint32_t t = static_cast<uint32_t>(p.tokens[gr]);
          if (t >= p.V0) t = 0;
          e0[i] = static_cast<const OutT*>(p.E0) + static_cast<int64_t>(t) * p.N;
        }
      }
      bool got = false;
      if (lane == 0) got = mbar_wait(tfull_bar(acc), (local >> 1) & 1u, abort_flag, p.status);
      if (!__shfl_sync(0xffffffffu, got, 0)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * L::kAccStride);
      constexpr int kChunks = BN / 32;
#pragma unroll 1
      for (int cc = 0; cc < kChunks; ++cc) {
        // the columns shared with the other accumulator first: its last 32 (accumulator 0)
        // or first 32 (accumulator 1)
        const int c = L::kOverlap && acc == 0 ? (cc == 0 ? kChunks - 1 : cc - 1) : cc;
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c * 32, v);
        tmem_wait_ld();
        if (L::kOverlap ? cc == 0 : cc + 1 == kChunks) {
          tc_fence_before();
          mbar_arrive_relaxed(tempty_bar(L::kOverlap ? 0 : acc));
        }
#pragma unroll
        for (int w = 0; w < 8; ++w)
          st_shared_v4(row_w + (static_cast<uint32_t>(w ^ (lane & 7)) << 4),
                       make_uint4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]));
        __syncwarp();
        const int col = n_blk * BN + c * 32 + u2 * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 lo = ld_shared_v4(rd_lo + i * 8 * 128);
          const uint4 hi = ld_shared_v4(rd_hi + i * 8 * 128);
          const int gr = row0 + i * 8 + rsub;
          if (gr < p.M && col < p.N) {
            const float x[8] = {__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                                __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)};
            mx4_store8<OutT>(static_cast<OutT*>(p.out) + static_cast<int64_t>(gr) * p.ldo + col, x,
                             e0[i] ? e0[i] + col : nullptr, p.scale, p.N - col, p.vec != 0);
          }
        }
        __syncwarp();  // the staging area is rewritten by the next chunk
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

}  // namespace ngram
