// Host side of the 4-bit table operators and of the table lookup with its gradient
// (included by ngram_embed.cu after its own helpers).
//
// All but the sort in tiles and the numbering after it are programmatic dependent launches: a
// kernel's set-up runs while the one before ends, and it waits for all of that before its first
// global access. With them (and with plain launches), in graphs: one token's projection 6.7 us
// (7.2), a decode step's layer 19.9 (21.1), the gradients of 32768 rows of 4096 columns 95.4
// (101.4) and of 641 rows 14.5 (16.1); one call after another: 10.9 (11.8), 20.6 (25.1), 96.8
// (107.0), 17.2 (24.0). The product, the
// lookup and the join do not let their own dependents start early: the projection of 1280 tokens
// took 17.5 us for 16.9, the gradient 118 for 97.
#pragma once

namespace {

// Runs `set` (a kernel's attributes) once a device, a bit of `done` each.
template <typename F>
int once_a_device(std::atomic<uint64_t>& done, F set) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return NGRAM_ERR_CUDA;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return NGRAM_OK;
  if (!set()) return NGRAM_ERR_CUDA;
  if (dev < 64) done.fetch_or(bit, std::memory_order_release);
  return NGRAM_OK;
}

// A kernel's shared memory beyond 48 KB.
template <typename K>
int opt_in_smem(K kern, int bytes, std::atomic<uint64_t>& done, bool wide_clusters = false) {
  return once_a_device(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
           (!wide_clusters || cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess);
  });
}

// Makes the device that owns `p` current for a call, and the caller's again after it. Calls
// without a plan take their device from a pointer; host memory is refused there.
struct DeviceScope {
  int prev = -1;
  bool changed = false;
  int rc = NGRAM_OK;
  explicit DeviceScope(const void* p) {
    cudaPointerAttributes a{};
    if (cudaGetDevice(&prev) != cudaSuccess || cudaPointerGetAttributes(&a, p) != cudaSuccess) {
      (void)cudaGetLastError();
      rc = NGRAM_ERR_CUDA;
      return;
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) {
      rc = NGRAM_ERR_INVALID_ARG;
      return;
    }
    enter(a.device);
  }
  explicit DeviceScope(const ngram_embed_plan* plan) {
    if (plan->device < 0 || cudaGetDevice(&prev) != cudaSuccess) {
      rc = NGRAM_ERR_CUDA;
      return;
    }
    enter(plan->device);
  }
  void enter(int dev) {
    if (dev == prev) return;
    if (cudaSetDevice(dev) != cudaSuccess) rc = NGRAM_ERR_CUDA;
    else changed = true;
  }
  ~DeviceScope() {
    if (changed) cudaSetDevice(prev);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
};

// A row stride of an array that is only read: of rows beside one another, or 0, one row for all.
bool read_stride_ok(int64_t stride, int64_t cols) { return stride == 0 || stride >= cols; }

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

int device_sms() {
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

size_t mx4_tiled_scale_bytes(int64_t rows, int64_t cols) {
  return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>((cols + 127) / 128) * kMxTileBytes;
}

// 2-D map over 4-bit codes: boxes of one 128-byte swizzle row (256 elements) x box_rows. Rows
// and bytes outside the array read zero codes.
int encode_codes(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return NGRAM_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols / 2)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NGRAM_OK : NGRAM_ERR_CUDA;
}

// 2-D map over scale tiles: [row blocks x kt * 128 words], boxes of two tiles x `blocks` row
// blocks. Tiles and row blocks outside the array read zeros.
int encode_scales(CUtensorMap* m, const void* base, int64_t rows, int64_t kt, int blocks) {
  auto fn = encode_fn();
  if (!fn) return NGRAM_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kt * 128), static_cast<cuuint64_t>((rows + 127) / 128)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kt * kMxTileBytes)};
  const cuuint32_t box[2] = {256, static_cast<cuuint32_t>(blocks)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NGRAM_OK : NGRAM_ERR_CUDA;
}

struct Mx4Operands {
  const uint8_t *A, *SA, *B, *SB;  // codes and scale tiles
};

// The maps of a product on tiles of layout L (see Mx4Maps).
template <typename L, int BN, int RANKS>
int encode_mx4(Mx4Maps* m, const Mx4Operands& o, const Mx4GemmParams& p) {
  const int64_t kt = (p.K + 127) / 128;
  int rc;
  if ((rc = encode_codes(&m->A, o.A, p.K, p.M, 128))) return rc;
  if ((rc = encode_codes(&m->B, o.B, p.K, p.N, L::part_rows(0)))) return rc;
  m->B1 = m->B;
  if (L::kParts > 1 && (rc = encode_codes(&m->B1, o.B, p.K, p.N, L::part_rows(1)))) return rc;
  m->At = m->A;
  m->Bt = m->B;
  if (p.M % 128 && (rc = encode_codes(&m->At, o.A, p.K, p.M, (p.M % 128 + 7) & ~7))) return rc;
  for (int part = 0; part < L::kParts; ++part)  // the one box that N ends inside
    for (int rank = 0; rank < RANKS; ++rank) {
      const int rows = p.N % BN - L::part_row(part, rank);
      if (rows > 0 && rows < L::part_rows(part) && (rc = encode_codes(&m->Bt, o.B, p.K, p.N, (rows + 7) & ~7))) return rc;
    }
  if ((rc = encode_scales(&m->SA, o.SA, p.M, kt, 1))) return rc;
  return encode_scales(&m->SB, o.SB, p.N, kt, L::kSfbRows);
}

template <int BN, int STAGES, typename OutT, bool PAIR>
int launch_mx4_tiles(Mx4GemmParams prm, const Mx4Operands& o, int sms, cudaStream_t st) {
  using L = Mx4Smem<BN, STAGES, PAIR>;
  static_assert(L::kLaunchBytes <= 232448, "4-bit product stages exceed 227 KB of shared memory");
  auto kern = mx4_gemm_kernel<BN, STAGES, OutT, PAIR>;
  static std::atomic<uint64_t> done{0};
  Mx4Maps maps;
  int rc = opt_in_smem(kern, L::kLaunchBytes, done);
  if (rc) return rc;
  if ((rc = (encode_mx4<L, BN, PAIR ? 2 : 1>(&maps, o, prm)))) return rc;
  constexpr int kRows = PAIR ? 256 : 128;
  prm.num_m_blocks = (prm.M + kRows - 1) / kRows;
  prm.num_n_blocks = (prm.N + BN - 1) / BN;
  prm.num_k_blocks = (prm.K + 255) / 256;
  const int64_t tiles = static_cast<int64_t>(prm.num_m_blocks) * prm.num_n_blocks;
  if (tiles > INT32_MAX / 2) return NGRAM_ERR_UNSUPPORTED;
  const int workers = PAIR ? sms / 2 : sms;
  const int grid = (tiles < workers ? static_cast<int>(tiles) : workers) * (PAIR ? 2 : 1);
  return launch(kern, dim3(static_cast<unsigned>(grid)), dim3(kMxThreads), L::kLaunchBytes, st, true, PAIR ? 2 : 1, maps,
                prm);
}

// Which tiles: CTA pairs on 256 x 256 (the fewest bytes for their products) or 256 x 320 (fewer
// tiles where those just exceed a wave, no overlap of a tile's epilogue with the next tile), or
// one CTA on 128 x 192, 128 or 64, whichever finishes its waves first by the times below: a wave
// of a form costs so many us a k-block and so many besides, and never less than its least.
// Measured on B200, bf16 out (us, 320 / 256 / 192 / 128 / 64; * taken):
//   32768 x 2048 x 2048   81.1  61.5* 72.4  82.9 150.4    1280 x 4096 x 4096  13.1* 17.0  16.0  18.8  27.2
//    4096 x 4096 x 4096   30.9  28.7* 33.8  39.3  71.4    1280 x 2048 x 2048   9.6   8.6   6.6*  8.7  10.4
//    8192 x 2048 x 2048   28.2  18.9* 19.6  22.9  39.7    1280 x 4096 x 1024   8.4  10.3   8.2*  8.8  10.4
//     512 x 8192 x 4096   12.7  11.7* 15.6  14.5  22.5     512 x 4096 x 4096  12.4  11.0   9.2   8.4* 12.6
//   37000 x  320 x 4096   24.6* 32.7  29.8  34.9  52.2   16384 x 1000 x  512     -  17.1  17.7  16.4* 19.5
//     512 x 10000 x 4096  12.5* 16.2  16.0  18.6  26.9     333 x 1111 x 2080     -  11.5  10.1   8.3   6.2*
//    9400 x  640 x 2048   10.0* 11.8  10.4  12.0  16.1       1 x 4096 x 4096     -  10.0   8.4   7.6   7.2*
struct Mx4Form {
  int rows, cols;              // of a tile
  double us_kb, us_tile, least, once;  // a wave's us: for a k-block, besides, at least; the call's besides
};
constexpr Mx4Form kMx4Forms[5] = {{256, 256, 0.32, 1.6, 3.1, 1.5},
                                  {256, 320, 0.39, 3.2, 4.8, 0.3},
                                  {128, 192, 0.30, 1.3, 2.5, 0.0},
                                  {128, 128, 0.26, 1.0, 1.75, 0.0},
                                  {128, 64, 0.27, 0.5, 1.25, 0.0}};
// 0: no tiles, a warp a column (mx4_few_kernel), for up to four rows where that is sooner: it costs
// an element of B so much a row and in any case, all of B on this many SMs, and a tile form about
// 1.7 us more than it before the first wave. 1 / 4 rows, us (tiles in brackets): 4096 x 4096
// 4.6 / 6.8 (7.2), 2048 x 2048 2.3 / 3.4 (4.9), 512 x 512 1.6 / 2.4 (3.1), 16384 x 16384 43 / 74
// (40); rows of B much shorter than the 4096 elements that a warp takes at a time leave lanes
// idle: 50000 x 1024 19 / 33 (12).
constexpr int kMx4FewRows = 4;
int mx4_few_rows(int M) { return M < 3 ? M : kMx4FewRows; }  // rows that the kernel for M computes
double mx4_few_us(int M, int N, int K, int sms) {
  const double elements = static_cast<double>(N) * ((K + 4095) / 4096) * 4096;
  return elements * (0.13 + 0.04 * mx4_few_rows(M)) * 1e-6 * 148 / sms - 1.7;
}
int mx4_tile_width(int M, int N, int K, int sms) {
  int width = -1;
  double best = 0;
  if (M <= kMx4FewRows) {
    width = 0;
    best = mx4_few_us(M, N, K, sms);
  }
  for (const Mx4Form& f : kMx4Forms) {
    const int64_t tiles = (static_cast<int64_t>(M) + f.rows - 1) / f.rows * ((static_cast<int64_t>(N) + f.cols - 1) / f.cols);
    const int64_t workers = sms * 128 / f.rows, waves = (tiles + workers - 1) / workers;
    const double wave = (K + 255) / 256 * f.us_kb + f.us_tile;
    const double us = f.once + static_cast<double>(waves) * (wave > f.least ? wave : f.least);
    if (width < 0 || us < best) {
      width = f.cols;
      best = us;
    }
  }
  return width;
}

template <int R, typename OutT>
int launch_mx4_few(const Mx4GemmParams& prm, const Mx4Operands& o, cudaStream_t st) {
  const Mx4FewParams p{prm, o.A, o.SA, o.B, o.SB};
  return launch(mx4_few_kernel<R, OutT>, dim3(static_cast<unsigned>((prm.N + 127) / 128 * 16)), dim3(32 * kMxFewWarps), 0, st,
                true, 1, p);
}

template <typename OutT>
int launch_mx4_gemm(const Mx4GemmParams& prm, const Mx4Operands& o, int sms, cudaStream_t st) {
  if (sms < 2) return NGRAM_ERR_CUDA;
  const int width = mx4_tile_width(prm.M, prm.N, prm.K, sms);
  if (width == 0)
    switch (mx4_few_rows(prm.M)) {
      case 1: return launch_mx4_few<1, OutT>(prm, o, st);
      case 2: return launch_mx4_few<2, OutT>(prm, o, st);
      default: return launch_mx4_few<kMx4FewRows, OutT>(prm, o, st);
    }
  switch (width) {
    case 320: return launch_mx4_tiles<320, 5, OutT, true>(prm, o, sms, st);
    case 256: return launch_mx4_tiles<256, 5, OutT, true>(prm, o, sms, st);
    case 192: return launch_mx4_tiles<192, 5, OutT, false>(prm, o, sms, st);
    case 128: return launch_mx4_tiles<128, 6, OutT, false>(prm, o, sms, st);
    default: return launch_mx4_tiles<64, 8, OutT, false>(prm, o, sms, st);
  }
}

// Workspace of the layer on 4-bit tables: [head | T x D / 2 codes | scale tiles]
struct Mx4LayerWs {
  uint8_t *G, *Gs;
  size_t bytes;
};
Mx4LayerWs mx4_layer_ws(const ngram_embed_plan* p, int64_t T, void* ws) {
  Mx4LayerWs w{};
  const size_t at_g = kHeadBytes;
  const size_t at_s = at_g + round256(static_cast<size_t>(T) * static_cast<size_t>(p->D) / 2);
  w.bytes = at_s + round256(mx4_tiled_scale_bytes(T, p->D));
  if (ws) {
    auto* b = static_cast<uint8_t*>(ws);
    w.G = b + at_g;
    w.Gs = b + at_s;
  }
  return w;
}

bool mx4_plan_ok(const ngram_embed_plan* p) { return p->S > 0 && p->d % kMxBlock == 0; }

int check_mx4_layer(const ngram_embed_plan* p, const int32_t* tokens, const void* E0, const ngram_mx4* E_nk,
                    const ngram_mx4* W, void* out) {
  if (!tokens || !E0 || !E_nk || !W || !W->codes || !W->scales || !out) return NGRAM_ERR_INVALID_ARG;
  if (!aligned16(E0) || !aligned16(out) || !aligned16(W->codes) || !aligned16(W->scales)) return NGRAM_ERR_MISALIGNED;
  for (int s = 0; s < p->S; ++s) {
    if (!E_nk[s].codes || !E_nk[s].scales) return NGRAM_ERR_INVALID_ARG;
    if (!aligned16(E_nk[s].codes)) return NGRAM_ERR_MISALIGNED;
  }
  return NGRAM_OK;
}

// The gather of the call's sub-rows (indices from idx, or hashed from h's sequences), then the
// product with E_0 added.
int project_mx4(const ngram_embed_plan* p, const HashParams& h, const int32_t* idx, const void* E0,
                const ngram_mx4* E_nk, const ngram_mx4* W, void* out, const Mx4LayerWs& w, cudaStream_t st) {
  if (p->sms < 2) return NGRAM_ERR_CUDA;
  const int64_t T = h.T;
  Mx4GatherParams g{};
  for (int s = 0; s < p->S; ++s) {
    g.E[s].codes = static_cast<const uint8_t*>(E_nk[s].codes);
    g.E[s].scales = static_cast<const uint8_t*>(E_nk[s].scales);
  }
  g.idx = idx;
  g.h = h;
  g.row_blocks = p->d / kMxBlock;
  g.kt = (p->D + 127) / 128;
  g.by_row.set(static_cast<uint32_t>(g.kt) * 4);
  g.by_sub.set(static_cast<uint32_t>(g.row_blocks));
  g.blocks = p->D / kMxBlock;
  g.G = w.G;
  g.Gs = w.Gs;
  // tokens a block: kMx4GatherUnroll vectors a thread where the call has blocks to spare
  static_assert(8 * kMaxS <= kMx4GatherThreads, "a block hashes its tokens' indices in one pass");
  int tokens = T < 32 * static_cast<int64_t>(p->sms) ? 8 : kMx4GatherThreads * kMx4GatherUnroll / static_cast<int>(g.by_row.d);
  if (tokens > kMx4GatherThreads / p->S) tokens = kMx4GatherThreads / p->S;
  if (tokens > kMx4GatherMaxTokens) tokens = kMx4GatherMaxTokens;
  g.tokens = tokens < 8 ? 8 : tokens;
  int rc = launch(mx4_gather_kernel, dim3(static_cast<unsigned>((T + g.tokens - 1) / g.tokens)), dim3(kMx4GatherThreads), 0,
                  st, true, 1, g);
  if (rc) return rc;
  Mx4GemmParams prm{};
  prm.M = static_cast<int>(T);
  prm.N = p->D;
  prm.K = p->D;
  prm.scale = p->out_scale / static_cast<float>(p->S + 1);
  prm.tokens = h.tokens;
  prm.E0 = E0;
  prm.V0 = static_cast<uint32_t>(p->V0);
  prm.out = out;
  prm.ldo = p->D;
  prm.vec16 = 1;  // rows of a multiple of 32 elements, out and E_0 16-byte aligned
  prm.vec32 = aligned32(out) && aligned32(E0) ? 1 : 0;
  prm.status = h.status;
  const Mx4Operands o{w.G, w.Gs, static_cast<const uint8_t*>(W->codes), static_cast<const uint8_t*>(W->scales)};
  return p->dtype == NGRAM_F32 ? launch_mx4_gemm<float>(prm, o, p->sms, st)
                               : launch_mx4_gemm<uint16_t>(prm, o, p->sms, st);
}

// ---- lookup and gradient of one table ----
struct GradWs {
  uint32_t *key[2], *counts, *totals, *tile_heads;
  int32_t *pos[2], *piece_run, *crossing, *lists;
  float* partial;
  size_t bytes;
};
// Positions a piece: 128 while that leaves 4096 warps, else 32 while that leaves 1024, else 8. Long
// pieces leave few partial sums of the frequent ids to join, which a run's block adds one after
// another (65536 Zipf ids over 100 of 256 columns, pieces of 8 / 32: 25 / 8 us for the join); short
// ones have their row loads in flight at once where the warps are few (641 ids of 136 columns,
// pieces of 32 / 8: 16 / 6 us for the sums).
struct GradPiece {
  int positions;
  int64_t warps;  // the fewest that it may leave
};
constexpr GradPiece kGradPieces[3] = {{128, 4096}, {32, 1024}, {8, 0}};
int64_t grad_warps(int64_t n, int64_t D, int piece) { return (n + piece - 1) / piece * ((D + 255) / 256); }
int grad_piece(int64_t n, int64_t D) {
  int k = 0;
  while (grad_warps(n, D, kGradPieces[k].positions) < kGradPieces[k].warps) ++k;
  return kGradPieces[k].positions;
}
// The most pieces that a call of up to n positions takes: fewer positions may take shorter ones,
// but only while the next longer ones leave too few warps.
int64_t grad_max_pieces(int64_t n, int64_t D) {
  const int64_t chunks = (D + 255) / 256;
  int64_t most = 0;
  for (int k = 0; k < 3; ++k) {
    int64_t m = n;  // positions that take this length
    if (k) {
      const int64_t limit = (kGradPieces[k - 1].warps + chunks - 1) / chunks * kGradPieces[k - 1].positions;
      if (limit < m) m = limit;
    }
    const int64_t pieces = (m + kGradPieces[k].positions - 1) / kGradPieces[k].positions;
    if (pieces > most) most = pieces;
  }
  return most;
}

// Sized for every call of up to n positions.
GradWs grad_ws(int64_t n, int64_t D, void* ws) {
  GradWs w{};
  size_t off = kHeadBytes;
  auto take = [&](size_t b) {
    const size_t at = off;
    off += round256(b);
    return at;
  };
  const size_t N = static_cast<size_t>(n);
  const size_t tiles = (N + kSortTile - 1) / kSortTile;
  const size_t pieces = static_cast<size_t>(grad_max_pieces(n, D));
  const size_t k0 = take(N * 4), k1 = take(N * 4), p0 = take(N * 4), p1 = take(N * 4);
  const size_t cn = take(tiles << (kSortMaxBits + 2)), to = take(4u << kSortMaxBits), th = take(tiles * 4);
  const size_t pr = take(pieces * 4), cr = take(8), li = take(pieces * 8), pa = take(pieces * 2 * static_cast<size_t>(D) * 4);
  w.bytes = off;
  if (ws) {
    auto* b = static_cast<uint8_t*>(ws);
    w.key[0] = reinterpret_cast<uint32_t*>(b + k0);
    w.key[1] = reinterpret_cast<uint32_t*>(b + k1);
    w.pos[0] = reinterpret_cast<int32_t*>(b + p0);
    w.pos[1] = reinterpret_cast<int32_t*>(b + p1);
    w.counts = reinterpret_cast<uint32_t*>(b + cn);
    w.totals = reinterpret_cast<uint32_t*>(b + to);
    w.tile_heads = reinterpret_cast<uint32_t*>(b + th);
    w.piece_run = reinterpret_cast<int32_t*>(b + pr);
    w.crossing = reinterpret_cast<int32_t*>(b + cr);
    w.lists = reinterpret_cast<int32_t*>(b + li);
    w.partial = reinterpret_cast<float*>(b + pa);
  }
  return w;
}

// The cluster that sorts n positions: `ctas` of them with `items` positions a thread, the fewest
// items first, of at most `limit` CTAs. {0, 0}: it holds too few, they are sorted in tiles.
struct ClusterForm {
  int items, ctas;
};
ClusterForm cluster_form(int64_t n, int limit) {
  for (int items = 1; items <= kClusterMaxItems; items *= 2) {
    int ctas = 1;
    while (ctas < limit && static_cast<int64_t>(ctas) * kClusterThreads * items < n) ctas *= 2;
    if (ctas <= limit && static_cast<int64_t>(ctas) * kClusterThreads * items >= n) return {items, ctas};
  }
  return {0, 0};
}

template <int ITEMS>
int opt_in_cluster_sort() {
  static std::atomic<uint64_t> done{0};
  return opt_in_smem(sort_cluster_kernel<ITEMS>, sizeof(ClusterSmem<ITEMS>), done, true);
}

// The most CTAs, up to kClusterCtas, of a cluster of the sort that the current device places:
// fewer than 16 on a part of a GPU whose SM groups are smaller, 0 for none. Asked once a device,
// for the form that takes the most shared memory. Negative on an error.
int cluster_limit() {
  static std::atomic<int> known[64];  // 1 + the answer
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return NGRAM_ERR_CUDA;
  if (dev < 64)
    if (const int k = known[dev].load(std::memory_order_acquire)) return k - 1;
  if (opt_in_cluster_sort<kClusterMaxItems>()) return NGRAM_ERR_CUDA;
  int limit = 0;
  for (int ctas = kClusterCtas; ctas && !limit; ctas /= 2) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = sizeof(ClusterSmem<kClusterMaxItems>);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, sort_cluster_kernel<kClusterMaxItems>, &cfg) != cudaSuccess)
      (void)cudaGetLastError();  // a size that the device does not know
    else if (fit > 0)
      limit = ctas;
  }
  if (dev < 64) known[dev].store(limit + 1, std::memory_order_release);
  return limit;
}

template <int ITEMS>
int launch_cluster_sort(const ClusterSortParams& a, int ctas, cudaStream_t st) {
  const int rc = opt_in_cluster_sort<ITEMS>();
  if (rc) return rc;
  return launch(sort_cluster_kernel<ITEMS>, dim3(static_cast<unsigned>(ctas)), dim3(kClusterThreads),
                sizeof(ClusterSmem<ITEMS>), st, true, ctas, a);
}

template <typename T>
int launch_grad_reduce(const GradParams& r, dim3 grid, cudaStream_t st) {
  if (r.piece == 128) return launch(grad_reduce_kernel<T, 128>, grid, dim3(256), 0, st, true, 1, r);
  if (r.piece == 32) return launch(grad_reduce_kernel<T, 32>, grid, dim3(256), 0, st, true, 1, r);
  return launch(grad_reduce_kernel<T, 8>, grid, dim3(256), 0, st, true, 1, r);
}

int embedding_bwd(const int32_t* ids, int64_t n, const void* g, int g_dtype, int64_t g_stride, int64_t V, int64_t D,
                  float scale, int64_t pad_id, int32_t* rows_out, int32_t* count_out, float* out, bool dense,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || n > INT32_MAX || V < 1 || V >= (int64_t(1) << 31) || D < 1 || D > INT32_MAX || !(scale - scale == 0.0f) ||
      (g_dtype != NGRAM_BF16 && g_dtype != NGRAM_F32) || !workspace || (!dense && !count_out) ||
      (n > 0 && (!ids || !g || !out || (!dense && !rows_out) || !read_stride_ok(g_stride, D))))
    return NGRAM_ERR_INVALID_ARG;
  if (D % 8 != 0) return NGRAM_ERR_UNSUPPORTED;
  const int elt = g_dtype == NGRAM_BF16 ? 2 : 4;
  if (!aligned16(workspace)) return NGRAM_ERR_MISALIGNED;
  if (n > 0 && (!aligned16(g) || !aligned16(out) || g_stride * elt % 16 != 0)) return NGRAM_ERR_MISALIGNED;
  const GradWs w = grad_ws(n, D, workspace);
  if (workspace_bytes < w.bytes) return NGRAM_ERR_WORKSPACE;
  const DeviceScope dev(workspace);
  if (dev.rc) return dev.rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (!dense && cudaMemsetAsync(count_out, 0, 4, st) != cudaSuccess) return NGRAM_ERR_CUDA;
    return NGRAM_OK;
  }
  // keys 0 .. V (V: a padded position) in equal digits
  int bits = 1;
  while ((V >> bits) != 0) ++bits;
  const int limit = n <= kClusterMax ? cluster_limit() : 0;
  if (limit < 0) return limit;
  const ClusterForm form = cluster_form(n, limit);
  const bool cluster = form.ctas > 0;
  const int max_bits = cluster ? kClusterMaxBits : kSortMaxBits;
  const int passes = (bits + max_bits - 1) / max_bits;
  SortParams s{};
  s.ids = ids;
  s.V = static_cast<uint32_t>(V);
  s.pad_id = pad_id;
  s.n = static_cast<uint32_t>(n);
  s.bits = (bits + passes - 1) / passes;
  s.tiles = static_cast<uint32_t>((n + kSortTile - 1) / kSortTile);
  s.counts = w.counts;
  s.totals = w.totals;
  s.status = status_ptr(workspace);
  GradParams r{};
  r.n = s.n;
  r.V = s.V;
  r.tiles = s.tiles;
  r.tile_heads = w.tile_heads;
  r.piece = static_cast<uint32_t>(grad_piece(n, D));
  r.piece_run = w.piece_run;
  r.rows_out = rows_out;
  r.count_out = count_out;
  r.g = g;
  r.g_stride = g_stride;
  r.D = static_cast<int>(D);
  r.chunks = static_cast<int>((D + 255) / 256);
  r.scale = scale;
  r.partial = w.partial;
  r.crossing = w.crossing;
  r.lists = w.lists;
  r.pieces = static_cast<uint32_t>((n + r.piece - 1) / r.piece);
  r.out = out;
  r.dense = dense ? 1 : 0;
  int rc;
  if (cluster) {
    s.key_out = w.key[0];
    s.pos_out = w.pos[0];
    r.key = w.key[0];
    r.pos = w.pos[0];
    const ClusterSortParams a{s, passes, r};
    rc = form.items == 1 ? launch_cluster_sort<1>(a, form.ctas, st)
                         : (form.items == 2 ? launch_cluster_sort<2>(a, form.ctas, st) : launch_cluster_sort<4>(a, form.ctas, st));
    if (rc) return rc;
  } else {
    int cur = 0;
    for (int k = 0; k < passes; ++k) {
      s.shift = k * s.bits;
      s.key_in = k ? w.key[cur ^ 1] : nullptr;
      s.pos_in = k ? w.pos[cur ^ 1] : nullptr;
      s.key_out = w.key[cur];
      s.pos_out = w.pos[cur];
      if ((rc = launch(sort_count_kernel, dim3(s.tiles), dim3(kSortThreads), 0, st, false, 1, s))) return rc;
      if ((rc = launch(sort_scan_kernel, dim3(1u << s.bits), dim3(kSortThreads), 0, st, false, 1, s))) return rc;
      if ((rc = launch(sort_scatter_kernel, dim3(s.tiles), dim3(kSortThreads), 0, st, false, 1, s))) return rc;
      cur ^= 1;
    }
    r.key = w.key[cur ^ 1];
    r.pos = w.pos[cur ^ 1];
    if ((rc = launch(grad_heads_kernel, dim3(r.tiles), dim3(kSortThreads), 0, st, false, 1, r))) return rc;
    if ((rc = launch(grad_number_kernel, dim3(r.tiles), dim3(kSortThreads), 0, st, false, 1, r))) return rc;
  }
  const int64_t items = static_cast<int64_t>(r.pieces) * r.chunks;
  if (items > int64_t(INT32_MAX) * 8) return NGRAM_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((items + 7) / 8));
  rc = g_dtype == NGRAM_BF16 ? launch_grad_reduce<uint16_t>(r, grid, st) : launch_grad_reduce<float>(r, grid, st);
  if (rc) return rc;
  // enough for every run that could cross pieces, at most a resident grid
  const int64_t most = static_cast<int64_t>(r.pieces) * ((D + 127) / 128), resident = int64_t(device_sms()) * kJoinBlocksPerSm;
  return launch(grad_join_kernel, dim3(static_cast<unsigned>(most < resident ? most : resident)), dim3(256), 0, st, true, 1,
                r);
}

dim3 row_map_grid(const RowMap& m) { return dim3((m.items + 7) / 8); }

template <int TABLE, typename OutT>
int launch_lookup(LookupParams& p, uint32_t rows, uint32_t vecs, cudaStream_t st) {
  const int U = RowMap::unroll(vecs);
  p.map.set(rows, vecs, U);
  const dim3 grid = row_map_grid(p.map);
  if (U == 4) return launch(lookup_kernel<TABLE, OutT, 4>, grid, dim3(256), 0, st, true, 1, p);
  if (U == 2) return launch(lookup_kernel<TABLE, OutT, 2>, grid, dim3(256), 0, st, true, 1, p);
  return launch(lookup_kernel<TABLE, OutT, 1>, grid, dim3(256), 0, st, true, 1, p);
}
template <int TABLE>
int launch_lookup_to(LookupParams& p, int out_dtype, uint32_t rows, uint32_t vecs, cudaStream_t st) {
  return out_dtype == NGRAM_BF16 ? launch_lookup<TABLE, uint16_t>(p, rows, vecs, st)
                                 : launch_lookup<TABLE, float>(p, rows, vecs, st);
}

template <typename T, bool VEC>
int launch_quantize(Mx4QuantParams& p, uint32_t rows, uint32_t vecs, cudaStream_t st) {
  const int U = RowMap::unroll(vecs);
  p.map.set(rows, vecs, U);
  const dim3 grid = row_map_grid(p.map);
  if (U == 4) return launch(mx4_quantize_kernel<T, VEC, 4>, grid, dim3(256), 0, st, true, 1, p);
  if (U == 2) return launch(mx4_quantize_kernel<T, VEC, 2>, grid, dim3(256), 0, st, true, 1, p);
  return launch(mx4_quantize_kernel<T, VEC, 1>, grid, dim3(256), 0, st, true, 1, p);
}

// Rows of a launch whose warps are numbered in 32 bits: at most 2^30 vectors of eight elements.
int64_t rows_per_launch(int64_t cols) {
  const int64_t r = (int64_t(1) << 30) / (cols / 8);
  return r < 1 ? 1 : r;
}

}  // namespace

extern "C" {

size_t ngram_mx4_scale_bytes(int64_t rows, int64_t cols, int layout) {
  if (rows < 0 || cols < 1 || cols % kMxBlock != 0 || (layout != NGRAM_MX4_ROWS && layout != NGRAM_MX4_TILES)) return 0;
  return layout == NGRAM_MX4_ROWS ? static_cast<size_t>(rows) * static_cast<size_t>(cols / kMxBlock)
                                  : mx4_tiled_scale_bytes(rows, cols);
}

int ngram_mx4_quantize(const void* src, int dtype, int64_t rows, int64_t cols, int64_t src_stride, void* codes,
                       void* scales, int layout, void* stream) {
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > INT32_MAX || (dtype != NGRAM_BF16 && dtype != NGRAM_F32) ||
      (layout != NGRAM_MX4_ROWS && layout != NGRAM_MX4_TILES) ||
      (rows > 0 && (!src || !codes || !scales || !read_stride_ok(src_stride, cols))))
    return NGRAM_ERR_INVALID_ARG;
  if (cols % kMxBlock != 0) return NGRAM_ERR_UNSUPPORTED;
  if (rows == 0) return NGRAM_OK;
  const int elt = dtype == NGRAM_BF16 ? 2 : 4;
  if (!aligned16(codes) || !aligned16(scales) || reinterpret_cast<uintptr_t>(src) % elt != 0) return NGRAM_ERR_MISALIGNED;
  const DeviceScope dev(codes);
  if (dev.rc) return dev.rc;
  const bool vec = aligned16(src) && src_stride * elt % 16 == 0;
  const int64_t step = rows_per_launch(cols);
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t r = rows - r0 < step ? rows - r0 : step;
    Mx4QuantParams p{};
    p.src = static_cast<const uint8_t*>(src) + r0 * src_stride * elt;
    p.src_stride = src_stride;
    p.row0 = r0;
    p.cols = static_cast<int>(cols);
    p.kt = static_cast<int>((cols + 127) / 128);
    p.codes = static_cast<uint8_t*>(codes) + r0 * (cols / 2);
    p.tiles = layout == NGRAM_MX4_TILES ? 1 : 0;
    p.scales = static_cast<uint8_t*>(scales) + (p.tiles ? 0 : r0 * (cols / kMxBlock));
    const uint32_t n = static_cast<uint32_t>(r), vecs = static_cast<uint32_t>(cols / 8);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc;
    if (dtype == NGRAM_BF16)
      rc = vec ? launch_quantize<uint16_t, true>(p, n, vecs, st) : launch_quantize<uint16_t, false>(p, n, vecs, st);
    else
      rc = vec ? launch_quantize<float, true>(p, n, vecs, st) : launch_quantize<float, false>(p, n, vecs, st);
    if (rc) return rc;
  }
  return NGRAM_OK;
}

int ngram_mx4_product_form(int64_t M, int64_t N, int64_t K, int sms) {
  if (M < 1 || M > INT32_MAX - 256 || N < 1 || N > INT32_MAX - 256 || K < 1 || K > INT32_MAX - 256 || sms < 2)
    return NGRAM_ERR_INVALID_ARG;
  return mx4_tile_width(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), sms);
}

size_t ngram_mx4_product_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 1) return 0;
  return kHeadBytes;
}

int ngram_mx4_product(const ngram_mx4* A, const ngram_mx4* B, int64_t M, int64_t N, int64_t K, float alpha, void* out,
                      int out_dtype, int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (!A || !B || M < 0 || M > INT32_MAX - 256 || N < 0 || N > INT32_MAX - 256 || K < 1 || K > INT32_MAX - 256 ||
      !(alpha - alpha == 0.0f) || (out_dtype != NGRAM_BF16 && out_dtype != NGRAM_F32) || !workspace ||
      out_stride < N)
    return NGRAM_ERR_INVALID_ARG;
  if (K % kMxBlock != 0) return NGRAM_ERR_UNSUPPORTED;
  if (!aligned16(workspace)) return NGRAM_ERR_MISALIGNED;
  if (workspace_bytes < ngram_mx4_product_workspace_bytes(M, N, K)) return NGRAM_ERR_WORKSPACE;
  if (M == 0 || N == 0) return NGRAM_OK;
  if (!A->codes || !A->scales || !B->codes || !B->scales || !out) return NGRAM_ERR_INVALID_ARG;
  const int elt = out_dtype == NGRAM_BF16 ? 2 : 4;
  if (!aligned16(A->codes) || !aligned16(A->scales) || !aligned16(B->codes) || !aligned16(B->scales) ||
      reinterpret_cast<uintptr_t>(out) % elt != 0)
    return NGRAM_ERR_MISALIGNED;
  const DeviceScope dev(workspace);
  if (dev.rc) return dev.rc;
  Mx4GemmParams prm{};
  prm.M = static_cast<int>(M);
  prm.N = static_cast<int>(N);
  prm.K = static_cast<int>(K);
  prm.scale = alpha;
  prm.out = out;
  prm.ldo = out_stride;
  prm.vec16 = aligned16(out) && out_stride * elt % 16 == 0 ? 1 : 0;
  prm.vec32 = aligned32(out) && out_stride * elt % 32 == 0 ? 1 : 0;
  prm.status = status_ptr(workspace);
  const Mx4Operands o{static_cast<const uint8_t*>(A->codes), static_cast<const uint8_t*>(A->scales),
                      static_cast<const uint8_t*>(B->codes), static_cast<const uint8_t*>(B->scales)};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return out_dtype == NGRAM_F32 ? launch_mx4_gemm<float>(prm, o, device_sms(), st)
                                : launch_mx4_gemm<uint16_t>(prm, o, device_sms(), st);
}

size_t ngram_embed_mx4_workspace_bytes(const ngram_embed_plan* plan, int64_t max_tokens) {
  if (!plan || max_tokens < 0 || !mx4_plan_ok(plan)) return 0;
  return mx4_layer_ws(plan, max_tokens, nullptr).bytes;
}

int ngram_embed_project_mx4(const ngram_embed_plan* plan, const int32_t* tokens, const int32_t* idx, int64_t num_tokens,
                            const void* E0, const ngram_mx4* E_nk, const ngram_mx4* W, void* out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!plan || !workspace || num_tokens < 0 || num_tokens > INT32_MAX - 256) return NGRAM_ERR_INVALID_ARG;
  if (!mx4_plan_ok(plan)) return NGRAM_ERR_UNSUPPORTED;
  if (!aligned16(workspace)) return NGRAM_ERR_MISALIGNED;
  const Mx4LayerWs w = mx4_layer_ws(plan, num_tokens, workspace);
  if (workspace_bytes < w.bytes) return NGRAM_ERR_WORKSPACE;
  if (num_tokens == 0) return NGRAM_OK;
  if (!idx) return NGRAM_ERR_INVALID_ARG;
  int rc = check_mx4_layer(plan, tokens, E0, E_nk, W, out);
  if (rc) return rc;
  const DeviceScope dev(plan);
  if (dev.rc) return dev.rc;
  return project_mx4(plan, hash_params(plan, tokens, nullptr, 0, num_tokens, nullptr, nullptr, workspace), idx, E0, E_nk, W,
                     out, w, static_cast<cudaStream_t>(stream));
}

int ngram_embed_fwd_mx4(const ngram_embed_plan* plan, const int32_t* tokens, const int32_t* seq_offsets,
                        int32_t num_seqs, int64_t num_tokens, const void* E0, const ngram_mx4* E_nk, const ngram_mx4* W,
                        const ngram_cache* cache, const int32_t* cache_slots, void* out, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!plan || !workspace || num_tokens < 0 || num_tokens > INT32_MAX - 256 || num_seqs < 0) return NGRAM_ERR_INVALID_ARG;
  if (!mx4_plan_ok(plan)) return NGRAM_ERR_UNSUPPORTED;
  if (!aligned16(workspace)) return NGRAM_ERR_MISALIGNED;
  const Mx4LayerWs w = mx4_layer_ws(plan, num_tokens, workspace);
  if (workspace_bytes < w.bytes) return NGRAM_ERR_WORKSPACE;
  if (num_tokens == 0) return NGRAM_OK;
  if (!seq_offsets || num_seqs == 0) return NGRAM_ERR_INVALID_ARG;
  int rc = check_mx4_layer(plan, tokens, E0, E_nk, W, out);
  if (rc) return rc;
  if (cache && (rc = validate_cache(plan, cache))) return rc;
  const DeviceScope dev(plan);
  if (dev.rc) return dev.rc;
  return project_mx4(plan, hash_params(plan, tokens, seq_offsets, num_seqs, num_tokens, cache, cache_slots, workspace),
                     nullptr, E0, E_nk, W, out, w, static_cast<cudaStream_t>(stream));
}

size_t ngram_embedding_workspace_bytes(int64_t max_ids, int64_t D) {
  if (max_ids < 0 || max_ids > INT32_MAX || D < 1 || D > INT32_MAX) return 0;
  return grad_ws(max_ids, D, nullptr).bytes;
}

int ngram_embedding_sort_ctas(int64_t n, int limit) {
  if (n < 1 || n > INT32_MAX || limit < 0) return NGRAM_ERR_INVALID_ARG;
  return cluster_form(n, limit < kClusterCtas ? limit : kClusterCtas).ctas;
}

int ngram_embedding_piece(int64_t n, int64_t D) {
  if (n < 1 || n > INT32_MAX || D < 1 || D > INT32_MAX) return NGRAM_ERR_INVALID_ARG;
  return grad_piece(n, D);
}

int ngram_embedding_fwd(const void* table, const void* table_scales, int table_dtype, int64_t V, int64_t D,
                        const int32_t* ids, int64_t n, float scale, int64_t pad_id, void* out, int out_dtype,
                        int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || n > INT32_MAX || V < 1 || V >= (int64_t(1) << 31) || D < 1 || D > INT32_MAX || !(scale - scale == 0.0f) ||
      (table_dtype != NGRAM_BF16 && table_dtype != NGRAM_F32 && table_dtype != NGRAM_MX4) ||
      (out_dtype != NGRAM_BF16 && out_dtype != NGRAM_F32) || !workspace || (!ids && n > V))
    return NGRAM_ERR_INVALID_ARG;
  if (D % (table_dtype == NGRAM_MX4 ? kMxBlock : 8) != 0) return NGRAM_ERR_UNSUPPORTED;
  if (!aligned16(workspace)) return NGRAM_ERR_MISALIGNED;
  if (workspace_bytes < kHeadBytes) return NGRAM_ERR_WORKSPACE;
  if (n == 0) return NGRAM_OK;
  if (!table || !out || out_stride < D || (table_dtype == NGRAM_MX4 && !table_scales)) return NGRAM_ERR_INVALID_ARG;
  const int elt = out_dtype == NGRAM_BF16 ? 2 : 4;
  if (!aligned16(table) || !aligned16(out) || out_stride * elt % 16 != 0) return NGRAM_ERR_MISALIGNED;
  const DeviceScope dev(workspace);
  if (dev.rc) return dev.rc;
  const int64_t step = rows_per_launch(D);
  for (int64_t r0 = 0; r0 < n; r0 += step) {
    const int64_t r = n - r0 < step ? n - r0 : step;
    LookupParams p{};
    p.table = table;
    p.scales = static_cast<const uint8_t*>(table_scales);
    p.ids = ids ? ids + r0 : nullptr;
    p.V = static_cast<uint32_t>(V);
    p.pad_id = pad_id;
    p.scale = scale;
    p.out = static_cast<uint8_t*>(out) + r0 * out_stride * elt;
    p.out_stride = out_stride;
    p.row0 = r0;
    p.pad_pos = !ids && pad_id >= r0 && pad_id - r0 < r ? static_cast<uint32_t>(pad_id - r0) : UINT32_MAX;
    p.status = status_ptr(workspace);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc;
    const uint32_t rows = static_cast<uint32_t>(r), vecs = static_cast<uint32_t>(D / 8);
    if (table_dtype == NGRAM_BF16) rc = launch_lookup_to<kTableBf16>(p, out_dtype, rows, vecs, st);
    else if (table_dtype == NGRAM_F32) rc = launch_lookup_to<kTableF32>(p, out_dtype, rows, vecs, st);
    else rc = launch_lookup_to<kTableMx4>(p, out_dtype, rows, vecs, st);
    if (rc) return rc;
  }
  return NGRAM_OK;
}

int ngram_embedding_bwd(const int32_t* ids, int64_t n, const void* grad_out, int grad_dtype, int64_t grad_stride,
                        int64_t V, int64_t D, float scale, int64_t pad_id, float* d_table, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return embedding_bwd(ids, n, grad_out, grad_dtype, grad_stride, V, D, scale, pad_id, nullptr, nullptr, d_table, true,
                       workspace, workspace_bytes, stream);
}

int ngram_embedding_bwd_rows(const int32_t* ids, int64_t n, const void* grad_out, int grad_dtype, int64_t grad_stride,
                             int64_t V, int64_t D, float scale, int64_t pad_id, int32_t* rows, int32_t* num_rows,
                             float* grads, void* workspace, size_t workspace_bytes, void* stream) {
  return embedding_bwd(ids, n, grad_out, grad_dtype, grad_stride, V, D, scale, pad_id, rows, num_rows, grads, false,
                       workspace, workspace_bytes, stream);
}

}  // extern "C"
