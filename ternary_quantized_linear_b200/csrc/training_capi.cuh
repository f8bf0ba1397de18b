// training_capi.cuh -- host side of the training operators (vocabulary cross
// entropy, orthogonalised updates): argument checks, workspace layouts,
// launch planning and the C entry points.  Included by bitnet_capi.cu, whose
// helpers it uses.
#pragma once

namespace bitnet {
namespace {

// The SM count that plans and workspace sizes assume (size queries run
// without a device).  A device with another count gets the same results.
constexpr int kPlanSms = 148;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// ------------------------------------------------------------ matrix product

// One operand: `rows` (m or n) x contraction, K-major (k contiguous) or
// MN-major as the epilogue's product has it, row stride ld and batch stride in
// elements.
struct TgOperand {
  const void* p = nullptr;
  const void* lo = nullptr;
  int64_t ld = 0, batch_stride = 0;
};

// A tensor of the epilogue: [batch][M][N] with row stride ld.
struct TgTensor {
  const void* p = nullptr;
  const void* lo = nullptr;
  int64_t ld = 0, batch_stride = 0, batch = 1;
  CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int block = 32;            // columns of a block: rows of 64 or 128 bytes
};

// How a product is cut: SM pairs on 256-row tiles (cg = 2) or single SMs on
// 128-row ones, bn columns a tile, and the CTAs of a cluster that share one
// tile's contraction.
struct TgPlan {
  int cg = 1, bn = 128, split = 1;
};

struct TgProblem {
  TgOperand a, b;
  TgTensor in, out;
  int64_t M = 0, N = 0, Kc = 0, batch = 1;
  bool sym = false;
  bool backwards = false;    // take the contraction from its end
  int passes = 1;
  int ksplit = 1;            // slices of the contraction as tiles of their own
  TgPlan plan;
};

// 3-D tensor [batch][rows][inner], boxes of box_inner x box_rows;
// out-of-range elements read as zero and are not written.
bool make_tmap_3d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int64_t inner,
                  int64_t rows, int64_t batch, int64_t ld, int64_t batch_stride, int box_inner,
                  int box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int64_t size = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(size * ld),
                           static_cast<cuuint64_t>(size * (batch > 1 ? batch_stride : ld * rows))};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_operand_map(CUtensorMap* map, const TgOperand& o, bool mn, const void* base, bool bf16,
                      int64_t rows, int64_t Kc, int64_t batch, int tile_rows) {
  const CUtensorMapDataType type =
      bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return mn ? make_tmap_3d(map, base, type, rows, Kc, batch, o.ld, o.batch_stride, 64, 64,
                             CU_TENSOR_MAP_SWIZZLE_128B)
              : make_tmap_3d(map, base, type, Kc, rows, batch, o.ld, o.batch_stride, 64,
                             tile_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Blocks of 32 rows, swizzled by their rows' 64 or 128 bytes.
bool make_tensor_maps(CUtensorMap* map, CUtensorMap* map_lo, const TgTensor& t, int64_t M,
                      int64_t N) {
  const int row = t.block * (t.type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2);
  const CUtensorMapSwizzle swz = row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                            : CU_TENSOR_MAP_SWIZZLE_64B;
  return (!t.p || make_tmap_3d(map, t.p, t.type, N, M, t.batch, t.ld, t.batch_stride, t.block, 32,
                               swz)) &&
         (!t.lo || make_tmap_3d(map_lo, t.lo, t.type, N, M, t.batch, t.ld, t.batch_stride,
                                t.block, 32, swz));
}

int64_t tg_tiles(int64_t M, int64_t N, int64_t batch, bool sym, int bm, int bn) {
  const int64_t mt = ceil_div(M, bm), nt = ceil_div(N, bn);
  return batch * (sym ? mt * (mt + 1) / 2 : mt * nt);
}

// Cycles that a plan needs, roughly: its waves of tiles, a tile's steps and
// its epilogue.  A pair's 64-k step takes 650 cycles (measured; the MMAs
// alone 512), a 128 x 128 step 570 (32 KiB at 64 bytes a cycle are 512; the
// MMAs 256); the epilogue and what a launch waits for come on top of each
// wave, and for a cluster's split the meeting of the parts (4 us).  Of clusters
// of two SMs 74 are resident at a time, of three 45, of four 33 (the occupancy
// query's answer on a B200: its SM groups do not divide into fours).
double tg_cost(int64_t M, int64_t N, int64_t batch, bool sym, int64_t steps, const TgPlan& pl) {
  const int64_t tiles = tg_tiles(M, N, batch, sym, 128 * pl.cg, pl.bn);
  const int64_t slots = pl.split == 4   ? 33
                        : pl.split == 3 ? 45
                                        : kPlanSms / std::max(pl.cg, pl.split);
  const double waves = static_cast<double>(ceil_div(tiles, slots));
  if (pl.cg == 2) return waves * (650.0 * static_cast<double>(steps) + 5000.0);
  return waves * (570.0 * static_cast<double>(ceil_div(steps, pl.split)) + 3000.0 +
                  (pl.split > 1 ? 7000.0 : 0.0));
}

// Pairs on 256 x 256 tiles, or single SMs on 128 x 128 tiles, each tile's
// steps shared by a cluster of up to max_split: whichever tg_cost prefers.
// Every CTA of a cluster needs a step of its own.  (Only X X^T asks for a split:
// by two, three or four it pays for the parts' meeting from 25, 19 or 17 steps
// on, and R R and Q X with as many, n = 1570, 1180 or 1050, have more tiles than
// clusters are resident.)
TgPlan tg_plan(int64_t M, int64_t N, int64_t batch, bool sym, int64_t steps, int passes,
               int max_split = 1) {
  TgPlan best{2, 256, 1};
  double cost = tg_cost(M, N, batch, sym, steps * passes, best);
  for (int s = 1; s <= max_split; ++s) {
    if ((s - 1) * ceil_div(steps, s) >= steps) continue;
    const TgPlan pl{1, 128, s};
    const double c = tg_cost(M, N, batch, sym, ceil_div(steps, s) * s * passes, pl);
    if (c < cost) {
      cost = c;
      best = pl;
    }
  }
  return best;
}

// Resident workers (pairs or single CTAs) of one kernel instance, per device;
// sets the kernel's shared-memory limit the first time.
template <int CG, int BN, int SPLIT, class Epi>
int tg_workers(int num_sms) {
  static std::once_flag once[kMaxDevices];
  static int workers[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::call_once(once[dev], [dev, num_sms]() {
    using C = TgCfg<CG, BN, Epi>;
    auto kernel = tc_gemm_kernel<CG, BN, SPLIT, Epi>;
    if (!set_smem(kernel, C::SMEM_DYN)) return;
    // (a split of registers that the launch does not have would wait for good)
    cudaFuncAttributes attr_of{};
    if (CG == 2 && Epi::kPairRun > 0 &&
        (cudaFuncGetAttributes(&attr_of, kernel) != cudaSuccess || attr_of.numRegs < kTgRegs))
      return;
    if (CG == 1) {
      workers[dev] = num_sms;
      return;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms / 2 * 2));
    cfg.blockDim = dim3(kTgThreads);
    cfg.dynamicSmemBytes = C::SMEM_DYN;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) workers[dev] = n;
  });
  return workers[dev];
}

// A product ready to launch: its tensor maps and shape (a step that comes
// again with the same tensors reuses them; encoding the six maps of one
// product takes the host as long as half a launch).
struct TgReady {
  bool done = false;
  TgMaps maps;
  TgShape shape;
  int workers = 0;
};

template <int CG, int BN, int SPLIT, class Epi>
bitnet_status prepare_tg(const DeviceState& ds, const TgProblem& g, TgReady& r) {
  using C = TgCfg<CG, BN, Epi>;
  r.workers = tg_workers<CG, BN, SPLIT, Epi>(ds.num_sms);
  if (r.workers < 1) return cuda_status(cudaErrorInvalidConfiguration);
  const int bn = g.plan.bn, b_rows = bn / CG;
  // A K-major operand of fewer rows is copied as far as it goes.
  const int a_rows =
      CG == 1 && !Epi::kAMn && g.M < 128 ? static_cast<int>(round_up(g.M, 8)) : 128;
  TgMaps& maps = r.maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!make_operand_map(&maps.a, g.a, Epi::kAMn, g.a.p, Epi::kBf16, g.M, g.Kc, g.batch, a_rows) ||
      !make_operand_map(&maps.b, g.b, Epi::kBMn, g.b.p, Epi::kBf16, g.N, g.Kc, g.batch, b_rows) ||
      !make_tensor_maps(&maps.in, &maps.in_lo, g.in, g.M, g.N) ||
      !make_tensor_maps(&maps.out, &maps.out_lo, g.out, g.M, g.N))
    return BITNET_ERR_CUDA;
  if (g.passes == 3 &&
      (!make_operand_map(&maps.a_lo, g.a, Epi::kAMn, g.a.lo, Epi::kBf16, g.M, g.Kc, g.batch,
                         a_rows) ||
       !make_operand_map(&maps.b_lo, g.b, Epi::kBMn, g.b.lo, Epi::kBf16, g.N, g.Kc, g.batch,
                         b_rows)))
    return BITNET_ERR_CUDA;
  TgShape& p = r.shape;
  p = TgShape{};
  p.M = static_cast<int>(g.M);
  p.N = static_cast<int>(g.N);
  p.bn = bn;
  p.a_rows = a_rows;
  // (the MMA reads 128 rows of A whatever was copied: within the ring)
  const int stage_bytes = (a_rows + b_rows) * 128;
  p.stages = std::min({kTgMaxStages, C::RING_BYTES / stage_bytes,
                       1 + (C::RING_BYTES - 16384) / stage_bytes});
  p.steps = static_cast<int>(ceil_div(g.Kc, kTgKStep));
  p.mt = static_cast<int>(ceil_div(g.M, 128 * CG));
  p.nt = static_cast<int>(ceil_div(g.N, bn));
  p.sym = g.sym ? 1 : 0;
  p.per_batch = static_cast<int>(tg_tiles(g.M, g.N, 1, g.sym, 128 * CG, bn));
  p.split_steps = static_cast<int>(ceil_div(p.steps, SPLIT > 1 ? SPLIT : g.ksplit));
  p.ksplit = g.ksplit;
  p.tiles = static_cast<int>(g.batch * p.per_batch * p.ksplit);
  // Tile rows that share a sweep over n: 8, or up to 16 while their rows of A
  // stay within 32 MiB of L2 (8192 tokens over 128000 x 4096: 8 rows 6.16 ms,
  // 16 6.01, 32 6.40).  A contraction of up to 128 is all writing: one, whole
  // rows of the output at a time (dW of 64 tokens over 50021 x 1608, whose rows
  // share lines, 8 % less than with 8; of 300 tokens 1 % more).
  p.group = g.Kc <= 128 ? 1
                        : static_cast<int>(std::max<int64_t>(
                              8, std::min<int64_t>(16, (32LL << 20) / (128LL * CG * 2 * g.Kc))));
  p.backwards = g.backwards ? 1 : 0;
  p.passes = g.passes;
  p.idesc = tg_idesc(128 * CG, bn, Epi::kBf16, Epi::kAMn, Epi::kBMn);
  p.status = ds.status;
  p.wait_limit_ns = kWaitLimitNs;
  r.done = true;
  return BITNET_OK;
}

template <int CG, int BN, int SPLIT, class Epi>
bitnet_status launch_tg_cfg(const DeviceState& ds, const TgProblem& g,
                            const typename Epi::Params& ep, cudaStream_t stream, TgReady* ready) {
  using C = TgCfg<CG, BN, Epi>;
  TgReady own;
  TgReady& r = ready ? *ready : own;
  if (!r.done) {
    const bitnet_status st = prepare_tg<CG, BN, SPLIT, Epi>(ds, g, r);
    if (st != BITNET_OK) return st;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(
      CG * SPLIT * (SPLIT > 1 ? r.shape.tiles : std::min(r.workers, r.shape.tiles))));
  cfg.blockDim = dim3(kTgThreads);
  cfg.dynamicSmemBytes = C::SMEM_DYN;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG * SPLIT;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG * SPLIT > 1 ? 2 : 1;
  return cuda_status(
      cudaLaunchKernelEx(&cfg, tc_gemm_kernel<CG, BN, SPLIT, Epi>, r.maps, r.shape, ep));
}

// Pairs of 256 columns, or single SMs with tiles of up to BN1.
template <int BN1, class Epi>
bitnet_status launch_tg(const DeviceState& ds, const TgProblem& g,
                        const typename Epi::Params& ep, cudaStream_t stream,
                        TgReady* ready = nullptr) {
  return g.plan.cg == 2 ? launch_tg_cfg<2, 256, 1, Epi>(ds, g, ep, stream, ready)
                        : launch_tg_cfg<1, BN1, 1, Epi>(ds, g, ep, stream, ready);
}

// A head's logits: pairs sum contractions of more than one run in runs.
template <class Epi>
bitnet_status launch_logits(const DeviceState& ds, const TgProblem& g,
                            const typename Epi::Params& ep, cudaStream_t stream) {
  if (g.plan.cg == 2 && ceil_div(g.Kc, kTgKStep) <= Epi::kPairRun)
    return launch_tg_cfg<2, 256, 1, CeWhole<Epi>>(ds, g, ep, stream, nullptr);
  return launch_tg<256, Epi>(ds, g, ep, stream);
}

// X X^T, whose contraction is the long side: a 128 x 128 tile's may be shared by
// a cluster.
bitnet_status launch_gram(const DeviceState& ds, const TgProblem& g, const OrthoGram::Params& ep,
                          cudaStream_t stream, TgReady* ready) {
  switch (g.plan.split) {
    case 2: return launch_tg_cfg<1, 128, 2, OrthoGram>(ds, g, ep, stream, ready);
    case 3: return launch_tg_cfg<1, 128, 3, OrthoGram>(ds, g, ep, stream, ready);
    case 4: return launch_tg_cfg<1, 128, 4, OrthoGram>(ds, g, ep, stream, ready);
    default: return launch_tg<128, OrthoGram>(ds, g, ep, stream, ready);
  }
}

template <typename... KArgs, typename... Args>
bitnet_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, unsigned threads,
                         cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...));
}

// ------------------------------------------------------------- cross entropy

// Limits: as the warm-up's, and tile indices in 32 bits.
bitnet_status check_ce_shape(int64_t M, int64_t V, int64_t K) {
  if (M < 0 || V < 0 || K < 0) return BITNET_ERR_INVALID_ARG;
  if (V < 1 || V > BITNET_MAX_N || K < 8 || K % 8 != 0 || K > BITNET_MAX_K || M > BITNET_MAX_M ||
      ceil_div(M, 128) * ceil_div(V, 128) > (1LL << 30))
    return BITNET_ERR_UNSUPPORTED_SHAPE;
  return BITNET_OK;
}

// The logits' product, x [M] by `cols` of W.  Up to 128 tokens it reads W
// once and that is its time: single SMs, and tiles as wide as spreads the
// columns evenly over all of them (a multiple of `unit`).
TgPlan ce_logits_plan(int64_t M, int64_t cols, int64_t K, int unit) {
  if (M > 128) {
    const TgPlan pl = tg_plan(M, cols, 1, false, ceil_div(K, kTgKStep), 1);
    return pl;
  }
  const int64_t rounds = ceil_div(cols, 256LL * kPlanSms);
  return TgPlan{1, static_cast<int>(round_up(ceil_div(cols, rounds * kPlanSms), unit)), 1};
}

struct CeFwdLayout {
  TgPlan plan;
  int64_t parts;
  size_t part, total;
};

CeFwdLayout ce_fwd_layout(int64_t M, int64_t V, int64_t K) {
  CeFwdLayout w{};
  w.plan = ce_logits_plan(M, V, K, 16);
  w.parts = 2 * ceil_div(V, w.plan.bn);
  w.part = 0;
  w.total = align256(static_cast<size_t>(8 * w.parts * M));
  return w;
}

// Bytes of g that one piece of the vocabulary may take.
constexpr int64_t kCePieceBytes = 256LL << 20;

struct CeBwdLayout {
  int64_t cols, pieces;      // vocabulary columns of a piece, number of pieces
  TgPlan dx_plan;
  int dx_split;
  size_t g, acc, part, logit, scale, total;
};

CeBwdLayout ce_bwd_layout(int64_t M, int64_t V, int64_t K) {
  CeBwdLayout w{};
  const int64_t most = std::max<int64_t>(256, kCePieceBytes / (2 * M) / 256 * 256);
  w.pieces = ceil_div(V, most);
  w.cols = round_up(ceil_div(V, w.pieces), 256);
  w.pieces = ceil_div(V, w.cols);
  // dx has few tiles and a long contraction: split it so that the last wave
  // of tiles is full (at most 16 slices, 4 steps each at least).
  w.dx_plan = M > 128 && K > 128 ? TgPlan{2, 256, 1} : TgPlan{1, 128, 1};
  const int64_t tiles = tg_tiles(M, K, 1, false, 128 * w.dx_plan.cg, w.dx_plan.bn);
  const int64_t slots = kPlanSms / w.dx_plan.cg;
  const int64_t steps = ceil_div(std::min(w.cols, V), kTgKStep);
  w.dx_split = 1;
  double best = static_cast<double>(ceil_div(tiles, slots));
  for (int s = 2; s <= 16 && steps / s >= 4 && tiles < 2 * slots; ++s) {
    const double cost = static_cast<double>(ceil_div(tiles * s, slots)) / s;
    if (cost < 0.9 * best) {
      best = cost;
      w.dx_split = s;
    }
  }
  // every slice has work: steps are dealt in equal parts, the last one short
  const int64_t per = ceil_div(steps, w.dx_split);
  w.dx_split = static_cast<int>(ceil_div(steps, per));
  size_t o = 0;
  auto take = [&o](int64_t bytes) {
    const size_t at = o;
    o = align256(o + static_cast<size_t>(bytes));
    return at;
  };
  w.g = take(2 * M * w.cols);
  w.acc = take(w.pieces > 1 ? 4 * M * K : 0);
  w.part = take(w.dx_split > 1 ? 4 * M * K * w.dx_split : 0);
  w.logit = take(4 * M);
  w.scale = take(4);
  w.total = o;
  return w;
}

// -------------------------------------------------------- orthogonalisation

constexpr int kOrthoMaxSteps = 32;
// Largest smaller side that runs on both halves of its operands.
constexpr int64_t kOrthoSplitN = 192;

// Updates that run in one launch: on clusters of up to eight CTAs, or of
// sixteen, of which seven are resident at a time, for two rounds of them at
// most (128 x 4096: 1 matrix 101 us, as products of their own 183; 7: 104 and
// 213; 14: 208 and 263; 16: 306 and 272).
constexpr int64_t kOsWideBatch = 14;

bool ortho_is_small(int64_t B, int64_t N, int64_t K) {
  const int64_t k = std::max(N, K);
  return std::min(N, K) <= 128 &&
         (k <= 8 * kOsMaxKs || (k <= kOsMaxCluster * kOsMaxKs && B <= kOsWideBatch));
}

// CTAs per matrix: one while it holds all columns; else four or eight of 128
// columns each while the whole batch is resident (128 x 512: 2 CTAs 89 us, 4
// 72; x 1024: 4 91, 8 76, 16 75; but 40 of the first 94 and 148, 30 of the
// second 96 and 166); else as few as hold them.
int ortho_small_cluster(int64_t B, int64_t k) {
  if (k <= kOsMaxKs) return 1;
  if (k <= 4 * 128 && B <= 33) return 4;
  if (k > 4 * 128 && k <= 8 * 128 && B <= 15) return 8;
  int cluster = 2;
  while (cluster * kOsMaxKs < k) cluster *= 2;
  return cluster;
}

bitnet_status check_ortho_shape(int64_t B, int64_t N, int64_t K) {
  if (B < 0 || N < 0 || K < 0) return BITNET_ERR_INVALID_ARG;
  const int64_t n = std::min(N, K), k = std::max(N, K);
  if (N < 1 || K < 1 || k > BITNET_MAX_K || B > 65535 ||
      ceil_div(n, 128) * ceil_div(k, 128) > (1LL << 30) / std::max<int64_t>(B, 1))
    return BITNET_ERR_UNSUPPORTED_SHAPE;
  return BITNET_OK;
}

struct OrthoLayout {
  int64_t n, k, ldx, ldr;
  bool split;
  int parts;                 // blocks of the norm, per matrix
  size_t norm, X[2], X_lo[2], R, R_lo, Q, Q_lo, D, E, total;
};

OrthoLayout ortho_layout(int64_t B, int64_t N, int64_t K) {
  OrthoLayout w{};
  w.n = std::min(N, K);
  w.k = std::max(N, K);
  w.ldx = round_up(w.k, 64);
  w.ldr = round_up(w.n, 64);
  w.split = w.n <= kOrthoSplitN;
  w.parts = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(ceil_div(N * K, 8 * kOrthoNormThreads), 4 * kPlanSms)));
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  const size_t x = static_cast<size_t>(2 * B * w.n * w.ldx);
  const size_t r = static_cast<size_t>(2 * B * w.n * w.ldr);
  w.norm = take(static_cast<size_t>(8 * B * w.parts));
  for (int i = 0; i < 2; ++i) {
    w.X[i] = take(x);
    w.X_lo[i] = take(x);
  }
  w.R = take(r);
  w.Q = take(r);
  w.R_lo = take(w.split ? r : 0);
  w.Q_lo = take(w.split ? r : 0);
  w.D = take(static_cast<size_t>(4 * B * w.n));
  w.E = take(static_cast<size_t>(4 * B * w.n));
  w.total = o;
  return w;
}

// The largest |a s + b s^3 + c s^5| and |b t + c t^2| for s in [0, top],
// t = s^2: bounds of the next X and of b A + c A A.
void ortho_bounds(double a, double b, double c, double top, double* next, double* poly) {
  auto value = [&](double s) { return std::fabs(s * (a + s * s * (b + c * s * s))); };
  double m = value(top);
  // stationary points: a + 3 b t + 5 c t^2 = 0
  auto at = [&](double t) {
    if (t > 0.0 && t <= top * top) m = std::max(m, value(std::sqrt(t)));
  };
  if (c != 0.0) {
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (disc >= 0.0) {
      at((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
      at((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
    }
  } else if (b != 0.0) {
    at(-a / (3.0 * b));
  }
  *next = m;
  const double t = top * top;
  double q = std::fabs(t * (b + c * t));
  if (c != 0.0) {
    const double v = -b / (2.0 * c);
    if (v > 0.0 && v < t) q = std::max(q, std::fabs(v * (b + c * v)));
  }
  *poly = q;
}

// The power of two that brings values up to `top` below 2^15 (fp16 ends at
// 65504; the slack covers the rounding that pushes a value past its bound).
int fp16_exponent(double top) {
  return top > 0.0 ? 14 - static_cast<int>(std::ceil(std::log2(top))) : 14;
}

// The factors of a step with coefficients c[3], and in *ex the exponent of the
// stored X: before the step's, then the next one's (0, the result, at the last).
// top, next: bounds of X before and after the step; poly: of b A + c A A.
OrthoStep ortho_step(const double* c, double top, double next, double poly, bool last, int* ex) {
  const int ey = last ? 0 : fp16_exponent(next), er = fp16_exponent(top * top);
  const int e = ey - *ex;
  const int eq = poly > 0.0 ? fp16_exponent(poly) : e;  // (no Q: any will do)
  auto times = [](double v, int power) { return static_cast<float>(std::ldexp(v, power)); };
  const OrthoStep f{times(1.0, er - 2 * *ex), times(c[2], eq - 2 * er), times(c[1], eq - er),
                    times(c[0], e),           times(c[1], e - er),      times(c[2], e - 2 * er),
                    times(1.0, e - eq)};
  *ex = ey;
  return f;
}

bitnet_status launch_ortho_small(const DeviceState& ds, const void* U, int u_bf16, int64_t B,
                                 int64_t N, int64_t K, int steps, const double* coefficients,
                                 const double* top, const double* poly, float eps, void* O,
                                 cudaStream_t stream) {
  static std::once_flag once[kMaxDevices];
  static bool ok[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return BITNET_ERR_CUDA;
  std::call_once(once[dev],
                 [dev]() {
                   // (clusters of sixteen are past the portable size)
                   ok[dev] = set_smem(ortho_small_kernel, OsSmem::SMEM_DYN) &&
                             cudaFuncSetAttribute(ortho_small_kernel,
                                                  cudaFuncAttributeNonPortableClusterSizeAllowed,
                                                  1) == cudaSuccess;
                 });
  if (!ok[dev]) return BITNET_ERR_CUDA;
  OsParams p{};
  p.U = U;
  p.out = static_cast<__nv_bfloat16*>(O);
  p.u_bf16 = u_bf16;
  p.n = static_cast<int>(std::min(N, K));
  p.k = static_cast<int>(std::max(N, K));
  p.tall = N > K ? 1 : 0;
  p.cluster = ortho_small_cluster(B, p.k);
  p.ks = static_cast<int>(round_up(ceil_div(p.k, p.cluster), 64));
  p.steps = steps;
  p.eps = eps;
  p.status = ds.status;
  p.wait_limit_ns = kWaitLimitNs;
  int ex = fp16_exponent(top[0]);
  p.scale = std::ldexp(1.0f, ex);
  for (int i = 0; i < steps; ++i)
    p.step[i] = ortho_step(coefficients + 3 * i, top[i], top[i + 1], poly[i], i == steps - 1, &ex);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(B * p.cluster));
  cfg.blockDim = dim3(kOsThreads);
  cfg.dynamicSmemBytes = OsSmem::SMEM_DYN;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, ortho_small_kernel, p));
}

}  // namespace
}  // namespace bitnet

extern "C" {

BITNET_API size_t bitnet_cross_entropy_forward_workspace_bytes(int64_t M, int64_t V, int64_t K) {
  if (check_ce_shape(M, V, K) != BITNET_OK || M == 0) return 0;
  return ce_fwd_layout(M, V, K).total;
}

BITNET_API bitnet_status bitnet_cross_entropy_forward(const void* x, const void* W,
                                                      const int64_t* targets, int64_t M,
                                                      int64_t V, int64_t K, float* loss,
                                                      float* lse, void* workspace,
                                                      size_t workspace_bytes,
                                                      bitnet_stream_t stream) {
  bitnet_status st = check_ce_shape(M, V, K);
  if (st != BITNET_OK) return st;
  if (M == 0) return BITNET_OK;
  if (!x || !W || !targets || !loss || !lse) return BITNET_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(targets, 8) || !aligned(loss, 4) ||
      !aligned(lse, 4))
    return BITNET_ERR_MISALIGNED;
  const CeFwdLayout L = ce_fwd_layout(M, V, K);
  if (!workspace || workspace_bytes < L.total) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_MISALIGNED;
  DeviceState* ds = device_state();
  if (!ds) return BITNET_ERR_CUDA;
  cudaStream_t s = as_stream(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TgProblem g;
  g.a.p = x;
  g.a.ld = K;
  g.b.p = W;
  g.b.ld = K;
  g.M = M;
  g.N = V;
  g.Kc = K;
  g.plan = L.plan;
  CeStats::Params ep{targets, reinterpret_cast<float2*>(ws + L.part)};
  st = launch_logits<CeStats>(*ds, g, ep, s);
  if (st != BITNET_OK) return st;
  // (256 rows: a block per row is two waves of them, and the wide cut's
  // neighbouring parts begin to count)
  const bool wide = M > 256;
  return launch_pdl(wide ? ce_join_kernel<true> : ce_join_kernel<false>,
                    dim3(static_cast<unsigned>(wide ? ceil_div(M, 32) : M)), wide ? 1024 : 256, s,
                    ep.part, static_cast<int>(L.parts), static_cast<const __nv_bfloat16*>(x),
                    static_cast<const __nv_bfloat16*>(W), targets, V, K, static_cast<int>(M),
                    loss, lse);
}

BITNET_API size_t bitnet_cross_entropy_backward_workspace_bytes(int64_t M, int64_t V, int64_t K) {
  if (check_ce_shape(M, V, K) != BITNET_OK || M == 0) return 0;
  return ce_bwd_layout(M, V, K).total;
}

BITNET_API bitnet_status bitnet_cross_entropy_backward(const void* x, const void* W,
                                                       const int64_t* targets, const float* lse,
                                                       const float* dloss, int64_t M, int64_t V,
                                                       int64_t K, void* dx, void* dW,
                                                       void* workspace, size_t workspace_bytes,
                                                       bitnet_stream_t stream) {
  bitnet_status st = check_ce_shape(M, V, K);
  if (st != BITNET_OK) return st;
  if (dW && !aligned(dW, 16)) return BITNET_ERR_MISALIGNED;
  cudaStream_t s = as_stream(stream);
  if (M == 0) {
    if (dW) return cuda_status(cudaMemsetAsync(dW, 0, 2 * static_cast<size_t>(V * K), s));
    return BITNET_OK;
  }
  if (!x || !W || !targets || !lse || !dloss) return BITNET_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(targets, 8) || !aligned(lse, 4) ||
      !aligned(dloss, 4) || (dx && !aligned(dx, 16)))
    return BITNET_ERR_MISALIGNED;
  const CeBwdLayout L = ce_bwd_layout(M, V, K);
  if (!workspace || workspace_bytes < L.total) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_MISALIGNED;
  if (!dx && !dW) return BITNET_OK;
  DeviceState* ds = device_state();
  if (!ds) return BITNET_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  __nv_bfloat16* gbuf = reinterpret_cast<__nv_bfloat16*>(ws + L.g);
  float* acc = reinterpret_cast<float*>(ws + L.acc);
  float* part = reinterpret_cast<float*>(ws + L.part);
  float* scale = reinterpret_cast<float*>(ws + L.scale);
  float* logit = reinterpret_cast<float*>(ws + L.logit);
  st = launch_pdl(ce_target_kernel, dim3(static_cast<unsigned>(ceil_div(M, 8))), 256, s,
                  static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(W),
                  targets, dloss, M, V, K, logit, scale);
  if (st != BITNET_OK) return st;
  for (int64_t i = 0; i < L.pieces; ++i) {
    const int64_t v0 = i * L.cols, cols = std::min(L.cols, V - v0);
    const __nv_bfloat16* Wi = static_cast<const __nv_bfloat16*>(W) + v0 * K;
    {  // g of the piece
      TgProblem g;
      g.a.p = x;
      g.a.ld = K;
      g.b.p = Wi;
      g.b.ld = K;
      g.out.p = gbuf;
      g.out.ld = L.cols;
      g.M = M;
      g.N = cols;
      g.Kc = K;
      g.plan = ce_logits_plan(M, cols, K, 32);
      // The product before left the ends of W's rows in L2 (64 tokens over
      // 32000 x 2048, loss and gradient: 150 us from the front, 145 from the end).
      g.backwards = true;
      CeGrad::Params ep{targets, lse, dloss, logit, scale, V, v0};
      st = launch_logits<CeGrad>(*ds, g, ep, s);
      if (st != BITNET_OK) return st;
    }
    if (dx) {  // dx (+)= g W_i
      const bool first = i == 0, last = i == L.pieces - 1;
      TgProblem g;
      g.a.p = gbuf;
      g.a.ld = L.cols;
      g.b.p = Wi;
      g.b.ld = K;
      g.M = M;
      g.N = K;
      g.Kc = cols;
      g.plan = L.dx_plan;
      const int64_t steps = ceil_div(cols, kTgKStep);
      const int64_t per = ceil_div(steps, L.dx_split);
      g.ksplit = static_cast<int>(ceil_div(steps, per));
      TgAccumulate::Params ep{};
      g.out.ld = K;
      g.out.type = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
      if (g.ksplit > 1) {
        g.out.p = part;
        g.out.batch = g.ksplit;
        g.out.batch_stride = M * K;
      } else {
        if (!first) {
          ep.add = 1;
          g.in.p = acc;
          g.in.ld = K;
          g.in.type = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
        }
        g.out.p = acc;
        if (last) {
          ep.to_bf16 = 1;
          ep.scale = scale;
          g.out.p = dx;
          g.out.type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        }
      }
      st = launch_tg<128, TgAccumulate>(*ds, g, ep, s);
      if (st != BITNET_OK) return st;
      if (g.ksplit > 1) {
        const int64_t n4 = M * K / 4;
        const int64_t blocks = std::min<int64_t>(ceil_div(n4, 256), 8LL * ds->num_sms);
        st = launch_pdl(ce_join_dx_kernel, dim3(static_cast<unsigned>(blocks)), 256, s, part,
                        g.ksplit, M * K, first ? nullptr : acc, n4, acc, scale,
                        last ? static_cast<__nv_bfloat16*>(dx) : nullptr);
        if (st != BITNET_OK) return st;
      }
    }
    if (dW) {  // dW_i = g^T x
      TgProblem g;
      g.a.p = gbuf;
      g.a.ld = L.cols;
      g.b.p = x;
      g.b.ld = K;
      g.out.p = static_cast<__nv_bfloat16*>(dW) + v0 * K;
      g.out.ld = K;
      g.out.block = 64;
      g.M = cols;
      g.N = K;
      g.Kc = M;
      g.plan = tg_plan(cols, K, 1, false, ceil_div(M, kTgKStep), 1);
      st = launch_tg<128, TgStoreBf16>(*ds, g, TgStoreBf16::Params{scale}, s);
      if (st != BITNET_OK) return st;
    }
  }
  return BITNET_OK;
}

BITNET_API size_t bitnet_orthogonalize_workspace_bytes(int64_t B, int64_t N, int64_t K) {
  if (check_ortho_shape(B, N, K) != BITNET_OK || B == 0 || ortho_is_small(B, N, K)) return 0;
  return ortho_layout(B, N, K).total;
}

BITNET_API bitnet_status bitnet_orthogonalize(const void* U, int u_dtype, int64_t B, int64_t N,
                                              int64_t K, int steps, const double* coefficients,
                                              float eps, void* O, void* workspace,
                                              size_t workspace_bytes, bitnet_stream_t stream) {
  bitnet_status st = check_ortho_shape(B, N, K);
  if (st != BITNET_OK) return st;
  if (steps < 1 || steps > kOrthoMaxSteps || !coefficients || !ok_dtype(u_dtype) ||
      !(eps >= 0.0f) || eps > 3.0e38f)
    return BITNET_ERR_INVALID_ARG;
  // The scales of every step, from what its singular values can reach.
  double top[kOrthoMaxSteps + 1], poly[kOrthoMaxSteps];
  top[0] = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double* c = coefficients + 3 * i;
    if (!std::isfinite(c[0]) || !std::isfinite(c[1]) || !std::isfinite(c[2]))
      return BITNET_ERR_INVALID_ARG;
    ortho_bounds(c[0], c[1], c[2], top[i], &top[i + 1], &poly[i]);
    if (!(top[i + 1] <= 1048576.0) || !(poly[i] <= 1048576.0)) return BITNET_ERR_INVALID_ARG;
  }
  if (B == 0) return BITNET_OK;
  if (!U || !O) return BITNET_ERR_INVALID_ARG;
  if (!aligned(U, 16) || !aligned(O, 16)) return BITNET_ERR_MISALIGNED;
  if (ortho_is_small(B, N, K)) {
    DeviceState* ds = device_state();
    if (!ds) return BITNET_ERR_CUDA;
    return launch_ortho_small(*ds, U, u_dtype == BITNET_BF16 ? 1 : 0, B, N, K, steps,
                              coefficients, top, poly, eps, O, as_stream(stream));
  }
  const OrthoLayout L = ortho_layout(B, N, K);
  if (!workspace || workspace_bytes < L.total) return BITNET_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return BITNET_ERR_MISALIGNED;
  DeviceState* ds = device_state();
  if (!ds) return BITNET_ERR_CUDA;
  cudaStream_t s = as_stream(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto half_at = [ws](size_t o) { return reinterpret_cast<uint16_t*>(ws + o); };
  const bool tall = N > K;
  const int u_bf16 = u_dtype == BITNET_BF16 ? 1 : 0;
  double* norm = reinterpret_cast<double*>(ws + L.norm);
  float* D = reinterpret_cast<float*>(ws + L.D);
  float* E = reinterpret_cast<float*>(ws + L.E);
  uint16_t* R_lo = L.split ? half_at(L.R_lo) : nullptr;
  uint16_t* Q_lo = L.split ? half_at(L.Q_lo) : nullptr;
  const int64_t xb = L.n * L.ldx, rb = L.n * L.ldr;

  st = launch_pdl(ortho_norm_kernel,
                  dim3(static_cast<unsigned>(L.parts), static_cast<unsigned>(B)),
                  kOrthoNormThreads, s, U, u_bf16, N * K, N * K % 8 == 0 ? 1 : 0, norm);
  if (st != BITNET_OK) return st;
  int ex = fp16_exponent(top[0]);
  const float scale = std::ldexp(1.0f, ex);
  if (tall) {
    st = launch_pdl(ortho_start_tall_kernel,
                    dim3(static_cast<unsigned>(ceil_div(N, 64)),
                         static_cast<unsigned>(ceil_div(K, 32)), static_cast<unsigned>(B)),
                    256, s, U, u_bf16, static_cast<int>(N), static_cast<int>(K), norm, L.parts,
                    eps, scale, half_at(L.X[0]), half_at(L.X_lo[0]), L.ldx);
  } else {
    const int64_t blocks = std::min<int64_t>(N, std::max<int64_t>(1, 16LL * ds->num_sms / B));
    st = launch_pdl(ortho_start_kernel,
                    dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(B)), 256, s, U,
                    u_bf16, N, K, K % 8 == 0 ? 1 : 0, norm, L.parts, eps, scale,
                    half_at(L.X[0]), half_at(L.X_lo[0]), L.ldx);
  }
  if (st != BITNET_OK) return st;

  const int passes = L.split ? 3 : 1;
  const int64_t n_steps = ceil_div(L.n, kTgKStep), k_steps = ceil_div(L.k, kTgKStep);
  const TgPlan gram_plan = tg_plan(L.n, L.n, B, !L.split, k_steps, passes, 4);
  const TgPlan poly_plan = tg_plan(L.n, L.n, B, !L.split, n_steps, passes);
  const TgPlan update_plan = tg_plan(L.n, L.k, B, false, n_steps, passes);
  // The result goes out by TMA where its rows are whole 16-byte pieces.
  const bool direct = !tall && L.k % 8 != 0;
  TgReady gram_ready[2], poly_ready, update_ready[2], last_ready;
  for (int i = 0; i < steps; ++i) {
    const int from = i & 1, to = from ^ 1;
    const bool last = i == steps - 1;
    const OrthoStep f =
        ortho_step(coefficients + 3 * i, top[i], top[i + 1], poly[i], last, &ex);
    TgProblem g;
    g.batch = B;
    g.passes = passes;
    // A = X X^T
    g.M = g.N = L.n;
    g.Kc = L.k;
    g.sym = !L.split;
    g.a.p = half_at(L.X[from]);
    g.a.lo = half_at(L.X_lo[from]);
    g.a.ld = L.ldx;
    g.a.batch_stride = xb;
    g.b = g.a;
    g.out.p = half_at(L.R);
    g.out.lo = R_lo;
    g.out.ld = L.ldr;
    g.out.batch_stride = rb;
    g.out.batch = B;
    g.out.type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    g.plan = gram_plan;
    OrthoGram::Params gram{D, L.split ? 1 : 0, f};
    st = launch_gram(*ds, g, gram, s, &gram_ready[from]);
    if (st != BITNET_OK) return st;
    // R R -> Q, E
    g.Kc = L.n;
    g.a.p = half_at(L.R);
    g.a.lo = R_lo;
    g.a.ld = L.ldr;
    g.a.batch_stride = rb;
    g.b = g.a;
    g.in = g.out;
    g.out.p = half_at(L.Q);
    g.out.lo = Q_lo;
    g.plan = poly_plan;
    OrthoPoly::Params poly_p{D, E, L.split ? 1 : 0, f};
    st = launch_tg<128, OrthoPoly>(*ds, g, poly_p, s, &poly_ready);
    if (st != BITNET_OK) return st;
    // X <- E X + Q X
    g.sym = false;
    g.N = L.k;
    g.a.p = half_at(L.Q);
    g.a.lo = Q_lo;
    g.b.p = half_at(L.X[from]);
    g.b.lo = half_at(L.X_lo[from]);
    g.b.ld = L.ldx;
    g.b.batch_stride = xb;
    g.in.p = g.b.p;
    g.in.lo = g.b.lo;
    g.in.ld = L.ldx;
    g.in.batch_stride = xb;
    g.out = g.in;
    g.out.p = half_at(L.X[to]);
    g.out.lo = half_at(L.X_lo[to]);
    if (last) {
      g.out = TgTensor{};
      if (!tall && !direct) {
        g.out.p = O;
        g.out.ld = L.k;
        g.out.batch_stride = L.n * L.k;
        g.out.batch = B;
      }
    }
    g.plan = update_plan;
    OrthoUpdate::Params up{E, last ? static_cast<__nv_bfloat16*>(O) : nullptr, tall ? 1 : 0,
                           direct ? 1 : 0, f.ku};
    st = launch_tg<128, OrthoUpdate>(*ds, g, up, s, last ? &last_ready : &update_ready[from]);
    if (st != BITNET_OK) return st;
  }
  return BITNET_OK;
}

}  // extern "C"
