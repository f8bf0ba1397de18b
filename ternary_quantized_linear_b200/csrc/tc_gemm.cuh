// tc_gemm.cuh -- the 16-bit matrix product behind the training operators
// (vocabulary cross entropy, orthogonalised updates): D = A B^T with fp32
// sums in TMEM and an epilogue of the operator's own, persistent and
// warp-specialised for sm_100a.
//
//   D[b][m][n] = sum_k A[b](m, k) B[b](n, k)
//
// A and B are bf16 or fp16 (both the same).  Each is either K-major (k
// contiguous in memory) or MN-major (m or n contiguous), so no product of the
// operators needs a transposed copy.  `passes` = 3 sums A B + A B_lo + A_lo B
// for operands held as a high and a low half.
//
// Layout of the work: an output tile is (128 CG) x BN.  CG = 2 pairs two SMs
// on one 256-row tile (cta_group::2): each CTA holds its own 128 rows of A
// and half of B's rows, so a byte of B in shared memory feeds twice the MMA
// work; CG = 1 is for outputs with few tiles.  Tiles are dealt round-robin to
// a grid of resident CTAs; the accumulator is double-buffered in TMEM, so a
// tile's epilogue runs under the next tile's MMAs.
//
// Warps: 0 copies (TMA, one thread, a ring of 64-k stages), 1 issues the MMAs
// (the pair's leader only), 2 owns TMEM, 4..11 run the epilogue: warp w reads
// TMEM lanes 32 (w % 4) .. +31, and columns [0, BN/2) for w < 8, else the
// other half.  Every wait is bounded; on a timeout the kernel records the
// failure, lets its copies land and exits.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace bitnet {

constexpr int kTgThreads = 384;
constexpr int kTgEpiWarps = 8;
constexpr int kTgKStep = 64;  // elements: one 128-byte swizzle row

template <int CG, int BN>
struct TgCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_ROWS = BN / CG;
  static constexpr int B_BYTES = B_ROWS * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 6;
  static constexpr uint32_t TMEM_COLS = 2 * BN;  // two accumulators
  static constexpr int OFF_BAR = STAGES * STAGE_BYTES;
  static constexpr int NBAR = 2 * STAGES + 5;    // full, empty, accfull[2], accempty[2], drain
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_DYN = OFF_MISC + 16 + 1024;
  static_assert(BN == 128 || BN == 256, "BN");
  static_assert(TMEM_COLS <= 512, "TMEM");
  static_assert(B_ROWS % 64 == 0, "MN-major boxes hold 64 rows");
  static_assert(SMEM_DYN <= 232448, "shared memory");
};

struct TgMaps {
  CUtensorMap a, b, a_lo, b_lo;
};

struct TgShape {
  int M, N;              // output rows and columns
  int steps;             // 64-k steps of the contraction
  int mt, nt;            // tiles
  int per_batch;         // tiles of one batch entry
  int ksplit, split_steps;
  int tiles;             // all: batch * per_batch * ksplit
  int sym;               // only tiles with m >= n (square output)
  int group;             // m tiles that share one sweep over n
  int passes;
  int a_mn, b_mn;
  uint32_t idesc;
  int* status;
  uint64_t wait_limit_ns;
};

struct TgTile {
  int b, m, n, split;    // batch entry, tile row and column, part of the contraction
};

__device__ __forceinline__ TgTile tg_tile(const TgShape& p, int t) {
  TgTile o;
  o.split = t % p.ksplit;
  t /= p.ksplit;
  o.b = t / p.per_batch;
  const int r = t - o.b * p.per_batch;
  if (p.sym) {
    int i = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
    while (static_cast<int64_t>(i + 1) * (i + 2) / 2 <= r) ++i;
    while (static_cast<int64_t>(i) * (i + 1) / 2 > r) --i;
    o.m = i;
    o.n = r - static_cast<int>(static_cast<int64_t>(i) * (i + 1) / 2);
  } else {
    // m varies fastest inside a group of `group` tile rows: B's tile stays
    // in L2 for all of them, A's group for the whole sweep.
    const int width = p.group * p.nt;
    const int g = r / width, w = r - g * width;
    const int first = g * p.group;
    const int rows = min(p.group, p.mt - first);
    o.n = w / rows;
    o.m = first + (w - o.n * rows);
  }
  return o;
}

// ------------------------------------------------------------- PTX wrappers

// 3-D tiled bulk tensor load; with CG = 2 `bar` may belong to the pair's
// other CTA (a shared::cluster address).
template <int CG>
__device__ __forceinline__ void tg_tma_load(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tg_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` (in both CTAs of a pair) once this thread's MMAs are done.
template <int CG>
__device__ __forceinline__ void tg_commit(uint64_t* bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    tc_commit(bar);
}

template <int CG>
__device__ __forceinline__ void tg_tmem_alloc(uint32_t* slot, uint32_t ncols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, ncols);
    tmem_relinquish();
  }
}

template <int CG>
__device__ __forceinline__ void tg_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
  else
    tmem_dealloc(taddr, ncols);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The shared::cluster address of `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// 32 lanes x 32 columns.
__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Matrix descriptor of an MN-major operand in the 128-byte swizzled layout:
// blocks of 64 (m or n) x 64 k, each k row 128 bytes; 8-k atoms of 1024 bytes
// (stride byte offset), the next 64 rows of the operand 8192 bytes on
// (leading byte offset).
__device__ __forceinline__ uint64_t umma_desc_sw128_mnmajor(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Instruction descriptor: kind::f16, fp32 sums; M = rows of the whole tile.
__host__ __device__ constexpr uint32_t tg_idesc(int M, int N, bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// One operand's part of a stage: `rows` rows from row0, 64 k from k0.
template <int CG>
__device__ __forceinline__ void tg_load(const CUtensorMap* map, bool mn, int rows, uint32_t dst,
                                        int row0, int k0, int b, uint32_t bar) {
  if (!mn) {
    tg_tma_load<CG>(dst, map, k0, row0, b, bar);
  } else {
    for (int i = 0; i < rows; i += 64)
      tg_tma_load<CG>(dst + i * 128, map, row0 + i, k0, b, bar);
  }
}

// What an epilogue knows about its part of a tile.
struct TgPart {
  TgTile tile;
  int row;       // output row of this thread
  int col0;      // first output column of this warp
  uint32_t tmem; // address of that column for this warp's lanes
  int half;      // column half
};

// ------------------------------------------------------------------- kernel

// Epi: struct with Params and template<int COLS> run(const Params&, const
// TgShape&, const TgPart&), which reads COLS columns of the warp's lanes.
template <int CG, int BN, class Epi>
__global__ void __launch_bounds__(kTgThreads, 1)
tc_gemm_kernel(const __grid_constant__ TgMaps maps, const TgShape p,
               const typename Epi::Params ep) {
  using C = TgCfg<CG, BN>;
  extern __shared__ uint8_t tg_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(tg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::STAGES;
  uint64_t* accfull = empty + C::STAGES;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const uint64_t limit = p.wait_limit_ns;
  const int worker = static_cast<int>(blockIdx.x) / CG;
  const int workers = static_cast<int>(gridDim.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], CG * kTgEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 2) tg_tmem_alloc<CG>(tmem_slot, C::TMEM_COLS);
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;  // stages issued
      bool ok = true;
      for (int t = worker; t < p.tiles && ok; t += workers) {
        const TgTile tile = tg_tile(p, t);
        const int k_lo = tile.split * p.split_steps;
        const int k_hi = min(p.steps, k_lo + p.split_steps);
        const int a0 = tile.m * 128 * CG + 128 * static_cast<int>(rank);
        const int b0 = tile.n * BN + C::B_ROWS * static_cast<int>(rank);
        for (int pass = 0; pass < p.passes && ok; ++pass) {
          const CUtensorMap* ma = pass == 2 ? &maps.a_lo : &maps.a;
          const CUtensorMap* mb = pass == 1 ? &maps.b_lo : &maps.b;
          for (int j = k_lo; j < k_hi; ++j, ++it) {
            const uint32_t s = it % C::STAGES, round = it / C::STAGES;
            if (round > 0 && !mbar_wait_bounded(&empty[s], (round - 1) & 1u, abort_flag, limit)) {
              *abort_flag = 1;
              record_failure(p.status, DEV_TIMEOUT_PRODUCER);
              ok = false;
              break;
            }
            const uint32_t dst = smem_u32(smem + s * C::STAGE_BYTES);
            uint32_t bar = smem_u32(&full[s]);
            if (CG == 2) bar = map_to_rank(bar, 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * C::STAGE_BYTES);
            tg_load<CG>(ma, p.a_mn, 128, dst, a0, j * kTgKStep, tile.b, bar);
            tg_load<CG>(mb, p.b_mn, C::B_ROWS, dst + C::A_BYTES, b0, j * kTgKStep, tile.b, bar);
          }
        }
      }
      // The last commits must have arrived before this CTA's barriers go away.
      const uint32_t from = it > static_cast<uint32_t>(C::STAGES) ? it - C::STAGES : 0u;
      for (uint32_t i = from; i < it && ok; ++i)
        if (!mbar_wait_bounded(&empty[i % C::STAGES], (i / C::STAGES) & 1u, abort_flag, limit)) {
          *abort_flag = 1;
          record_failure(p.status, DEV_TIMEOUT_PRODUCER);
          ok = false;
        }
      // After a timeout, let the copies in flight land first (otherwise the
      // MMAs have consumed them all).
      if (*abort_flag && rank == 0)
        for (uint32_t i = from; i < it; ++i)
          if (!mbar_wait_bounded(&full[i % C::STAGES], (i / C::STAGES) & 1u, nullptr, limit))
            record_failure(p.status, DEV_TIMEOUT_DRAIN);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t it = 0;
      int local = 0;
      bool ok = true;
      for (int t = worker; t < p.tiles && ok; t += workers, ++local) {
        const int buf = local & 1;
        const TgTile tile = tg_tile(p, t);
        const int k_lo = tile.split * p.split_steps;
        const int k_hi = min(p.steps, k_lo + p.split_steps);
        const int n_it = (k_hi - k_lo) * p.passes;
        if (local >= 2 && !mbar_wait_bounded(&accempty[buf],
                                             static_cast<uint32_t>((local >> 1) - 1) & 1u,
                                             abort_flag, limit)) {
          *abort_flag = 1;
          record_failure(p.status, DEV_TIMEOUT_MMA);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
        for (int j = 0; j < n_it; ++j, ++it) {
          const uint32_t s = it % C::STAGES;
          if (!mbar_wait_bounded(&full[s], (it / C::STAGES) & 1u, abort_flag, limit)) {
            *abort_flag = 1;
            record_failure(p.status, DEV_TIMEOUT_MMA);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a = smem_u32(smem + s * C::STAGE_BYTES);
          const uint32_t b = a + C::A_BYTES;
#pragma unroll
          for (int kk = 0; kk < kTgKStep / 16; ++kk) {
            const uint64_t da = p.a_mn ? umma_desc_sw128_mnmajor(a + 2048 * kk)
                                       : umma_desc_sw128_kmajor(a + 32 * kk);
            const uint64_t db = p.b_mn ? umma_desc_sw128_mnmajor(b + 2048 * kk)
                                       : umma_desc_sw128_kmajor(b + 32 * kk);
            tg_mma<CG>(d, da, db, p.idesc, (j > 0 || kk > 0) ? 1u : 0u);
          }
          tg_commit<CG>(&empty[s]);
        }
        if (ok) tg_commit<CG>(&accfull[buf]);
      }
      if (*abort_flag) {  // the MMAs issued so far still read shared memory
        tg_commit<CG>(drain);
        if (!mbar_wait_bounded(drain, 0u, nullptr, limit))
          record_failure(p.status, DEV_TIMEOUT_DRAIN);
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    int local = 0;
    for (int t = worker; t < p.tiles; t += workers, ++local) {
      const int buf = local & 1;
      const bool ok = __all_sync(
          0xFFFFFFFFu, mbar_wait_bounded(&accfull[buf], static_cast<uint32_t>(local >> 1) & 1u,
                                         abort_flag, limit));
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) record_failure(p.status, DEV_TIMEOUT_EPILOGUE);
        break;
      }
      tc_fence_after_sync();
      TgPart part;
      part.tile = tg_tile(p, t);
      part.row = part.tile.m * 128 * CG + 128 * static_cast<int>(rank) + 32 * q + lane;
      part.col0 = part.tile.n * BN + half * (BN / 2);
      part.tmem = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                  static_cast<uint32_t>(buf * BN + half * (BN / 2));
      part.half = half;
      Epi::template run<BN / 2>(ep, p, part);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(map_to_rank(smem_u32(&accempty[buf]), 0));
        else
          mbar_arrive(&accempty[buf]);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 2) {
    tc_fence_after_sync();
    tg_tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------ epilogue tools

// Store 32 consecutive 16-bit values of one row (two per word); vec when the
// address is 16-byte aligned and all 32 fit, else n of them one by one.
__device__ __forceinline__ void store_row32_16(uint16_t* dst, const uint32_t (&w)[16], bool vec,
                                               int n) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) dst[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(a))) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(b))) << 16);
}

// D to memory: fp32 (plus `add` when given; the part's own slice for a split
// contraction) or bf16.
struct TgStore {
  struct Params {
    float* f32;           // fp32 out, or
    __nv_bfloat16* bf16;  // bf16 out
    const float* add;     // fp32 [M][ld] added first, or null
    int64_t ld;           // of f32 and add
    int64_t ld_out;       // of bf16
    int64_t split_stride; // elements between the slices of a split contraction
    const float* scale;   // device scalar times the bf16 result, or null
  };
  template <int COLS>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgPart& t) {
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      const int col = t.col0 + c;
      if (col >= p.N) break;  // the same for all of the warp
      uint32_t r[32];
      tmem_ld_32x32b_x32(t.tmem + c, r);
      tmem_ld_wait();
      if (t.row < p.M) {
        const int n = min(32, p.N - col);
        if (e.add) {
          const float* s = e.add + t.row * e.ld + col;
          if (n == 32 && (e.ld & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = *reinterpret_cast<const float4*>(s + 4 * i);
              r[4 * i] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i]), v.x));
              r[4 * i + 1] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i + 1]), v.y));
              r[4 * i + 2] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i + 2]), v.z));
              r[4 * i + 3] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i + 3]), v.w));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < n) r[i] = __float_as_uint(__fadd_rn(__uint_as_float(r[i]), s[i]));
          }
        }
        if (e.bf16) {
          uint32_t w[16];
          const float f = e.scale ? __ldg(e.scale) : 1.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = pack_bf16x2(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
          store_row32_16(reinterpret_cast<uint16_t*>(e.bf16) + t.row * e.ld_out + col, w,
                         n == 32 && (e.ld_out & 7) == 0, n);
        } else {
          float* d = e.f32 + t.tile.split * e.split_stride + t.row * e.ld + col;
          if (n == 32 && (e.ld & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(d)[i] =
                  make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < n) d[i] = __uint_as_float(r[i]);
          }
        }
      }
    }
  }
};

}  // namespace bitnet
