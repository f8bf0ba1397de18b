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
// Layout of the work: an output tile is (128 CG) x bn, bn <= BN.  CG = 2 pairs
// two SMs on one 256-row tile (cta_group::2): each CTA holds its own 128 rows
// of A and half of B's rows, so a byte of B in shared memory feeds twice the
// MMA work; CG = 1 is for outputs with few tiles.  An SM takes 64 bytes a
// cycle from L2, and a 64-k step of a 256 x 256 pair tile needs 32 KiB per SM
// and 512 cycles of MMA: both just meet, while a 128 x 128 tile, with as many
// bytes for half the MMA work, runs at half the rate.  SPLIT = 2 to 4 (CG = 1,
// X X^T) lets a cluster of CTAs share one tile's contraction: each sums its
// part, the parts meet through distributed shared memory, added in rank
// order, and each CTA finishes its share of the columns.
//
// Tiles are dealt round-robin to a grid of resident CTAs; the accumulator is
// double-buffered in TMEM, so a tile's epilogue runs under the next tile's
// MMAs.
//
// Warps: 0 copies (TMA, one thread, a ring of 64-k stages), 1 issues the MMAs
// (the pair's leader only), 2 owns TMEM, 4..11 run the epilogue: warp w has
// TMEM lanes 32 (w % 4) .. +31, and every other chunk of 32 columns.  The
// epilogue's tensors pass through shared memory in 32 x 32 blocks, copied by
// TMA: a warp's own loads and stores, one row per lane, cost 32 transactions
// each and took longer than the MMAs of a short contraction.
//
// A kernel's first pass through its epilogue waits for its instructions to
// arrive, about 5 us; the epilogue warps take that pass on an empty tile
// (`dry`) while the first copies and MMAs are under way.
//
// The tensor cores truncate every sum: 16 terms at a time, half a unit of the
// last place off toward zero on average, so a logit of 4096 terms comes out
// some 1e-5 of itself too small.  An epilogue that needs better (kRun, kPairRun)
// has the contraction in runs of so many steps, which its warps add up with
// rounding: on single SMs in the second accumulator; a pair's tile fills TMEM
// with its two, which its runs take in turn, and the sums are held in registers,
// 128 a thread.  Terms of one sign, logits of 40, 256 tokens over 40000 entries:
// the loss is off by 1.2e-5, 4.0e-5 and 1.2e-4 of itself for 2048, 4096 and 8192
// terms in one go, by 3.9e-6 for each in runs of 16 steps (fp32 torch 2.7e-6,
// 3.4e-6, 5.6e-6).
//
// A product of fewer than 128 rows copies only those (rounded up to 8): the
// MMA then takes whatever follows in the ring for the missing rows, whose sums
// nobody reads, and the ring holds more stages.  Reading a head for one token
// needs them: a 224 x 64 piece of it takes 3.6 us to arrive when all SMs ask.
//
// Every wait on a barrier in shared memory is bounded; on a timeout the kernel
// records the failure, lets its copies land and exits.  Cluster barriers and
// the wait for the launch before have no limit of their own: they end because
// the peers' and that launch's waits do.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace bitnet {

constexpr int kTgThreads = 384;
constexpr int kTgEpiWarps = 8;
constexpr int kTgKStep = 64;  // elements: one 128-byte swizzle row

constexpr int kTgMaxStages = 16;

// Registers of a thread at launch (65536 over 384 threads, a multiple of 8), and
// after the split where the epilogue keeps sums in them: warps 0 to 3 need 40,
// the rest goes to the epilogue (216, with 72 for the others, spills).
constexpr int kTgRegs = 168, kTgLightRegs = 40, kTgEpiRegs = 232;
static_assert(128 * kTgLightRegs + 32 * kTgEpiWarps * kTgEpiRegs <= kTgThreads * kTgRegs,
              "the split may not ask for more than the block was launched with");

// Epi::kSlots blocks of Epi::kSlotBytes per epilogue warp for its tensors; the
// rest of shared memory is the ring.
template <int CG, int BN, class Epi>
struct TgCfg {
  static constexpr int EPI_BYTES = kTgEpiWarps * Epi::kSlots * Epi::kSlotBytes;
  static constexpr int RING_BYTES = (232448 - 2048 - EPI_BYTES) / 1024 * 1024;
  static constexpr uint32_t PAIR_STAGES =
      RING_BYTES / ((128 + BN / 2) * 128) < 6 ? RING_BYTES / ((128 + BN / 2) * 128) : 6;
  static constexpr uint32_t TMEM_COLS = 2 * BN;  // two accumulators
  static constexpr int OFF_EPI = RING_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + EPI_BYTES;
  // full, empty, accfull[2], accempty[2], drain, parts, one per epilogue block
  static constexpr int NBAR = 2 * kTgMaxStages + 6 + kTgEpiWarps * Epi::kSlots;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_DYN = OFF_MISC + 16 + 1024;
  static_assert(BN == 128 || BN == 256, "BN");
  static_assert(RING_BYTES >= 4 * (128 + BN / CG) * 128, "ring");
  static_assert(TMEM_COLS <= 512, "TMEM");
  static_assert(SMEM_DYN <= 232448, "shared memory");
};

// Operands, and the epilogue's tensors (32 x 32 boxes; unused ones are zero).
struct TgMaps {
  CUtensorMap a, b, a_lo, b_lo;
  CUtensorMap in, in_lo, out, out_lo;
};

struct TgShape {
  int M, N;              // output rows and columns
  int bn;                // columns of a tile
  int a_rows;            // rows of A that a stage holds (128, or fewer when M is smaller)
  int stages;            // of the ring (single SMs)
  int steps;             // 64-k steps of the contraction
  int mt, nt;            // tiles
  int per_batch;         // tiles of one batch entry
  int ksplit, split_steps;  // slices of the contraction (tiles of their own, or a cluster's CTAs)
  int tiles;             // all: batch * per_batch * ksplit
  int sym;               // only tiles with m >= n (square output)
  int group;             // m tiles that share one sweep over n
  int backwards;         // the contraction runs from its end
  int passes;
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
    // Bands of 8 tile rows; a band is swept over n with m fastest (its square
    // part, then the triangle on the diagonal), so that tiles under way
    // together share rows of both operands.  Before band t: 32 t^2 + 4 t.
    int t8 = static_cast<int>((sqrtf(16.0f + 128.0f * static_cast<float>(r)) - 4.0f) / 64.0f);
    while (static_cast<int64_t>(t8 + 1) * (32LL * (t8 + 1) + 4) <= r) ++t8;
    while (static_cast<int64_t>(t8) * (32LL * t8 + 4) > r) --t8;
    const int first = 8 * t8, rows = min(8, p.mt - first);
    int w = r - static_cast<int>(static_cast<int64_t>(t8) * (32LL * t8 + 4));
    if (w < rows * first) {
      o.n = w / rows;
      o.m = first + (w - o.n * rows);
    } else {
      w -= rows * first;
      int i = 0;
      while (w > i) w -= ++i;  // row i of the triangle has i + 1 tiles
      o.m = first + i;
      o.n = first + w;
    }
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

// Give back registers, or take more (waits until others gave theirs back): all
// warps of a warpgroup.
template <int N, bool kMore>
__device__ __forceinline__ void set_max_regs() {
  if constexpr (kMore)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// True in one lane of the warp, the same one every time; all lanes call it.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}" : "=r"(one)::"memory");
  return one != 0;
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
template <int CG, bool MN>
__device__ __forceinline__ void tg_load(const CUtensorMap* map, int rows, uint32_t dst, int row0,
                                        int k0, int b, uint32_t bar) {
  if constexpr (!MN) {
    tg_tma_load<CG>(dst, map, k0, row0, b, bar);
  } else {
    for (int i = 0; i < rows; i += 64)
      tg_tma_load<CG>(dst + i * 128, map, row0 + i, k0, b, bar);
  }
}

// ------------------------------------------------------- epilogue machinery

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(src)
      : "memory");
}

__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// At most `n` of this thread's store groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// What an epilogue knows about its part of a tile.
struct TgPart {
  TgTile tile;
  int row0, row;        // first output row of the warp, row of this thread
  int col0, col_end;    // the tile's columns [col0, col_end)
  int first, step;      // the warp's chunks: columns col0 + first + i * step, 32 each
  bool dry;             // an empty pass: no tensor is read or written
  bool live;            // this thread's row exists (never in a dry pass)
  bool any;             // the warp's first row does: there is something to store

  __device__ __forceinline__ int chunks() const {
    const int w = col_end - col0 - first;
    return w <= 0 ? 0 : (w + step - 1) / step;
  }
};

// A warp's blocks of shared memory, used in turn; `seq` counts blocks.
// 16-bit tensors: 32 rows of 64 bytes, 64-byte swizzle (16-byte piece j of
// row r at piece j ^ ((r >> 1) & 3)); fp32: 32 rows of 128 bytes, 128-byte
// swizzle (piece j at j ^ (r & 7)).  Either way the lanes of a quarter warp,
// one row each, hit all banks once.
struct TgStage {
  uint8_t* base;
  uint64_t* bars;
  uint32_t seq;
  int lane;
  volatile int* abort_flag;
  int* status;
  uint64_t limit;
  float pre[2];         // values that begin() loads ahead for run()
};

__device__ __forceinline__ uint32_t block16_piece(int lane, int j) {
  return static_cast<uint32_t>(lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t block32_piece(int lane, int j) {
  return static_cast<uint32_t>(lane * 128 + ((j ^ (lane & 7)) << 4));
}

__device__ __forceinline__ void block16_write(uint8_t* blk, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(blk + block16_piece(lane, j)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

__device__ __forceinline__ void block16_read(const uint8_t* blk, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = *reinterpret_cast<const uint4*>(blk + block16_piece(lane, j));
    w[4 * j] = v.x;
    w[4 * j + 1] = v.y;
    w[4 * j + 2] = v.z;
    w[4 * j + 3] = v.w;
  }
}

// Loads of the epilogue's input blocks, two chunks ahead, for an Epi with
// three slots whose outputs replace the inputs in place.
template <class Epi>
struct TgInput {
  // Chunk i of the part into the slot of block seq + i.
  static __device__ __forceinline__ void issue(TgStage& st, const TgMaps& m, const TgPart& t,
                                               int i, uint32_t seq, bool two, uint32_t bytes) {
    const uint32_t s = seq % Epi::kSlots;
    uint8_t* blk = st.base + s * Epi::kSlotBytes;
    const int col = t.col0 + t.first + i * t.step;
    mbar_arrive_expect_tx(&st.bars[s], two ? 2 * bytes : bytes);
    const uint32_t bar = smem_u32(&st.bars[s]);
    tg_tma_load<1>(smem_u32(blk), &m.in, col, t.row0, t.tile.b, bar);
    if (two) tg_tma_load<1>(smem_u32(blk + bytes), &m.in_lo, col, t.row0, t.tile.b, bar);
  }
  static __device__ __forceinline__ void begin(TgStage& st, const TgMaps& m, const TgPart& t,
                                               bool two, uint32_t bytes) {
    if (st.lane == 0 && !t.dry) {
      bulk_wait_read<0>();
      const int n = t.chunks();
      if (n > 0) issue(st, m, t, 0, st.seq, two, bytes);
      if (n > 1) issue(st, m, t, 1, st.seq + 1, two, bytes);
    }
  }
  // Wait for the current block; on a timeout also for the one behind it.
  static __device__ __forceinline__ bool wait(TgStage& st, const TgPart& t, int i) {
    if (t.dry) return true;
    const uint32_t s = st.seq % Epi::kSlots, ph = (st.seq / Epi::kSlots) & 1u;
    if (__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&st.bars[s], ph, nullptr, st.limit)))
      return true;
    *st.abort_flag = 1;
    if (st.lane == 0) {
      record_failure(st.status, DEV_TIMEOUT_EPILOGUE);
      if (i + 1 < t.chunks()) {
        const uint32_t s1 = (st.seq + 1) % Epi::kSlots, p1 = ((st.seq + 1) / Epi::kSlots) & 1u;
        if (!mbar_wait_bounded(&st.bars[s1], p1, nullptr, st.limit))
          record_failure(st.status, DEV_TIMEOUT_DRAIN);
      }
    }
    __syncwarp();
    return false;
  }
  // Loads that begin() issued for a part that is not run.
  static __device__ __forceinline__ void abandon(TgStage& st, const TgPart& t) {
    if (st.lane != 0) return;
    for (int i = 0; i < 2 && i < t.chunks(); ++i) {
      const uint32_t s = (st.seq + i) % Epi::kSlots, ph = ((st.seq + i) / Epi::kSlots) & 1u;
      if (!mbar_wait_bounded(&st.bars[s], ph, nullptr, st.limit))
        record_failure(st.status, DEV_TIMEOUT_DRAIN);
    }
  }
  // After the store of chunk i was committed: fetch chunk i + 2 into the slot
  // that the store before it has finished reading.
  static __device__ __forceinline__ void next(TgStage& st, const TgMaps& m, const TgPart& t,
                                              int i, bool two, uint32_t bytes) {
    if (st.lane == 0 && !t.dry && i + 2 < t.chunks()) {
      bulk_wait_read<1>();
      issue(st, m, t, i + 2, st.seq + 2, two, bytes);
    }
    ++st.seq;
  }
};

// The block for the next output of an Epi without inputs: the store before
// the last kSlots - 1 has been read out.
template <class Epi>
__device__ __forceinline__ uint8_t* tg_out_block(TgStage& st) {
  if (st.lane == 0) bulk_wait_read<Epi::kSlots - 1>();
  __syncwarp();
  return st.base + (st.seq++ % Epi::kSlots) * Epi::kSlotBytes;
}

// Accumulator values of this thread's row, 32 columns from column c of the
// tile: from TMEM, or the sum over the CTAs of a cluster.
struct TgTmemSrc {
  static constexpr bool kRegs = false;
  uint32_t addr;
  __device__ __forceinline__ void load(int c, uint32_t (&r)[32]) const {
    tmem_ld_32x32b_x32(addr + c, r);
    tmem_ld_wait();
  }
};

// A pair's sums of runs, in the epilogue's registers: 4 chunks of 32 columns of
// a thread's row.  Registers have no indexes, so the chunks come to the front
// one after another (unrolled instead, the epilogue is four times as much code
// to arrive on its first pass, which is longer than the two runs it may take).
struct TgRegSrc {
  static constexpr bool kRegs = true;
  float (&sum)[128];
};

// Calls f(k, r) for the part's chunks: r holds 32 columns from first + k * step.
template <class Src, class F>
__device__ __forceinline__ void tg_chunks(const TgPart& t, const Src& src, F&& f) {
  const int n = t.chunks();
#pragma unroll 1
  for (int k = 0; k < n; ++k) {
    uint32_t r[32];
    if constexpr (Src::kRegs) {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(src.sum[i]);
#pragma unroll
      for (int i = 0; i < 96; ++i) src.sum[i] = src.sum[i + 32];
    } else {
      src.load(t.first + k * t.step, r);
    }
    f(k, r);
  }
}

// The last run of a contraction and the sum of those before it (none: !more).
struct TgRunSrc {
  static constexpr bool kRegs = false;
  uint32_t addr, sum;
  bool more;
  __device__ __forceinline__ void load(int c, uint32_t (&r)[32]) const {
    TgTmemSrc{addr}.load(c, r);
    if (more) {
      uint32_t s[32];
      TgTmemSrc{sum}.load(c, s);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        r[i] = __float_as_uint(__fadd_rn(__uint_as_float(s[i]), __uint_as_float(r[i])));
    }
  }
  // Add this run to the sum: the columns of a part.
  __device__ __forceinline__ void add(const TgPart& t) const {
    const int n = t.any ? t.chunks() : 0;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      uint32_t r[32];
      load(t.first + k * t.step, r);
      tmem_st_32x32b_x32(sum + t.first + k * t.step, r);
    }
    tmem_st_wait();
  }
};

// Parts of a cluster's CTAs of one chunk, [SPLIT][32 columns][128 rows] fp32
// in this CTA's shared memory, added in rank order.
template <int SPLIT>
struct TgClusterSrc {
  const float* parts;  // of this thread's row
  __device__ __forceinline__ void load(int, uint32_t (&r)[32]) const {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float v = parts[i * 128];
#pragma unroll
      for (int s = 1; s < SPLIT; ++s) v = __fadd_rn(v, parts[s * 4096 + i * 128]);
      r[i] = __float_as_uint(v);
    }
  }
};

// Copy shared memory to another CTA of the cluster, counted on its barrier.
__device__ __forceinline__ void dsmem_copy(uint32_t dst_cluster, uint32_t src, uint32_t bytes,
                                           uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(dst_cluster),
      "r"(src), "r"(bytes), "r"(bar_cluster)
      : "memory");
}

// ------------------------------------------------------------------- kernel

// Epi: struct with Params, kAMn and kBMn (which operands are MN-major) and
// kBf16 (else fp16), kRun, kSlots, kSlotBytes, begin(...) (called before the
// accumulator is waited for), run(...), which takes the part's chunks, and
// abandon(...) for a part that was begun and is not run.
template <int CG, int BN, int SPLIT, class Epi>
__global__ void __launch_bounds__(kTgThreads, 1)
tc_gemm_kernel(const __grid_constant__ TgMaps maps, const TgShape p,
               const typename Epi::Params ep) {
  using C = TgCfg<CG, BN, Epi>;
  static_assert(SPLIT == 1 || (CG == 1 && BN == 128 &&
                               C::RING_BYTES >= 65536 + ((3 + SPLIT) / SPLIT) * SPLIT * 16384),
                "split");
  extern __shared__ uint8_t tg_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(tg_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + kTgMaxStages;
  uint64_t* accfull = empty + kTgMaxStages;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint64_t* parts_bar = drain + 1;
  uint64_t* epi_bars = parts_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int CLUSTER = CG * SPLIT;
  // Steps that the tensor cores sum before the epilogue warps add the run up;
  // 0: all of them.  On single SMs one accumulator holds the run, the other the
  // sum; a pair's runs alternate between the two and its sums are in registers.
  constexpr int RUN = SPLIT > 1 ? 0 : CG == 2 ? Epi::kPairRun : Epi::kRun;
  constexpr bool kRegs = CG == 2 && RUN > 0;
  constexpr bool kOneBuf = CG == 1 && RUN > 0;
  const uint32_t rank = CLUSTER > 1 ? cluster_rank() : 0u;
  const uint32_t half_rank = CG == 2 ? rank : 0u;  // which half of the pair's tile
  const uint64_t limit = p.wait_limit_ns;
  const int worker = static_cast<int>(blockIdx.x) / CLUSTER;
  const int workers = static_cast<int>(gridDim.x) / CLUSTER;
  // Pairs always take whole 256 x 256 tiles.
  const int a_rows = CG == 2 ? 128 : p.a_rows;
  const int b_rows = CG == 2 ? BN / 2 : p.bn;
  const uint32_t a_bytes = static_cast<uint32_t>(a_rows) * 128u;
  const uint32_t stage_bytes = static_cast<uint32_t>(a_rows + b_rows) * 128u;
  const uint32_t stages = CG == 2 ? C::PAIR_STAGES : static_cast<uint32_t>(p.stages);
  const uint32_t stage_tx = CG * stage_bytes;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], CG * kTgEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(parts_bar, 1);
    for (int i = 0; i < kTgEpiWarps * Epi::kSlots; ++i) mbar_init(&epi_bars[i], 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    if (p.passes == 3) {
      tma_prefetch_desc(&maps.a_lo);
      tma_prefetch_desc(&maps.b_lo);
    }
  }
  if (warp == 2) tg_tmem_alloc<CG>(tmem_slot, C::TMEM_COLS);
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CLUSTER > 1) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;

  // Contraction steps of a tile's slice that this CTA (or pair) takes.
  auto k_range = [&](int split, int& lo, int& hi) {
    const int slice = SPLIT > 1 ? static_cast<int>(rank) : split;
    lo = slice * p.split_steps;
    hi = min(p.steps, lo + p.split_steps);
  };
  auto part_of = [&](const TgTile& tile, int q, int half) {
    TgPart t;
    t.tile = tile;
    t.row0 = tile.m * 128 * CG + 128 * static_cast<int>(half_rank) + 32 * q;
    t.row = t.row0 + lane;
    t.col0 = tile.n * (CG == 2 ? BN : p.bn);
    t.col_end = min(p.N, t.col0 + (CG == 2 ? BN : p.bn));
    t.first = 32 * half;
    t.step = 64;
    t.dry = false;
    t.live = t.row < p.M;
    t.any = t.row0 < p.M;
    return t;
  };
  const int q = warp & 3, half = (warp - 4) >> 2;
  TgStage st;
  st.base = smem + C::OFF_EPI + (warp - 4) * Epi::kSlots * Epi::kSlotBytes;
  st.bars = epi_bars + (warp - 4) * Epi::kSlots;
  st.seq = 0;
  st.lane = lane;
  st.abort_flag = abort_flag;
  st.status = p.status;
  st.limit = limit;
  st.pre[0] = st.pre[1] = 0.0f;
  const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16);

  if (warp < 4) {
    if constexpr (kRegs) set_max_regs<kTgLightRegs, false>();
    if (warp == 0) {
      if (lane == 0) {
        uint32_t it = 0, s = 0, round = 0;  // stages issued, the ring's place
        bool ok = true;
        // The first tile's place is worked out before the launch before has
        // ended (its divisions take 1500 cycles with cold instructions).
        int t = worker;
        TgTile tile = tg_tile(p, t);
        int k_lo, k_hi;
        k_range(tile.split, k_lo, k_hi);
        pdl_wait_prior_grid();
        pdl_launch_dependents();
        while (true) {
          const int a0 = tile.m * 128 * CG + 128 * static_cast<int>(half_rank);
          const int b0 = tile.n * (CG * b_rows) + b_rows * static_cast<int>(half_rank);
          for (int pass = 0; pass < p.passes && ok; ++pass) {
            const CUtensorMap* ma = pass == 2 ? &maps.a_lo : &maps.a;
            const CUtensorMap* mb = pass == 1 ? &maps.b_lo : &maps.b;
            for (int j = k_lo; j < k_hi; ++j, ++it) {
              if (round > 0 && !mbar_wait_bounded(&empty[s], (round - 1) & 1u, abort_flag, limit)) {
                *abort_flag = 1;
                record_failure(p.status, DEV_TIMEOUT_PRODUCER);
                ok = false;
                break;
              }
              const uint32_t dst = smem_u32(smem) + s * stage_bytes;
              uint32_t bar = smem_u32(&full[s]);
              if (CG == 2) bar = map_to_rank(bar, 0);
              if (half_rank == 0) mbar_arrive_expect_tx(&full[s], stage_tx);
              const int k0 = (p.backwards ? k_hi - 1 - (j - k_lo) : j) * kTgKStep;
              tg_load<CG, Epi::kAMn>(ma, a_rows, dst, a0, k0, tile.b, bar);
              tg_load<CG, Epi::kBMn>(mb, b_rows, dst + a_bytes, b0, k0, tile.b, bar);
              if (++s == stages) {
                s = 0;
                ++round;
              }
            }
          }
          t += workers;
          if (t >= p.tiles || !ok) break;
          tile = tg_tile(p, t);
          k_range(tile.split, k_lo, k_hi);
        }
        // The last commits must have arrived before this CTA's barriers go away.
        const uint32_t from = it > stages ? it - stages : 0u;
        for (uint32_t i = from; i < it && ok; ++i)
          if (!mbar_wait_bounded(&empty[i % stages], (i / stages) & 1u, abort_flag, limit)) {
            *abort_flag = 1;
            record_failure(p.status, DEV_TIMEOUT_PRODUCER);
            ok = false;
          }
        // After a timeout, let the copies in flight land first (otherwise the
        // MMAs have consumed them all).
        if (*abort_flag && half_rank == 0)
          for (uint32_t i = from; i < it; ++i)
            if (!mbar_wait_bounded(&full[i % stages], (i / stages) & 1u, nullptr, limit))
              record_failure(p.status, DEV_TIMEOUT_DRAIN);
      }
    } else if (warp == 1) {
      if (half_rank == 0) {
        // This warp feeds the tensor cores of the pair, a step of 512 cycles:
        // whatever it need not compute per step is outside the loop or a constant
        // (operand layouts as run-time choices cost 8 % of the rate), and the
        // whole warp takes the loop, one lane of it issuing, so that addresses are
        // uniform values.  With one lane in the loop a run's end cost some 1000
        // cycles: 8192 tokens over 128000 x 4096 in runs of 16 steps 6.51 ms, so 6.01.
        const uint32_t a = smem_u32(smem);
        const uint64_t desc_a = Epi::kAMn ? umma_desc_sw128_mnmajor(a) : umma_desc_sw128_kmajor(a);
        const uint64_t desc_b = Epi::kBMn ? umma_desc_sw128_mnmajor(a + a_bytes)
                                          : umma_desc_sw128_kmajor(a + a_bytes);
        const uint32_t idesc =
            CG == 2 ? tg_idesc(256, BN, Epi::kBf16, Epi::kAMn, Epi::kBMn) : p.idesc;
        // (one answer for all lanes: they go on, or stop, together)
        auto there = [&](uint64_t* bar, uint32_t parity) {
          if (__all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, limit)))
            return true;
          *abort_flag = 1;
          if (lane == 0) record_failure(p.status, DEV_TIMEOUT_MMA);
          return false;
        };
        uint32_t s = 0, ph = 0;
        int local = 0;
        bool ok = true;
        for (int t = worker; t < p.tiles && ok; t += workers) {
          int k_lo, k_hi;
          k_range(p.ksplit > 1 ? t % p.ksplit : 0, k_lo, k_hi);
          const int n_it = (k_hi - k_lo) * p.passes;
          int j = 0;
          do {
            const int buf = kOneBuf ? 0 : local & 1;
            const int start = RUN > 0 ? j : 0, end = RUN > 0 ? min(n_it, j + RUN) : n_it;
            const bool used = local >= (kOneBuf ? 1 : 2);
            const uint32_t before = static_cast<uint32_t>(kOneBuf ? local - 1 : (local >> 1) - 1);
            ok = !used || there(&accempty[buf], before & 1u);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
            for (; j < end; ++j) {
              ok = there(&full[s], ph);
              if (!ok) break;
              tc_fence_after_sync();
              // (start addresses stay below 2^18: adding to the field is safe)
              const uint64_t at = s * (stage_bytes >> 4);
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTgKStep / 16; ++kk)
                  tg_mma<CG>(d, desc_a + at + (Epi::kAMn ? 128 : 2) * kk,
                             desc_b + at + (Epi::kBMn ? 128 : 2) * kk, idesc,
                             (kk > 0 || j > start) ? 1u : 0u);
                tg_commit<CG>(&empty[s]);
              }
              __syncwarp();
              if (++s == stages) {
                s = 0;
                ph ^= 1u;
              }
            }
            if (ok && elect_one()) tg_commit<CG>(&accfull[buf]);
            __syncwarp();
            ++local;
          } while (RUN > 0 && ok && j < n_it);
        }
        if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) {
          // The MMAs issued so far still read shared memory.
          if (elect_one()) tg_commit<CG>(drain);
          __syncwarp();
          if (!mbar_wait_bounded(drain, 0u, nullptr, limit) && lane == 0)
            record_failure(p.status, DEV_TIMEOUT_DRAIN);
        }
      }
    }
  } else {
    // This warp has read accumulator `buf`.
    auto release = [&](int buf) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(map_to_rank(smem_u32(&accempty[buf]), 0));
        else
          mbar_arrive(&accempty[buf]);
      }
    };
    // The next turn of accumulator `buf` has its sums.
    auto summed = [&](int buf, int turn) {
      return __all_sync(0xFFFFFFFFu,
                        mbar_wait_bounded(&accfull[buf], static_cast<uint32_t>(turn) & 1u,
                                          abort_flag, limit));
    };
    auto give_up = [&](const TgPart& part) {
      *abort_flag = 1;
      if (lane == 0) record_failure(p.status, DEV_TIMEOUT_EPILOGUE);
      if constexpr (SPLIT == 1) Epi::abandon(st, ep, part);
    };
    TgPart part = part_of(TgTile{0, 0, 0, 0}, q, half);
    part.dry = true;
    part.live = part.any = false;
    part.first = 0;
    part.col_end = min(part.col_end, 32);
    if constexpr (kRegs) {
      set_max_regs<kTgEpiRegs, true>();
      int local = 0;
      for (int t = worker; t < p.tiles;) {
        float sum[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) sum[i] = 0.0f;
        bool ok = true;
        if (!part.dry) {
          Epi::begin(st, maps, ep, p, part);
#pragma unroll 1
          for (int j = 0; j < p.steps; j += RUN, ++local) {
            const int buf = local & 1;
            ok = summed(buf, local >> 1);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t r[32];
              TgTmemSrc{lanes + static_cast<uint32_t>(buf * BN + 32 * half)}.load(64 * k, r);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                sum[32 * k + i] = __fadd_rn(sum[32 * k + i], __uint_as_float(r[i]));
            }
            release(buf);
          }
        }
        if (!ok) {
          give_up(part);
          break;
        }
        Epi::run(ep, p, maps, part, st, TgRegSrc{sum});
        const bool dry = part.dry;
        if (!dry) t += workers;
        if (t < p.tiles) part = part_of(tg_tile(p, t), q, half);
        if (dry) {
          st.seq = 0;
          pdl_wait_prior_grid();
        }
      }
    } else {
      if constexpr (SPLIT > 1)
        Epi::run(ep, p, maps, part, st, TgClusterSrc<SPLIT>{reinterpret_cast<const float*>(smem)});
      else if constexpr (kOneBuf)
        Epi::run(ep, p, maps, part, st, TgRunSrc{lanes, lanes + BN, false});
      else
        Epi::run(ep, p, maps, part, st, TgTmemSrc{lanes});
      st.seq = 0;
      part = part_of(tg_tile(p, worker), q, half);
      pdl_wait_prior_grid();
      int local = 0;
      for (int t = worker; t < p.tiles; ++local) {
        const int buf = kOneBuf ? 0 : local & 1;
        if constexpr (SPLIT == 1) Epi::begin(st, maps, ep, p, part);
        bool ok = true, more = false;
        if constexpr (kOneBuf) {
          for (int j = RUN; j < p.steps && ok; j += RUN) {  // all runs but the last
            ok = summed(0, local);
            if (!ok) break;
            tc_fence_after_sync();
            TgRunSrc{lanes, lanes + BN, more}.add(part);
            more = true;
            release(0);
            ++local;
          }
        }
        ok = ok && summed(buf, kOneBuf ? local : local >> 1);
        if (!ok) {
          give_up(part);
          break;
        }
        tc_fence_after_sync();
        const uint32_t acc = lanes + static_cast<uint32_t>(buf * BN);
        if constexpr (SPLIT == 1) {
          if constexpr (kOneBuf)
            Epi::run(ep, p, maps, part, st, TgRunSrc{acc, acc + BN, more});
          else
            Epi::run(ep, p, maps, part, st, TgTmemSrc{acc});
        } else {
          // This CTA's part, [column][row] fp32, over the ring (all consumed).
          float* part_sum = reinterpret_cast<float*>(smem);
#pragma unroll 1
          for (int c = 32 * half; c < BN; c += 64) {
            uint32_t r[32];
            TgTmemSrc{acc}.load(c, r);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              part_sum[(c + i) * 128 + 32 * q + lane] = __uint_as_float(r[i]);
          }
        }
        release(buf);
        t += workers;
        if (t < p.tiles) part = part_of(tg_tile(p, t), q, half);
      }
    }
  }
  __syncwarp();
  if constexpr (SPLIT > 1) {
    // One tile per cluster: CTA r finishes the chunks of 32 columns r and, if
    // there is one, r + SPLIT, one per half of its warps.  The ring's first 64
    // KiB hold this CTA's part, behind them it receives its chunks of every part.
    constexpr uint32_t kChunk = 16384;  // bytes: 32 columns, 128 rows
    const int mine = static_cast<int>(rank) + SPLIT < 4 ? 2 : 1;
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) mbar_arrive_expect_tx(parts_bar, mine * SPLIT * kChunk);
    cluster_sync();
    if (threadIdx.x == 0) {
      const uint32_t base = smem_u32(smem);
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c)
        dsmem_copy(map_to_rank(base + 65536u + ((c / SPLIT) * SPLIT + rank) * kChunk, c % SPLIT),
                   base + c * kChunk, kChunk, map_to_rank(smem_u32(parts_bar), c % SPLIT));
    }
    if (warp >= 4 && half < mine) {
      TgPart part = part_of(tg_tile(p, worker), q, half);
      part.first = 32 * (static_cast<int>(rank) + half * SPLIT);
      part.step = 1 << 20;
      const bool run = *abort_flag == 0;
      if (run) Epi::begin(st, maps, ep, p, part);
      const bool ok = __all_sync(0xFFFFFFFFu,
                                 mbar_wait_bounded(parts_bar, 0u, nullptr, limit));
      if (!ok && lane == 0) record_failure(p.status, DEV_TIMEOUT_EPILOGUE);
      if (run && ok)
        Epi::run(ep, p, maps, part, st,
                 TgClusterSrc<SPLIT>{reinterpret_cast<const float*>(smem) + 16384 +
                                     half * SPLIT * 4096 + 32 * q + lane});
      else if (run)
        Epi::abandon(st, ep, part);
    }
    __syncwarp();
  }
  if (warp >= 4 && lane == 0) bulk_wait_all();
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CLUSTER > 1) cluster_sync();
  if (warp == 2) {
    tc_fence_after_sync();
    tg_tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------ epilogue tools

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(a))) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(b))) << 16);
}

// Store a chunk's block and count it as one group of this warp.
__device__ __forceinline__ void tg_store_block(const TgStage& st, const CUtensorMap* map,
                                               const uint8_t* blk, int col, const TgPart& t) {
  if (st.lane == 0 && t.any) tma_store_3d(map, smem_u32(blk), col, t.row0, t.tile.b);
}

// D to bf16, times a device scalar when given.  Blocks of 32 x 64 (rows of 128
// bytes, 128-byte swizzle): a short contraction is all writing, and with rows
// of 64 bytes the copy engine took 5 % longer for it (dW of 64 tokens over
// 32000 x 2048 at 2.9 TB/s; a plain fill of that size reaches 3.5).
struct TgStoreBf16 {
  static constexpr bool kAMn = true, kBMn = true, kBf16 = true;
  static constexpr int kRun = 0, kPairRun = 0, kSlots = 2, kSlotBytes = 4096;
  struct Params {
    const float* scale;
  };
  static __device__ __forceinline__ void begin(TgStage&, const TgMaps&, const Params&,
                                               const TgShape&, const TgPart&) {}
  static __device__ __forceinline__ void abandon(TgStage&, const Params&, const TgPart&) {}
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape&, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const float f = e.scale && !t.dry ? __ldcg(e.scale) : 1.0f;
    // every other pair of chunks
#pragma unroll 1
    for (int c = 2 * t.first; t.col0 + c < t.col_end; c += 128) {
      uint8_t* blk = tg_out_block<TgStoreBf16>(st);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32], w[16];
        src.load(c + 32 * h, r);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[j] = pack_bf16x2(__uint_as_float(r[2 * j]) * f, __uint_as_float(r[2 * j + 1]) * f);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(blk + block32_piece(st.lane, 4 * h + j)) =
              make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      tg_store_block(st, &m.out, blk, t.col0 + c, t);
      if (st.lane == 0) bulk_commit();
    }
  }
};

// D (+ an fp32 tensor) to fp32, or times a device scalar to bf16; a slice of
// a split contraction goes to its own [M][N] of the output.
struct TgAccumulate {
  static constexpr bool kAMn = false, kBMn = true, kBf16 = true;
  static constexpr int kRun = 0, kPairRun = 0, kSlots = 3, kSlotBytes = 4096;
  struct Params {
    int add;             // add `in`
    int to_bf16;         // `out` is bf16 (else fp32)
    const float* scale;  // for bf16
  };
  using In = TgInput<TgAccumulate>;
  static __device__ __forceinline__ void begin(TgStage& st, const TgMaps& m, const Params& e,
                                               const TgShape&, const TgPart& t) {
    if (e.add)
      In::begin(st, m, t, false, 4096);
    else if (st.lane == 0)
      bulk_wait_read<0>();
    __syncwarp();
  }
  static __device__ __forceinline__ void abandon(TgStage& st, const Params& e, const TgPart& t) {
    if (e.add) In::abandon(st, t);
  }
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape&, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const float f = e.to_bf16 && !t.dry ? __ldcg(e.scale) : 1.0f;
    TgPart o = t;             // slices are the output's batch entries
    o.tile.b = t.tile.split;
    const int n = t.chunks();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int c = t.first + i * t.step;
      uint8_t* blk = st.base + (st.seq % kSlots) * kSlotBytes;
      if (e.add && !In::wait(st, t, i)) break;
      uint32_t r[32];
      src.load(c, r);
      if (e.add) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(blk + block32_piece(st.lane, j));
          r[4 * j] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * j]), v.x));
          r[4 * j + 1] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * j + 1]), v.y));
          r[4 * j + 2] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * j + 2]), v.z));
          r[4 * j + 3] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * j + 3]), v.w));
        }
      }
      if (e.to_bf16) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[j] = pack_bf16x2(__uint_as_float(r[2 * j]) * f, __uint_as_float(r[2 * j + 1]) * f);
        __syncwarp();  // the whole block was read
        block16_write(blk, st.lane, w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(blk + block32_piece(st.lane, j)) =
              make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      tg_store_block(st, &m.out, blk, t.col0 + c, o);
      if (st.lane == 0) {
        bulk_commit();
        if (!e.add) bulk_wait_read<2>();  // the next block's slot is free again
      }
      if (e.add) {
        In::next(st, m, t, i, false, 4096);
      } else {
        ++st.seq;
        __syncwarp();
      }
    }
  }
};

}  // namespace bitnet
