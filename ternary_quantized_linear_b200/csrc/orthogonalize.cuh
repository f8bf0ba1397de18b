// orthogonalize.cuh -- Newton-Schulz orthogonalisation of a weight update.
//
//   X = U / (||U||_F + eps), transposed when U is taller than wide, n <= k
//   steps times:  A = X X^T,  X <- a X + (b A + c A A) X
//
// Precision.  The products run on the tensor cores in fp16, and the map
// multiplies what it has not yet orthogonalised by up to a per step: noise
// that a rounding of X itself spreads over all directions grows with them
// (an update of rank one ends 75 % off with bf16 iterates, 10 % with fp16).
// So nothing that is added is rounded to 16 bits:
//   X is held as a high and a low fp16 half (22 bits), the products read the
//   high half, and a X is formed from both;
//   the diagonals of A and of b A + c A A, which are as large as all the rest
//   of their rows, stay apart in fp32: with A = D + R,
//     A A          = D D + D R + R D + R R
//     b A + c A A  = E + Q,  Q_ij = b R_ij + c ((D_i + D_j) R_ij + (R R)_ij),
//                            E_i  = b D_i + c (D_i^2 + (R R)_ii)
//     X           <- (a + E_i) X_ij + (Q X)_ij
//   and only the hollow matrices R and Q, which are small, are fp16 operands.
// What is left is below the rounding of the bf16 result.  Small matrices
// (n <= kOrthoSplitN) have little to average over; R, Q and X enter their
// products with both halves (three products of fp16 for one of 22 bits).
//
// fp16 has too little range for entries near 1 / n, so X, R and Q are stored
// times powers of two that the host takes from the largest singular value
// that each step can reach (D as R is, E as the factor from one stored X to the
// next).  The powers and the coefficients meet on the host, in fp64, so that
// iterates may shrink or grow as they like: what the kernels multiply by
// stays near 1.
#pragma once

#include "tc_gemm.cuh"

namespace bitnet {

constexpr int kOrthoNormThreads = 256;

// v as the sum of two fp16 values.
__device__ __forceinline__ void split_half(float v, uint16_t& hi, uint16_t& lo) {
  const __half h = __float2half_rn(v);
  hi = __half_as_ushort(h);
  lo = __half_as_ushort(__float2half_rn(v - __half2float(h)));
}

__device__ __forceinline__ float ortho_load(const void* U, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(U)[i])
              : static_cast<const float*>(U)[i];
}

// Eight entries of U from `at` on, the first `n` of them (0 beyond); vec: all
// eight, 16-byte aligned.
__device__ __forceinline__ void ortho_load8(const void* U, bool bf16, int64_t at, bool vec, int n,
                                            float (&v)[8]) {
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? ortho_load(U, bf16, at + j) : 0.0f;
  } else if (bf16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(U) + at));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32(ws[j] & 0xFFFFu);
      v[2 * j + 1] = bf16_bits_to_f32(ws[j] >> 16);
    }
  } else {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(U) + at);
    const float4 x = __ldg(src), y = __ldg(src + 1);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
}

__device__ __forceinline__ double ortho_squares(const float (&v)[8]) {
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += static_cast<double>(v[j]) * static_cast<double>(v[j]);
  return s;
}

// scale / norm as power * mantissa * power, each within fp32's range, so that
// updates far from 1 keep their digits; norm = 0 (eps = 0 and U = 0): 0.
struct OrthoFactor {
  float p1, man, p2;
  __device__ __forceinline__ float operator()(float v) const { return v * p1 * man * p2; }
};

__device__ __forceinline__ OrthoFactor ortho_factor(double norm, float scale) {
  int e = 0;
  const float man = norm > 0.0 ? static_cast<float>(frexp(1.0 / norm, &e)) : 0.0f;
  return OrthoFactor{exp2f(static_cast<float>(e / 2)), man,
                     exp2f(static_cast<float>(e - e / 2)) * scale};
}

// Sum of squares of one block's share of a matrix, in fp64 (the squares of
// fp32 values neither overflow nor vanish there), in a fixed order.  vec: the
// matrices' sizes are multiples of 8.
__global__ void __launch_bounds__(kOrthoNormThreads)
ortho_norm_kernel(const void* __restrict__ U, int u_bf16, int64_t size, int vec,
                  double* __restrict__ part) {
  __shared__ double red[kOrthoNormThreads / 32];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * size;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  double s = 0.0;
  const int64_t eights = (size + 7) >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kOrthoNormThreads;
  const int64_t me = blockIdx.x * static_cast<int64_t>(kOrthoNormThreads) + threadIdx.x;
#pragma unroll 4
  for (int64_t i = me; i < eights; i += step) {
    float v[8];
    ortho_load8(U, u_bf16 != 0, base + 8 * i, vec != 0,
                static_cast<int>(min(static_cast<int64_t>(8), size - 8 * i)), v);
    s += ortho_squares(v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < kOrthoNormThreads / 32; ++i) s += red[i];
    part[blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x] = s;
  }
}

// ||U||_F + eps of matrix b from the blocks' sums, in a fixed order; all 256
// threads of a block.
__device__ __forceinline__ double ortho_norm_of(const double* part, int parts, int b, float eps,
                                                double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256)
    s += __ldcg(part + static_cast<int64_t>(b) * parts + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
  return sqrt(s) + static_cast<double>(eps);
}

// X = U / (||U||_F + eps) times `scale`, as two halves, [n][ldx], from a wide
// U [n][k]: a block takes rows, a thread eight entries at a time (U's rows
// 16-byte aligned when `vec`; the last columns of a row may be padding of X).
__global__ void __launch_bounds__(256)
ortho_start_kernel(const void* __restrict__ U, int u_bf16, int64_t n, int64_t k, int vec,
                   const double* __restrict__ part, int parts, float eps, float scale,
                   uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, int64_t ldx) {
  __shared__ double red[8];
  const int b = blockIdx.y;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const OrthoFactor f = ortho_factor(ortho_norm_of(part, parts, b, eps, red), scale);
  for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
    const int64_t from = (static_cast<int64_t>(b) * n + r) * k;
    const int64_t to = (static_cast<int64_t>(b) * n + r) * ldx;
#pragma unroll 2
    for (int64_t c = 8 * threadIdx.x; c < k; c += 8 * 256) {
      float v[8];
      ortho_load8(U, u_bf16 != 0, from + c, vec != 0,
                  static_cast<int>(min(static_cast<int64_t>(8), k - c)), v);
      __align__(16) uint16_t h[8], l[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) split_half(f(v[j]), h[j], l[j]);
      *reinterpret_cast<uint4*>(hi + to + c) = *reinterpret_cast<const uint4*>(h);
      *reinterpret_cast<uint4*>(lo + to + c) = *reinterpret_cast<const uint4*>(l);
    }
  }
}

// The same, transposed, from a tall U [rows][cols]: 64 x 32 tiles through
// shared memory (64 rows of U become 64 neighbouring entries of X's rows).
__global__ void __launch_bounds__(256)
ortho_start_tall_kernel(const void* __restrict__ U, int u_bf16, int rows, int cols,
                        const double* __restrict__ part, int parts, float eps, float scale,
                        uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, int64_t ldx) {
  __shared__ double red[8];
  __shared__ float tile[32][65];
  const int b = blockIdx.z;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const OrthoFactor f = ortho_factor(ortho_norm_of(part, parts, b, eps, red), scale);
  const int64_t base = static_cast<int64_t>(b) * rows * cols;
  const int r0 = blockIdx.x * 64, c0 = blockIdx.y * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
#pragma unroll
  for (int i = ty; i < 64; i += 8) {
    const int r = r0 + i, c = c0 + tx;
    tile[tx][i] = r < rows && c < cols
                      ? ortho_load(U, u_bf16 != 0, base + static_cast<int64_t>(r) * cols + c)
                      : 0.0f;
  }
  __syncthreads();
#pragma unroll
  for (int i = ty; i < 32; i += 8) {
    const int c = c0 + i, r = r0 + 2 * tx;
    if (c < cols && r < rows) {  // rows past the last one are padding of X
      uint16_t h[2], l[2];
      split_half(f(tile[i][2 * tx]), h[0], l[0]);
      split_half(f(tile[i][2 * tx + 1]), h[1], l[1]);
      const int64_t o = (static_cast<int64_t>(b) * cols + c) * ldx + r;
      *reinterpret_cast<uint32_t*>(hi + o) = h[0] | (static_cast<uint32_t>(h[1]) << 16);
      *reinterpret_cast<uint32_t*>(lo + o) = l[0] | (static_cast<uint32_t>(l[1]) << 16);
    }
  }
}

// Transposed entries straight to memory: lanes hold neighbouring rows, so a
// store of one column is 64 contiguous bytes.
__device__ __forceinline__ void ortho_store_mirror(uint16_t* base, int64_t ld, int row, int col,
                                                   const uint32_t (&w)[16], int n) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < n)
      base[static_cast<int64_t>(col + i) * ld + row] =
          static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

// Entry `at` (0..31) of a chunk's accumulators, by selects.
__device__ __forceinline__ float chunk_pick(const uint32_t (&r)[32], int at) {
  uint32_t v = 0u;
#pragma unroll
  for (int i = 0; i < 32; ++i) v = i == at ? r[i] : v;
  return __uint_as_float(v);
}

__device__ __forceinline__ void ortho_pack(const float (&v)[32], uint32_t (&hi)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    hi[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ float2 half2_bits_to_f32(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// What v has beyond hi.
__device__ __forceinline__ void ortho_pack_rest(const float (&v)[32], const uint32_t (&hi)[16],
                                                uint32_t (&lo)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 f = half2_bits_to_f32(hi[i]);
    const __half2 h = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    lo[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// A block out by TMA, with the low halves behind it (low), or with its mirror
// image behind it (mirror, a tile below the diagonal of a symmetric product):
// element (r, j) of the chunk goes to piece r / 8 of row j there.
__device__ __forceinline__ void ortho_store(TgStage& st, const TgMaps& m, const TgPart& t,
                                            uint8_t* blk, int col, const float (&v)[32],
                                            bool low, bool mirror) {
  uint32_t w[16];
  ortho_pack(v, w);
  block16_write(blk, st.lane, w);
  if (low) {
    uint32_t lo[16];
    ortho_pack_rest(v, w, lo);
    block16_write(blk + 2048, st.lane, lo);
  } else if (mirror) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      *reinterpret_cast<uint16_t*>(blk + 2048 + j * 64 +
                                   (((st.lane >> 3) ^ ((j >> 1) & 3)) << 4) +
                                   (st.lane & 7) * 2) =
          static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (st.lane == 0 && t.any) {
    tma_store_3d(&m.out, smem_u32(blk), col, t.row0, t.tile.b);
    if (low)
      tma_store_3d(&m.out_lo, smem_u32(blk + 2048), col, t.row0, t.tile.b);
    else if (mirror)
      tma_store_3d(&m.out, smem_u32(blk + 2048), t.row0, col, t.tile.b);
  }
  if (st.lane == 0) bulk_commit();
}

// The factors of one step, between values as they are stored.
struct OrthoStep {
  float to_R;            // X X^T's accumulator -> R and D
  float kr, kb;          // R R's accumulator, and D R -> Q; R -> Q
  float ea, eb, ec;      // a + E from 1, D, and D^2 + (R R)_ii
  float ku;              // Q X's accumulator -> X
};

// A = X X^T: its diagonal to D (fp32), the rest to R (fp16, and its low half
// where the products take it).
struct OrthoGram {
  static constexpr bool kAMn = false, kBMn = false, kBf16 = false;
  static constexpr int kRun = 0, kPairRun = 0, kSlots = 2, kSlotBytes = 4096;
  struct Params {
    float* D;              // [batch][n]
    int low;               // R's low half too (then not symmetric tiles)
    OrthoStep f;
  };
  static __device__ __forceinline__ void begin(TgStage&, const TgMaps&, const Params&,
                                               const TgShape&, const TgPart&) {}
  static __device__ __forceinline__ void abandon(TgStage&, const Params&, const TgPart&) {}
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const bool mirror = p.sym && t.tile.m != t.tile.n;
    const int n = t.chunks();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int c = t.first + k * t.step, col = t.col0 + c;
      uint32_t r[32];
      src.load(c, r);
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * e.f.to_R;
      if (t.row0 < col + 32 && col < t.row0 + 32) {  // the diagonal passes this chunk
        const int at = t.row - col;
        const float d = chunk_pick(r, at);
        if (t.live && at >= 0 && at < 32)
          e.D[static_cast<int64_t>(t.tile.b) * p.M + t.row] = d * e.f.to_R;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i == at ? 0.0f : v[i];
      }
      ortho_store(st, m, t, tg_out_block<OrthoGram>(st), col, v, e.low != 0, mirror);
    }
  }
};

// R R, and from it Q (fp16) and a + E (fp32, the factor of X).
struct OrthoPoly {
  static constexpr bool kAMn = false, kBMn = false, kBf16 = false;
  static constexpr int kRun = 0, kPairRun = 0, kSlots = 3, kSlotBytes = 4096;
  struct Params {
    const float* D;
    float* E;              // [batch][n]: a + b D + c (D^2 + (R R)_ii)
    int low;               // R and Q with their low halves (then not symmetric tiles)
    OrthoStep f;
  };
  using In = TgInput<OrthoPoly>;
  // D of this thread's row, and of the lane's column of the first chunk.
  static __device__ __forceinline__ void begin(TgStage& st, const TgMaps& m, const Params& e,
                                               const TgShape& p, const TgPart& t) {
    In::begin(st, m, t, e.low != 0, 2048);
    const float* D = e.D + static_cast<int64_t>(t.tile.b) * p.M;
    st.pre[0] = t.live ? __ldcg(D + t.row) : 0.0f;
    const int col = t.col0 + t.first + st.lane;
    st.pre[1] = col < p.N ? __ldcg(D + col) : 0.0f;
  }
  static __device__ __forceinline__ void abandon(TgStage& st, const Params&, const TgPart& t) {
    In::abandon(st, t);
  }
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const bool mirror = p.sym && t.tile.m != t.tile.n, low = e.low != 0;
    const float* D = e.D + static_cast<int64_t>(t.tile.b) * p.M;
    const float di = st.pre[0];
    float dl_next = st.pre[1];
    // Q = c R R + (b + c (D_i + D_j)) R
    const float kr = e.f.kr, ki = __fmaf_rn(kr, di, e.f.kb);
    const int n = t.chunks();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int c = t.first + k * t.step, col = t.col0 + c;
      const float dl = dl_next;
      if (k + 1 < n && col + t.step + st.lane < p.N) dl_next = __ldcg(D + col + t.step + st.lane);
      uint8_t* blk = st.base + (st.seq % kSlots) * kSlotBytes;
      if (!In::wait(st, t, k)) break;
      uint32_t r[32], w[16];
      block16_read(blk, st.lane, w);
      float v[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = half2_bits_to_f32(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
      if (low) {
        block16_read(blk + 2048, st.lane, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f = half2_bits_to_f32(w[i]);
          v[2 * i] += f.x;
          v[2 * i + 1] += f.y;
        }
      }
      src.load(c, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float dj = __shfl_sync(0xFFFFFFFFu, dl, i);
        v[i] = __fmaf_rn(__fmaf_rn(kr, dj, ki), v[i], __uint_as_float(r[i]) * kr);
      }
      if (t.row0 < col + 32 && col < t.row0 + 32) {  // the diagonal passes this chunk
        const int at = t.row - col;
        const float rr = chunk_pick(r, at);
        if (t.live && at >= 0 && at < 32)
          e.E[static_cast<int64_t>(t.tile.b) * p.M + t.row] =
              e.f.ea + __fmaf_rn(e.f.ec, __fmaf_rn(di, di, rr), e.f.eb * di);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i == at ? 0.0f : v[i];
      }
      __syncwarp();  // the whole block was read
      ortho_store(st, m, t, blk, col, v, low, mirror);
      In::next(st, m, t, k, low, 2048);
    }
  }
};

// X <- (a + E_i) X + Q X: the next X as two halves, or the result in bf16
// (transposed back for a tall update).
struct OrthoUpdate {
  static constexpr bool kAMn = false, kBMn = true, kBf16 = false;
  static constexpr int kRun = 0, kPairRun = 0, kSlots = 3, kSlotBytes = 4096;
  struct Params {
    const float* E;
    __nv_bfloat16* out;    // last step: [batch][n][k], or [batch][k][n] when tall; else null
    int tall;
    int direct;            // store the result without `maps.out` (rows of odd length)
    float ku;              // accumulator -> the next X, or the result
  };
  using In = TgInput<OrthoUpdate>;
  static __device__ __forceinline__ void begin(TgStage& st, const TgMaps& m, const Params& e,
                                               const TgShape& p, const TgPart& t) {
    In::begin(st, m, t, true, 2048);
    st.pre[0] = t.live ? __ldcg(e.E + static_cast<int64_t>(t.tile.b) * p.M + t.row) : 0.0f;
  }
  static __device__ __forceinline__ void abandon(TgStage& st, const Params&, const TgPart& t) {
    In::abandon(st, t);
  }
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const float ei = st.pre[0], ku = e.ku;
    const int n = t.chunks();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int c = t.first + k * t.step, col = t.col0 + c;
      uint8_t* blk = st.base + (st.seq % kSlots) * kSlotBytes;
      if (!In::wait(st, t, k)) break;
      uint32_t r[32], w[16], l[16];
      float v[32];
      block16_read(blk, st.lane, w);
      block16_read(blk + 2048, st.lane, l);
      src.load(c, r);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 h = half2_bits_to_f32(w[i]), g = half2_bits_to_f32(l[i]);
        v[2 * i] = __fmaf_rn(ei, h.x, __fmaf_rn(ei, g.x, __uint_as_float(r[2 * i]) * ku));
        v[2 * i + 1] =
            __fmaf_rn(ei, h.y, __fmaf_rn(ei, g.y, __uint_as_float(r[2 * i + 1]) * ku));
      }
      __syncwarp();  // the whole block was read
      if (!e.out) {
        ortho_store(st, m, t, blk, col, v, true, false);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        uint16_t* out = reinterpret_cast<uint16_t*>(e.out) +
                        static_cast<int64_t>(t.tile.b) * p.M * p.N;
        const int cols = min(32, p.N - col);
        if (e.tall) {
          if (t.live) ortho_store_mirror(out, p.M, t.row, col, w, cols);
        } else if (e.direct) {
          if (t.live) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < cols)
                out[static_cast<int64_t>(t.row) * p.N + col + i] =
                    static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
          }
        } else {
          block16_write(blk, st.lane, w);
          fence_proxy_async_smem();
          __syncwarp();
          tg_store_block(st, &m.out, blk, col, t);
        }
        if (st.lane == 0) bulk_commit();
      }
      In::next(st, m, t, k, true, 2048);
    }
  }
};

// ------------------------------------------------- small updates in one launch

// n <= 128 and k <= 2048, or k <= 4096 for batches of up to kOsWideBatch: all
// steps in one launch, X, R and Q in shared memory.  As products of their own,
// seventeen launches, a 128 x 128 update takes 109 us, so 44.
//
// A cluster of `cluster` CTAs holds one matrix, each CTA `ks` columns of X
// (K-major for A = X X^T; the same bytes are the MN-major operand of Q X).
// Per step: each CTA's part of A goes to the CTAs that own its columns, which
// add the parts in rank order and copy their rows of R (columns, by symmetry:
// whole 128-byte rows) and D to all; every CTA forms Q for itself (128^3 is
// cheaper than an exchange) and updates its own columns.
// The products take both halves of their operands (three MMAs for one).
// Threads: 16 warps; warp w has TMEM lanes 32 (w % 4) .. +31, a row each, and
// the columns of group w / 4.  Thread 0 issues the MMAs.

constexpr int kOsThreads = 512;
constexpr int kOsMaxKs = 256;
constexpr int kOsMaxCluster = 16;

struct OsParams {
  const void* U;
  __nv_bfloat16* out;
  int u_bf16, n, k, tall, cluster, ks, steps;
  float eps, scale;              // of the first X
  int* status;
  uint64_t wait_limit_ns;
  OrthoStep step[32];
};

struct OsSmem {
  static constexpr int OFF_X = 0;                         // hi: ks / 64 blocks of 128 x 64
  static constexpr int OFF_X_LO = kOsMaxKs / 64 * 16384;
  static constexpr int OFF_R = 2 * OFF_X_LO;              // hi: 2 blocks; the parts before it
  static constexpr int OFF_R_LO = OFF_R + 32768;
  static constexpr int OFF_D = OFF_R + 65536;
  static constexpr int OFF_E = OFF_D + 512;
  static constexpr int OFF_RED = OFF_E + 512;             // 16 + 16 doubles
  static constexpr int OFF_BAR = OFF_RED + 256;           // MMAs, received rows
  static constexpr int SMEM_DYN = OFF_BAR + 32 + 1024;
  static_assert(SMEM_DYN <= 232448, "shared memory");
};

// Byte of element (row, col) in 128-byte swizzled blocks of 128 rows x 64.
__device__ __forceinline__ int os_at(int row, int col) {
  return (col >> 6) * 16384 + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

// MN-major descriptor of such blocks (64 columns of the block are the MN
// extent, its 128 rows the contraction): the next 64 columns 16384 bytes on.
__device__ __forceinline__ uint64_t os_desc_mn(uint32_t smem_addr) {
  uint64_t d = umma_desc_sw128_mnmajor(smem_addr);
  d &= ~(static_cast<uint64_t>(0x3FFF) << 16);
  return d | (static_cast<uint64_t>(16384u >> 4) << 16);
}

__device__ __forceinline__ void os_read16(const uint8_t* hi, const uint8_t* lo, int row, int col,
                                          float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 h = *reinterpret_cast<const uint4*>(hi + os_at(row, col + 8 * j));
    const uint4 l = *reinterpret_cast<const uint4*>(lo + os_at(row, col + 8 * j));
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = half2_bits_to_f32(hw[i]), b = half2_bits_to_f32(lw[i]);
      v[8 * j + 2 * i] = a.x + b.x;
      v[8 * j + 2 * i + 1] = a.y + b.y;
    }
  }
}

__device__ __forceinline__ void os_write16(uint8_t* hi, uint8_t* lo, int row, int col,
                                           const float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[8 * j + 2 * i], y = v[8 * j + 2 * i + 1];
      const __half2 p = __floats2half2_rn(x, y);
      h[i] = *reinterpret_cast<const uint32_t*>(&p);
      const float2 f = __half22float2(p);
      const __half2 q = __floats2half2_rn(x - f.x, y - f.y);
      l[i] = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint4*>(hi + os_at(row, col + 8 * j)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo + os_at(row, col + 8 * j)) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// r[at] as a float (0 outside), by selects.
__device__ __forceinline__ float os_pick(const uint32_t (&r)[16], int at) {
  uint32_t v = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) v = i == at ? r[i] : v;
  return __uint_as_float(v);
}

// All writes to shared memory (of this or another CTA) before, all operand
// reads after.
__device__ __forceinline__ void os_sync(bool cluster) {
  asm volatile("fence.proxy.async;" ::: "memory");
  tc_fence_before_sync();
  if (cluster)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
}

__global__ void __launch_bounds__(kOsThreads, 1)
ortho_small_kernel(const __grid_constant__ OsParams p) {
  using L = OsSmem;
  extern __shared__ uint8_t os_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(os_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *Xh = smem + L::OFF_X, *Xl = smem + L::OFF_X_LO;
  uint8_t *Rh = smem + L::OFF_R, *Rl = smem + L::OFF_R_LO;
  float* D = reinterpret_cast<float*>(smem + L::OFF_D);
  float* E = reinterpret_cast<float*>(smem + L::OFF_E);
  double* red = reinterpret_cast<double*>(smem + L::OFF_RED);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* got = bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + 20);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, grp = warp >> 2;
  const int row = 32 * q + lane;
  const bool many = p.cluster > 1;
  const uint32_t rank = many ? cluster_rank() : 0u;
  const int64_t b = blockIdx.x / p.cluster;
  const int c0 = static_cast<int>(rank) * p.ks;

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(got, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (many) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  // ||U||_F: fp64 squares, a fixed order inside the CTA, then rank order.
  const int64_t base = b * p.n * p.k;
  const int width = max(0, min(p.ks, p.k - c0));  // this CTA's columns of X
  auto u_at = [&](int r, int c) {                  // X's element (r, c0 + c) in U
    return p.tall ? base + static_cast<int64_t>(c0 + c) * p.n + r
                  : base + static_cast<int64_t>(r) * p.k + c0 + c;
  };
  // Threads take eight neighbours of U at a time: columns of a row of X, or
  // for a tall U rows of a column.
  const int fast = p.tall ? p.n : width;
  const int per = (fast + 7) >> 3;                 // eights in a line
  const int units = width > 0 ? per * (p.tall ? width : p.n) : 0;
  const bool vec = ((p.tall ? p.n : p.k) & 7) == 0;  // every eight is whole and aligned
  auto each = [&](auto&& use) {
#pragma unroll 2
    for (int u = tid; u < units; u += kOsThreads) {
      const int slow = u / per, f = (u - slow * per) * 8;
      const int r = p.tall ? f : slow, c = p.tall ? slow : f;
      const int64_t at = u_at(r, c);
      float v[8];
      ortho_load8(p.U, p.u_bf16 != 0, at, vec, fast - f, v);
      use(r, c, v);
    }
  };
  double s = 0.0;
  each([&](int, int, const float (&v)[8]) { s += ortho_squares(v); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) red[warp] = s;
  // X starts as zeros: rows past n and columns past k stay so.
  for (int i = tid; i < p.ks / 64 * 1024; i += kOsThreads) {
    reinterpret_cast<uint4*>(Xh)[i] = make_uint4(0u, 0u, 0u, 0u);
    reinterpret_cast<uint4*>(Xl)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (tid == 0) {
    s = 0.0;
    for (int i = 0; i < kOsThreads / 32; ++i) s += red[i];
    if (!many) {
      red[16] = s;
    } else {
      for (int i = 0; i < p.cluster; ++i)
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                         map_to_rank(smem_u32(red + 16 + rank), i)),
                     "d"(s)
                     : "memory");
    }
  }
  os_sync(many);
  s = 0.0;
  for (int i = 0; i < p.cluster; ++i) s += red[16 + i];
  const OrthoFactor factor = ortho_factor(sqrt(s) + static_cast<double>(p.eps), p.scale);
  each([&](int r, int c, const float (&v)[8]) {
    __align__(16) uint16_t h[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split_half(factor(v[j]), h[j], l[j]);
    if (!p.tall) {  // (columns past the last one get their zeros again)
      *reinterpret_cast<uint4*>(Xh + os_at(r, c)) = *reinterpret_cast<const uint4*>(h);
      *reinterpret_cast<uint4*>(Xl + os_at(r, c)) = *reinterpret_cast<const uint4*>(l);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        *reinterpret_cast<uint16_t*>(Xh + os_at(r + j, c)) = h[j];
        *reinterpret_cast<uint16_t*>(Xl + os_at(r + j, c)) = l[j];
      }
    }
  });
  os_sync(false);

  uint32_t phase = 0;
  auto wait_mma = [&]() {
    if (*abort_flag == 0 && !mbar_wait_bounded(bar, phase, abort_flag, p.wait_limit_ns)) {
      *abort_flag = 1;
      record_failure(p.status, DEV_TIMEOUT_MMA);
    }
    phase ^= 1u;
    __syncwarp();
    tc_fence_after_sync();
  };
  // D[tmem + col] = sum over the contraction of A B^T, hi hi + hi lo + lo hi;
  // A K-major at a_hi / a_lo, B K-major or MN-major.
  auto issue = [&](uint32_t col, const uint8_t* a_hi, const uint8_t* a_lo, const uint8_t* b_hi,
                   const uint8_t* b_lo, int k16, bool b_mn, uint32_t idesc) {
    for (int pass = 0; pass < 3; ++pass) {
      const uint32_t a = smem_u32(pass == 2 ? a_lo : a_hi), bb = smem_u32(pass == 1 ? b_lo : b_hi);
      for (int i = 0; i < k16; ++i) {
        const uint32_t off = (i >> 2) * 16384 + (i & 3) * 32;  // K-major: 16 columns on
        tg_mma<1>(tmem + col, umma_desc_sw128_kmajor(a + off),
                  b_mn ? os_desc_mn(bb + i * 2048) : umma_desc_sw128_kmajor(bb + off), idesc,
                  (pass > 0 || i > 0) ? 1u : 0u);
      }
    }
    tc_commit(bar);
  };
  constexpr uint32_t kGramCol = 0, kPolyCol = 128, kUpdCol = 256;
  const uint32_t sq_desc = tg_idesc(128, 128, false, false, false);
  const uint32_t upd_desc = tg_idesc(128, p.ks, false, false, true);

  for (int it = 0; it < p.steps; ++it) {
    const OrthoStep& c = p.step[it];
    // A = X X^T, this CTA's columns of X
    if (tid == 0) issue(kGramCol, Xh, Xl, Xh, Xl, p.ks / 16, false, sq_desc);
    wait_mma();
    if (!many) {
#pragma unroll 1
      for (int j = 32 * grp; j < 32 * grp + 32; j += 16) {
        uint32_t r[16];
        float v[16];
        tmem_ld_32x32b_x16(lanes + kGramCol + j, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]) * c.to_R;
        os_write16(Rh, Rl, row, j, v);
        const float d = os_pick(r, row - j);
        if (row >= j && row < j + 16) {  // the diagonal
          D[row] = d * c.to_R;
          *reinterpret_cast<uint16_t*>(Rh + os_at(row, row)) = 0;
          *reinterpret_cast<uint16_t*>(Rl + os_at(row, row)) = 0;
        }
      }
      os_sync(false);
    } else {
      // Part `rank` of columns [share * o, +share) to CTA o, four columns of a
      // row together: [rank][column / 4][row][4].
      const int share = 128 / p.cluster;
#pragma unroll 1
      for (int j = 32 * grp; j < 32 * grp + 32; j += 16) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(lanes + kGramCol + j, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = (j + 4 * i) / share, at = (j + 4 * i) % share;
          // (column / 4) * 128 rows * 16 bytes = column * 512: 128 * 4 bytes a column
          const uint32_t to = map_to_rank(
              smem_u32(Rh) + static_cast<uint32_t>(((static_cast<int>(rank) * share + at) * 32 +
                                                    row) * 16),
              static_cast<uint32_t>(o));
          asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to),
                       "r"(r[4 * i]), "r"(r[4 * i + 1]), "r"(r[4 * i + 2]), "r"(r[4 * i + 3])
                       : "memory");
        }
      }
      os_sync(true);
      // The sums of this CTA's columns, in rank order; thread (row, grp) has
      // share / 4 of them, or four (and the last groups none).
      const int each4 = max(4, share / 4), first = grp * each4;
      const int mine = first < share ? each4 : 0;
      const float4* parts = reinterpret_cast<const float4*>(Rh);
      float sum[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (4 * i < mine) {
          v = parts[((first >> 2) + i) * 128 + row];
          for (int o = 1; o < p.cluster; ++o) {
            const float4 w = parts[(((o * share + first) >> 2) + i) * 128 + row];
            v.x = __fadd_rn(v.x, w.x);
            v.y = __fadd_rn(v.y, w.y);
            v.z = __fadd_rn(v.z, w.z);
            v.w = __fadd_rn(v.w, w.w);
          }
        }
        sum[4 * i] = v.x;
        sum[4 * i + 1] = v.y;
        sum[4 * i + 2] = v.z;
        sum[4 * i + 3] = v.w;
      }
      // The rows that the other CTAs send: [share o, +share) of both blocks,
      // both halves, and of D.
      if (tid == 0)
        mbar_arrive_expect_tx(got, static_cast<uint32_t>((p.cluster - 1) * share * (4 * 128 + 4)));
      os_sync(true);  // the parts were read everywhere: R may take their place
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < mine) {
          const int col = static_cast<int>(rank) * share + first + i;
          uint16_t h, l;
          split_half(col == row ? 0.0f : sum[i] * c.to_R, h, l);
          // R is symmetric: (col, row), so that lanes are neighbours
          const int at = os_at(col, row);
          *reinterpret_cast<uint16_t*>(Rh + at) = h;
          *reinterpret_cast<uint16_t*>(Rl + at) = l;
          if (col == row) D[row] = sum[i] * c.to_R;
        }
      os_sync(false);
      if (tid < p.cluster && tid != static_cast<int>(rank)) {
        const uint32_t o = static_cast<uint32_t>(tid), there = map_to_rank(smem_u32(got), o);
        const uint32_t bytes = static_cast<uint32_t>(share) * 128u;
        const uint32_t at = smem_u32(Rh) + rank * bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // blocks 0, 1 of the high half, then of the low
          dsmem_copy(map_to_rank(at + i * 16384u, o), at + i * 16384u, bytes, there);
        const uint32_t d = smem_u32(D) + rank * static_cast<uint32_t>(share) * 4u;
        dsmem_copy(map_to_rank(d, o), d, static_cast<uint32_t>(share) * 4u, there);
      }
      if (*abort_flag == 0 && !mbar_wait_bounded(got, it & 1, abort_flag, p.wait_limit_ns)) {
        *abort_flag = 1;
        record_failure(p.status, DEV_TIMEOUT_EPILOGUE);
      }
      __syncwarp();
      os_sync(true);  // every copy has arrived: Q may take R's place
    }
    // R R, and Q and a + E in its place
    if (tid == 0) issue(kPolyCol, Rh, Rl, Rh, Rl, 8, false, sq_desc);
    const float di = D[row];
    const float kr = c.kr, ki = __fmaf_rn(kr, di, c.kb);
    wait_mma();
#pragma unroll 1
    for (int j = 32 * grp; j < 32 * grp + 32; j += 16) {
      uint32_t r[16];
      float v[16];
      tmem_ld_32x32b_x16(lanes + kPolyCol + j, r);
      os_read16(Rh, Rl, row, j, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 d4 = *reinterpret_cast<const float4*>(D + j + i);
        const float dj[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
        for (int h = 0; h < 4; ++h)  // Q = c R R + (b + c (D_i + D_j)) R
          v[i + h] = __fmaf_rn(__fmaf_rn(kr, dj[h], ki), v[i + h],
                               __uint_as_float(r[i + h]) * kr);
      }
      os_write16(Rh, Rl, row, j, v);
      const float rr = os_pick(r, row - j);
      if (row >= j && row < j + 16) {  // the diagonal
        E[row] = c.ea + __fmaf_rn(c.ec, __fmaf_rn(di, di, rr), c.eb * di);
        *reinterpret_cast<uint16_t*>(Rh + os_at(row, row)) = 0;
        *reinterpret_cast<uint16_t*>(Rl + os_at(row, row)) = 0;
      }
    }
    os_sync(false);
    // X <- E X + Q X
    if (tid == 0) issue(kUpdCol, Rh, Rl, Xh, Xl, 8, true, upd_desc);
    const bool last = it == p.steps - 1;
    const float ei = E[row], ku = c.ku;
    wait_mma();
    const int quarter = p.ks / 4;
#pragma unroll 1
    for (int j = quarter * grp; j < quarter * grp + quarter; j += 16) {
      uint32_t r[16];
      float v[16];
      tmem_ld_32x32b_x16(lanes + kUpdCol + j, r);
      os_read16(Xh, Xl, row, j, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = __fmaf_rn(ei, v[i], __uint_as_float(r[i]) * ku);
      if (!last) {
        os_write16(Xh, Xl, row, j, v);
      } else if (row < p.n) {
        if (!p.tall && (p.k & 7) == 0 && j + 16 <= width) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          uint4* o = reinterpret_cast<uint4*>(p.out + u_at(row, j));
          o[0] = make_uint4(w[0], w[1], w[2], w[3]);
          o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j + i < width) p.out[u_at(row, j + i)] = __float2bfloat16_rn(v[i]);
        }
      }
    }
    os_sync(many);  // Q was read everywhere: the next parts may take its place
  }
  if (many) cluster_sync();  // no CTA leaves while another may still reach it
  if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace bitnet
