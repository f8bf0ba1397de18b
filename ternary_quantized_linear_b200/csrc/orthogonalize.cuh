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
// that each step can reach.
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

__device__ __forceinline__ float half_bits_to_f32(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}

__device__ __forceinline__ float ortho_load(const void* U, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(U)[i])
              : static_cast<const float*>(U)[i];
}

// Sum of squares of one block's share of a matrix, in fp64 (the squares of
// fp32 values neither overflow nor vanish there), in a fixed order.
__global__ void __launch_bounds__(kOrthoNormThreads)
ortho_norm_kernel(const void* __restrict__ U, int u_bf16, int64_t size,
                  double* __restrict__ part) {
  __shared__ double red[kOrthoNormThreads];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * size;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  double s = 0.0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kOrthoNormThreads;
  const int64_t me = blockIdx.x * static_cast<int64_t>(kOrthoNormThreads) + threadIdx.x;
  for (int64_t i = me; i < size; i += step) {
    const double v = ortho_load(U, u_bf16 != 0, base + i);
    s += v * v;
  }
  red[threadIdx.x] = s;
  __syncthreads();
  for (int h = kOrthoNormThreads / 2; h > 0; h >>= 1) {
    if (threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x] = red[0];
}

// 1 / (||U||_F + eps) of matrix b from the blocks' sums, in a fixed order;
// all 256 threads of a block.
__device__ __forceinline__ double ortho_inverse_norm(const double* part, int parts, int b,
                                                     float eps, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256)
    s += __ldcg(part + static_cast<int64_t>(b) * parts + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
  const double norm = sqrt(s) + static_cast<double>(eps);
  return norm > 0.0 ? 1.0 / norm : 0.0;  // eps = 0 and U = 0: X = 0
}

// X = U / (||U||_F + eps) times `scale`, as two halves, [n][ldx], from a wide
// U [n][k]: eight elements per thread and round (U's rows 16-byte aligned when
// `vec`; the last columns of a row may be padding of X).
__global__ void __launch_bounds__(256)
ortho_start_kernel(const void* __restrict__ U, int u_bf16, int64_t n, int64_t k, int vec,
                   const double* __restrict__ part, int parts, float eps, float scale,
                   uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, int64_t ldx) {
  __shared__ double red[8];
  const int b = blockIdx.y;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const double inv = ortho_inverse_norm(part, parts, b, eps, red);
  const int64_t per_row = (k + 7) >> 3, total = n * per_row;
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += 256LL * gridDim.x) {
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    const int64_t at = (static_cast<int64_t>(b) * n + r) * k + c;
    float v[8];
    if (vec) {
      if (u_bf16) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(U) + at));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = bf16_bits_to_f32(ws[j] & 0xFFFFu);
          v[2 * j + 1] = bf16_bits_to_f32(ws[j] >> 16);
        }
      } else {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(U) + at);
        const float4 x = __ldg(s), y = __ldg(s + 1);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < k ? ortho_load(U, u_bf16 != 0, at + j) : 0.0f;
    }
    __align__(16) uint16_t h[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      split_half(static_cast<float>(v[j] * inv) * scale, h[j], l[j]);
    const int64_t o = (static_cast<int64_t>(b) * n + r) * ldx + c;
    *reinterpret_cast<uint4*>(hi + o) = *reinterpret_cast<const uint4*>(h);
    *reinterpret_cast<uint4*>(lo + o) = *reinterpret_cast<const uint4*>(l);
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
  const double inv = ortho_inverse_norm(part, parts, b, eps, red);
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
      split_half(static_cast<float>(tile[i][2 * tx] * inv) * scale, h[0], l[0]);
      split_half(static_cast<float>(tile[i][2 * tx + 1] * inv) * scale, h[1], l[1]);
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
                                            bool low, bool mirror, int rows) {
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
  if (st.lane == 0 && !t.dry) {
    tma_store_3d(&m.out, smem_u32(blk), col, t.row0, t.tile.b);
    if (low)
      tma_store_3d(&m.out_lo, smem_u32(blk + 2048), col, t.row0, t.tile.b);
    else if (mirror && t.row0 < rows)
      tma_store_3d(&m.out, smem_u32(blk + 2048), t.row0, col, t.tile.b);
  }
  if (st.lane == 0) bulk_commit();
}

// A = X X^T: its diagonal to D (fp32), the rest to R (fp16, and its low half
// where the products take it).
struct OrthoGram {
  static constexpr int kSlots = 2, kSlotBytes = 4096;
  struct Params {
    float* D;              // [batch][n]
    int low;               // R's low half too (then not symmetric tiles)
    float to_true, to_R;   // accumulator -> A, accumulator -> stored R
  };
  static __device__ __forceinline__ void begin(TgStage&, const TgMaps&, const Params&,
                                               const TgPart&) {}
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
      float v[32], d = 0.0f;
      const int at = t.row - col;  // the diagonal's place in the chunk
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float z = __uint_as_float(r[i]);
        if (i == at) d = z;
        v[i] = i == at ? 0.0f : z * e.to_R;
      }
      if (t.live && at >= 0 && at < 32)
        e.D[static_cast<int64_t>(t.tile.b) * p.M + t.row] = d * e.to_true;
      ortho_store(st, m, t, tg_out_block<OrthoGram>(st), col, v, e.low != 0, mirror, p.M);
    }
  }
};

// R R, and from it Q (fp16) and a + E (fp32, the factor of X).
struct OrthoPoly {
  static constexpr int kSlots = 3, kSlotBytes = 4096;
  struct Params {
    const float* D;
    float* E;              // [batch][n]: a + b D + c (D^2 + (R R)_ii)
    int low;               // R and Q with their low halves (then not symmetric tiles)
    float a, b, c;
    float acc_true, r_true, to_Q;
  };
  using In = TgInput<OrthoPoly>;
  static __device__ __forceinline__ void begin(TgStage& st, const TgMaps& m, const Params& e,
                                               const TgPart& t) {
    In::begin(st, m, t, e.low != 0, 2048);
  }
  static __device__ __forceinline__ void abandon(TgStage& st, const Params&, const TgPart& t) {
    In::abandon(st, t);
  }
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const bool mirror = p.sym && t.tile.m != t.tile.n, low = e.low != 0;
    const float* D = e.D + static_cast<int64_t>(t.tile.b) * p.M;
    const float di = t.live ? __ldcg(D + t.row) : 0.0f;
    const int n = t.chunks();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int c = t.first + k * t.step, col = t.col0 + c;
      const float dl = !t.dry && col + st.lane < p.N ? __ldcg(D + col + st.lane) : 0.0f;
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
      const int at = t.row - col;  // the diagonal's place in the chunk
      float rr_ii = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float rr = __uint_as_float(r[i]) * e.acc_true;
        const float x = v[i] * e.r_true;
        const float dj = __shfl_sync(0xFFFFFFFFu, dl, i);
        if (i == at) rr_ii = rr;
        v[i] = i == at ? 0.0f
                       : __fmaf_rn(e.c, __fmaf_rn(di + dj, x, rr), e.b * x) * e.to_Q;
      }
      if (t.live && at >= 0 && at < 32)
        e.E[static_cast<int64_t>(t.tile.b) * p.M + t.row] =
            e.a + __fmaf_rn(e.c, __fmaf_rn(di, di, rr_ii), e.b * di);
      __syncwarp();  // the whole block was read
      ortho_store(st, m, t, blk, col, v, low, mirror, p.M);
      In::next(st, m, t, k, low, 2048);
    }
  }
};

// X <- (a + E_i) X + Q X: the next X as two halves, or the result in bf16
// (transposed back for a tall update).
struct OrthoUpdate {
  static constexpr int kSlots = 3, kSlotBytes = 4096;
  struct Params {
    const float* E;
    __nv_bfloat16* out;    // last step: [batch][n][k], or [batch][k][n] when tall; else null
    int tall;
    int direct;            // store the result without `maps.out` (rows of odd length)
    float acc_true, x_true, to_Y;
  };
  using In = TgInput<OrthoUpdate>;
  static __device__ __forceinline__ void begin(TgStage& st, const TgMaps& m, const Params&,
                                               const TgPart& t) {
    In::begin(st, m, t, true, 2048);
  }
  static __device__ __forceinline__ void abandon(TgStage& st, const Params&, const TgPart& t) {
    In::abandon(st, t);
  }
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    const float ei =
        t.live ? __ldcg(e.E + static_cast<int64_t>(t.tile.b) * p.M + t.row) * e.x_true : 0.0f;
    const int n = t.chunks();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int c = t.first + k * t.step, col = t.col0 + c;
      uint8_t* blk = st.base + (st.seq % kSlots) * kSlotBytes;
      if (!In::wait(st, t, k)) break;
      uint32_t r[32], w[16];
      float v[32];
      block16_read(blk, st.lane, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = half2_bits_to_f32(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
      block16_read(blk + 2048, st.lane, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = half2_bits_to_f32(w[i]);
        v[2 * i] += f.x;
        v[2 * i + 1] += f.y;
      }
      src.load(c, r);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[i] = __fmaf_rn(ei, v[i], __uint_as_float(r[i]) * e.acc_true);
      __syncwarp();  // the whole block was read
      if (!e.out) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= e.to_Y;
        ortho_store(st, m, t, blk, col, v, true, false, p.M);
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

}  // namespace bitnet
