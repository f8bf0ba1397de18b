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

// X = U / (||U||_F + eps) times `scale`, as two halves, [n][ldx], from U
// [rows][cols] (transposed when `tall`), one 32 x 32 tile per block.
__global__ void __launch_bounds__(256)
ortho_start_kernel(const void* __restrict__ U, int u_bf16, int rows, int cols, int tall,
                   const double* __restrict__ part, int parts, float eps, float scale,
                   uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, int64_t ldx,
                   int64_t x_batch) {
  __shared__ double red[256];
  __shared__ float tile[32][33];
  const int b = blockIdx.z;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) s += part[static_cast<int64_t>(b) * parts + i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if (threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
    __syncthreads();
  }
  const double norm = sqrt(red[0]) + static_cast<double>(eps);
  const double inv = norm > 0.0 ? 1.0 / norm : 0.0;  // eps = 0 and U = 0: X = 0
  const int64_t base = static_cast<int64_t>(b) * rows * cols;
  const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  for (int i = ty; i < 32; i += 8) {
    const int r = r0 + i, c = c0 + tx;
    float v = 0.0f;
    if (r < rows && c < cols)
      v = static_cast<float>(ortho_load(U, u_bf16 != 0, base + static_cast<int64_t>(r) * cols + c) *
                             inv) *
          scale;
    tile[i][tx] = v;
  }
  __syncthreads();
  for (int i = ty; i < 32; i += 8) {
    const int r = tall ? c0 + i : r0 + i, c = tall ? r0 + tx : c0 + tx;
    if (r < (tall ? cols : rows) && c < (tall ? rows : cols)) {
      const int64_t o = b * x_batch + static_cast<int64_t>(r) * ldx + c;
      split_half(tall ? tile[tx][i] : tile[i][tx], hi[o], lo[o]);
    }
  }
}

// A symmetric product's tile: its rows, and for a tile below the diagonal the
// mirrored ones (lanes hold neighbouring rows, so a mirrored store of one
// column is 64 contiguous bytes).
__device__ __forceinline__ void ortho_store_sym(uint16_t* base, int64_t ld, int row, int col,
                                                const uint32_t (&w)[16], int n, int M,
                                                bool mirror) {
  if (row < M) {
    // ld is a multiple of 32: the chunk's last columns may be padding.
    store_row32_16(base + row * ld + col, w, true, 32);
    if (mirror) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n)
          base[static_cast<int64_t>(col + i) * ld + row] =
              static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

__device__ __forceinline__ void ortho_pack(const float (&v)[32], uint32_t (&hi)[16],
                                           uint32_t (&lo)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint16_t h0, l0, h1, l1;
    split_half(v[2 * i], h0, l0);
    split_half(v[2 * i + 1], h1, l1);
    hi[i] = h0 | (static_cast<uint32_t>(h1) << 16);
    lo[i] = l0 | (static_cast<uint32_t>(l1) << 16);
  }
}

// A = X X^T: its diagonal to D (fp32), the rest to R (fp16, and its low half
// where the products take it).
struct OrthoGram {
  struct Params {
    float* D;              // [batch][n]
    uint16_t *R, *R_lo;    // [batch][n][ld]; R_lo may be null
    int64_t ld, batch;     // row stride, batch stride (elements)
    float to_true, to_R;   // accumulator -> A, accumulator -> stored R
  };
  template <int COLS>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgPart& t) {
    const bool mirror = t.tile.m != t.tile.n;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      const int col = t.col0 + c;
      if (col >= p.N) break;  // the same for all of the warp
      uint32_t r[32];
      tmem_ld_32x32b_x32(t.tmem + c, r);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float z = __uint_as_float(r[i]);
        const bool diag = col + i == t.row;
        if (diag && t.row < p.M)
          e.D[static_cast<int64_t>(t.tile.b) * p.M + t.row] = z * e.to_true;
        v[i] = diag ? 0.0f : z * e.to_R;
      }
      uint32_t hi[16], lo[16];
      ortho_pack(v, hi, lo);
      const int n = min(32, p.N - col);
      ortho_store_sym(e.R + t.tile.b * e.batch, e.ld, t.row, col, hi, n, p.M, mirror);
      if (e.R_lo)
        ortho_store_sym(e.R_lo + t.tile.b * e.batch, e.ld, t.row, col, lo, n, p.M, mirror);
    }
  }
};

// R R, and from it Q (fp16) and a + E (fp32, the factor of X).
struct OrthoPoly {
  struct Params {
    const float* D;
    float* E;              // [batch][n]: a + b D + c (D^2 + (R R)_ii)
    const uint16_t *R, *R_lo;
    uint16_t *Q, *Q_lo;    // Q_lo may be null
    int64_t ld, batch;
    float a, b, c;
    float acc_true, r_true, to_Q;
  };
  template <int COLS>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgPart& t) {
    const bool mirror = t.tile.m != t.tile.n;
    const bool live = t.row < p.M;
    const float* D = e.D + static_cast<int64_t>(t.tile.b) * p.M;
    const float di = live ? D[t.row] : 0.0f;
    const int64_t base = t.tile.b * e.batch;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      const int col = t.col0 + c;
      if (col >= p.N) break;  // the same for all of the warp
      uint32_t rh[16], rl[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) rh[i] = rl[i] = 0u;
      if (live) {
        const uint4* s = reinterpret_cast<const uint4*>(e.R + base + t.row * e.ld + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = s[i];
          rh[4 * i] = w.x; rh[4 * i + 1] = w.y; rh[4 * i + 2] = w.z; rh[4 * i + 3] = w.w;
        }
        if (e.R_lo) {
          const uint4* sl = reinterpret_cast<const uint4*>(e.R_lo + base + t.row * e.ld + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w = sl[i];
            rl[4 * i] = w.x; rl[4 * i + 1] = w.y; rl[4 * i + 2] = w.z; rl[4 * i + 3] = w.w;
          }
        }
      }
      uint32_t r[32];
      tmem_ld_32x32b_x32(t.tmem + c, r);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint32_t sh = 16 * (i & 1);
        const float rr = __uint_as_float(r[i]) * e.acc_true;
        const float x = (half_bits_to_f32((rh[i >> 1] >> sh) & 0xFFFFu) +
                         half_bits_to_f32((rl[i >> 1] >> sh) & 0xFFFFu)) * e.r_true;
        const float dj = col + i < p.N ? __ldg(D + col + i) : 0.0f;
        const bool diag = col + i == t.row;
        const float q = __fmaf_rn(e.c, __fmaf_rn(di + dj, x, rr), e.b * x);
        if (diag && live)
          e.E[static_cast<int64_t>(t.tile.b) * p.M + t.row] =
              e.a + __fmaf_rn(e.c, __fmaf_rn(di, di, rr), e.b * di);
        v[i] = diag ? 0.0f : q * e.to_Q;
      }
      uint32_t hi[16], lo[16];
      ortho_pack(v, hi, lo);
      const int n = min(32, p.N - col);
      ortho_store_sym(e.Q + base, e.ld, t.row, col, hi, n, p.M, mirror);
      if (e.Q_lo) ortho_store_sym(e.Q_lo + base, e.ld, t.row, col, lo, n, p.M, mirror);
    }
  }
};

// X <- (a + E_i) X + Q X: the next X as two halves, or the result in bf16
// (transposed back for a tall update).
struct OrthoUpdate {
  struct Params {
    const float* E;
    const uint16_t *X, *X_lo;
    uint16_t *Y, *Y_lo;    // next X, or null for the last step
    int64_t ld, batch;     // of X and Y
    __nv_bfloat16* out;    // last step: [batch][n][k], or [batch][k][n] when tall
    int tall;
    float acc_true, x_true, to_Y;
  };
  template <int COLS>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgPart& t) {
    const bool live = t.row < p.M;
    const float ei = live ? e.E[static_cast<int64_t>(t.tile.b) * p.M + t.row] : 0.0f;
    const int64_t base = t.tile.b * e.batch;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      const int col = t.col0 + c;
      if (col >= p.N) break;  // the same for all of the warp
      uint32_t xh[16], xl[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) xh[i] = xl[i] = 0u;
      if (live) {
        const uint4* s = reinterpret_cast<const uint4*>(e.X + base + t.row * e.ld + col);
        const uint4* sl = reinterpret_cast<const uint4*>(e.X_lo + base + t.row * e.ld + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = s[i], u = sl[i];
          xh[4 * i] = w.x; xh[4 * i + 1] = w.y; xh[4 * i + 2] = w.z; xh[4 * i + 3] = w.w;
          xl[4 * i] = u.x; xl[4 * i + 1] = u.y; xl[4 * i + 2] = u.z; xl[4 * i + 3] = u.w;
        }
      }
      uint32_t r[32];
      tmem_ld_32x32b_x32(t.tmem + c, r);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint32_t sh = 16 * (i & 1);
        const float x = (half_bits_to_f32((xh[i >> 1] >> sh) & 0xFFFFu) +
                         half_bits_to_f32((xl[i >> 1] >> sh) & 0xFFFFu)) * e.x_true;
        v[i] = __fmaf_rn(ei, x, __uint_as_float(r[i]) * e.acc_true);
      }
      const int n = min(32, p.N - col);
      if (e.Y) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= e.to_Y;
        ortho_pack(v, hi, lo);
        if (live) {
          store_row32_16(e.Y + base + t.row * e.ld + col, hi, true, 32);
          store_row32_16(e.Y_lo + base + t.row * e.ld + col, lo, true, 32);
        }
      } else {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        uint16_t* out = reinterpret_cast<uint16_t*>(e.out) +
                        static_cast<int64_t>(t.tile.b) * p.M * p.N;
        if (live && !e.tall) {
          store_row32_16(out + static_cast<int64_t>(t.row) * p.N + col, w,
                         n == 32 && (p.N & 7) == 0, n);
        } else if (live) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < n)
              out[static_cast<int64_t>(col + i) * p.M + t.row] =
                  static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
      }
    }
  }
};

}  // namespace bitnet
