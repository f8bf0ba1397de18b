// cross_entropy.cuh -- softmax cross entropy of an output head over its whole
// vocabulary, with its gradient, without keeping the logits.
//
//   z      = x W^T                       x [M][K], W [V][K] bf16, fp32 sums
//   lse_m  = log sum_v exp(z_mv)
//   loss_m = lse_m - z_m,t(m)            t(m) in [0, V); otherwise 0
//   g_mv   = dloss_m (exp(z_mv - lse_m) - [v = t(m)]), 0 where t(m) is not in [0, V)
//   dx = g W,  dW = g^T x
//
// Forward: one product whose epilogue keeps, per row and column half of a
// tile, the running maximum and the sum of exp(z - maximum) (fp32), and the
// target's logit; a second kernel joins them.  The logits never leave the SM.
// Backward: the vocabulary is taken in pieces; the same product forms g of a
// piece (bf16, in the workspace) from the saved lse, and two more give dx
// (summed over the pieces in fp32) and the piece's rows of dW.
//
// g is rounded to bf16 because it is a tensor-core operand next to bf16 x and
// W (the MMA takes operands of one type, and fp16 cannot hold a weight's
// range); every sum over it is fp32.  What is rounded is g / max|dloss|, the
// common factor being put back in fp32 at the end: for a mean every dloss is
// the same, and the entries of most tokens, near -1 from below, then round by
// half as much as at an arbitrary factor's place between powers of two.
#pragma once

#include "tc_gemm.cuh"

namespace bitnet {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x on the special-function unit (2 ulp; results below 2^-126 are 0, which
// a sum of probabilities cannot see).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct CeStats {
  struct Params {
    const int64_t* targets;
    float2* part;          // [2 nt][M]: maximum, sum of exp(z - maximum)
    float* target_logit;   // [M], written for valid targets only
  };
  template <int COLS>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgPart& t) {
    const bool live = t.row < p.M;
    const int64_t target = live ? __ldg(e.targets + t.row) : -1;
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      const int col = t.col0 + c;
      if (col >= p.N) break;  // the same for all of the warp
      uint32_t r[32];
      tmem_ld_32x32b_x32(t.tmem + c, r);
      tmem_ld_wait();
      if (col + 32 > p.N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i >= p.N) r[i] = 0xFF800000u;  // -inf: past the vocabulary
      }
      float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(r[i]));
      const float m_new = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      const float shift = m_new * kLog2e;
      float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 32; ++i)
        s4[i & 3] += exp2_approx(__fmaf_rn(__uint_as_float(r[i]), kLog2e, -shift));
      // A row of -inf so far: nothing to sum, and no inf - inf.
      if (m_new != -INFINITY) {
        sum = __fmaf_rn(sum, exp2_approx(__fmaf_rn(mx, kLog2e, -shift)),
                        (s4[0] + s4[1]) + (s4[2] + s4[3]));
        mx = m_new;
      }
      if (target >= col && target < col + 32 && target < p.N) {
        const int at = static_cast<int>(target) - col;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i == at) z = __uint_as_float(r[i]);
        e.target_logit[t.row] = z;
      }
    }
    if (live)
      e.part[(2 * static_cast<int64_t>(t.tile.n) + t.half) * p.M + t.row] = make_float2(mx, sum);
  }
};

// Joins the parts of each row: 32 rows x 32 lanes of parts per block (parts
// of neighbouring rows are neighbours in memory).
__global__ void __launch_bounds__(1024)
ce_join_kernel(const float2* __restrict__ part, int parts, const float* __restrict__ target_logit,
               const int64_t* __restrict__ targets, int64_t V, int M, float* __restrict__ loss,
               float* __restrict__ lse) {
  __shared__ float smx[32][33], ssum[32][33];
  const int r = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 32 + r;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  float mx = -INFINITY, sum = 0.0f;
  auto join = [&](float pm, float ps) {
    const float m_new = fmaxf(mx, pm);
    if (m_new != -INFINITY) {
      sum = __fmaf_rn(sum, exp2_approx((mx - m_new) * kLog2e),
                      ps * exp2_approx((pm - m_new) * kLog2e));
      mx = m_new;
    }
  };
  if (m < M)
    for (int i = w; i < parts; i += 32) {
      const float2 v = part[static_cast<int64_t>(i) * M + m];
      join(v.x, v.y);
    }
  smx[w][r] = mx;
  ssum[w][r] = sum;
  __syncthreads();
  if (w == 0 && m < M) {
    for (int i = 1; i < 32; ++i) join(smx[i][r], ssum[i][r]);
    const float l = mx + logf(sum);
    lse[m] = l;
    const int64_t t = targets[m];
    loss[m] = (t >= 0 && t < V) ? l - target_logit[m] : 0.0f;
  }
}

// scale = max |dloss| over the tokens that have a target; one block.
__global__ void __launch_bounds__(1024)
ce_scale_kernel(const float* __restrict__ dloss, const int64_t* __restrict__ targets, int64_t V,
                int64_t M, float* __restrict__ scale) {
  __shared__ float red[32];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  float a = 0.0f;
  for (int64_t m = threadIdx.x; m < M; m += 1024) {
    const int64_t t = targets[m];
    if (t >= 0 && t < V) a = fmaxf(a, fabsf(dloss[m]));  // NaN: its own row carries it
  }
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    a = red[threadIdx.x];
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    if (threadIdx.x == 0) *scale = a;
  }
}

struct CeGrad {
  struct Params {
    const int64_t* targets;
    const float* lse;
    const float* dloss;
    const float* scale;    // max |dloss|: g is formed relative to it
    int64_t V;             // of the whole vocabulary
    int64_t v0;            // first column of this piece
    __nv_bfloat16* g;      // [M][ld], ld a multiple of 32 and >= the piece
    int64_t ld;
  };
  template <int COLS>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgPart& t) {
    const bool live = t.row < p.M;
    int64_t target = live ? __ldg(e.targets + t.row) : -1;
    const bool valid = target >= 0 && target < e.V;
    const float top = __ldg(e.scale);
    const float dl = valid ? __ldg(e.dloss + t.row) : 0.0f;
    const float d = dl == 0.0f ? 0.0f : __fdiv_rn(dl, top);
    const float shift = valid ? __ldg(e.lse + t.row) * kLog2e : 0.0f;
    target = valid ? target - e.v0 : -1;
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      const int col = t.col0 + c;
      if (col >= p.N) break;  // the same for all of the warp
      uint32_t r[32];
      tmem_ld_32x32b_x32(t.tmem + c, r);
      tmem_ld_wait();
      const bool here = target >= col && target < col + 32;
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        r[i] = __float_as_uint(
            exp2_approx(__fmaf_rn(__uint_as_float(r[i]), kLog2e, -shift)));
      if (here) {
        const int at = static_cast<int>(target) - col;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i == at) r[i] = __float_as_uint(__fadd_rn(__uint_as_float(r[i]), -1.0f));
      }
      // A row without a target has no gradient, whatever its logits hold.
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = valid ? pack_bf16x2(__uint_as_float(r[2 * i]) * d, __uint_as_float(r[2 * i + 1]) * d)
                     : 0u;
      if (live)
        store_row32_16(reinterpret_cast<uint16_t*>(e.g) + t.row * e.ld + col, w, true, 32);
    }
  }
};

// dx of a split contraction: add + the slices in order, in fp32, or times
// `scale` in bf16; 4 per thread.
__global__ void __launch_bounds__(256)
ce_join_dx_kernel(const float* __restrict__ part, int slices, int64_t stride,
                  const float* __restrict__ add, int64_t n4, float* __restrict__ f32,
                  const float* __restrict__ scale, __nv_bfloat16* __restrict__ out) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const float f = *scale;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n4;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float4 s = add ? reinterpret_cast<const float4*>(add)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < slices; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(part + k * stride + 4 * i);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    if (out)
      reinterpret_cast<uint2*>(out)[i] = 
          make_uint2(pack_bf16x2(s.x * f, s.y * f), pack_bf16x2(s.z * f, s.w * f));
    else
      reinterpret_cast<float4*>(f32)[i] = s;
  }
}

}  // namespace bitnet
