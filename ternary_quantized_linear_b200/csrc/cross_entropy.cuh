// cross_entropy.cuh -- softmax cross entropy of an output head over its whole
// vocabulary, with its gradient, without keeping the logits.
//
//   z      = x W^T                       x [M][K], W [V][K] bf16, fp32 sums
//   lse_m  = log sum_v exp(z_mv)
//   loss_m = lse_m - z_m,t(m)            t(m) in [0, V); otherwise 0
//   g_mv   = dloss_m (exp(z_mv - lse_m) - [v = t(m)]), 0 where t(m) is not in [0, V)
//   dx = g W,  dW = g^T x
//
// Forward: one product whose epilogue keeps, per row and half of a tile's
// columns, the running maximum and the sum of exp(z - maximum) (fp32) of all
// but the target's logit; a second kernel joins them.  The logits never leave
// the SM.  The target's logit is a dot product of its own, in fp32 with
// rounded sums (the tensor cores truncate theirs, which at 4096 terms of one
// sign makes a logit 1e-5 of itself too small): with s the sum of exp(z_v - z_t) over the
// others, loss = log(1 + s) has no cancellation for a confident token, and
// the target's entry of the gradient is exp(z_t - lse) - 1 by expm1.  lse comes
// back in fp32, so that entry is good to half a unit of lse's last place, 1e-6
// for logits near 30: a token whose loss is no larger has no better gradient.
// Backward: the vocabulary is taken in pieces; the same product forms g of a
// piece (bf16, in the workspace) from the saved lse, and two more give dx
// (summed over the pieces in fp32) and the piece's rows of dW.
//
// g is rounded to bf16 because it is a tensor-core operand next to bf16 x and
// W (the MMA takes operands of one type, and fp16 cannot hold a weight's
// range); every sum over it is fp32.  What is rounded is g / max|dloss| (of the
// finite ones), the common factor being put back in fp32 at the end: for a
// mean every dloss is the same, and the entries of most tokens, near -1 from
// below, then round by half as much as at an arbitrary factor's place between
// powers of two.
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

// Logit of one row's target, by one warp: products of bf16 are exact in fp32,
// each lane sums its own 8-element pieces in order.
__device__ __forceinline__ float ce_target_dot(const __nv_bfloat16* __restrict__ x,
                                               const __nv_bfloat16* __restrict__ w, int64_t K,
                                               int lane) {
  float s = 0.0f;
  for (int64_t i = lane; i < (K >> 3); i += 32) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(x) + i);
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(w) + i);
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s = __fmaf_rn(bf16_bits_to_f32(av[j] & 0xFFFFu), bf16_bits_to_f32(bv[j] & 0xFFFFu), s);
      s = __fmaf_rn(bf16_bits_to_f32(av[j] >> 16), bf16_bits_to_f32(bv[j] >> 16), s);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// The statistics of a row over half a tile's columns, the target's left out.
// The tensor cores sum runs of 8 steps, 512 terms, on single SMs, and of 16 on
// pairs, where a run has to outlast half of the epilogue (8 there: 8192 tokens
// over 128000 x 4096 6.35 ms, 16: 6.01).  100 tokens over 2000 x 4096, all
// terms positive: lse off by 1.4e-5 instead of 4.4e-4, and one token's loss by
// 1e-7 of itself instead of 1e-6, in the same time (51 us over 32000 x 4096);
// 256 tokens over 40000 x 4096: 4.2e-5 instead of 4.2e-4.  The loss takes the
// target's logit from a sum of its own, so what the others lose stays in it.
// CeGrad forms its logits in runs as short (from the other end of the
// contraction: other roundings), since e^(z - lse) wants both off alike.
struct CeStats {
  static constexpr bool kAMn = false, kBMn = false, kBf16 = true;
  static constexpr int kRun = 8, kPairRun = 16, kSlots = 0, kSlotBytes = 0;
  struct Params {
    const int64_t* targets;
    float2* part;          // [2 nt][M]: maximum, sum of exp(z - maximum)
  };
  static __device__ __forceinline__ void begin(TgStage&, const TgMaps&, const Params&,
                                               const TgShape&, const TgPart&) {}
  static __device__ __forceinline__ void abandon(TgStage&, const Params&, const TgPart&) {}
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape& p, const TgMaps&,
                                             const TgPart& t, TgStage&, Src src) {
    const int64_t target = t.live ? __ldg(e.targets + t.row) : -1;
    float mx = -INFINITY, sum = 0.0f;
    tg_chunks(t, src, [&](int k, uint32_t (&r)[32]) {
      const int col = t.col0 + t.first + k * t.step;
      if (col + 32 > t.col_end) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i >= t.col_end) r[i] = 0xFF800000u;  // -inf: not this tile's
      }
      if (target >= col && target < t.col_end && target < col + 32) {
        const int at = static_cast<int>(target) - col;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i == at) r[i] = 0xFF800000u;
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
      if (m_new != -INFINITY) {
        sum = __fmaf_rn(sum, exp2_approx(__fmaf_rn(mx, kLog2e, -shift)),
                        (s4[0] + s4[1]) + (s4[2] + s4[3]));
        mx = m_new;
      } else {  // -inf and NaN only: no inf - inf, but NaN stays
        float nan = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (__uint_as_float(r[i]) != -INFINITY) nan = __uint_as_float(r[i]);
        sum += nan;
      }
    });
    if (t.live)
      e.part[(2 * static_cast<int64_t>(t.tile.n) + (t.first >> 5)) * p.M + t.row] =
          make_float2(mx, sum);
  }
};

// The statistics (maximum, sum) of two sets of entries as those of both.
__device__ __forceinline__ void ce_join(float& mx, float& sum, float pm, float ps) {
  const float m_new = fmaxf(mx, pm);
  if (m_new != -INFINITY) {
    sum = __fmaf_rn(sum, exp2_approx((mx - m_new) * kLog2e),
                    ps * exp2_approx((pm - m_new) * kLog2e));
    mx = m_new;
  } else {
    sum += ps;  // 0, or NaN
  }
}

// Loss and lse of a row from the statistics of all entries but the target's.
// A target at -inf has no weight in lse and a loss of inf; one at +inf gives
// inf - inf.
__device__ __forceinline__ void ce_finish(float mx, float sum, bool valid, float z, float* loss,
                                          float* lse) {
  if (!valid) {
    *loss = 0.0f;
    *lse = mx + logf(sum);
    return;
  }
  if (z == -INFINITY) {
    *lse = mx + logf(sum);
    *loss = *lse - z;
    return;
  }
  const float d = mx - z;  // loss = log(1 + sum exp(mx - z))
  float l;
  if (mx == -INFINITY && sum == 0.0f)
    l = z - z;  // no other entry with any weight (NaN for a non-finite z)
  else
    l = d <= 0.0f ? log1pf(sum * expf(d)) : d + logf(sum + expf(-d));
  *loss = z < INFINITY ? l : z - z;
  *lse = z + l;
}

// Joins the parts of each row.  kWide (many rows): 32 rows x 32 lanes of parts
// per block, neighbouring rows' parts being neighbours in memory; warp w also
// forms the target's logit of row w.  Else a block of 8 warps per row, its
// threads over the parts: one token's 286 parts were 9 dependent loads and 31
// dependent joins with the other cut (8 us; 4 with this one).  The target's
// logit depends on the inputs alone and is formed while the product runs.
template <bool kWide>
__global__ void __launch_bounds__(kWide ? 1024 : 256)
ce_join_kernel(const float2* __restrict__ part, int parts, const __nv_bfloat16* __restrict__ x,
               const __nv_bfloat16* __restrict__ W, const int64_t* __restrict__ targets,
               int64_t V, int64_t K, int M, float* __restrict__ loss, float* __restrict__ lse) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if constexpr (kWide) {
    __shared__ float smx[32][33], ssum[32][33], slogit[32];
    const int64_t m = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    {
      const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + w;
      const int64_t t = row < M ? targets[row] : -1;
      float z = 0.0f;
      if (t >= 0 && t < V) z = ce_target_dot(x + row * K, W + t * K, K, lane);
      if (lane == 0) slogit[w] = z;
    }
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    float mx = -INFINITY, sum = 0.0f;
    if (m < M)
#pragma unroll 4
      for (int i = w; i < parts; i += 32) {
        const float2 v = __ldcg(part + static_cast<int64_t>(i) * M + m);
        ce_join(mx, sum, v.x, v.y);
      }
    smx[w][lane] = mx;
    ssum[w][lane] = sum;
    __syncthreads();
    if (w == 0 && m < M) {
      for (int i = 1; i < 32; ++i) ce_join(mx, sum, smx[i][lane], ssum[i][lane]);
      const int64_t t = targets[m];
      ce_finish(mx, sum, t >= 0 && t < V, slogit[lane], loss + m, lse + m);
    }
  } else {
    __shared__ float smx[8], ssum[8];
    const int64_t m = blockIdx.x;
    const int64_t t = targets[m];
    const bool valid = t >= 0 && t < V;
    float z = 0.0f;
    if (w == 0 && valid) z = ce_target_dot(x + m * K, W + t * K, K, lane);
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    float mx = -INFINITY, sum = 0.0f;
    for (int i = threadIdx.x; i < parts; i += 256) {
      const float2 v = __ldcg(part + static_cast<int64_t>(i) * M + m);
      ce_join(mx, sum, v.x, v.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)  // the lower lane's first, as in the wide cut
      ce_join(mx, sum, __shfl_down_sync(0xFFFFFFFFu, mx, o),
              __shfl_down_sync(0xFFFFFFFFu, sum, o));
    if (lane == 0) {
      smx[w] = mx;
      ssum[w] = sum;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) ce_join(mx, sum, smx[i], ssum[i]);
      ce_finish(mx, sum, valid, z, loss + m, lse + m);
    }
  }
}

// Per row: the target's logit.  Block 0 also: max |dloss| over the rows that
// have a target and a finite one (1 where that is 0): an infinite dloss as the
// common factor would make every other row 0 times infinity.
__global__ void __launch_bounds__(256)
ce_target_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ W,
                 const int64_t* __restrict__ targets, const float* __restrict__ dloss, int64_t M,
                 int64_t V, int64_t K, float* __restrict__ logit, float* __restrict__ scale) {
  __shared__ float red[8];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + w;
  if (row < M) {
    const int64_t t = targets[row];
    if (t >= 0 && t < V) {
      const float z = ce_target_dot(x + row * K, W + t * K, K, lane);
      if (lane == 0) logit[row] = z;
    }
  }
  if (blockIdx.x != 0) return;
  float a = 0.0f;
  for (int64_t m = threadIdx.x; m < M; m += 256) {
    const int64_t t = targets[m];
    if (t >= 0 && t < V) {
      const float d = fabsf(dloss[m]);
      if (d < INFINITY) a = fmaxf(a, d);  // inf and NaN: their own rows carry them
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if (lane == 0) red[w] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) a = fmaxf(a, red[i]);
    *scale = a > 0.0f ? a : 1.0f;
  }
}

struct CeGrad {
  static constexpr bool kAMn = false, kBMn = false, kBf16 = true;
  static constexpr int kRun = CeStats::kRun, kPairRun = CeStats::kPairRun;
  static constexpr int kSlots = 2, kSlotBytes = 2048;
  struct Params {
    const int64_t* targets;
    const float* lse;
    const float* dloss;
    const float* logit;    // of the target
    const float* scale;    // max finite |dloss|: g is formed relative to it
    int64_t V;             // of the whole vocabulary
    int64_t v0;            // first column of this piece
  };
  static __device__ __forceinline__ void begin(TgStage&, const TgMaps&, const Params&,
                                               const TgShape&, const TgPart&) {}
  static __device__ __forceinline__ void abandon(TgStage&, const Params&, const TgPart&) {}
  template <class Src>
  static __device__ __forceinline__ void run(const Params& e, const TgShape&, const TgMaps& m,
                                             const TgPart& t, TgStage& st, Src src) {
    int64_t target = t.live ? __ldg(e.targets + t.row) : -1;
    const bool valid = target >= 0 && target < e.V;
    float d = 0.0f, shift = 0.0f, at_target = 0.0f;
    if (valid) {
      const float dl = __ldg(e.dloss + t.row), l = __ldg(e.lse + t.row);
      d = __fdiv_rn(dl, __ldcg(e.scale));
      shift = l * kLog2e;
      at_target = expm1f(__ldcg(e.logit + t.row) - l);
      target -= e.v0;
    }
    tg_chunks(t, src, [&](int k, uint32_t (&r)[32]) {
      const int col = t.col0 + t.first + k * t.step;
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        r[i] = __float_as_uint(
            exp2_approx(__fmaf_rn(__uint_as_float(r[i]), kLog2e, -shift)));
      if (valid && target >= col && target < col + 32) {
        const int at = static_cast<int>(target) - col;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i == at) r[i] = __float_as_uint(at_target);
      }
      // A row without a target has no gradient, whatever its logits hold.
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = valid ? pack_bf16x2(__uint_as_float(r[2 * i]) * d, __uint_as_float(r[2 * i + 1]) * d)
                     : 0u;
      uint8_t* blk = tg_out_block<CeGrad>(st);
      block16_write(blk, st.lane, w);
      fence_proxy_async_smem();
      __syncwarp();
      tg_store_block(st, &m.out, blk, col, t);
      if (st.lane == 0) bulk_commit();
    });
  }
};

// The same on pairs whose contraction is one run: straight from TMEM (1024
// tokens over 32000 x 512: the statistics 34 us, 40 through registers).
template <class Epi>
struct CeWhole : Epi {
  static constexpr int kPairRun = 0;
};

// dx of a split contraction: add + the slices in order, in fp32, or times
// `scale` in bf16; 4 per thread.
__global__ void __launch_bounds__(256)
ce_join_dx_kernel(const float* __restrict__ part, int slices, int64_t stride,
                  const float* __restrict__ add, int64_t n4, float* __restrict__ f32,
                  const float* __restrict__ scale, __nv_bfloat16* __restrict__ out) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const float f = __ldcg(scale);
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n4;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float4 s = add ? __ldcg(reinterpret_cast<const float4*>(add) + i)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < slices; ++k) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part + k * stride) + i);
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
