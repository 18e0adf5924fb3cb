// norm.cu -- RMS norm with the residual's addition and an 8-bit output.
//
//   r = bf16(x + res)                    (r = x without a residual; stored on request)
//   y = r / sqrt(mean(r^2) + eps) * (w + w_off)     in fp32, never rounded to bf16
//   q, s = the quantisation of y: 1 x group_k groups (INT8, FP8: s = amax / Q,
//   as the activation quantiser) or MXFP8 groups of 32 with an E8M0 scale.
// The norm is taken of the rounded r, which is what the next layer adds to, so
// the stored residual and the normalised row agree.  The codes come from the
// fp32 y: the bf16 rounding between a separate norm and quantiser is left out.
// The sum of squares is fp32 (a product of two bf16 is exact in it).
#include <algorithm>

#include "bq_common.cuh"
#include "layer_ops.h"

namespace bq {

namespace {

constexpr int kAnyThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// E8M0 exponent (unbiased) of a group from its amax, as bq_mx_quant_act.
__device__ __forceinline__ int mx_exponent(float amax) {
  const int ef = (int)((__float_as_uint(amax) >> 23) & 0xFFu);
  return ef == 0 ? -127 : max(-127, min(127, ef - 127 - 8));
}

// Byte of (row, group of 32) in the scale atoms (tensor-core layout of gemm_mx.cu).
__device__ __forceinline__ int64_t mx_sf_index(int64_t r, int64_t g, int64_t K) {
  return ((r / 128) * (K / 128) + g / 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) / 32) + g % 4;
}

// Any width, group, stride and alignment: a CTA per row, the row's r in shared
// memory as bf16 (exactly what res_out holds), a warp per group.
template <int DT>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(const NormArgs a) {
  extern __shared__ uint16_t row[];
  __shared__ float red[kAnyThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t groups = (a.K + a.group - 1) / a.group;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    float sum = 0.f;
    for (int64_t k = tid; k < a.K; k += kAnyThreads) {
      uint16_t b = a.x[m * a.ldx + k];
      if (a.res)
        b = float_to_bf16_bits(bf16_bits_to_float(b) + bf16_bits_to_float(a.res[m * a.ldr + k]));
      if (a.res_out) a.res_out[m * a.ldro + k] = b;
      row[k] = b;
      const float r = bf16_bits_to_float(b);
      sum = fmaf(r, r, sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kAnyThreads / 32; ++i) sum += red[i];
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)a.K) + a.eps));
    for (int64_t g = warp; g < groups; g += kAnyThreads / 32) {
      const int64_t k0 = g * a.group, k1 = min(k0 + a.group, a.K);
      float amax = 0.f;
      for (int64_t k = k0 + lane; k < k1; k += 32)
        amax = fmaxf(amax, fabsf(bf16_bits_to_float(row[k]) * rstd *
                                 (bf16_bits_to_float(a.w[k]) + a.w_off)));
      amax = warp_max(amax);
      float sc = 0.f, inv = 0.f;
      if (DT == kMxFp8) {
        const int se = mx_exponent(amax);
        inv = __uint_as_float((uint32_t)(127 - se) << 23);   // 2^-se, exact
        if (lane == 0) a.sf[mx_sf_index(m, g, a.K)] = (uint8_t)(se + 127);
      } else {
        sc = group_scale<DT>(amax);
        if (lane == 0) a.s[g * a.M + m] = sc;
      }
      for (int64_t k = k0 + lane; k < k1; k += 32) {
        const float y = bf16_bits_to_float(row[k]) * rstd *
                        (bf16_bits_to_float(a.w[k]) + a.w_off);
        if (DT == kMxFp8)
          a.q[m * a.ldq + k] = (uint8_t)(e4m3x2_code(y * inv, 0.f, 1.0f) & 0xFFu);
        else
          a.q[m * a.ldq + k] = one_code<DT>(y, sc);
        if (a.h) a.h[m * a.ldh + k] = float_to_bf16_bits(y);
      }
    }
    __syncthreads();
  }
}

template <int DT>
cudaError_t launch_any(const NormArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)a.K * 2;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        norm_any_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kNormMaxK * 2));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(a.M, 148 * 16));
  cfg.blockDim = dim3(kAnyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_any_kernel<DT>, a);
}

template <int DT>
cudaError_t launch_dt(const NormArgs& a, cudaStream_t st) {
  return launch_any<DT>(a, st);
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormArgs& a, cudaStream_t st) {
  if (a.M == 0 || a.K == 0) return cudaSuccess;
  if (a.dtype == kMxFp8) return launch_dt<kMxFp8>(a, st);
  if (a.dtype == kInt8) return launch_dt<kInt8>(a, st);
  return launch_dt<kFp8>(a, st);
}

}  // namespace bq
