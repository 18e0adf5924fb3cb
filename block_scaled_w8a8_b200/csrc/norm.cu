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
// INT8, FP8: a group with a y that is not a number has a scale that is not one.  MXFP8:
// the codes are e4m3's NaN, and the scale is that of the other values.
#include <algorithm>

#include "bq_common.cuh"
#include "layer_ops.h"
#include "sm100.cuh"

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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 in one register pair, for the instructions that take two.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t both(uint32_t bf16x2) {
  return pair(bf16x2 << 16, bf16x2 & 0xFFFF0000u);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// t = r (w + w_off) of eight elements, r and w as packed bf16: exact in fp32 for
// w_off = 0.
__device__ __forceinline__ void weighted(const uint4& r, const uint4& w, float w_off,
                                         float (&t)[8]) {
  const uint32_t rr[4] = {r.x, r.y, r.z, r.w}, ww[4] = {w.x, w.y, w.z, w.w};
  const uint64_t off = pair(__float_as_uint(w_off), __float_as_uint(w_off));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t x = mul2(both(rr[e]), sm100::add2(both(ww[e]), off));
    t[2 * e] = __uint_as_float((uint32_t)x);
    t[2 * e + 1] = __uint_as_float((uint32_t)(x >> 32));
  }
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a / b from r = 1 / b, correctly rounded: the quotient's remainder is exact in one FMA,
// and the quotient corrected by it is the correctly rounded one (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990; checked for every mantissa of a with b = 127 and 448).  For operands far from
// the ends of fp32.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

// 1 / sqrt(x): a Newton step on the approximation, its residual 1 - x r^2 with the
// rounding of x r put back.
__device__ __forceinline__ float inv_sqrt(float x) {
  if (!(x >= 0x1p-100f && x <= 0x1p100f)) return __fdiv_rn(1.0f, __fsqrt_rn(x));
  const float r = rsqrtf(x), h = x * r;
  const float e = fmaf(-fmaf(x, r, -h), r, fmaf(-h, r, 1.0f));
  return fmaf(0.5f * r, e, r);
}

// The running largest magnitude of a group, as the type's scale wants it.
template <int DT>
__device__ __forceinline__ float largest(float amax, float v) {
  return DT == kMxFp8 ? fmaxf(amax, fabsf(v)) : max_nan(amax, fabsf(v));
}

__device__ __forceinline__ uint32_t e4m3x4(const float* y, float inv) {
  unsigned short lo, hi;     // the first source operand lands in the upper byte
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1] * inv), "f"(y[0] * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3] * inv), "f"(y[2] * inv));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Q / max |t| in two parts.  t f is then correctly rounded, so that a quotient that lies
// in the middle between two codes is exactly there and goes to the even one; with one
// part all such values of a group went the way of its rounding.  (4096 x 4096 to
// INT8: 23.2 us with one part, 23.7 with two.)
struct Factor {
  float hi, lo;
};

__device__ __forceinline__ float times(float t, const Factor& f) {
  return fmaf(t, f.hi, __fmul_rn(t, f.lo));
}

__device__ __forceinline__ uint64_t times2(const float* t, const Factor& f) {
  const uint64_t x = pair(__float_as_uint(t[0]), __float_as_uint(t[1]));
  return sm100::fma2(x, pair(__float_as_uint(f.hi), __float_as_uint(f.hi)),
                     mul2(x, pair(__float_as_uint(f.lo), __float_as_uint(f.lo))));
}

// Four codes of t f, |t f| <= Q: round to nearest even.  INT8: the sum with 1.5 * 2^23
// leaves the code in the low byte, with no conversion unit involved.
__device__ __forceinline__ uint32_t int8x4(const float* t, const Factor& f) {
  constexpr uint32_t kMagic = 0x4B400000u;
  const uint64_t a = sm100::add2(times2(t, f), pair(kMagic, kMagic));
  const uint64_t b = sm100::add2(times2(t + 2, f), pair(kMagic, kMagic));
  return __byte_perm(__byte_perm((uint32_t)a, (uint32_t)(a >> 32), 0x0040),
                     __byte_perm((uint32_t)b, (uint32_t)(b >> 32), 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t e4m3x4(const float* t, const Factor& f) {
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const uint64_t x = times2(t + e, f);
    q[e] = __uint_as_float((uint32_t)x);
    q[e + 1] = __uint_as_float((uint32_t)(x >> 32));
  }
  return e4m3x4(q, 1.0f);
}

// Scale of an INT8 or FP8 group and the factor of its codes from amax = max |t|, where
// y = t rstd and t = r (w + w_off): rstd falls out of y / s, so the codes are those of
// t Q / max |t|, and the scale is max |t| rstd / Q.  Both kernels go by it, so that codes
// do not depend on the order of a row's sum, nor on strides and alignment.  False where
// the factor may not be a number; the codes are then those of y / s, divided.
template <int DT>
__device__ __forceinline__ bool group_factor(float amax, float rstd, float& sc, Factor& f) {
  constexpr float kQ = DT == kInt8 ? 127.0f : 448.0f;
  const float top = amax * rstd;
  // a NaN fails, which may be in either
  if (amax >= 0x1p-100f && top >= 0x1p-100f && amax <= 0x1p100f && top <= 0x1p100f) {
    sc = quotient(top, kQ, 1.0f / kQ);
    const float r = rcp(amax);
    // kQ r is off by at most 3 units in the last place (r by one); from below, so that
    // the rest is positive and a zero keeps its sign
    f.hi = __uint_as_float(__float_as_uint(kQ * r) - 4);
    f.lo = fmaf(-f.hi, amax, kQ) * r;
    return true;
  }
  sc = group_scale<DT>(top);
  return false;
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
        amax = largest<DT>(amax, bf16_bits_to_float(row[k]) *
                                     (bf16_bits_to_float(a.w[k]) + a.w_off));
      amax = warp_max_nan(amax);                                   // of t, y = t rstd
      float sc = 0.f, inv = 0.f;
      Factor f{};
      bool fast = false;
      if (DT == kMxFp8) {
        const int se = mx_exponent(fmaxf(amax * rstd, 0.f));       // 0 for a row that is all NaN
        inv = __uint_as_float((uint32_t)(127 - se) << 23);   // 2^-se, exact
        if (lane == 0) a.sf[mx_sf_index(m, g, a.K)] = (uint8_t)(se + 127);
      } else {
        fast = group_factor<DT>(amax, rstd, sc, f);
        if (lane == 0) a.s[g * a.M + m] = sc;
      }
      for (int64_t k = k0 + lane; k < k1; k += 32) {
        const float t = bf16_bits_to_float(row[k]) * (bf16_bits_to_float(a.w[k]) + a.w_off);
        const float y = t * rstd;
        if (DT == kMxFp8)
          a.q[m * a.ldq + k] = (uint8_t)(e4m3x2_code(y * inv, 0.f, 1.0f) & 0xFFu);
        else if (DT == kInt8 && fast)
          a.q[m * a.ldq + k] = (uint8_t)__float_as_uint(__fadd_rn(times(t, f), 12582912.0f));
        else
          a.q[m * a.ldq + k] = fast ? one_code<DT>(times(t, f), 1.0f) : one_code<DT>(y, sc);
        if (a.h) a.h[m * a.ldh + k] = float_to_bf16_bits(y);
      }
    }
    __syncthreads();
  }
}

// Rows of whole 16-byte vectors, groups of 8 lanes' worth of a power of two (or
// the whole row): a CTA per row, V vectors of 8 elements a thread, everything in
// registers, one barrier a row.  Memory-bound: x and the residual are read once,
// the sum, the codes and the scales written once; the next row is under way while
// one is reduced (up to 16384 columns).  With a residual, 4096 x 4096 to INT8: 23.7 us,
// 5.0 TB/s; 2047 x 14336 to MXFP8: 35.8 us, 5.7 TB/s: what it issues (three quarters
// of the issue slots) stands in the way of the rest.  In place is safe: a row is loaded
// and stored by one CTA, each element by one thread, loads first.
template <int DT, int V>
__global__ void __launch_bounds__(V <= 2 ? 1024 : 512)
norm_vec_kernel(const NormArgs a, const int lpg) {       // lpg: lanes of a group, 0 = the row
  __shared__ float red[2][2][32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int nvec = (int)(a.K / 8);
  const float inv_k = __fdiv_rn(1.0f, (float)a.K);
  uint4 wv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * nt + tid;
    wv[i] = v < nvec ? __ldg(reinterpret_cast<const uint4*>(a.w) + v) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint4 nx[V], ns[V];                       // the next row, under way while this one is reduced
  auto load = [&](int64_t m) {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + m * a.ldx);
    const uint4* res = reinterpret_cast<const uint4*>(a.res + m * a.ldr);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * nt + tid;
      nx[i] = ns[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < nvec) {
        nx[i] = x[v];
        if (a.res) ns[i] = res[v];
      }
    }
  };
  constexpr bool kAhead = V <= 2;           // wider rows have no registers for it
  if (kAhead && blockIdx.x < a.M) load(blockIdx.x);
  int parity = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, parity ^= 1) {
    uint4 rv[V], sv[V];
    if (!kAhead) load(m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rv[i] = nx[i];
      sv[i] = ns[i];
    }
    if (kAhead && m + gridDim.x < a.M) load(m + gridDim.x);
    uint64_t sums = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint32_t* r = reinterpret_cast<uint32_t*>(&rv[i]);
      const uint32_t* t = reinterpret_cast<const uint32_t*>(&sv[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (a.res) {
          const uint64_t x = sm100::add2(both(r[e]), both(t[e]));
          r[e] = pack_bf16(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
        }
        sums = sm100::fma2(both(r[e]), both(r[e]), sums);
      }
      const int v = i * nt + tid;
      if (a.res_out && v < nvec) reinterpret_cast<uint4*>(a.res_out + m * a.ldro)[v] = rv[i];
    }
    float sum = warp_sum(__uint_as_float((uint32_t)sums) + __uint_as_float((uint32_t)(sums >> 32)));
    if (lane == 0) red[parity][0][warp] = sum;
    __syncthreads();
    sum = lane < nw ? red[parity][0][lane] : 0.f;
    sum = warp_sum(sum);
    const float rstd = inv_sqrt(fmaf(sum, inv_k, a.eps));
    float row_max = 0.f;
    if (lpg == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float t[8];
        weighted(rv[i], wv[i], a.w_off, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) row_max = largest<DT>(row_max, t[e]);
      }
      row_max = warp_max_nan(row_max);
      if (lane == 0) red[parity][1][warp] = row_max;
      __syncthreads();
      row_max = warp_max_nan(lane < nw ? red[parity][1][lane] : 0.f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = i * nt + tid;
      float t[8];
      weighted(rv[i], wv[i], a.w_off, t);
      float amax = 0.f;                        // of t
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = largest<DT>(amax, t[e]);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1)
        if (o < lpg) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (lpg == 0) amax = row_max;
      if (v >= nvec) continue;                 // no shuffle below
      const bool first = lpg == 0 ? v == 0 : (v & (lpg - 1)) == 0;
      const int64_t g = lpg == 0 ? 0 : v / lpg;
      uint2 q;
      if (DT == kMxFp8) {
        const int se = mx_exponent(fmaxf(amax * rstd, 0.f));     // 0 for a row that is all NaN
        const float inv = __uint_as_float((uint32_t)(127 - se) << 23);   // 2^-se, exact
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = t[e] * rstd;
        q.x = e4m3x4(y, inv);
        q.y = e4m3x4(y + 4, inv);
        if (first) a.sf[mx_sf_index(m, g, a.K)] = (uint8_t)(se + 127);
      } else {
        float sc;
        Factor f;
        if (group_factor<DT>(amax, rstd, sc, f)) {
          q.x = DT == kInt8 ? int8x4(t, f) : e4m3x4(t, f);
          q.y = DT == kInt8 ? int8x4(t + 4, f) : e4m3x4(t + 4, f);
        } else {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = t[e] * rstd;
          q.x = pack4_codes<DT == kMxFp8 ? kFp8 : DT>(y, sc);
          q.y = pack4_codes<DT == kMxFp8 ? kFp8 : DT>(y + 4, sc);
        }
        if (first) a.s[g * a.M + m] = sc;
      }
      *reinterpret_cast<uint2*>(a.q + m * a.ldq + 8 * (int64_t)v) = q;
      if (a.h)
        reinterpret_cast<uint4*>(a.h + m * a.ldh)[v] =
            make_uint4(pack_bf16(t[0] * rstd, t[1] * rstd), pack_bf16(t[2] * rstd, t[3] * rstd),
                       pack_bf16(t[4] * rstd, t[5] * rstd), pack_bf16(t[6] * rstd, t[7] * rstd));
    }
  }
}

// Lanes of a group for the vector kernel, 0 for the whole row, -1 if it does not fit.
int group_lanes(const NormArgs& a) {
  if (a.group >= a.K) return 0;
  const int64_t l = a.group / 8;
  return a.group % 8 == 0 && l <= 32 && (l & (l - 1)) == 0 ? (int)l : -1;
}

bool vec_ok(const NormArgs& a) {
  auto al = [](const void* p, int64_t ld, int n, int bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 && ld % n == 0);
  };
  return a.K % 8 == 0 && a.K <= 32768 && group_lanes(a) >= 0 && al(a.x, a.ldx, 8, 16) &&
         al(a.res, a.ldr, 8, 16) && al(a.w, 0, 8, 16) && al(a.res_out, a.ldro, 8, 16) &&
         al(a.h, a.ldh, 8, 16) && al(a.q, a.ldq, 8, 8);
}

template <int DT, int V>
cudaError_t launch_vec(const NormArgs& a, cudaStream_t st) {
  const int64_t nvec = a.K / 8;
  const int nt = (int)((nvec + 32 * V - 1) / (32 * V)) * 32;
  const int64_t fit = std::max(1, 1024 / nt);            // CTAs of an SM: 64 registers a thread
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(a.M, 148 * fit));
  cfg.blockDim = dim3((unsigned)nt);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_vec_kernel<DT, V>, a, group_lanes(a));
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
  // odd widths, strides and groups (4096 x 4096: 89 us, the vector kernel 24 us)
  if (!vec_ok(a)) return launch_any<DT>(a, st);
  // Few rows: a vector a thread, for latency; many: more loads in flight a thread
  // (1, 2 vectors: 16 x 2048 2.1, 2.5 us, 148 x 4096 2.5, 2.8 us, 148 x 8192 3.4, 3.4 us,
  // 4096 x 2048 13.9, 13.5 us, 4096 x 8192 47, 44 us).  A CTA of 1024 threads ends at
  // 16384 elements; the wider rows' eight vectors cost up to half more where both
  // could be taken (4096 x 14336: 114, 76 us), a fifth of the other kernel's time (2048 x
  // 32768: 121, 567 us).
  if (a.M <= 148 && a.K <= 4096) return launch_vec<DT, 1>(a, st);
  return a.K <= 16384 ? launch_vec<DT, 2>(a, st) : launch_vec<DT, 8>(a, st);
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormArgs& a, cudaStream_t st) {
  if (a.M == 0 || a.K == 0) return cudaSuccess;
  if (a.dtype == kMxFp8) return launch_dt<kMxFp8>(a, st);
  if (a.dtype == kInt8) return launch_dt<kInt8>(a, st);
  return launch_dt<kFp8>(a, st);
}

}  // namespace bq
