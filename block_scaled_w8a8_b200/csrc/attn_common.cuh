// attn_common.cuh -- device helpers shared by the attention kernels: which keys
// a row sees, how the keys are split, codes to fp16, and a row's result.
#pragma once

#include "bq_common.cuh"
#include "kv_common.cuh"
#include "layer_ops.h"

namespace bq {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;

struct Range { int lo, hi; };

// Keys [lo, hi) that row i of sequence s sees (hi <= lo: none).
__device__ __forceinline__ void row_range(const AttnArgs& a, const kv::Seq& s, int i, int& lo,
                                          int& hi) {
  const int pos = s.len - s.n + i;
  hi = a.causal ? min(pos + 1, s.len) : s.len;
  lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// Keys that some row of i_lo .. i_hi sees: both ends grow with the row.
__device__ __forceinline__ Range tile_range(const AttnArgs& a, const kv::Seq& s, int i_lo,
                                            int i_hi) {
  Range r;
  int unused;
  row_range(a, s, i_lo, r.lo, unused);
  row_range(a, s, i_hi, unused, r.hi);
  if (r.hi < r.lo) r.hi = r.lo;
  return r;
}

// Where the keys of a sequence begin to be split, in chunks of `chunk` tokens: the
// first key that any row of it sees, rounded down to the 128 keys of a tile.
__device__ __forceinline__ int split_base(const AttnArgs& a, const kv::Seq& s) {
  int lo, hi;
  row_range(a, s, 0, lo, hi);
  return lo / 128 * 128;
}

// The keys of `all` in chunk number i; may be empty.  A chunk is a multiple of the
// kernels' key tiles, and so is its start, that of `all` rounded down included.
__device__ __forceinline__ Range split_range(const Range& all, int base, int i, int chunk) {
  Range r;
  const int64_t lo = base + (int64_t)i * chunk;
  r.lo = (int)max((int64_t)all.lo / 128 * 128, min(lo, (int64_t)all.hi));
  r.hi = (int)min((int64_t)all.hi, lo + chunk);
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x 2^d for d <= 0, in two steps: the factor alone may be below fp32's smallest where
// the product is not (sums whose references lie more than 2^126 apart).
__device__ __forceinline__ float times_ex2(float x, float d) {
  const float h = ex2(0.5f * d);
  return x * h * h;
}

// The value scale as the kernels that fold it into the exponent take it (weight
// 2^(y - mo) with y = z + lg2 vs, mo within 15 of the row's largest y; the sum's term
// weight / vs).  A weight leaves fp32 below 2^-126, and its key's term with it: with
// scales within a factor of 2^100 of one another that is a term below 2^-41 of the sum.
// Scales below 2^-70, those of zero values among them, count as 2^-70 (their values are
// below 2^-61), which leaves room for scales up to 2^30.  A NaN stays one.
__device__ __forceinline__ float value_scale(float vs) { return max_nan(vs, 0x1p-70f); }

// A running maximum as the reference of a difference: 0 while nothing was seen.
__device__ __forceinline__ float finite(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ uint4 ld_codes16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The D / 8 code bytes of one token that a lane of the value product holds.
template <int D>
__device__ __forceinline__ void ld_codes(const uint8_t* p, uint32_t (&w)[D / 32]) {
  if constexpr (D == 64)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes (byte i = code i) as two fp16 pairs, exactly.
template <int DT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (DT == kInt8) {
    // q + 128 as the low byte of the fp16 number 1024 + (q + 128), less 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// Powers of two that bring a row of largest magnitude amax to 2^14 .. 2^15 and
// back; 1 for a row of zeros or one that is not finite.
__device__ __forceinline__ void row_power(float amax, float& up, float& down) {
  const int ef = (int)(__float_as_uint(amax) >> 23);
  int k = (ef == 0 || ef >= 255) ? 0 : min(14 - (ef - 127), 126);
  up = __uint_as_float((uint32_t)(127 + k) << 23);
  down = __uint_as_float((uint32_t)(127 - k) << 23);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4],
                                        const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The 8 x 8 matrix of 16-bit elements that a warp holds (lane 4 i + j: row i,
// columns 2j, 2j + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// out[tok, head, d] and, from the thread of d = 0, lse: from l = sum 2^(z - mo)
// and acc = O in units of 2^mo.
__device__ __forceinline__ void write_row(const AttnArgs& a, int64_t tok, int head, int d, float l,
                                          float mo, float acc) {
  // l == 0: the row saw no key; a NaN stays one
  a.out[tok * a.ldo + (int64_t)head * a.ho + d] =
      float_to_bf16_bits(l == 0.f ? 0.f : __fdiv_rn(acc, l));
  if (a.lse && d == 0)
    a.lse[tok * a.Hq + head] = l == 0.f ? -INFINITY : (mo + log2f(l)) * 0.6931471805599453f;
}

}  // namespace attn
}  // namespace bq
