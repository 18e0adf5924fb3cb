// rope.cu -- rotary positions.
//
// Pair i of the first rot dimensions of a head, (a, b) = (x[i], x[i + rot/2])
// (half layout) or (x[2i], x[2i+1]) (interleaved), is turned by the angle
// 2 pi * pos * turns[i] and scaled by mscale:
//   a' = mscale * (a cos - b sin),  b' = mscale * (b cos + a sin)
// and the dimensions past rot are copied.  Frequencies are fp64 turns per
// position: pos * turns is formed in fp64 and its whole turns are dropped
// there, so that the angle of position 10^6 is as exact as that of position 1
// (in fp32 the product alone would be off by 0.06 rad); the remaining
// fraction, below half a turn, goes to fp32 sine and cosine.
#include <algorithm>
#include <cstdint>

#include "bq_common.cuh"
#include "layer_ops.h"

namespace bq {

namespace {

// sin and cos of 2 pi * pos * turns, times mscale.
__device__ __forceinline__ void turn_of(int32_t pos, double turns, float mscale, float& sn,
                                        float& cs) {
  const double t = (double)pos * turns;
  const float f = (float)(t - rint(t));
  sincospif(2.0f * f, &sn, &cs);
  sn *= mscale;
  cs *= mscale;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A pair turned; the same roundings wherever it is done, so that the kernels
// agree to the bit.
__device__ __forceinline__ float turned_a(float a, float b, float c, float s) {
  return fmaf(a, c, -__fmul_rn(b, s));
}
__device__ __forceinline__ float turned_b(float a, float b, float c, float s) {
  return fmaf(b, c, __fmul_rn(a, s));
}

// Any rot, strides and alignment: a thread per pair or copied element.
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t half = a.rot / 2, per = half + (a.D - a.rot);
  const int64_t total = a.T * a.H * per;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t th = i / per, e = i - th * per;
    const int64_t t = th / a.H, h = th - t * a.H;
    const uint16_t* x = a.x + t * a.ldt + h * a.ldh;
    uint16_t* o = a.out + t * a.ldot + h * a.ldoh;
    if (e >= half) {
      o[e + half] = x[e + half];
      continue;
    }
    const int64_t ia = a.interleaved ? 2 * e : e, ib = a.interleaved ? 2 * e + 1 : e + half;
    const float va = bf16_bits_to_float(x[ia]), vb = bf16_bits_to_float(x[ib]);
    float sn, cs;
    turn_of(a.pos[t], a.turns[e], a.mscale, sn, cs);
    o[ia] = float_to_bf16_bits(turned_a(va, vb, cs, sn));
    o[ib] = float_to_bf16_bits(turned_b(va, vb, cs, sn));
  }
}

// Rows of whole 16-byte vectors: a CTA has TT tokens; its threads form the
// rot / 2 sines and cosines of each token once (the fp64 product is all that a
// pair costs beyond fp32), then turn 16 bytes of each half (or four neighbouring
// pairs) of all heads; the first of them are under way while the angles are formed.
// Memory-bound: every byte is read and written once.  8191 tokens x 40 heads of 128:
// neighbouring pairs 31.0 us, 5.4 TB/s, half layout 38.6 us, 4.3 TB/s; half of each head
// turned 32.2 and 40.5 us; 8 heads of 64 6.6 us (half layout).
constexpr int kVecThreads = 256;

template <bool INTER>
__global__ void __launch_bounds__(kVecThreads) rope_vec_kernel(const RopeArgs a, const int TT) {
  extern __shared__ float2 cs[];               // [TT][rot / 2] {cos, sin}
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int half = (int)(a.rot / 2), H = (int)a.H, tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const int nt = (int)min((int64_t)TT, a.T - t0);
  // vectors of a head: those with pairs, then those that are copied; a thread has
  // the same one of all its heads, so its sines and cosines are read once a token.
  // Few heads: several tokens side by side.
  const int np = INTER ? (int)a.rot / 8 : half / 8;
  const int nc = a.out == a.x ? 0 : (int)(a.D - a.rot) / 8, per = np + nc;
  const int lanes = min(kVecThreads / per, H);    // heads side by side
  const int tokens = kVecThreads / (per * lanes);
  const int e = tid % per, h0 = tid / per % lanes, first = tid / (per * lanes);
  const bool on = first < tokens && first < nt, copy = e >= np;
  const int64_t at = copy ? a.rot + 8 * (e - np) : 8 * e;
  // kBatch heads at a time: all their loads before the first store, which may be
  // to the same buffer (every element is read and written by one thread)
  constexpr int kBatch = INTER ? 6 : 4;
  uint4 va[kBatch], vb[INTER ? 1 : kBatch];
  auto load = [&](int t, int hb) {
    const uint16_t* xt = a.x + (t0 + t) * a.ldt + at;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = hb + i * lanes;
      if (h >= H) break;
      va[i] = *reinterpret_cast<const uint4*>(xt + h * a.ldh);
      if (!INTER && !copy)
        vb[INTER ? 0 : i] = *reinterpret_cast<const uint4*>(xt + h * a.ldh + half);
    }
  };
  if (on) load(first, h0);                     // under way while the angles are formed
  for (int e = tid; e < nt * half; e += kVecThreads) {
    const int t = e / half;
    float sn, c;
    turn_of(a.pos[t0 + t], a.turns[e - t * half], a.mscale, sn, c);
    cs[e] = make_float2(c, sn);
  }
  __syncthreads();
  if (!on) return;
  for (int t = first; t < nt; t += tokens) {
    uint16_t* ot = a.out + (t0 + t) * a.ldot + at;
    float4 f[INTER ? 2 : 4];
    if (!copy) {
#pragma unroll
      for (int k = 0; k < (INTER ? 2 : 4); ++k)
        f[k] = reinterpret_cast<const float4*>(cs + t * half + (INTER ? 4 : 8) * e)[k];
    }
    for (int hb = h0; hb < H; hb += kBatch * lanes) {
      if (t != first || hb != h0) load(t, hb);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = hb + i * lanes;
        if (h >= H) break;
        uint32_t* wa = reinterpret_cast<uint32_t*>(&va[i]);
        uint32_t* wb = reinterpret_cast<uint32_t*>(&vb[INTER ? 0 : i]);
        if (!copy) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 q = f[INTER ? k >> 1 : k];
            const float a0 = __uint_as_float(wa[k] << 16);
            const float a1 = __uint_as_float(wa[k] & 0xFFFF0000u);
            if (INTER) {
              const float c = k & 1 ? q.z : q.x, s = k & 1 ? q.w : q.y;
              wa[k] = pack_bf16(turned_a(a0, a1, c, s), turned_b(a0, a1, c, s));
            } else {
              const float b0 = __uint_as_float(wb[k] << 16);
              const float b1 = __uint_as_float(wb[k] & 0xFFFF0000u);
              wa[k] = pack_bf16(turned_a(a0, b0, q.x, q.y), turned_a(a1, b1, q.z, q.w));
              wb[k] = pack_bf16(turned_b(a0, b0, q.x, q.y), turned_b(a1, b1, q.z, q.w));
            }
          }
          if (!INTER) *reinterpret_cast<uint4*>(ot + h * a.ldoh + half) = vb[INTER ? 0 : i];
        }
        *reinterpret_cast<uint4*>(ot + h * a.ldoh) = va[i];
      }
    }
  }
}

bool vec_ok(const RopeArgs& a) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const int64_t unit = a.interleaved ? 8 : 16;           // of rot
  return al(a.x) && al(a.out) && a.ldt % 8 == 0 && a.ldh % 8 == 0 && a.ldot % 8 == 0 &&
         a.ldoh % 8 == 0 && a.D % 8 == 0 && a.rot % unit == 0 && a.D <= 1024 && a.D >= 8 &&
         (a.rot > 0 || a.out != a.x) && a.H * a.D <= (1 << 22);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.T == 0 || a.H == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (vec_ok(a)) {
    // many tokens: as many a CTA as one round of its threads has angles for (one token a
    // CTA: 8191 x 40 heads, half layout 48.8 us instead of 38.6, neighbouring pairs, half
    // turned 34.3 instead of 32.1, 8 heads of 64 26.1 instead of 6.6)
    const int64_t half = std::max<int64_t>(1, a.rot / 2);
    int64_t tt = std::max<int64_t>(1, kVecThreads / half);
    tt = std::min<int64_t>(tt, std::max<int64_t>(1, a.T / (148 * 8)));
    const int64_t grid = (a.T + tt - 1) / tt;
    if (grid <= INT32_MAX) {
      cfg.gridDim = dim3((unsigned)grid);
      cfg.blockDim = dim3(kVecThreads);
      cfg.dynamicSmemBytes = (size_t)(tt * half) * sizeof(float2);
      return a.interleaved ? cudaLaunchKernelEx(&cfg, rope_vec_kernel<true>, a, (int)tt)
                           : cudaLaunchKernelEx(&cfg, rope_vec_kernel<false>, a, (int)tt);
    }
  }
  // odd widths and strides (8191 tokens x 40 heads, 24 of 128 dimensions turned in half
  // layout: 216 us, 64 of them in the vector kernel 40 us)
  const int64_t work = a.T * a.H * (a.D - a.rot / 2);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((work + 255) / 256, 148 * 16));
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, rope_any_kernel, a);
}

}  // namespace bq
