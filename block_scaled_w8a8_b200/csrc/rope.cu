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
    o[ia] = float_to_bf16_bits(va * cs - vb * sn);
    o[ib] = float_to_bf16_bits(vb * cs + va * sn);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.T == 0 || a.H == 0) return cudaSuccess;
  const int64_t work = a.T * a.H * (a.D - a.rot / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((work + 255) / 256, 148 * 16));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_any_kernel, a);
}

}  // namespace bq
