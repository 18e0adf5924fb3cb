// kv_append.cu -- new keys and values into the paged 8-bit cache, with one
// scale for each block of bt tokens of a head.
//
// For a block that holds n_old tokens before the call and gets new ones:
//   s' = max(s_old, amax(new) / Q)        (s_old counts as 0 when n_old = 0)
//   new codes = code(x / s');
//   if s' > s_old and n_old > 0: old codes = code((q_old * s_old) / s').
// code() and the division are those of the activation quantiser (IEEE fp32,
// round to nearest even).  A block whose new tokens fit the old scale keeps its
// old codes, so writing the same tokens again changes nothing.  Slots behind
// the last token keep what they hold.
#include <algorithm>

#include "bq_common.cuh"
#include "kv_common.cuh"
#include "layer_ops.h"

namespace bq {

namespace {

constexpr int kAnyThreads = 128;

template <int DT>
__device__ __forceinline__ float code_value(uint8_t c) {
  return DT == kInt8 ? (float)(int8_t)c : e4m3_to_float(c);
}

// What one unit writes: tokens [t0, t1) of sequence b, all in one block; the
// block's earlier tokens begin at token tb.
struct Unit {
  int b, tb, t0, t1, row0;     // row0: the row of token t0
  int64_t page;
};

// Called by whole warps.
__device__ __forceinline__ bool find_unit(const AppendArgs& a, int64_t u, Unit& w) {
  const int bt = a.c.bt, lane = threadIdx.x & 31;
  w.b = kv::last_at_most(a.b.B, u, [&](int i) { return kv::first_unit(a.b, bt, i); });
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, w.b, s) || s.len < s.n) {
    if (lane == 0) record_status(a.status, kStatusBadInput, 0x601u);
    return false;
  }
  const int64_t j = u - kv::first_unit(a.b, bt, w.b);
  const int first = s.len - s.n;
  if (s.n == 0 || j < 0 || j > (s.len - 1) / bt - first / bt) return false;
  w.tb = (int)(first / bt + j) * bt;
  w.t0 = max(first, w.tb);
  w.t1 = min(s.len, w.tb + bt);
  w.row0 = s.row0 + (w.t0 - first);
  w.page = kv::page_of(a.b, a.c, w.b, w.tb);
  if (w.page < 0) {
    if (lane == 0) record_status(a.status, kStatusBadInput, 0x602u);
    return false;
  }
  return true;
}

// Any block size, head size, stride and alignment: a CTA per (unit, head, K or V).
template <int DT>
__global__ void __launch_bounds__(kAnyThreads) append_any_kernel(const AppendArgs a) {
  __shared__ float red[kAnyThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.y, tid = threadIdx.x, D = a.c.D;
  const bool is_v = blockIdx.z != 0;
  Unit w;
  if (!find_unit(a, blockIdx.x, w)) return;
  const int64_t ph = w.page * a.c.H + h;
  const int in_page = w.tb % a.c.page;
  uint8_t* codes = (is_v ? a.c.v : a.c.k) + (ph * a.c.page + in_page) * D;   // of token tb
  float* scale = (is_v ? a.c.vs : a.c.ks) + ph * (a.c.page / a.c.bt) + in_page / a.c.bt;
  const int64_t ld = is_v ? a.ldv : a.ldk;
  const uint16_t* x = (is_v ? a.v + h * a.hv : a.k + h * a.hk) + w.row0 * ld;   // of token t0
  const int n_old = w.t0 - w.tb, n_new = w.t1 - w.t0;
  float amax = 0.f;
  for (int e = tid; e < n_new * D; e += kAnyThreads)
    amax = fmaxf(amax, fabsf(bf16_bits_to_float(x[(e / D) * ld + e % D])));
  amax = warp_max(amax);
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  const float s_old = n_old > 0 ? *scale : 0.f;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float s_new = fmaxf(s_old, group_scale<DT>(amax));
  for (int e = tid; e < n_new * D; e += kAnyThreads)
    codes[n_old * D + e] = one_code<DT>(bf16_bits_to_float(x[(e / D) * ld + e % D]), s_new);
  if (s_new > s_old) {
    for (int e = tid; e < n_old * D; e += kAnyThreads)
      codes[e] = one_code<DT>(code_value<DT>(codes[e]) * s_old, s_new);
  }
  // every thread read the old scale before the barrier above
  if (tid == 0) *scale = s_new;
}

// Blocks of up to 8 * 8 * 256 elements in 16-byte vectors: NW warps have one (unit,
// head, K or V), up to 8 vectors of new elements a lane, read once and kept in
// registers between the maximum and the codes.  NW = 1: four items a CTA.
constexpr int kVecs = 8;

template <int DT>
__global__ void __launch_bounds__(256) append_vec_kernel(const AppendArgs a, const int NW) {
  __shared__ float red[8];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = NW == 1 ? (int)(blockDim.x >> 5) : 1;         // items of a CTA
  const int item = blockIdx.y * per + (NW == 1 ? warp : 0);     // 2 head + (K or V)
  const int nt = 32 * NW, tid = NW == 1 ? lane : (int)threadIdx.x;
  if (item >= 2 * a.c.H) return;                                // whole warps of NW = 1
  const int h = item >> 1, D = a.c.D, dv = D / 8;
  const bool is_v = item & 1;
  Unit w;
  if (!find_unit(a, blockIdx.x, w)) return;
  const int64_t ph = w.page * a.c.H + h;
  const int in_page = w.tb % a.c.page;
  uint8_t* codes = (is_v ? a.c.v : a.c.k) + (ph * a.c.page + in_page) * D;   // of token tb
  float* scale = (is_v ? a.c.vs : a.c.ks) + ph * (a.c.page / a.c.bt) + in_page / a.c.bt;
  const int64_t ld = is_v ? a.ldv : a.ldk;
  const uint16_t* x = (is_v ? a.v + h * a.hv : a.k + h * a.hk) + w.row0 * ld;   // of token t0
  const int n_old = w.t0 - w.tb, nv = (w.t1 - w.t0) * dv;
  const float s_old = n_old > 0 ? *scale : 0.f;
  uint4 v[kVecs];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int e = i * nt + tid;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (e < nv) v[i] = *reinterpret_cast<const uint4*>(x + (e / dv) * ld + 8 * (e % dv));
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[e] << 16)),
                               fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
  }
  amax = warp_max(amax);
  if (NW > 1) {
    if (lane == 0) red[warp] = amax;
    __syncthreads();
    amax = 0.f;
    for (int i = 0; i < NW; ++i) amax = fmaxf(amax, red[i]);
  }
  const float s_new = fmaxf(s_old, group_scale<DT>(amax));
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int e = i * nt + tid;
    if (e >= nv) break;
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
    *reinterpret_cast<uint2*>(codes + n_old * D + 8 * e) =
        make_uint2(pack4_codes<DT>(f, s_new), pack4_codes<DT>(f + 4, s_new));
  }
  if (s_new > s_old) {
    for (int e = tid; e < n_old * dv; e += nt) {
      uint2 c = *reinterpret_cast<const uint2*>(codes + 8 * e);
      uint32_t* p = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float f[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = code_value<DT>((uint8_t)(p[k] >> (8 * b))) * s_old;
        p[k] = pack4_codes<DT>(f, s_new);
      }
      *reinterpret_cast<uint2*>(codes + 8 * e) = c;
    }
  }
  // NW > 1: every thread read the old scale before the barrier above
  __syncwarp();
  if (tid == 0) *scale = s_new;
}

bool vec_ok(const AppendArgs& a) {
  auto al = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  return a.c.D % 8 == 0 && (int64_t)a.c.bt * a.c.D <= 8 * kVecs * 256 && al(a.k, 16) &&
         al(a.v, 16) && al(a.c.k, 8) && al(a.c.v, 8) && a.ldk % 8 == 0 && a.hk % 8 == 0 &&
         a.ldv % 8 == 0 && a.hv % 8 == 0;
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  const int64_t units = kv::unit_bound(a.b.T, a.b.B, a.c.bt);
  if (units == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (vec_ok(a)) {
    const int64_t lanes = ((int64_t)a.c.bt * a.c.D / 8 + kVecs - 1) / kVecs;
    const int nw = (int)((lanes + 31) / 32);
    const int per = nw == 1 ? 4 : 1;
    cfg.gridDim = dim3((unsigned)units, (unsigned)((2 * a.c.H + per - 1) / per));
    cfg.blockDim = dim3((unsigned)(nw == 1 ? 128 : 32 * nw));
    return a.c.dtype == kInt8 ? cudaLaunchKernelEx(&cfg, append_vec_kernel<kInt8>, a, nw)
                              : cudaLaunchKernelEx(&cfg, append_vec_kernel<kFp8>, a, nw);
  }
  cfg.gridDim = dim3((unsigned)units, (unsigned)a.c.H, 2);
  cfg.blockDim = dim3(kAnyThreads);
  if (a.c.dtype == kInt8) return cudaLaunchKernelEx(&cfg, append_any_kernel<kInt8>, a);
  return cudaLaunchKernelEx(&cfg, append_any_kernel<kFp8>, a);
}

}  // namespace bq
