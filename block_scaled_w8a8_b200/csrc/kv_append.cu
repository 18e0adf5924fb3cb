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

__device__ __forceinline__ bool find_unit(const AppendArgs& a, int64_t u, Unit& w) {
  const int bt = a.c.bt;
  w.b = kv::last_at_most(a.b.B, u, [&](int i) { return kv::first_unit(a.b, bt, i); });
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, w.b, s) || s.len < s.n) {
    if (threadIdx.x == 0) record_status(a.status, kStatusBadInput, 0x601u);
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
    if (threadIdx.x == 0) record_status(a.status, kStatusBadInput, 0x602u);
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

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  const int64_t units = kv::unit_bound(a.b.T, a.b.B, a.c.bt);
  if (units == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units, (unsigned)a.c.H, 2);
  cfg.blockDim = dim3(kAnyThreads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (a.c.dtype == kInt8) return cudaLaunchKernelEx(&cfg, append_any_kernel<kInt8>, a);
  return cudaLaunchKernelEx(&cfg, append_any_kernel<kFp8>, a);
}

}  // namespace bq
