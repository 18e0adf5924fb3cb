// attn.cu -- attention over the paged 8-bit cache: the dispatch, and the
// CUDA-core kernel that takes any head size and stride.
//
// For row i of sequence b at position p_i = len_b - n_b + i, query head h and
// its key head h / (Hq / Hkv):
//   s_j = scale * ks[block(j)] * (q . k_code[j])         for the keys j it sees
//   out = sum_j softmax(s)_j * vs[block(j)] * v_code[j],  lse = ln sum_j exp(s_j)
// A causal row sees j <= p_i, with a window W only j > p_i - W; otherwise it
// sees the whole sequence.  A row that sees nothing gives zeros and lse = -inf.
// Keys that no row may see are never read into a sum, whatever bytes they hold.
#include <algorithm>

#include "bq_common.cuh"
#include "kv_common.cuh"
#include "layer_ops.h"

namespace bq {

namespace {

constexpr int kAnyWarps = 4;
constexpr int kMaxD = 256;

template <int DT>
__device__ __forceinline__ float code_value(uint8_t c) {
  return DT == kInt8 ? (float)(int8_t)c : e4m3_to_float(c);
}

// A warp per (row, query head): lane l holds dimensions l, l + 32, ...; one
// key at a time, running maximum and sum in fp32.
template <int DT>
__global__ void __launch_bounds__(kAnyWarps * 32) attn_any_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPer = kMaxD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kAnyWarps + (threadIdx.x >> 5);
  const int64_t t = item / a.Hq;
  const int h = (int)(item - t * a.Hq);
  if (t >= a.b.T) return;
  const int b = kv::last_at_most(a.b.B, t, [&](int i) { return (int64_t)a.b.off[i]; });
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, b, s) || s.n > a.max_q || s.len > a.max_kv) {
    if (lane == 0) record_status(a.status, kStatusBadInput, 0x701u);
    return;
  }
  if (t < s.row0 || t >= s.row0 + s.n) return;      // a row behind the last sequence
  const int pos = s.len - s.n + (int)(t - s.row0);
  const int hi = a.causal ? min(pos + 1, s.len) : s.len;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int hk = h / (a.Hq / a.c.H), D = a.c.D;
  const uint16_t* q = a.q + t * a.ldq + h * a.hq;
  float qv[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    qv[i] = lane + 32 * i < D ? bf16_bits_to_float(q[lane + 32 * i]) : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int64_t page = kv::page_of(a.b, a.c, b, j);
    if (page < 0) {
      if (lane == 0) record_status(a.status, kStatusBadInput, 0x702u);
      continue;
    }
    const int64_t ph = page * a.c.H + hk;
    const int in_page = j % a.c.page;
    const int64_t row = (ph * a.c.page + in_page) * D;
    const int64_t blk = ph * (a.c.page / a.c.bt) + in_page / a.c.bt;
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < D) d = fmaf(qv[i], code_value<DT>(a.c.k[row + lane + 32 * i]), d);
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o2);
    const float sc = d * (a.c.ks[blk] * a.scale);
    const float mn = fmaxf(m, sc);
    // a first score of -inf would make the difference below NaN
    const float base = mn == -INFINITY ? 0.f : mn;
    const float keep = __expf(m - base), p = __expf(sc - base);
    l = l * keep + p;
    const float pv = p * a.c.vs[blk];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < D)
        o[i] = fmaf(pv, code_value<DT>(a.c.v[row + lane + 32 * i]), o[i] * keep);
    m = mn;
  }
  uint16_t* out = a.out + t * a.ldo + h * a.ho;
  const float inv = l > 0.f ? __fdiv_rn(1.0f, l) : (l == 0.f ? 0.f : l);   // a NaN stays one
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < D) out[lane + 32 * i] = float_to_bf16_bits(o[i] * inv);
  if (a.lse && lane == 0) a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attn_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                            int64_t, int64_t) {
  return 0;
}

cudaError_t launch_kv_attention(const AttnArgs& a, void* ws, cudaStream_t st) {
  (void)ws;
  const int64_t items = a.b.T * a.Hq;
  if (items == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items + kAnyWarps - 1) / kAnyWarps));
  cfg.blockDim = dim3(kAnyWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (a.c.dtype == kInt8) return cudaLaunchKernelEx(&cfg, attn_any_kernel<kInt8>, a);
  return cudaLaunchKernelEx(&cfg, attn_any_kernel<kFp8>, a);
}

}  // namespace bq
