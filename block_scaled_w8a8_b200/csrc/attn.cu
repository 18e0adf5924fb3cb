// attn.cu -- attention over the paged 8-bit cache: the dispatch, the join of
// split keys, and the CUDA-core kernel that takes any head size and stride.
//
// For row i of sequence b at position p_i = len_b - n_b + i, query head h and
// its key head h / (Hq / Hkv):
//   s_j = scale * ks[block(j)] * (q . k_code[j])         for the keys j it sees
//   out = sum_j softmax(s)_j * vs[block(j)] * v_code[j],  lse = ln sum_j exp(s_j)
// A causal row sees j <= p_i, with a window W only j > p_i - W; otherwise it
// sees the whole sequence.  A row that sees nothing gives zeros and lse = -inf.
// Keys that no row may see are never read into a sum, whatever bytes they hold.
#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"
#include "bq_common.cuh"
#include "kv_common.cuh"

namespace bq {

namespace {

using attn::row_range;

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
  const int b = kv::seq_of(a.b, t);
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, b, s) || s.n > a.max_q || s.len > a.max_kv) {
    if (lane == 0) record_status(a.status, kStatusBadInput, 0x701u);
    return;
  }
  if (t < s.row0 || t >= s.row0 + s.n) return;      // a row behind the last sequence
  int lo, hi;
  row_range(a, s, (int)(t - s.row0), lo, hi);
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

// Joins the splits of a row: NW warps per (row, query head) take the splits in
// turn, and their sums are joined in warp order.  NW = 1 up to 4 splits, 8 above:
// the splits' rows are loaded side by side instead of one latency each.
template <int NW>
__global__ void __launch_bounds__(128 * (NW > 4 ? 2 : 1))
attn_merge_kernel(const AttnArgs a, const AttnParts p) {
  __shared__ float so[NW][kMaxD];
  __shared__ float sl[NW];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = NW > 1 ? warp : 0;
  const int64_t item = NW > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + warp;
  const int64_t t = item / a.Hq;
  const int h = (int)(item - t * a.Hq), D = a.c.D;
  if (t >= a.b.T) return;
  const int b = kv::seq_of(a.b, t);
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, b, s) || s.n > a.max_q || s.len > a.max_kv || t < s.row0 ||
      t >= s.row0 + s.n)
    return;                          // recorded by the kernel before, or nobody's row
  const float2* stat = reinterpret_cast<const float2*>(p.stat) + item * p.splits;
  // the splits that hold keys this row sees
  int lo, hi;
  row_range(a, s, (int)(t - s.row0), lo, hi);
  const int first = attn::first_split(a, s, p.chunk);
  const int i0 = hi > lo ? lo / p.chunk - first : 0;
  const int i1 = hi > lo ? (hi - 1) / p.chunk - first + 1 : 0;
  float mo = -INFINITY;
  for (int i = i0 + lane; i < i1; i += 32) mo = fmaxf(mo, stat[i].y);
  mo = warp_max(mo);
  float l = 0.f, acc[kMaxD / 32] = {};
#pragma unroll 4
  for (int i = i0 + w; i < i1; i += NW) {
    const float2 x = stat[i];
    if (x.x == 0.f) continue;
    const float f = attn::ex2(x.y - attn::finite(mo));
    l += x.x * f;
    const float* o = p.o + (item * p.splits + i) * D;
#pragma unroll
    for (int e = 0; e < kMaxD / 32; ++e)
      if (lane + 32 * e < D) acc[e] = fmaf(o[lane + 32 * e], f, acc[e]);
  }
  if constexpr (NW == 1) {
#pragma unroll
    for (int e = 0; e < kMaxD / 32; ++e)
      if (lane + 32 * e < D) attn::write_row(a, t, h, lane + 32 * e, l, mo, acc[e]);
  } else {
    if (lane == 0) sl[w] = l;
#pragma unroll
    for (int e = 0; e < kMaxD / 32; ++e)
      if (lane + 32 * e < D) so[w][lane + 32 * e] = acc[e];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 32 * NW) {
      float sum = 0.f, v = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        sum += sl[i];
        v += so[i][d];
      }
      attn::write_row(a, t, h, d, sum, mo, v);
    }
  }
}

template <class... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), int64_t grid, int threads, cudaStream_t st,
                       Args... args) {
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The kernel of a call and how it splits the keys, from the call's sizes alone.
enum class Path { kAny, kDecode, kTc };

// Rows per key head up to which the streaming kernel is taken; it reads the codes
// once for 8 rows, the tensor core kernel once for 256 but with a dearer start.  16
// sequences of 8192 keys: 16 rows 121 and 163 us, 24 rows 156 and 163; 1 of 65536:
// 16 rows 75 and 88, 24 rows 94 and 88; 1 of 4096: 24 rows 17 and 22 us.
constexpr int64_t kDecodeRows = 24;

Path plan_path(int64_t D, int64_t page, int64_t rows) {
  if (rows > kDecodeRows && attn_tc_takes(D, page)) return Path::kTc;
  return attn_decode_takes(D, page) ? Path::kDecode : Path::kAny;
}

// Chunk of keys and most chunks that the keys of one sequence's rows lie in.
void plan_splits(Path path, int64_t B, int64_t Hq, int64_t Hkv, int64_t max_q, int64_t max_kv,
                 AttnParts& p) {
  p.splits = 1;
  p.chunk = 1 << 30;
  const int64_t g = Hq / Hkv;
  if (path == Path::kTc) p.chunk = attn_tc_chunk(B, Hkv, max_q, g, max_kv);
  if (path == Path::kDecode) p.chunk = attn_decode_chunk(B, Hkv, max_q * g, max_kv);
  p.splits = (int)std::max<int64_t>(1, (max_kv + p.chunk - 1) / p.chunk);
}

}  // namespace

size_t attn_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            int64_t max_q, int64_t max_kv, int64_t page, int64_t bt) {
  (void)bt;
  AttnParts p{};
  plan_splits(plan_path(D, page, max_q * (Hq / Hkv)), B, Hq, Hkv, max_q, max_kv, p);
  return attn_part_bytes(T * Hq, p.splits, D);
}

cudaError_t launch_attn_merge(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const int64_t items = a.b.T * a.Hq;
  return p.splits <= 4 ? launch_pdl(attn_merge_kernel<1>, (items + 3) / 4, 128, st, a, p)
                       : launch_pdl(attn_merge_kernel<8>, items, 256, st, a, p);
}

cudaError_t launch_kv_attention(const AttnArgs& a, void* ws, cudaStream_t st) {
  const int64_t items = a.b.T * a.Hq;
  const bool aligned = ((reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v)) &
                        15) == 0;
  const Path path = plan_path(a.c.D, a.c.page, (int64_t)a.max_q * (a.Hq / a.c.H));
  if (aligned && a.max_q > 0 && path != Path::kAny) {
    AttnParts p{};
    plan_splits(path, a.b.B, a.Hq, a.c.H, a.max_q, a.max_kv, p);
    if (p.splits > 1) {
      p.stat = static_cast<float*>(ws);
      p.o = p.stat + (2 * items * p.splits + 3) / 4 * 4;
    }
    cudaError_t e =
        path == Path::kTc ? launch_attn_tc(a, p, st) : launch_attn_decode(a, p, st);
    if (e == cudaSuccess && p.splits > 1) e = launch_attn_merge(a, p, st);
    return e;
  }
  const int64_t grid = (items + kAnyWarps - 1) / kAnyWarps;
  return a.c.dtype == kInt8 ? launch_pdl(attn_any_kernel<kInt8>, grid, kAnyWarps * 32, st, a)
                            : launch_pdl(attn_any_kernel<kFp8>, grid, kAnyWarps * 32, st, a);
}

}  // namespace bq
