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
// the last token keep what they hold.  Both maxima carry a NaN on: a block with one
// has a NaN scale, until its first token is written anew, instead of finite codes
// for a scale that left the NaN out.
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

// Which unit it is; its page is looked up by page_of_unit, so that what needs only
// the rows can go first.  Called by whole warps: each lane reads the offsets and
// lengths of up to four sequences at once, so that 128 sequences cost one memory
// latency.
__device__ __forceinline__ bool find_unit(const AppendArgs& a, int64_t u, Unit& w) {
  const int bt = a.c.bt, lane = threadIdx.x & 31;
  constexpr int kRounds = 4;
  kv::Seq s;
  bool ok = false;
  if (a.b.B <= 32 * kRounds) {
    kv::Seq x[kRounds];
    bool good[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
      if (32 * k < a.b.B)
        good[k] = kv::load_seq(a.b, a.c.page, min(32 * k + lane, a.b.B - 1), x[k]);
    w.b = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      if (32 * k >= a.b.B) break;
      const int i = 32 * k + lane;
      const unsigned before = __ballot_sync(
          0xffffffffu, i < a.b.B && (int64_t)(x[k].row0 / bt) + 2 * (int64_t)i <= u);
      if (k == 0 || before) {
        const int src = max(0, __popc(before) - 1);
        w.b = 32 * k + src;
        s.row0 = __shfl_sync(0xffffffffu, x[k].row0, src);
        s.n = __shfl_sync(0xffffffffu, x[k].n, src);
        s.len = __shfl_sync(0xffffffffu, x[k].len, src);
        ok = __shfl_sync(0xffffffffu, good[k] ? 1 : 0, src) != 0;
      }
    }
  } else {
    w.b = kv::last_at_most(a.b.B, u, [&](int i) { return kv::first_unit(a.b, bt, i); });
    ok = kv::load_seq(a.b, a.c.page, w.b, s);
  }
  if (!ok || s.len < s.n) {
    if (lane == 0) record_status(a.status, kStatusBadInput, 0x601u);
    return false;
  }
  const int64_t j = u - ((int64_t)(s.row0 / bt) + 2 * (int64_t)w.b);
  const int first = s.len - s.n;
  if (s.n == 0 || j < 0 || j > (s.len - 1) / bt - first / bt) return false;
  w.tb = (int)(first / bt + j) * bt;
  w.t0 = max(first, w.tb);
  w.t1 = min(s.len, w.tb + bt);
  w.row0 = s.row0 + (w.t0 - first);
  return true;
}

__device__ __forceinline__ bool page_of_unit(const AppendArgs& a, Unit& w) {
  w.page = kv::page_of(a.b, a.c, w.b, w.tb);
  if (w.page < 0 && (threadIdx.x & 31) == 0) record_status(a.status, kStatusBadInput, 0x602u);
  return w.page >= 0;
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
  if (!find_unit(a, blockIdx.x, w) || !page_of_unit(a, w)) return;
  const int64_t ph = w.page * a.c.H + h;
  const int in_page = w.tb % a.c.page;
  uint8_t* codes = (is_v ? a.c.v : a.c.k) + (ph * a.c.page + in_page) * D;   // of token tb
  float* scale = (is_v ? a.c.vs : a.c.ks) + ph * (a.c.page / a.c.bt) + in_page / a.c.bt;
  const int64_t ld = is_v ? a.ldv : a.ldk;
  const uint16_t* x = (is_v ? a.v + h * a.hv : a.k + h * a.hk) + w.row0 * ld;   // of token t0
  const int n_old = w.t0 - w.tb, n_new = w.t1 - w.t0;
  float amax = 0.f;
  for (int e = tid; e < n_new * D; e += kAnyThreads)
    amax = max_nan(amax, fabsf(bf16_bits_to_float(x[(e / D) * ld + e % D])));
  amax = warp_max_nan(amax);
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  const float s_old = n_old > 0 ? *scale : 0.f;
  __syncthreads();
  amax = max_nan(max_nan(red[0], red[1]), max_nan(red[2], red[3]));
  const float s_new = max_nan(s_old, group_scale<DT>(amax));
  for (int e = tid; e < n_new * D; e += kAnyThreads)
    codes[n_old * D + e] = one_code<DT>(bf16_bits_to_float(x[(e / D) * ld + e % D]), s_new);
  if (s_new > s_old) {
    for (int e = tid; e < n_old * D; e += kAnyThreads)
      codes[e] = one_code<DT>(code_value<DT>(codes[e]) * s_old, s_new);
  }
  // every thread read the old scale before the barrier above
  if (tid == 0) *scale = s_new;
}

// pack4_codes of v for a scale s in [2^-80, inf) with rs = 1 / s correctly
// rounded, without four divisions: q = v rs, its remainder q s - v (exact in one
// FMA), q - remainder * rs, is the correctly rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), as long as the remainder does not underflow: a code other than zero
// needs |v| > s 2^-11, far above that for such s.  The remainder's sign is taken so
// that a zero keeps its own: -0 gives -0 - (+0), where v - q s would give -0 + (+0).
template <int DT>
__device__ __forceinline__ uint32_t pack4_recip(const float v[4], float s, float rs) {
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q0 = v[i] * rs;
    q[i] = fmaf(-fmaf(q0, s, -v[i]), rs, q0);
  }
  if (DT == kInt8) {
    uint32_t b[4];               // round to nearest even; the code in the low byte
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 12582912.0f);
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  unsigned short lo, hi;         // the first source operand lands in the upper byte
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[1]), "f"(q[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[3]), "f"(q[2]));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Blocks of up to 8 * 4 * 512 elements in 16-byte vectors: NW warps have one (unit,
// head), keys and values, up to 4 vectors of new elements of each a lane, read once
// and kept in registers between the maximum and the codes.  A CTA has as many such
// items as make about 256 threads, each with a barrier of its own.  What bounds
// it is the chain of loads (lengths, rows and page, scale), so both arrays go
// through it together.  64 tokens x 8 heads of 128: 5.2 us (one item a CTA: 6.1 us);
// four prompts of up to 2731 tokens: 17.5 us, 3.1 TB/s.
constexpr int kVecs = 4;
constexpr int kVecThreads = 512;

template <int DT>
__global__ void __launch_bounds__(kVecThreads, 1)
append_vec_kernel(const AppendArgs a, const int NW) {
  __shared__ uint32_t red[2][kVecThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nt = 32 * NW, group = (int)threadIdx.x / nt, tid = (int)threadIdx.x - group * nt;
  const int h = blockIdx.y * ((int)blockDim.x / nt) + group, D = a.c.D, dv = D / 8;
  if (h >= a.c.H) return;
  Unit w;
  if (!find_unit(a, blockIdx.x, w)) return;
  const int n_old = w.t0 - w.tb, nv = (w.t1 - w.t0) * dv;
  uint4 v[2][kVecs];
  {
    const uint16_t* xk = a.k + h * a.hk + w.row0 * a.ldk;      // of token t0
    const uint16_t* xv = a.v + h * a.hv + w.row0 * a.ldv;
    int row = tid / dv, col = tid - row * dv;
    const int drow = nt / dv, dcol = nt - drow * dv;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      v[0][i] = v[1][i] = make_uint4(0u, 0u, 0u, 0u);
      if (i * nt + tid < nv) {
        v[0][i] = *reinterpret_cast<const uint4*>(xk + row * a.ldk + 8 * col);
        v[1][i] = *reinterpret_cast<const uint4*>(xv + row * a.ldv + 8 * col);
      }
      row += drow;
      col += dcol;
      if (col >= dv) {
        col -= dv;
        ++row;
      }
    }
  }
  if (!page_of_unit(a, w)) return;
  const int64_t ph = w.page * a.c.H + h;
  const int in_page = w.tb % a.c.page;
  const int64_t code0 = (ph * a.c.page + in_page) * D;          // of token tb
  const int64_t blk = ph * (a.c.page / a.c.bt) + in_page / a.c.bt;
  float s_old[2] = {0.f, 0.f};
  uint32_t amax[2];
  if (n_old > 0) {
    s_old[0] = a.c.ks[blk];
    s_old[1] = a.c.vs[blk];
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    // magnitudes compare as whole numbers, bf16 two at a time; a NaN's is the largest
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      top = __vimax3_u16x2(top, v[c][i].x & 0x7FFF7FFFu, v[c][i].y & 0x7FFF7FFFu);
      top = __vimax3_u16x2(top, v[c][i].z & 0x7FFF7FFFu, v[c][i].w & 0x7FFF7FFFu);
    }
    amax[c] = __reduce_max_sync(0xffffffffu, max(top << 16, top & 0xFFFF0000u));
    if (NW > 1 && lane == 0) red[c][warp] = amax[c];
  }
  if (NW > 1) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(nt) : "memory");
    amax[0] = amax[1] = 0;
    for (int i = 0; i < NW; ++i) {
      amax[0] = max(amax[0], red[0][group * NW + i]);
      amax[1] = max(amax[1], red[1][group * NW + i]);
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint8_t* codes = (c ? a.c.v : a.c.k) + code0;
    const float s_new = max_nan(s_old[c], group_scale<DT>(__uint_as_float(amax[c])));
    const bool fast = s_new >= 0x1p-80f && s_new < INFINITY;
    const float rs = fast ? __fdiv_rn(1.0f, s_new) : 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = i * nt + tid;
      if (e >= nv) break;
      const uint32_t u[4] = {v[c][i].x, v[c][i].y, v[c][i].z, v[c][i].w};
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(u[k] << 16);
        f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
      *reinterpret_cast<uint2*>(codes + n_old * D + 8 * e) =
          fast ? make_uint2(pack4_recip<DT>(f, s_new, rs), pack4_recip<DT>(f + 4, s_new, rs))
               : make_uint2(pack4_codes<DT>(f, s_new), pack4_codes<DT>(f + 4, s_new));
    }
    if (s_new > s_old[c]) {
      for (int e = tid; e < n_old * dv; e += nt) {
        uint2 old = *reinterpret_cast<const uint2*>(codes + 8 * e);
        uint32_t* p = reinterpret_cast<uint32_t*>(&old);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) f[b] = code_value<DT>((uint8_t)(p[k] >> (8 * b))) * s_old[c];
          p[k] = pack4_codes<DT>(f, s_new);
        }
        *reinterpret_cast<uint2*>(codes + 8 * e) = old;
      }
    }
    // every thread of the item read the old scale before the barrier (or this sync)
    __syncwarp();
    if (tid == 0) (c ? a.c.vs : a.c.ks)[blk] = s_new;
  }
}

bool vec_ok(const AppendArgs& a) {
  auto al = [](const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
  };
  return a.c.D % 8 == 0 && (int64_t)a.c.bt * a.c.D <= 8 * kVecs * kVecThreads && al(a.k, 16) &&
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
    const int per = std::max(1, 8 / nw);                 // items of a CTA
    cfg.gridDim = dim3((unsigned)units, (unsigned)((a.c.H + per - 1) / per));
    cfg.blockDim = dim3((unsigned)(32 * nw * per));
    return a.c.dtype == kInt8 ? cudaLaunchKernelEx(&cfg, append_vec_kernel<kInt8>, a, nw)
                              : cudaLaunchKernelEx(&cfg, append_vec_kernel<kFp8>, a, nw);
  }
  // odd widths and strides, long blocks (four prompts of 2731 tokens: 108 us, the
  // vector kernel 18 us)
  cfg.gridDim = dim3((unsigned)units, (unsigned)a.c.H, 2);
  cfg.blockDim = dim3(kAnyThreads);
  if (a.c.dtype == kInt8) return cudaLaunchKernelEx(&cfg, append_any_kernel<kInt8>, a);
  return cudaLaunchKernelEx(&cfg, append_any_kernel<kFp8>, a);
}

}  // namespace bq
