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

using attn::Range;
using attn::row_range;

constexpr int kAnyWarps = 4, kAnyRows = 4;
constexpr int kMaxD = 256;

// Four codes of a row as fp32; `n` of them are there, read at once if `words`.
template <int DT>
__device__ __forceinline__ void load4(const uint8_t* p, bool words, int n, float (&f)[4]) {
  uint32_t w = 0, lo, hi;
  if (words) {
    w = *reinterpret_cast<const uint32_t*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) w |= (uint32_t)p[e] << (8 * e);
  }
  attn::codes_to_f16<DT>(w, lo, hi);
  const float2 a = __half22float2(reinterpret_cast<const __half2&>(lo));
  const float2 b = __half22float2(reinterpret_cast<const __half2&>(hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// CUDA cores, any head size, page and alignment.  A CTA works on four rows (tokens x
// heads of one key head's group) and one part of the keys; a warp takes 32 keys at a
// time.  Scores: a lane per key, whose codes it reads four at a time where they are
// aligned, against the four queries in shared memory; values: four dimensions a lane
// (128 i + 4 lane), the keys in turn.  A code is so read and converted once for four rows.  The
// softmax runs in fp32, in units of 2^m.  Bound by its instructions, some ten of a
// warp for a key and row: 1 x 4096 keys, 32 heads over 8, pages of 8: 32 us (12 us where
// the streaming kernel takes the page), 64 x 2048 keys of dim 80: 265 us, a prompt of
// 2048 of dim 96: 2.7 ms.
template <int DT>
__global__ void __launch_bounds__(kAnyWarps * 32)
attn_any_kernel(const AttnArgs a, const AttnParts parts, const int row_tiles) {
  __shared__ float4 sq[kMaxD];                           // of the four rows
  __shared__ float4 sw[kAnyWarps][32];                   // weights of a warp's keys
  __shared__ int64_t sr[kAnyWarps][32];                  // where their codes lie, or -1
  __shared__ float so[kAnyWarps][kAnyRows][kMaxD], ss[kAnyWarps][kAnyRows][2];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPer = kMaxD / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.c.D;
  int idx = (int)blockIdx.x;
  const int rt = idx % row_tiles;
  idx /= row_tiles;
  const int split = idx % parts.splits, b = idx / parts.splits, hk = blockIdx.y;
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, b, s) || s.n > a.max_q || s.len > a.max_kv) {
    if (threadIdx.x == 0) record_status(a.status, kStatusBadInput, 0x701u);
    return;
  }
  const int g = a.Hq / a.c.H, R0 = rt * kAnyRows, n_rows = s.n * g;
  if (R0 >= n_rows) return;
  const int i_hi = min(s.n - 1, (R0 + kAnyRows - 1) / g);
  const Range all = attn::tile_range(a, s, R0 / g, i_hi);
  const Range part = attn::split_range(all, attn::split_base(a, s), split, parts.chunk);
  if (parts.splits > 1 && part.hi <= part.lo) return;    // the join does not look at it
  int lo[kAnyRows], hi[kAnyRows];
  float m[kAnyRows], l[kAnyRows], o[kAnyRows][kPer];
#pragma unroll
  for (int r = 0; r < kAnyRows; ++r) {
    // rows behind the last stand in for it: nothing of them is written
    row_range(a, s, min((R0 + r) / g, s.n - 1), lo[r], hi[r]);
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[r][i] = 0.f;
  }
  for (int d = threadIdx.x; d < D; d += kAnyWarps * 32) {
    float x[kAnyRows];
#pragma unroll
    for (int r = 0; r < kAnyRows; ++r) {
      const int row = min(R0 + r, n_rows - 1);
      x[r] = bf16_bits_to_float(
          a.q[(int64_t)(s.row0 + row / g) * a.ldq + (int64_t)(hk * g + row % g) * a.hq + d]);
    }
    sq[d] = make_float4(x[0], x[1], x[2], x[3]);
  }
  __syncthreads();
  const bool words = D % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.c.k) |
                                     reinterpret_cast<uintptr_t>(a.c.v)) & 3) == 0;
  const float scale = a.scale * attn::kLog2e;
  for (int t = part.lo + 32 * warp; t < part.hi; t += 32 * kAnyWarps) {
    const int tok = t + lane;
    int64_t row = -1;
    float z[kAnyRows] = {}, vs = 0.f;
    if (tok >= all.lo && tok < part.hi) {
      const int64_t page = kv::page_of(a.b, a.c, b, tok);
      if (page < 0) {
        record_status(a.status, kStatusBadInput, 0x702u);
      } else {
        const int64_t ph = page * a.c.H + hk;
        const int slot = tok % a.c.page;
        const int64_t blk = ph * (a.c.page / a.c.bt) + slot / a.c.bt;
        row = (ph * a.c.page + slot) * D;
        vs = a.c.vs[blk];
        const uint8_t* k = a.c.k + row;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float f[4];
          load4<DT>(k + d, words, D - d, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (d + e >= D) break;
            const float4 q = sq[d + e];
            z[0] = fmaf(q.x, f[e], z[0]);
            z[1] = fmaf(q.y, f[e], z[1]);
            z[2] = fmaf(q.z, f[e], z[2]);
            z[3] = fmaf(q.w, f[e], z[3]);
          }
        }
        const float f = a.c.ks[blk] * scale;
#pragma unroll
        for (int r = 0; r < kAnyRows; ++r) z[r] *= f;
      }
    }
    float p[kAnyRows];
#pragma unroll
    for (int r = 0; r < kAnyRows; ++r) {
      if (row < 0 || tok < lo[r] || tok >= hi[r]) z[r] = -INFINITY;
      const float mn = fmaxf(m[r], warp_max(z[r]));
      // while every score is -inf the reference is 0, not a difference of infinities
      const float keep = attn::ex2(m[r] - attn::finite(mn));
      p[r] = attn::ex2(z[r] - attn::finite(mn));
      l[r] = fmaf(l[r], keep, p[r]);
      // a key of weight 0 adds nothing, whatever its value is
      p[r] = p[r] == 0.f ? 0.f : p[r] * vs;
      m[r] = mn;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[r][i] *= keep;
    }
    sw[warp][lane] = make_float4(p[0], p[1], p[2], p[3]);
    sr[warp][lane] = row;
    __syncwarp();
    const int n = min(32, part.hi - t);
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const int64_t at = sr[warp][j];
      if (at < 0) continue;
      const float4 w = sw[warp][j];
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const int d = 4 * lane + 32 * i;
        if (d < D) {
          float f[4];
          load4<DT>(a.c.v + at + d, words, D - d, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (w.x != 0.f) o[0][i + e] = fmaf(w.x, f[e], o[0][i + e]);
            if (w.y != 0.f) o[1][i + e] = fmaf(w.y, f[e], o[1][i + e]);
            if (w.z != 0.f) o[2][i + e] = fmaf(w.z, f[e], o[2][i + e]);
            if (w.w != 0.f) o[3][i + e] = fmaf(w.w, f[e], o[3][i + e]);
          }
        }
      }
    }
    __syncwarp();
  }
  // the four warps' parts, joined in warp order
#pragma unroll
  for (int r = 0; r < kAnyRows; ++r) {
    float sum = l[r];
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    if (lane == 0) {
      ss[warp][r][0] = sum;
      ss[warp][r][1] = m[r];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) so[warp][r][4 * lane + 32 * (i & ~3) + (i & 3)] = o[r][i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kAnyRows * D; e += kAnyWarps * 32) {
    const int r = e / D, d = e % D;
    if (R0 + r >= n_rows) break;
    float M = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) M = fmaxf(M, ss[w][r][1]);
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) {
      const float f = attn::ex2(ss[w][r][1] - attn::finite(M));
      sum = fmaf(ss[w][r][0], f, sum);
      acc = fmaf(so[w][r][d], f, acc);
    }
    const int64_t tok = s.row0 + (R0 + r) / g;
    const int head = hk * g + (R0 + r) % g;
    if (parts.splits == 1) {
      attn::write_row(a, tok, head, d, sum, M, acc);
    } else {
      const int64_t at = (tok * a.Hq + head) * parts.splits + split;
      if (sum != 0.f) parts.o[at * D + d] = acc;
      if (d == 0) *reinterpret_cast<float2*>(parts.stat + 2 * at) = make_float2(sum, M);
    }
  }
}

// CTAs of at least 128 keys, about sixteen for each of the 148 SMs.
int attn_any_chunk(int64_t B, int64_t Hkv, int64_t rows, int64_t span) {
  const int64_t units = std::max<int64_t>(1, B * Hkv * ((rows + kAnyRows - 1) / kAnyRows));
  const int64_t c = units * span / (148 * 16);
  return (int)std::min<int64_t>(1 << 24, std::max<int64_t>(128, (c + 127) / 128 * 128));
}

// Joins the splits of a row: NW warps per (row, query head) take the splits in
// turn, and their sums are joined in warp order.  NW = 1 up to 4 splits, 8 above:
// the splits' rows are loaded side by side instead of one latency each (attention and
// join, 1, 8 warps: 32 rows of 16 splits 23, 13 us; 512 rows of 4 25, 24 us; 49248 rows of
// 2 173, 288 us).
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
  const int base = attn::split_base(a, s);
  const int i0 = hi > lo ? (lo - base) / p.chunk : 0;
  const int i1 = hi > lo ? (hi - 1 - base) / p.chunk + 1 : 0;
  float mo = -INFINITY;
  for (int i = i0 + lane; i < i1; i += 32) mo = fmaxf(mo, stat[i].y);
  mo = warp_max(mo);
  float l = 0.f, acc[kMaxD / 32] = {};
#pragma unroll 4
  for (int i = i0 + w; i < i1; i += NW) {
    const float2 x = stat[i];
    if (x.x == 0.f) continue;
    const float f = attn::ex2(x.y - attn::finite(mo));
    l += attn::times_ex2(x.x, x.y - attn::finite(mo));
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
cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t st,
                       Args... args) {
  if (grid.x > (unsigned)INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_any(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.c.H);
  const int64_t tiles = std::max<int64_t>(1, (rows + kAnyRows - 1) / kAnyRows);
  const dim3 grid((unsigned)attn_grid({tiles, a.b.B, p.splits}), (unsigned)a.c.H);
  return a.c.dtype == kInt8
             ? launch_pdl(attn_any_kernel<kInt8>, grid, kAnyWarps * 32, st, a, p, (int)tiles)
             : launch_pdl(attn_any_kernel<kFp8>, grid, kAnyWarps * 32, st, a, p, (int)tiles);
}

// The kernel of a call and how it splits the keys, from the call's sizes alone.
enum class Path { kAny, kDecode, kTc };

// Rows per key head up to which the streaming kernel is taken; it reads the codes
// once for 8 rows, the tensor core kernel once for 256 but with a dearer start.  16
// sequences of 8192 keys: 16 rows 125 and 165 us, 24 rows 163 and 165, 32 rows 217 and
// 165; 1 of 65536: 16 rows 69 and 88, 24 rows 97 and 88; 1 of 4096: 24 rows 17 and 22 us.
constexpr int64_t kDecodeRows = 24;

Path plan_path(int64_t D, int64_t page, int64_t rows) {
  if (rows > kDecodeRows && attn_tc_takes(D, page)) return Path::kTc;
  return attn_decode_takes(D, page) ? Path::kDecode : Path::kAny;
}

// Chunk of keys, and how many chunks the keys of one sequence's rows lie in.  With a
// window they are a stretch of window + max_q keys; it is split as finely as the
// workspace, which knows of no window, has room for.
void plan_splits(Path path, int64_t B, int64_t Hq, int64_t Hkv, int64_t max_q, int64_t max_kv,
                 int64_t window, AttnParts& p) {
  const int64_t g = Hq / Hkv;
  auto plan = [&](int64_t span) {
    p.chunk = path == Path::kTc       ? attn_tc_chunk(B, Hkv, max_q, g, span)
              : path == Path::kDecode ? attn_decode_chunk(B, Hkv, max_q * g, span)
                                      : attn_any_chunk(B, Hkv, max_q * g, span);
    p.splits = (int)std::max<int64_t>(1, (span + p.chunk - 1) / p.chunk);
  };
  plan(max_kv);
  const int64_t seen = window + max_q + 127;      // from a multiple of 128 on
  if (window == 0 || seen >= max_kv) return;
  const int64_t most = p.splits;
  plan(seen);
  if (p.splits <= most) return;
  p.chunk = (int)(((seen + most - 1) / most + 127) / 128 * 128);
  p.splits = (int)((seen + p.chunk - 1) / p.chunk);
}

}  // namespace

size_t attn_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            int64_t max_q, int64_t max_kv, int64_t page, int64_t bt) {
  (void)bt;
  AttnParts p{};
  plan_splits(plan_path(D, page, max_q * (Hq / Hkv)), B, Hq, Hkv, max_q, max_kv, 0, p);
  return attn_part_bytes(T * Hq, p.splits, D);
}

cudaError_t launch_attn_merge(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const int64_t items = a.b.T * a.Hq;
  const bool few = p.splits <= 4;
  const int64_t ctas = few ? (items + 3) / 4 : items;
  const dim3 grid((unsigned)std::min<int64_t>(ctas, (int64_t)INT32_MAX + 1));
  return few ? launch_pdl(attn_merge_kernel<1>, grid, 128, st, a, p)
             : launch_pdl(attn_merge_kernel<8>, grid, 256, st, a, p);
}

cudaError_t launch_kv_attention(const AttnArgs& a, void* ws, cudaStream_t st) {
  const int64_t items = a.b.T * a.Hq;
  const bool aligned = ((reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v)) &
                        15) == 0;
  const Path path = plan_path(a.c.D, a.c.page, (int64_t)a.max_q * (a.Hq / a.c.H));
  AttnParts p{};
  plan_splits(path, a.b.B, a.Hq, a.c.H, a.max_q, a.max_kv, a.window, p);
  if (p.splits > 1) {
    p.stat = static_cast<float*>(ws);
    p.o = p.stat + (2 * items * p.splits + 3) / 4 * 4;
  }
  cudaError_t e;
  if (!aligned || a.max_q == 0 || path == Path::kAny) e = launch_any(a, p, st);
  else e = path == Path::kTc ? launch_attn_tc(a, p, st) : launch_attn_decode(a, p, st);
  if (e == cudaSuccess && p.splits > 1) e = launch_attn_merge(a, p, st);
  return e;
}

}  // namespace bq
