// attn_decode.cu -- attention over the paged 8-bit cache for few query rows
// per key head (decoding): bound by the stream of codes from memory.
//
// A CTA works on up to 8 NR rows (tokens x heads of one key head's group) and
// one part of the keys; its four warps take groups of 16 NG tokens in turn.
// Codes go from global memory straight into the registers that the matrix
// instruction wants, with no pass through shared memory:
//   S^T = K Q^T   A = 16 tokens x 16 dims.  Which dims a k-step takes is free
//                 as long as Q agrees, so lane (r, c) = (lane / 4, lane % 4)
//                 loads 16 consecutive code bytes of tokens r and r + 8
//                 (4 lanes = 64 contiguous bytes), a word per k-step.
//   O^T = V^T P^T A = 16 dims x 16 tokens.  Lane (r, c) loads the D / 8 bytes of
//                 dims from r D / 8 on, of tokens 2c, 2c+1, 2c+8, 2c+9 (8 lanes =
//                 one row of D bytes); a byte permute pairs two tokens' codes.
//                 P^T is S^T's accumulator, transposed in registers (movmatrix).
// The next group's codes are requested before this group's are used.
//
// Precision.  Codes are exact in fp16 (INT8: 1152 is subtracted from the
// fp16 number 1024 + 128 + q; e4m3: the hardware conversion).  A query row is
// scaled by a power of two to a largest magnitude of 2^14 .. 2^15 and is then
// exact in fp16 too (8 significant bits), but for elements below 2^-29 of the
// row's largest.  Scores, running maxima and sums are fp32.  The weights are
// rounded to fp16 (half a step: 2^-11): they include the value's block scale,
// 2^(z + lg2 vs - mo) with mo the running maximum of that exponent, so the
// largest is 1 whatever the scales are; l = sum 2^(z - m) has its own maximum.
// Masked weights are set to zero, and the codes of values outside the rows'
// range are replaced by zero before the product, so no stale byte enters a sum.
#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"
#include "bq_common.cuh"
#include "kv_common.cuh"

namespace bq {

namespace {

using namespace attn;

constexpr int kWarps = 4;

template <int D>
struct VWords {                 // code bytes of one token that a lane holds: D / 8
  uint32_t w[D / 32];
};

template <int D>
__device__ __forceinline__ VWords<D> load_v(const uint8_t* p) {
  VWords<D> v;
  if constexpr (D == 64) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.w[0]), "=r"(v.w[1]) : "l"(p));
  } else {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "l"(p));
  }
  return v;
}

// One group of 16 tokens as it comes from memory.
template <int D>
struct Group {
  uint4 k[2][D / 64];           // tokens r, r + 8
  VWords<D> v[4];               // tokens 2c, 2c + 1, 2c + 8, 2c + 9
  float ks[2], vs[2];           // scales of tokens r, r + 8
  bool ok;                      // the group's page exists (warp-uniform)
};

template <int DT, int D, int NR>
__global__ void __launch_bounds__(kWarps * 32)
attn_decode_kernel(const AttnArgs a, const AttnParts parts, const int row_tiles) {
  constexpr int NG = 128 / D;              // groups of 16 tokens in flight: 4 KB of codes a warp
  constexpr int KS = D / 16;               // k-steps of the score product
  constexpr int R = 8 * NR;
  __shared__ float so[kWarps][R][D + 4];
  __shared__ float st[kWarps][R][3];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int split = (int)(blockIdx.x % (unsigned)parts.splits);
  const int bt_ = (int)(blockIdx.x / (unsigned)parts.splits);
  const int rt = bt_ % row_tiles, b = bt_ / row_tiles, hk = blockIdx.y;
  const int g = a.Hq / a.c.H;
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, b, s) || s.n > a.max_q || s.len > a.max_kv) {
    if (threadIdx.x == 0) record_status(a.status, kStatusBadInput, 0x711u);
    return;
  }
  const int R0 = rt * R, n_rows = s.n * g;
  if (R0 >= n_rows) return;
  // keys that some row of this tile sees, and this split's part of them
  const int i_lo = R0 / g, i_hi = min(s.n - 1, (R0 + R - 1) / g);
  const Range all = tile_range(a, s, i_lo, i_hi);
  const Range part = split_range(all, split, parts.splits, 16 * NG);

  // queries: row R0 + 8 nt + r of lane (r, c), dims 64 i + 16 c .. + 15
  uint32_t qf[NR][KS][2];
  float rowfac[NR][2];
  int row_lo[NR][2], row_hi[NR][2];        // of the rows 2c, 2c + 1 whose scores this lane gets
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
    const int row = R0 + 8 * nt + r;
    float v[KS][4], amax = 0.f;
    const bool on = row < n_rows;
    const uint16_t* q = a.q + (int64_t)(s.row0 + (on ? row / g : 0)) * a.ldq +
                        (int64_t)(hk * g + (on ? row % g : 0)) * a.hq;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[ks][e] = on ? bf16_bits_to_float(q[64 * (ks >> 2) + 16 * c + 4 * (ks & 3) + e]) : 0.f;
        amax = fmaxf(amax, fabsf(v[ks][e]));
      }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float up, down;
    row_power(amax, up, down);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qf[nt][ks][0] = pack_f16(v[ks][0] * up, v[ks][1] * up);
      qf[nt][ks][1] = pack_f16(v[ks][2] * up, v[ks][3] * up);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      rowfac[nt][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j)) * (a.scale * kLog2e);
      const int i = min((R0 + 8 * nt + 2 * c + j) / g, s.n - 1);
      row_range(a, s, i, row_lo[nt][j], row_hi[nt][j]);
    }
  }
  // every row of the tile sees the tokens of [in_lo, in_hi)
  int dummy, in_lo, in_hi;
  row_range(a, s, i_hi, in_lo, dummy);
  row_range(a, s, i_lo, dummy, in_hi);

  float o[NR][KS][4], m[NR][2], l[NR][2], mo[NR][2];
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    m[nt][0] = m[nt][1] = mo[nt][0] = mo[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  const int page = a.c.page, bt = a.c.bt, nblk = page / bt;
  const unsigned bt_inv = bt > 1 ? (unsigned)(0x100000000ull / (unsigned)bt + 1) : 0u;
  auto page_at = [&](int t) -> int64_t {
    return t < part.hi ? kv::page_of(a.b, a.c, b, t) : -1;
  };
  auto load = [&](Group<D>& G, int t0, int64_t pg) {
    G.ok = pg >= 0;
    if (!G.ok) {
      if (t0 < part.hi && lane == 0) record_status(a.status, kStatusBadInput, 0x712u);
      return;
    }
    const int64_t ph = pg * a.c.H + hk;
    const int in_page = t0 % page;
    const uint8_t* kp = a.c.k + (ph * page + in_page + r) * D + 16 * c;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) G.k[h][i] = ld_codes16(kp + h * 8 * D + 64 * i);
    const uint8_t* vp = a.c.v + (ph * page + in_page + 2 * c) * D + r * (D / 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) G.v[e] = load_v<D>(vp + ((e & 1) + 8 * (e >> 1)) * D);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned x = (unsigned)(in_page + r + 8 * h);
      const int64_t blk = ph * nblk + (bt > 1 ? __umulhi(x, bt_inv) : x);
      G.ks[h] = a.c.ks[blk];
      G.vs[h] = a.c.vs[blk];
    }
  };

  constexpr int STEP = 16 * NG;
  int t = part.lo + warp * STEP;
  Group<D> cur[NG];
  int64_t pg[NG];
#pragma unroll
  for (int u = 0; u < NG; ++u) load(cur[u], t + 16 * u, page_at(t + 16 * u));
#pragma unroll
  for (int u = 0; u < NG; ++u) pg[u] = page_at(t + kWarps * STEP + 16 * u);
  for (; t < part.hi; t += kWarps * STEP) {
    Group<D> nxt[NG];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      const int tn = t + kWarps * STEP + 16 * u;
      load(nxt[u], tn, pg[u]);
      pg[u] = page_at(tn + kWarps * STEP);
    }
    const bool whole = t >= in_lo && t + STEP <= in_hi;
    // scores
    float z[NR][NG][4];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[nt][u][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t f[4];
        codes_to_f16<DT>(word_of(cur[u].k[0][ks >> 2], ks & 3), f[0], f[2]);
        codes_to_f16<DT>(word_of(cur[u].k[1][ks >> 2], ks & 3), f[1], f[3]);
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) mma_f16(z[nt][u], f, qf[nt][ks]);
      }
    }
    // weights: e = 0, 1 rows 2c, 2c + 1 of token r; e = 2, 3 of token r + 8
    uint32_t pf[NR][NG][2];
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      float zo[NG][4], mx[2] = {-INFINITY, -INFINITY}, mxo[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ks = cur[u].ks[h], lv = lg2(cur[u].vs[h]);
          const int tok = t + 16 * u + r + 8 * h;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = z[nt][u][2 * h + j] * (ks * rowfac[nt][j]), y = x + lv;
            if (!whole || !cur[u].ok) {
              const bool on = cur[u].ok && tok >= row_lo[nt][j] && tok < row_hi[nt][j];
              x = on ? x : -INFINITY;
              y = on ? y : -INFINITY;
            }
            z[nt][u][2 * h + j] = x;
            zo[u][2 * h + j] = y;
            mx[j] = fmaxf(mx[j], x);
            mxo[j] = fmaxf(mxo[j], y);
          }
        }
      float keep[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int sh = 4; sh <= 16; sh <<= 1) {
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], sh));
          mxo[j] = fmaxf(mxo[j], __shfl_xor_sync(0xffffffffu, mxo[j], sh));
        }
        mx[j] = fmaxf(mx[j], m[nt][j]);
        mxo[j] = fmaxf(mxo[j], mo[nt][j]);
        l[nt][j] *= ex2(m[nt][j] - finite(mx[j]));
        keep[j] = ex2(mo[nt][j] - finite(mxo[j]));
        m[nt][j] = mx[j];
        mo[nt][j] = mxo[j];
        mx[j] = finite(mx[j]);
        mxo[j] = finite(mxo[j]);
      }
      if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] *= keep[e & 1];
      }
#pragma unroll
      for (int u = 0; u < NG; ++u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float p[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            l[nt][j] += ex2(z[nt][u][2 * h + j] - mx[j]);
            p[j] = ex2(zo[u][2 * h + j] - mxo[j]);
          }
          pf[nt][u][h] = transpose8(pack_f16(p[0], p[1]));
        }
      }
    }
    // values
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      if (t + 16 * u < part.lo || t + 16 * u + 16 > part.hi || !cur[u].ok || t + 16 * u < all.lo) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = t + 16 * u + 2 * c + (e & 1) + 8 * (e >> 1);
          const bool on = cur[u].ok && tok >= all.lo && tok < part.hi;
#pragma unroll
          for (int w = 0; w < D / 32; ++w) cur[u].v[e].w[w] = on ? cur[u].v[e].w[w] : 0u;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t f0[4], f1[4];           // m-tiles 2w, 2w + 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = cur[u].v[2 * h].w[w], y = cur[u].v[2 * h + 1].w[w];
          codes_to_f16<DT>(__byte_perm(x, y, 0x5140), f0[2 * h], f0[2 * h + 1]);
          codes_to_f16<DT>(__byte_perm(x, y, 0x7362), f1[2 * h], f1[2 * h + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          mma_f16(o[nt][2 * w], f0, pf[nt][u]);
          mma_f16(o[nt][2 * w + 1], f1, pf[nt][u]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NG; ++u) cur[u] = nxt[u];
  }

  // the four warps' parts, joined in warp order
#pragma unroll
  for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x = l[nt][j];
#pragma unroll
      for (int sh = 4; sh <= 16; sh <<= 1) x += __shfl_xor_sync(0xffffffffu, x, sh);
      const int row = 8 * nt + 2 * c + j;
      if (r == 0) {
        st[warp][row][0] = m[nt][j];
        st[warp][row][1] = x;
        st[warp][row][2] = mo[nt][j];
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        so[warp][row][r * (D / 8) + 2 * i] = o[nt][i][j];
        so[warp][row][r * (D / 8) + 2 * i + 1] = o[nt][i][2 + j];
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * D; e += kWarps * 32) {
    const int row = e / D, d = e % D;
    if (R0 + row >= n_rows) break;
    float M = -INFINITY, MO = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      M = fmaxf(M, st[w][row][0]);
      MO = fmaxf(MO, st[w][row][2]);
    }
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += st[w][row][1] * ex2(st[w][row][0] - finite(M));
      acc += so[w][row][d] * ex2(st[w][row][2] - finite(MO));
    }
    const int64_t tok = s.row0 + (R0 + row) / g;
    const int head = hk * g + (R0 + row) % g;
    if (parts.splits == 1) {
      write_row(a, tok, head, d, M, sum, MO, acc);
    } else {
      const int64_t p = (tok * a.Hq + head) * parts.splits + split;
      if (sum != 0.f) parts.o[p * D + d] = acc;
      if (d == 0)
        *reinterpret_cast<float4*>(parts.stat + 4 * p) = make_float4(M, sum, MO, 0.f);
    }
  }
}

template <int DT, int D, int NR>
cudaError_t launch_t(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.c.H);
  const int64_t tiles = (rows + 8 * NR - 1) / (8 * NR);
  const int64_t x = tiles * a.b.B * p.splits;
  if (x > INT32_MAX || tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)x, (unsigned)a.c.H);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<DT, D, NR>, a, p, (int)tiles);
}

template <int DT>
cudaError_t launch_dt(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const bool few = (int64_t)a.max_q * (a.Hq / a.c.H) <= 8;
  if (a.c.D == 64)
    return few ? launch_t<DT, 64, 1>(a, p, st) : launch_t<DT, 64, 2>(a, p, st);
  return few ? launch_t<DT, 128, 1>(a, p, st) : launch_t<DT, 128, 2>(a, p, st);
}

}  // namespace

bool attn_decode_takes(int64_t D, int64_t page) {
  return (D == 64 || D == 128) && page % 16 == 0;
}

// Enough CTAs to fill 148 SMs a few times over (sequences of different lengths
// even out), but at least 256 keys for a CTA.
int attn_decode_splits(int64_t B, int64_t Hkv, int64_t rows, int64_t max_kv) {
  const int64_t units = std::max<int64_t>(1, B * Hkv * ((rows + 15) / 16));
  const int64_t want = (148 * 12 + units - 1) / units;
  const int64_t most = std::max<int64_t>(1, max_kv / 256);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 256}));
}

cudaError_t launch_attn_decode(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  return a.c.dtype == kInt8 ? launch_dt<kInt8>(a, p, st) : launch_dt<kFp8>(a, p, st);
}

}  // namespace bq
