// attn_decode.cu -- attention over the paged 8-bit cache for few query rows
// per key head (decoding): bound by the stream of codes from memory.
//
// A CTA works on 8 rows (tokens x heads of one key head's group) and one part
// of the keys; its four warps take groups of 16 NG tokens in turn.
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
// More rows are more row tiles, side by side in the grid, whose codes come from L2:
// 16 x 8192 keys, 8 rows 73 us, 16 rows 124 us (two row tiles in one CTA, whose
// registers leave room for half as many warps: slower by a tenth).
// 64 x up to 8192 keys, 32 heads over 8 of dim 128: 142 us, 4.7 TB/s.
// A group's registers take the next group's codes as soon as the product that
// reads them has been issued, so a warp has about 4 KB under way and needs no
// second set of registers.
//
// Precision.  Codes are exact in fp16 (INT8: 1152 is subtracted from the
// fp16 number 1024 + 128 + q; e4m3: the hardware conversion).  A query row is
// scaled by a power of two to a largest magnitude of 2^14 .. 2^15 and is then
// exact in fp16 too (8 significant bits), but for elements below 2^-29 of the
// row's largest.  Scores and sums are fp32.  The weights are rounded to fp16; as in
// attn_tc.cu they include the value's block scale, 2^(y - mo) with y = z + lg2 vs,
// and l += weight / vs.  mo is set 11 below the row's largest y of the first keys a
// warp sees; later weights are formed with it as it stands, and only where one passes
// 2^15 (fp16 ends at 2^16) is mo raised and O rescaled, so that a group of keys
// costs no search for a maximum across lanes.  A weight is so off by at most half a
// step (2^-11 of it) within 2^-25 of the row's largest, and by at most 2^-36 of the
// largest below that.
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

constexpr int kWarps = 4, R = 8;        // R: rows of a CTA
// The reference of a row is set kBelow (log2) under the largest y, and raised when y
// passes it by kTop: see the precision note above.
constexpr float kBelow = 11.0f, kTop = 15.0f;

// One group of 16 tokens as it comes from memory.
template <int D, int UNI>
struct Group {
  uint4 k[2][D / 64];           // tokens r, r + 8
  uint32_t v[4][D / 32];        // tokens 2c, 2c + 1, 2c + 8, 2c + 9: D / 8 bytes each
  float ks[UNI ? 1 : 2], vs[UNI ? 1 : 2];   // scales of tokens r, r + 8 (UNI: of all)
};

// Where a group of 16 tokens lies: its page of the sequence and its first slot
// there, moved on by a fixed number of tokens without a division.
struct Place {
  int idx, slot;
};

// UNI: what of the tokens shares its scales and its page: 16 a group (block_t a
// multiple of 16), 32 a step of two groups (block_t a multiple of 32), 0 nothing.  2 x
// up to 131071 keys of dim 64, block_t 32: 69, 65, 57 us with 0, 16, 32.  Dim 128, with
// one group a step, has no use for it (64 x up to 8192 keys, block_t 64: 141.4, 142.6 us
// with 0, 16; 16 x 8192, block_t 16: 73, 75 us).
template <int DT, int D, int UNI>
__global__ void __launch_bounds__(kWarps * 32, 4)
attn_decode_kernel(const AttnArgs a, const AttnParts parts, const int row_tiles) {
  constexpr int NG = 128 / D;              // groups of 16 tokens in flight: 4 KB of codes a warp
  constexpr int KS = D / 16;               // k-steps of the score product
  constexpr int SC = UNI ? 1 : 2;
  constexpr int NP = UNI == 32 ? NG / 2 : NG, TP = 16 * NG / NP;   // places of a step, their tokens
  __shared__ float so[kWarps][R][D + 4];
  __shared__ float st[kWarps][R][2];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  // row tiles of the same keys side by side: the second one's codes come from L2
  const int rt = (int)(blockIdx.x % (unsigned)row_tiles);
  const int bs = (int)(blockIdx.x / (unsigned)row_tiles);
  const int split = bs % parts.splits, b = bs / parts.splits, hk = blockIdx.y;
  const int g = a.Hq / a.c.H, page = a.c.page;
  const int32_t* table = a.b.table + (int64_t)b * a.b.ld_table;
  constexpr int STEP = 16 * NG, STRIDE = kWarps * STEP;
  // without a window a split begins at a place known beforehand: its first pages
  // are asked for together with the sequence's length
  Place at[2][NP];                         // of the next two rounds' groups
  int32_t pg[2][NP];                       // their pages
  auto pages = [&](int t, int end) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const int64_t tu = (int64_t)t + h * STRIDE + TP * u;
        const int idx = (int)(tu / page);
        at[h][u] = {idx, (int)(tu - (int64_t)idx * page)};
        pg[h][u] = tu < end ? table[idx] : -1;
      }
  };
  const int64_t guess = (int64_t)split * parts.chunk + warp * STEP;
  const int held = a.b.table_cols * page;
  const bool early = a.window == 0 && guess < held;
  if (early) pages((int)guess, held);
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
  const Range part = split_range(all, split_base(a, s), split, parts.chunk);
  if (parts.splits > 1 && part.hi <= part.lo) return;      // the join does not look at it

  const int bt = a.c.bt, nblk = page / bt;
  const unsigned bt_inv = bt > 1 ? (unsigned)(0x100000000ull / (unsigned)bt + 1) : 0u;
  const int stride_idx = STRIDE / page, stride_slot = STRIDE % page;
  const uint8_t* kbase = a.c.k + r * D + 16 * c;
  const uint8_t* vbase = a.c.v + 2 * c * D + r * (D / 8);
  int t = part.lo + warp * STEP;
  if (!early) pages(t, part.hi);
  // (page, key head) of the next round's place u, which begins at token tok, or -1;
  // pages wholly before the first key in sight need not exist
  auto row_of = [&](int u, int tok) -> int64_t {
    if (tok >= part.hi) return -1;
    const int64_t p = pg[0][u];
    if (p >= 0 && p < a.c.n_pages) return p * a.c.H + hk;
    if (lane == 0 && tok + TP > all.lo) record_status(a.status, kStatusBadInput, 0x712u);
    return -1;
  };
  Group<D, UNI> G[NG];
  bool ok[NP];                             // the group's page exists (warp-uniform)
  auto load_k = [&](int u, int64_t ph) {
    const int slot = at[0][u * NP / NG].slot + (16 * u) % TP;
    if (ph < 0) return;
    const uint8_t* p = kbase + (ph * page + slot) * D;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) G[u].k[h][i] = ld_codes16(p + h * 8 * D + 64 * i);
    if ((16 * u) % TP) return;             // the place's scales are there already
#pragma unroll
    for (int h = 0; h < SC; ++h) {
      const unsigned x = (unsigned)(slot + (UNI ? 0 : r + 8 * h));
      G[u].ks[h] = a.c.ks[ph * nblk + (bt > 1 ? __umulhi(x, bt_inv) : x)];
    }
  };
  auto load_v = [&](int u, int64_t ph) {
    const int slot = at[0][u * NP / NG].slot + (16 * u) % TP;
    if (ph < 0) return;
    const uint8_t* p = vbase + (ph * page + slot) * D;
#pragma unroll
    for (int e = 0; e < 4; ++e) ld_codes<D>(p + ((e & 1) + 8 * (e >> 1)) * D, G[u].v[e]);
    if ((16 * u) % TP) return;
#pragma unroll
    for (int h = 0; h < SC; ++h) {
      const unsigned x = (unsigned)(slot + (UNI ? 0 : r + 8 * h));
      G[u].vs[h] = a.c.vs[ph * nblk + (bt > 1 ? __umulhi(x, bt_inv) : x)];
    }
  };
  int64_t ph[NP];
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    ph[u] = row_of(u, t + TP * u);
    ok[u] = ph[u] >= 0;
  }
#pragma unroll
  for (int u = 0; u < NG; ++u) {
    load_k(u, ph[u * NP / NG]);
    load_v(u, ph[u * NP / NG]);
  }

  // queries: row R0 + r of lane (r, c), dims 64 i + 16 c .. + 15
  uint32_t qf[KS][2];
  float rowfac[2];
  const int row = R0 + r;
  const bool on = row < n_rows;
  const uint16_t* q = a.q + (int64_t)(s.row0 + (on ? row / g : 0)) * a.ldq +
                      (int64_t)(hk * g + (on ? row % g : 0)) * a.hq;
  uint32_t w[KS][2];                     // bf16 pairs: word 2 (k-step) + e of the row's part
  const bool vec = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
#pragma unroll
  for (int ks = 0; ks < KS; ks += 2) {
    const uint16_t* p = q + 64 * (ks >> 2) + 16 * c + 4 * (ks & 3);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (on && vec) x = *reinterpret_cast<const uint4*>(p);
    else if (on)
      x = make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16,
                     p[4] | (uint32_t)p[5] << 16, p[6] | (uint32_t)p[7] << 16);
    w[ks][0] = x.x; w[ks][1] = x.y; w[ks + 1][0] = x.z; w[ks + 1][1] = x.w;
  }
  float amax = 0.f;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[ks][e] << 16)),
                               fabsf(__uint_as_float(w[ks][e] & 0xFFFF0000u))));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  float up, down;
  row_power(amax, up, down);
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      qf[ks][e] = pack_f16(__uint_as_float(w[ks][e] << 16) * up,
                               __uint_as_float(w[ks][e] & 0xFFFF0000u) * up);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    rowfac[j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j)) * (a.scale * kLog2e);
  }
  // every row of the tile sees the tokens of [in_lo, in_hi)
  int unused, in_lo, in_hi;
  row_range(a, s, i_hi, in_lo, unused);
  row_range(a, s, i_lo, unused, in_hi);

  float o[KS][4], l[2], mo[2];
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  mo[0] = mo[1] = -INFINITY;
  l[0] = l[1] = 0.f;

  for (; t < part.hi; t += STRIDE) {
    // the next round's pages are here; those of the one after it are asked for
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      at[0][u] = at[1][u];
      pg[0][u] = pg[1][u];
      at[1][u].idx += stride_idx;
      at[1][u].slot += stride_slot;
      if (at[1][u].slot >= page) {
        at[1][u].slot -= page;
        ++at[1][u].idx;
      }
      pg[1][u] = (int64_t)t + 2 * STRIDE + TP * u < part.hi ? table[at[1][u].idx] : -1;
    }
    bool whole = t >= in_lo && t + STEP <= in_hi;
#pragma unroll
    for (int u = 0; u < NP; ++u) whole = whole && ok[u];
    // scores, then y: e = 0, 1 rows 2c, 2c + 1 of token r; e = 2, 3 of token r + 8
    float y[NG][4];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[u][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t f[4];
        codes_to_f16<DT>(word_of(G[u].k[0][ks >> 2], ks & 3), f[0], f[2]);
        codes_to_f16<DT>(word_of(G[u].k[1][ks >> 2], ks & 3), f[1], f[3]);
        mma_f16(y[u], f, qf[ks]);
      }
    }
    float iv[NP][SC], lv[NP][SC];
#pragma unroll
    for (int u = 0; u < NP; ++u)
#pragma unroll
      for (int h = 0; h < SC; ++h) {
        const float vs = ok[u] ? value_scale(G[u * NG / NP].vs[h]) : 1.f;
        lv[u][h] = lg2(vs);
        iv[u][h] = rcp(vs);
      }
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      const int w = u * NP / NG;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[u][e] = fmaf(y[u][e], G[w * NG / NP].ks[UNI ? 0 : e >> 1] * rowfac[e & 1],
                           lv[w][UNI ? 0 : e >> 1]);
    }
    // keys of the group after next are under way from here on
    int64_t ph_next[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) ph_next[u] = row_of(u, t + STRIDE + TP * u);
#pragma unroll
    for (int u = 0; u < NG; ++u) load_k(u, ph_next[u * NP / NG]);
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // the range of row 2c + j, whose scores this lane has; rows behind the last
        // stand in for it (their queries are zero, nothing is written)
        int lo, hi;
        row_range(a, s, min((R0 + 2 * c + j) / g, s.n - 1), lo, hi);
#pragma unroll
        for (int u = 0; u < NG; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int tok = t + 16 * u + r + 8 * h;
            if (!ok[u * NP / NG] || tok < lo || tok >= hi) y[u][2 * h + j] = -INFINITY;
          }
      }
      // scales that belong to no key in sight may be anything, NaN among it
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int h = 0; h < SC; ++h) {
          const int tok = t + TP * u + (UNI ? TP - 1 : r + 8 * h);
          if (tok < all.lo || (!UNI && tok >= part.hi)) iv[u][h] = 0.f;
        }
    }
    // weights
    uint32_t pf[NG][2];
    bool far = false;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = y[0][j];
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) mx = fmaxf(mx, y[u][2 * h + j]);
      // the first keys of a row, or one far above its reference
      far = far || mx > mo[j] + kTop;
    }
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = mo[j];
#pragma unroll
        for (int u = 0; u < NG; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) mx = fmaxf(mx, y[u][2 * h + j]);
#pragma unroll
        for (int sh = 4; sh <= 16; sh <<= 1)
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        // another row's keys may have led here: a reference is never lowered
        mx = fmaxf(mx - kBelow, mo[j]);
        const float keep = ex2(mo[j] - finite(mx));
        l[j] = times_ex2(l[j], mo[j] - finite(mx));
        mo[j] = mx;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          o[i][j] *= keep;
          o[i][2 + j] *= keep;
        }
      }
    }
    const float ref[2] = {finite(mo[0]), finite(mo[1])};
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = ex2(y[u][e] - ref[e & 1]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        l[j] = UNI ? fmaf(p[j] + p[2 + j], iv[u * NP / NG][0], l[j])
                       : fmaf(p[j], iv[u * NP / NG][0],
                              fmaf(p[2 + j], iv[u * NP / NG][SC - 1], l[j]));
      pf[u][0] = transpose8(pack_f16(p[0], p[1]));
      pf[u][1] = transpose8(pack_f16(p[2], p[3]));
    }
    // values
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      if (!ok[u * NP / NG] || t + 16 * u < all.lo || t + 16 * u + 16 > part.hi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = t + 16 * u + 2 * c + (e & 1) + 8 * (e >> 1);
          const bool on = ok[u * NP / NG] && tok >= all.lo && tok < part.hi;
#pragma unroll
          for (int w = 0; w < D / 32; ++w) G[u].v[e][w] = on ? G[u].v[e][w] : 0u;
        }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t f0[4], f1[4];           // m-tiles 2w, 2w + 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = G[u].v[2 * h][w], z = G[u].v[2 * h + 1][w];
          codes_to_f16<DT>(__byte_perm(x, z, 0x5140), f0[2 * h], f0[2 * h + 1]);
          codes_to_f16<DT>(__byte_perm(x, z, 0x7362), f1[2 * h], f1[2 * h + 1]);
        }
        mma_f16(o[2 * w], f0, pf[u]);
        mma_f16(o[2 * w + 1], f1, pf[u]);
      }
      load_v(u, ph_next[u * NP / NG]);
    }
#pragma unroll
    for (int u = 0; u < NP; ++u) ok[u] = ph_next[u] >= 0;
  }

  // the four warps' parts, joined in warp order
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float x = l[j];
#pragma unroll
    for (int sh = 4; sh <= 16; sh <<= 1) x += __shfl_xor_sync(0xffffffffu, x, sh);
    const int row = 2 * c + j;
    if (r == 0) {
      st[warp][row][0] = x;
      st[warp][row][1] = mo[j];
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      so[warp][row][r * (D / 8) + 2 * i] = o[i][j];
      so[warp][row][r * (D / 8) + 2 * i + 1] = o[i][2 + j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * D; e += kWarps * 32) {
    const int row = e / D, d = e % D;
    if (R0 + row >= n_rows) break;
    float MO = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) MO = fmaxf(MO, st[w][row][1]);
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(st[w][row][1] - finite(MO));
      sum += times_ex2(st[w][row][0], st[w][row][1] - finite(MO));
      acc += so[w][row][d] * f;
    }
    const int64_t tok = s.row0 + (R0 + row) / g;
    const int head = hk * g + (R0 + row) % g;
    if (parts.splits == 1) {
      write_row(a, tok, head, d, sum, MO, acc);
    } else {
      const int64_t p = (tok * a.Hq + head) * parts.splits + split;
      if (sum != 0.f) parts.o[p * D + d] = acc;
      if (d == 0) *reinterpret_cast<float2*>(parts.stat + 2 * p) = make_float2(sum, MO);
    }
  }
}

template <int DT, int D, int UNI>
cudaError_t launch_t(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.c.H);
  const int64_t tiles = (rows + R - 1) / R;
  const int64_t x = attn_grid({tiles, a.b.B, p.splits});
  if (x > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)x, (unsigned)a.c.H);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<DT, D, UNI>, a, p, (int)tiles);
}

template <int DT, int D>
cudaError_t launch_d(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  if constexpr (D == 64) {
    if (a.c.bt % 32 == 0) return launch_t<DT, D, 32>(a, p, st);
    if (a.c.bt % 16 == 0) return launch_t<DT, D, 16>(a, p, st);
  }
  return launch_t<DT, D, 0>(a, p, st);
}

template <int DT>
cudaError_t launch_dt(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  return a.c.D == 64 ? launch_d<DT, 64>(a, p, st) : launch_d<DT, 128>(a, p, st);
}

}  // namespace

bool attn_decode_takes(int64_t D, int64_t page) {
  return (D == 64 || D == 128) && page % 16 == 0;
}

// Long keys: about sixteen CTAs for each of the 148 SMs.  A CTA's start and end cost
// as much as some ten groups of 16 keys of a warp, but few long ones end unevenly
// (8, 16, 24 CTAs an SM: 2 x up to 131071 keys of dim 64 58, 57, 67 us, 64 x up to
// 8192 keys of dim 128 161, 144, 144 us).  Where that would leave a CTA 512 keys or
// fewer, as many as run at once, four an SM, with 256 to 1152 keys each (chunks of 256,
// 512, 1152: 64 x 1152 keys 56, 46, 32 us, 32 x 1001 keys 30, 25, 30 us, 4 x 2001 keys
// 15, 19, 23 us).
int attn_decode_chunk(int64_t B, int64_t Hkv, int64_t rows, int64_t span) {
  const int64_t units = std::max<int64_t>(1, B * Hkv * ((rows + 7) / 8));
  int64_t c = units * span / (148 * 16);
  if (c <= 512) {
    const int64_t parts = std::max<int64_t>(1, 148 * 4 / units);
    c = std::min<int64_t>(1152, std::max<int64_t>(256, (span + parts - 1) / parts));
  }
  return (int)std::min<int64_t>(1 << 24, (c + 127) / 128 * 128);
}

cudaError_t launch_attn_decode(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  return a.c.dtype == kInt8 ? launch_dt<kInt8>(a, p, st) : launch_dt<kFp8>(a, p, st);
}

}  // namespace bq
