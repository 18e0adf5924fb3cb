// attn_tc.cu -- attention over the paged 8-bit cache for many query rows per
// key head (prompts, chunks of prompts) on the 5th-generation tensor cores.
//
// A CTA holds 256 rows (tokens x heads of one key head's group) as two tiles of
// 128 and walks the keys in tiles of 128 tokens:
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread per row reads its 128
//                   scores from tensor memory, writes the weights back as fp16
//                   over them, and at the end divides the output row;
//   warps 8-11      converters: codes from memory (requested a tile ahead) to
//                   fp16 tiles in shared memory, K and V each twice buffered,
//                   and the tile's scales;
//   warp 12         issues the products: S_a = Q_a K^T (both operands in shared
//                   memory) and O_a += P_a V (P_a from tensor memory, V as it
//                   lies, its rows running along the reduction).
// The issue order O_0(j), S_0(j+1), O_1(j), S_1(j+1) keeps the tensor cores on
// one row tile while the other's softmax runs.
// Tensor memory: S_0, S_1 (128 columns each, P_a in the first 64 of S_a), O_0, O_1.
//
// Weights: with y = z + lg2 vs (z the score in log2 units, vs the value's block
// scale) and mo a bound on the row's y so far, the weight is 2^(y - mo), so the
// product with the bare codes is the value sum in units of 2^mo whatever the
// scales are, and l += weight / vs is the softmax sum in the same units: one
// exponential serves both.  Value scales below 2^-100 count as 2^-100 there.
// mo is raised (and O rescaled) only when y passes it by more than 8: weights
// stay below 2^8, far from fp16's end, and a rescale is rare.  The fp16
// rounding of a weight is half a step of 2^-11; scores, sums and O are fp32.
// Queries are scaled per row by a power of two and exact in fp16, as in
// attn_decode.cu.  Keys that no row of the CTA sees have zero codes and lg2 vs =
// -inf, so no stale byte enters a sum.
//
// Every wait is bounded (2 s); on expiry the CTA records a timeout in the
// device status word, drains its MMAs, frees its tensor memory and exits.
#include <algorithm>

#include "attn.h"
#include "attn_common.cuh"
#include "bq_common.cuh"
#include "kv_common.cuh"
#include "sm100.cuh"

namespace bq {

namespace {

using namespace attn;
using namespace sm100;

constexpr int kThreads = 512;
constexpr int BM = 128;                 // rows of a row tile
constexpr int BN = 128;                 // tokens of a key tile
// Register split (setmaxnreg): 256 x 184 + 128 x 104 + 128 x 40 = 65536, what 512
// threads at 128 each are launched with (checked before the first launch).
constexpr int kSoftRegs = 184, kConvRegs = 104, kMmaRegs = 40;
constexpr int kSplitRegs = 256 * kSoftRegs + 128 * kConvRegs + 128 * kMmaRegs;
static_assert(kSplitRegs <= 65536, "register file");
constexpr float kLazy = 8.0f;           // how far y may pass its reference (log2)
constexpr float kMinVs = 0x1p-100f;

template <int D>
struct Lay {
  static constexpr uint32_t kHalf = BN * 128;           // 128 rows of 64 fp16, 128-byte swizzle
  static constexpr uint32_t kTile = kHalf * (D / 64);
  static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kSc = 6 * kTile;
  static constexpr uint32_t kScSlot = 3 * BN * 4;       // cs, lv, iv of a tile
  static constexpr uint32_t kBar = kSc + 4 * kScSlot;
  static constexpr uint32_t kNumBars = 4 + 8 + 6 + 1;
  static constexpr uint32_t kTotal = 1024 + kBar + kNumBars * 8 + 16;
  static constexpr uint32_t kS = 0, kO = 2 * BN;        // tensor memory columns
};
static_assert(Lay<128>::kTotal <= 227u * 1024u, "shared memory");

// Byte of 16-byte unit `unit` (of 8) of row `row` in a half tile.
__device__ __forceinline__ uint32_t sw128(int row, int unit) {
  return (uint32_t)row * 128u + ((uint32_t)(unit ^ (row & 7)) << 4);
}

// Descriptor of a tile whose reduction runs along its rows: 64 columns (128
// bytes, 128-byte swizzle) x 8 rows are an atom; the next 8 rows are 1024 bytes
// on, the next 64 columns a half tile on.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(half_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// fp16 x fp16 -> fp32, M = 128; b_rows: B's reduction runs along its rows.
constexpr uint32_t idesc_f16(int N, bool b_rows) {
  return (1u << 4) | (b_rows ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(BM >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ void ld_shared2x2(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const AttnArgs a, const AttnParts parts, const int row_tiles) {
  using L = Lay<D>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the tiles with the most keys first: later rows see more
  int idx = blockIdx.x;
  const int hk = idx % a.c.H;
  idx /= a.c.H;
  const int split = idx % parts.splits;
  idx /= parts.splits;
  const int b = idx % a.b.B;
  const int rt = row_tiles - 1 - idx / a.b.B;
  const int g = a.Hq / a.c.H;
  kv::Seq s;
  if (!kv::load_seq(a.b, a.c.page, b, s) || s.n > a.max_q || s.len > a.max_kv) {
    if (tid == 0) record_status(a.status, kStatusBadInput, 0x721u);
    return;
  }
  const int R0 = rt * 2 * BM, n_rows = s.n * g;
  if (R0 >= n_rows) return;
  const bool two = R0 + BM < n_rows;      // the second row tile has rows
  const int i_lo = R0 / g, i_hi = min(s.n - 1, (R0 + 2 * BM - 1) / g);
  const Range all = tile_range(a, s, i_lo, i_hi);
  const Range part = split_range(all, split, parts.splits, BN);
  const int nt = part.hi > part.lo ? (part.hi - part.lo + BN - 1) / BN : 0;

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t *k_full = bars, *v_full = bars + 2, *k_empty = bars + 4, *v_empty = bars + 6,
           *sc_full = bars + 8, *s_full = bars + 12, *p_ready = bars + 14, *o_done = bars + 16,
           *drain = bars + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&k_full[i]), 4);
      mbar_init(smem_u32(&v_full[i]), 4);
      mbar_init(smem_u32(&k_empty[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), 1);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), 4);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sc_full[i]), 4);
    mbar_init(smem_u32(&drain[0]), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(smem_u32(tmem_slot), 512);

  // queries: a thread per row, scaled by a power of two, fp16, swizzled
  const int row = R0 + tid;               // of warps 0-7
  const bool row_on = warp < 8 && row < n_rows;
  float rd = 1.f;
  if (warp < 8) {
    const uint16_t* q = a.q + (int64_t)(s.row0 + (row_on ? row / g : 0)) * a.ldq +
                        (int64_t)(hk * g + (row_on ? row % g : 0)) * a.hq;
    const uint32_t dst = sbase + L::kQ + (uint32_t)(tid >> 7) * L::kTile;
    const bool vec = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
    float amax = 0.f;
    uint32_t w[D / 2];
#pragma unroll
    for (int u = 0; u < D / 8; ++u) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (row_on) {
        if (vec) {
          x = *reinterpret_cast<const uint4*>(q + 8 * u);
        } else {
          const uint16_t* e = q + 8 * u;
          x = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                         e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
        }
      }
      w[4 * u] = x.x; w[4 * u + 1] = x.y; w[4 * u + 2] = x.z; w[4 * u + 3] = x.w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[4 * u + e] << 16)),
                                 fabsf(__uint_as_float(w[4 * u + e] & 0xFFFF0000u))));
    }
    float up;
    row_power(amax, up, rd);
#pragma unroll
    for (int u = 0; u < D / 8; ++u) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        h[e] = pack_f16(__uint_as_float(w[4 * u + e] << 16) * up,
                        __uint_as_float(w[4 * u + e] & 0xFFFF0000u) * up);
      st_shared16(dst + (uint32_t)(u >> 3) * L::kHalf + sw128(tid & 127, u & 7), h[0], h[1], h[2],
                  h[3]);
    }
    fence_async_shared();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 12) {
    // ---------------- products ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kMmaRegs) : "memory");
    if (warp == 12 && lane == 0 && nt > 0) {
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) {
        ok = ok && mbar_wait(smem_u32(bar), parity, abort_flag, a.status, site);
        return ok;
      };
      auto scores = [&](int t, int j) {
        const uint32_t qa = sbase + L::kQ + (uint32_t)t * L::kTile;
        const uint32_t ka = sbase + L::kK + (uint32_t)(j & 1) * L::kTile;
#pragma unroll
        for (uint32_t h = 0; h < D / 64; ++h)
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            mma_ss(tmem + L::kS + t * BN, smem_desc_k128(qa + h * L::kHalf) + 2ull * k,
                   smem_desc_k128(ka + h * L::kHalf) + 2ull * k, idesc_f16(BN, false),
                   (h | k) != 0);
        mma_commit(smem_u32(&s_full[t]));
      };
      auto values = [&](int t, int j) {
        const uint32_t va = sbase + L::kV + (uint32_t)(j & 1) * L::kTile;
#pragma unroll
        for (uint32_t k = 0; k < BN / 16; ++k)
          mma_ts(tmem + L::kO + t * D, tmem + L::kS + t * BN + 8 * k,
                 desc_rows(va + 2048u * k, L::kHalf), idesc_f16(D, true), (j > 0 || k > 0));
        mma_commit(smem_u32(&o_done[t]));
      };
      if (wait(&k_full[0], 0, 0x731u)) {
        tc_fence_after();
        scores(0, 0);
        if (two) scores(1, 0);
        mma_commit(smem_u32(&k_empty[0]));
      }
      for (int j = 0; j < nt && ok; ++j) {
        const bool more = j + 1 < nt;
        if (!wait(&v_full[j & 1], (j >> 1) & 1, 0x732u)) break;
        if (!wait(&p_ready[0], j & 1, 0x733u)) break;
        tc_fence_after();
        values(0, j);
        if (!two) mma_commit(smem_u32(&v_empty[j & 1]));
        if (more) {
          if (!wait(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, 0x734u)) break;
          tc_fence_after();
          scores(0, j + 1);
        }
        if (two) {
          if (!wait(&p_ready[1], j & 1, 0x735u)) break;
          tc_fence_after();
          values(1, j);
          mma_commit(smem_u32(&v_empty[j & 1]));
          if (more) scores(1, j + 1);
        }
        if (more) mma_commit(smem_u32(&k_empty[(j + 1) & 1]));
      }
      if (!ok) {
        mma_commit(smem_u32(&drain[0]));
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&drain[0]), 0) && globaltimer() - t0 < 100000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---------------- converters ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kConvRegs) : "memory");
    constexpr int CH = D / 16;                   // 16-code chunks of a token
    constexpr int NL = CH;                       // loads of a thread: 128 CH chunks / 128 threads
    constexpr int TPL = 128 / CH;                // tokens that one load of all threads covers
    const int ct = tid - 256, ch = ct % CH, tk = ct / CH;
    const int page = a.c.page, bt = a.c.bt, nblk = page / bt;
    // pages of the tile's eight groups of 16 tokens, in lanes 0-7
    auto pages = [&](int t0) -> int {
      int64_t pg = -1;
      const int t = t0 + 16 * lane;
      if (lane < 8 && t < part.hi && t + 16 > all.lo) {
        pg = kv::page_of(a.b, a.c, b, t);
        if (pg < 0) record_status(a.status, kStatusBadInput, 0x722u);
      }
      return (int)pg;
    };
    auto load = [&](uint4 (&x)[NL], const uint8_t* codes, int t0, int pgs) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int tl = i * TPL + tk, t = t0 + tl;
        const int pg = __shfl_sync(0xffffffffu, pgs, tl >> 4);
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (pg >= 0 && t >= all.lo && t < part.hi)
          x[i] = ld_codes16(codes + (((int64_t)pg * a.c.H + hk) * page + t % page) * D + 16 * ch);
      }
    };
    auto store = [&](const uint4 (&x)[NL], uint32_t dst) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int tl = i * TPL + tk;
        uint32_t f[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) codes_to_f16<DT>(word_of(x[i], w), f[2 * w], f[2 * w + 1]);
        const uint32_t base = dst + (uint32_t)(ch >> 2) * L::kHalf;
        // lanes of the second half store their units in the other order: no bank conflict
        const bool odd = (ch >> 2) & 1;
        const int u = 2 * (ch & 3);
        st_shared16(base + sw128(tl, odd ? u + 1 : u), odd ? f[4] : f[0], odd ? f[5] : f[1],
                    odd ? f[6] : f[2], odd ? f[7] : f[3]);
        st_shared16(base + sw128(tl, odd ? u : u + 1), odd ? f[0] : f[4], odd ? f[1] : f[5],
                    odd ? f[2] : f[6], odd ? f[3] : f[7]);
      }
    };
    // scale of keys and values of token t0 + ct; ok: some row may see it
    auto scales = [&](int t0, int pgs, float& ks, float& vs) -> bool {
      const int t = t0 + ct, pg = __shfl_sync(0xffffffffu, pgs, ct >> 4);
      ks = 0.f;
      vs = 1.f;
      if (pg < 0 || t < all.lo || t >= part.hi) return false;
      const int64_t blk = ((int64_t)pg * a.c.H + hk) * nblk + (t % page) / bt;
      ks = a.c.ks[blk];
      vs = a.c.vs[blk];
      return true;
    };
    uint4 kx[NL], vx[NL];
    float ks = 0.f, vs = 1.f;
    bool on = false;
    if (nt > 0) {
      const int pgs = pages(part.lo);
      load(kx, a.c.k, part.lo, pgs);
      on = scales(part.lo, pgs, ks, vs);
      load(vx, a.c.v, part.lo, pgs);
    }
    for (int j = 0; j < nt; ++j) {
      const int t1 = part.lo + (j + 1) * BN;
      const bool more = j + 1 < nt;
      const int pgs = more ? pages(t1) : -1;
      const uint32_t parity = ((j >> 1) & 1) ^ 1;
      if (!warp_wait(smem_u32(&k_empty[j & 1]), parity, abort_flag, a.status, 0x736u)) break;
      float* sc = reinterpret_cast<float*>(smem + L::kSc + (uint32_t)(j & 3) * L::kScSlot);
      vs = fmaxf(vs, kMinVs);
      sc[ct] = ks * (a.scale * kLog2e);
      sc[BN + ct] = on ? lg2(vs) : -INFINITY;
      sc[2 * BN + ct] = on ? __fdividef(1.f, vs) : 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sc_full[j & 3]));
      store(kx, sbase + L::kK + (uint32_t)(j & 1) * L::kTile);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&k_full[j & 1]));
      if (more) {
        load(kx, a.c.k, t1, pgs);
        on = scales(t1, pgs, ks, vs);
      }
      if (!warp_wait(smem_u32(&v_empty[j & 1]), parity, abort_flag, a.status, 0x737u)) break;
      store(vx, sbase + L::kV + (uint32_t)(j & 1) * L::kTile);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&v_full[j & 1]));
      if (more) load(vx, a.c.v, t1, pgs);
    }
  } else {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs) : "memory");
    const int t = warp >> 2;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t st = tmem + quad + L::kS + t * BN, ot = tmem + quad + L::kO + t * D;
    const bool idle = t == 1 && !two;
    int row_lo = 0, row_hi = 0, in_lo, in_hi, unused;
    if (row_on) row_range(a, s, row / g, row_lo, row_hi);
    // tokens that every row of this row tile sees
    const int i0 = min(s.n - 1, (R0 + t * BM) / g), i1 = min(s.n - 1, (R0 + t * BM + BM - 1) / g);
    row_range(a, s, i1, in_lo, unused);
    row_range(a, s, i0, unused, in_hi);
    float mo = -INFINITY, l = 0.f;
    const uint64_t rd2 = pack2(rd, rd);
    bool ok = true;
    for (int j = 0; j < nt && !idle; ++j) {
      const int t0 = part.lo + j * BN;
      ok = warp_wait(smem_u32(&sc_full[j & 3]), (j >> 2) & 1, abort_flag, a.status, 0x738u) &&
           warp_wait(smem_u32(&s_full[t]), j & 1, abort_flag, a.status, 0x739u);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sc = sbase + L::kSc + (uint32_t)(j & 3) * L::kScSlot;
      uint64_t y[BN / 2];
      float mx = -INFINITY;
      {
        uint32_t r[2][32];               // two chunks of 32 scores in flight
        tmem_ld32(st, r[0]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_ld_wait();
          if (q < 3) tmem_ld32(st + 32 * (q + 1), r[(q + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint64_t c0, c1, v0, v1;
            ld_shared2x2(sc + 128 * q + 16 * i, c0, c1);
            ld_shared2x2(sc + 4 * BN + 128 * q + 16 * i, v0, v1);
            const uint32_t* w = &r[q & 1][4 * i];
            y[16 * q + 2 * i] = fma2(mul2((uint64_t)w[1] << 32 | w[0], c0), rd2, v0);
            y[16 * q + 2 * i + 1] = fma2(mul2((uint64_t)w[3] << 32 | w[2], c1), rd2, v1);
          }
        }
      }
      if (t0 < in_lo || t0 + BN > in_hi) {
        const int a0 = row_lo - t0, a1 = row_hi - t0;
#pragma unroll
        for (int i = 0; i < BN / 2; ++i)
          y[i] = pack2(2 * i >= a0 && 2 * i < a1 ? lo2(y[i]) : -INFINITY,
                       2 * i + 1 >= a0 && 2 * i + 1 < a1 ? hi2(y[i]) : -INFINITY);
      }
#pragma unroll
      for (int i = 0; i < BN / 2; ++i) mx = fmaxf(mx, fmaxf(lo2(y[i]), hi2(y[i])));
      const bool up = mx > mo + kLazy || (mo == -INFINITY && mx != -INFINITY);
      if (__any_sync(0xffffffffu, up)) {
        const float f = up ? ex2(mo - mx) : 1.f;     // 0 for the first keys seen
        if (up) mo = mx;
        l *= f;
        if (j > 0) {
          if (!warp_wait(smem_u32(&o_done[t]), (j - 1) & 1, abort_flag, a.status, 0x73Au)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t r[32];
            tmem_ld32(ot + 32 * q, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st32(ot + 32 * q, r);
          }
        }
      }
      const float neg = -finite(mo);
      const uint64_t neg2 = pack2(neg, neg);
      uint64_t l2 = pack2(l, 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint64_t v0, v1;
          ld_shared2x2(sc + 8 * BN + 256 * h + 16 * i, v0, v1);
          const uint64_t d0 = add2(y[32 * h + 2 * i], neg2), d1 = add2(y[32 * h + 2 * i + 1], neg2);
          const float p0 = ex2(lo2(d0)), p1 = ex2(hi2(d0)), p2 = ex2(lo2(d1)), p3 = ex2(hi2(d1));
          l2 = fma2(pack2(p0, p1), v0, l2);
          l2 = fma2(pack2(p2, p3), v1, l2);
          p[2 * i] = pack_f16(p0, p1);
          p[2 * i + 1] = pack_f16(p2, p3);
        }
        tmem_st32(st + 32 * h, p);
      }
      l = lo2(l2) + hi2(l2);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_ready[t]));
    }
    if (nt > 0 && !idle && ok)
      ok = warp_wait(smem_u32(&o_done[t]), (nt - 1) & 1, abort_flag, a.status, 0x73Bu);
    if (ok && !idle) {
      tc_fence_after();
      const int64_t tok = s.row0 + (row_on ? row / g : 0);
      const int head = hk * g + (row_on ? row % g : 0);
      const bool whole = parts.splits == 1;
      const int64_t pi = (tok * a.Hq + head) * parts.splits + split;
      const float f = whole ? (l == 0.f ? 0.f : __fdiv_rn(1.f, l)) : 1.f;
      uint16_t* out = a.out + tok * a.ldo + (int64_t)head * a.ho;
      const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t r[32];
        if (nt > 0) {
          tmem_ld32(ot + 32 * q, r);
          tmem_ld_wait();
        }
        if (!row_on) continue;
        if (!whole) {
          if (l != 0.f) {
            float4* o = reinterpret_cast<float4*>(parts.o + pi * D + 32 * q);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                 __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
          }
          continue;
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x0 = l == 0.f ? 0.f : __uint_as_float(r[2 * e]) * f;
          const float x1 = l == 0.f ? 0.f : __uint_as_float(r[2 * e + 1]) * f;
          w[e] = (uint32_t)float_to_bf16_bits(x0) | (uint32_t)float_to_bf16_bits(x1) << 16;
        }
        if (vec) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(out + 32 * q + 8 * e) =
                make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            out[32 * q + 2 * e] = (uint16_t)w[e];
            out[32 * q + 2 * e + 1] = (uint16_t)(w[e] >> 16);
          }
        }
      }
      if (row_on) {
        if (!whole)
          *reinterpret_cast<float4*>(parts.stat + 4 * pi) = make_float4(mo, l, mo, 0.f);
        else if (a.lse)
          a.lse[tok * a.Hq + head] =
              l == 0.f ? -INFINITY : (mo + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DT, int D>
cudaError_t launch_t(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  auto kern = attn_tc_kernel<DT, D>;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Lay<D>::kTotal);
    if (e != cudaSuccess) return e;
    // the register split must fit what the CTA is launched with, or the
    // softmax warps' setmaxnreg.inc would never be satisfied
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kThreads < kSplitRegs) return cudaErrorInvalidConfiguration;
    ready[dev] = true;
  }
  const int64_t tiles = attn_tc_tiles(a.max_q, a.Hq / a.c.H);
  const int64_t grid = tiles * a.b.B * p.splits * a.c.H;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<D>::kTotal;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, p, (int)tiles);
}

}  // namespace

int64_t attn_tc_tiles(int64_t max_q, int64_t group) {
  return (max_q * group + 2 * BM - 1) / (2 * BM);
}

bool attn_tc_takes(int64_t D, int64_t page) { return (D == 64 || D == 128) && page % 16 == 0; }

// One CTA runs on an SM: fill the 148, with at least 512 keys for a CTA.
int attn_tc_splits(int64_t B, int64_t Hkv, int64_t max_q, int64_t group, int64_t max_kv) {
  const int64_t units = std::max<int64_t>(1, B * Hkv * attn_tc_tiles(max_q, group));
  const int64_t most = std::max<int64_t>(1, max_kv / 512);
  return (int)std::max<int64_t>(1, std::min<int64_t>({148 / units, most, 64}));
}

cudaError_t launch_attn_tc(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  if (a.c.dtype == kInt8)
    return a.c.D == 64 ? launch_t<kInt8, 64>(a, p, st) : launch_t<kInt8, 128>(a, p, st);
  return a.c.D == 64 ? launch_t<kFp8, 64>(a, p, st) : launch_t<kFp8, 128>(a, p, st);
}

}  // namespace bq
