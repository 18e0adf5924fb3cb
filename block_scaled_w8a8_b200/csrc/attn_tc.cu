// attn_tc.cu -- attention over the paged 8-bit cache for many query rows per
// key head (prompts, chunks of prompts) on the 5th-generation tensor cores.
//
// A CTA holds 256 rows (tokens x heads of one key head's group) as two tiles of
// 128 and walks the keys in tiles of 128 tokens:
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread per row reads its 64
//                   scores of a block from tensor memory, writes the weights back as fp16
//                   over them, and at the end divides the output row;
//   warps 8-11      keys: codes from memory (requested a tile ahead) to fp16
//                   tiles in shared memory, twice buffered, and the scales of
//                   the tile's keys and values;
//   warps 13-15     values: the same;
//   warp 12         issues the products: S_a = Q_a K^T (both operands in shared
//                   memory) and O_a += P_a V (P_a from tensor memory, V as it
//                   lies, its rows running along the reduction).
// Scores are formed 64 keys at a time and each row tile has two such blocks, so
// that the next block's scores and the last one's value product run on the
// tensor cores while a block is in the softmax: neither waits for the other.
// Tensor memory: four score blocks of 64 columns (the weights in the first 32 of
// each), O_0, O_1.
//
// Weights: with y = z + lg2 vs (z the score in log2 units, vs the value's block
// scale) and mo a reference of the row, the weight is 2^(y - mo), so the product
// with the bare codes is the value sum in units of 2^mo whatever the scales are,
// and l += weight / vs is the softmax sum in the same units: one exponential
// serves both (value_scale in attn_common.cuh: for which scales).  Scores, sums and
// O are fp32; the weights are fp16, the type of the codes they are multiplied with.
// mo is set 8 below the largest y, and raised (and O rescaled) only when y passes it
// by more than 15: weights end at 2^15, fp16 at 2^16, and a rescale is rare.  So a
// weight is off by at most half a step (2^-11 of it) if it is within 2^-22 of the
// row's largest, and by at most 2^-33 of the largest below that: a long flat tail
// under one dominating key keeps its sum.
// Queries are scaled per row by a power of two and exact in fp16, as in
// attn_decode.cu.  Keys that no row of the CTA sees have zero codes and lg2 vs =
// -inf, so no stale byte enters a sum.
//
// Measured: a prompt of 8192 tokens (32 heads over 8, dim 128) 633 us, 869 TFLOP/s
// of the two products over the pairs that causality leaves, for some milliseconds of
// calls one behind the other; 677 us, 812 TFLOP/s, in a run of hundreds, in which the
// card's power limit lowers its clock.  Bound by the tensor cores as they are fed: with
// neither softmax nor conversion in the way the products alone take 508 us, since a
// score product of 64 keys reads as much of Q from shared memory as one of 128 would.
// 128 scores at a time halve that, but tensor memory then holds one block a row tile,
// so that the products wait for the softmax and the other way round (723 us).  The
// softmax adds 85 us, the conversion 60 us (measured at 645 us in all); a CTA's start
// and end cost about two key tiles of 2.7 us.
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
constexpr int SN = 64;                  // tokens of a score block
// Register split (setmaxnreg): 256 x 152 + 256 x 104 = 65536, what 512 threads at
// 128 each are launched with (checked before the first launch).
constexpr int kSoftRegs = 152, kConvRegs = 104;
constexpr int kSplitRegs = 256 * kSoftRegs + 256 * kConvRegs;
static_assert(kSplitRegs <= 65536, "register file");
// The reference of a row is set kBelow (log2) under the largest y, so that the largest
// weight is 2^8 and those down to 2^-22 of it have all of fp16's bits; y may then pass
// the reference by 15 before it is raised (fp16 ends at 2^16).
constexpr float kBelow = 8.0f, kTop = 15.0f;

template <int D>
struct Lay {
  static constexpr uint32_t kHalf = BN * 128;           // 128 rows of 64 fp16, 128-byte swizzle
  static constexpr uint32_t kTile = kHalf * (D / 64);
  static constexpr uint32_t kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kSc = 6 * kTile;
  static constexpr uint32_t kScSlot = 3 * BN * 4;       // cs, lv, iv of a tile
  static constexpr uint32_t kBar = kSc + 4 * kScSlot;
  static constexpr uint32_t kNumBars = 8 + 4 + 10 + 1 + 4;
  static constexpr uint32_t kTotal = 1024 + kBar + kNumBars * 8 + 16;
  static constexpr uint32_t kS = 0, kO = 2 * BN;        // tensor memory columns
};
static_assert(Lay<128>::kTotal <= 227u * 1024u, "shared memory");

// Byte of 16-byte unit `unit` (of 8) of row `row` in a half tile.
__device__ __forceinline__ uint32_t sw128(int row, int unit) {
  return (uint32_t)row * 128u + ((uint32_t)(unit ^ (row & 7)) << 4);
}

// Descriptors (128-byte swizzle, 8-row groups 1024 bytes apart): the low word
// has the address and the leading offset, the high word is a constant.  A tile
// read along its rows (K, Q) needs no leading offset; one whose reduction runs
// across its rows (V) has 64 columns x 8 rows as its atom, and the next 64
// columns a half tile on.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
  return ((saddr >> 4) & 0x3FFFu) | (leading >> 4) << 16;
}

// fp16 x fp16 -> fp32, M = 128; b_rows: B's reduction runs along its rows.
constexpr uint32_t idesc_f16(int N, bool b_rows) {
  return (1u << 4) | (b_rows ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(BM >> 4) << 24);
}

// The products are issued by a whole warp in step, one lane (`on`) doing it, so
// that descriptors and addresses stay in uniform registers: under a divergent
// branch every operand is moved there anew, 80 cycles an instruction, more than
// the product itself takes.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b),
      "r"(idesc), "r"(acc), "r"(kDescHi), "r"(on)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a),
      "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi), "r"(on)
      : "memory");
}

__device__ __forceinline__ void commit_if(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(on)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// tmem_ld32 into part of a longer array.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  sm100::tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(r));
}

__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)),
      "f"(__uint_as_float(c)));
  return d;
}

__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

// warp_wait, with the clock of its bound left alone while the wait is an ordinary
// one: reading %globaltimer costs more than most waits here last.
__device__ __forceinline__ bool wait_bar(const uint64_t* bar, uint32_t parity,
                                         volatile int* abort_flag, unsigned* status,
                                         unsigned site) {
  const uint32_t b = smem_u32(bar);
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
  return warp_wait(b, parity, abort_flag, status, site);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ void ld_shared4(const float4* p, float (&v)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(smem_u32(p)));
}

// Scales of a group of 16 tokens: y = c s + lv for a score product s of a row
// with power rd, and 1 / vs.  c is kept above zero, so that a masked score of
// -inf stays one (codes under a zero scale are zero, and so are their products); a
// NaN stays one too.
__device__ __forceinline__ void group_scales(const float4* sc, float rd, float& c, float& lv,
                                             float& iv) {
  const float4 x = *sc;
  c = max_nan(x.x * rd, 1e-37f);
  lv = x.y;
  iv = x.z;
}

// y of one token (own scales): c = cs, lv = lg2 vs.
__device__ __forceinline__ float token_y(uint32_t s, float cs, float rd, float lv) {
  return fmaf(__uint_as_float(s), max_nan(cs * rd, 1e-37f), lv);
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// UNI: aligned tokens that share their scales: 64 (a score block), 16 or 0, as
// block_t is a multiple of them.  With 16 the scales of a tile are eight entries
// {cs, lg2 vs, 1 / vs, -}, with 64 a score block has one of them.  Prompt of 8192,
// block_t 64: 902, 688, 631 us with 0, 16, 64; three chunks of 513 over 6000 keys,
// block_t 16: 215, 174 us with 0, 16.
template <int DT, int D, int UNI>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const AttnArgs a, const AttnParts parts, const int row_tiles) {
  using L = Lay<D>;
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);    // known to be uniform
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
  const Range part = split_range(all, split_base(a, s), split, parts.chunk);
  if (parts.splits > 1 && part.hi <= part.lo) return;      // the join does not look at it
  const int keys = max(part.hi - part.lo, 0);
  const int nt = (keys + BN - 1) / BN, nb = (keys + SN - 1) / SN;   // key tiles, score blocks

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t *k_full = bars, *v_full = bars + 2, *k_empty = bars + 4, *v_empty = bars + 6,
           *sc_full = bars + 8, *s_full = bars + 12, *p_ready = bars + 16, *o_done = bars + 20,
           *drain = bars + 22, *q_full = bars + 23, *o_last = bars + 25;
  // s_full, p_ready: [row tile][block & 1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&k_full[i]), 4);
      mbar_init(smem_u32(&v_full[i]), 3);
      mbar_init(smem_u32(&k_empty[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), 1);
      mbar_init(smem_u32(&q_full[i]), 4);
      mbar_init(smem_u32(&o_last[i]), 1);
      mbar_init(smem_u32(&o_done[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sc_full[i]), 4);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_ready[i]), 4);
    }
    mbar_init(smem_u32(&drain[0]), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(smem_u32(tmem_slot), 512);

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kConvRegs) : "memory");
  }
  if (warp == 12) {
    // ---------------- products ----------------
    const int n = __shfl_sync(0xffffffffu, nb, 0);
    const bool both = __shfl_sync(0xffffffffu, two ? 1 : 0, 0) != 0;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), on = elect_one();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) {
      ok = ok && wait_bar(bar, parity, abort_flag, a.status, site);
      return ok;
    };
    // low words of the descriptors; the high word is the same for all
    const uint32_t qd = desc_lo(sbase + L::kQ, 16), kd = desc_lo(sbase + L::kK, 16),
                   vd = desc_lo(sbase + L::kV, L::kHalf);
    auto scores = [&](int t, int i) {                // block i
      const uint32_t q = qd + (uint32_t)t * (L::kTile >> 4);
      const uint32_t k = kd + (uint32_t)((i >> 1) & 1) * (L::kTile >> 4) +
                         (uint32_t)(i & 1) * (SN * 128 >> 4);
#pragma unroll
      for (uint32_t h = 0; h < D / 64; ++h)
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
          mma_ss(tm + L::kS + 2 * SN * t + SN * (i & 1), q + h * (L::kHalf >> 4) + 2 * u,
                 k + h * (L::kHalf >> 4) + 2 * u, idesc_f16(SN, false), (h | u) != 0, on);
      commit_if(smem_u32(&s_full[2 * t + (i & 1)]), on);
    };
    auto values = [&](int t, int i) {
      const uint32_t v = vd + (uint32_t)((i >> 1) & 1) * (L::kTile >> 4) +
                         (uint32_t)(i & 1) * (SN * 128 >> 4);
#pragma unroll
      for (uint32_t u = 0; u < SN / 16; ++u)
        mma_ts(tm + L::kO + t * D, tm + L::kS + 2 * SN * t + SN * (i & 1) + 8 * u, v + 128u * u,
               idesc_f16(D, true), u > 0 || i > 0, on);
      commit_if(smem_u32(i == n - 1 ? &o_last[t] : &o_done[t]), on);
    };
    // a block's score buffer is free once the block two before it has been
    // through the value product, which is issued ahead of it
    auto next_scores = [&](int i) {
      if ((i & 1) == 0 && !wait(&k_full[(i >> 1) & 1], (i >> 2) & 1, 0x731u)) return;
      tc_fence_after();
      scores(0, i);
      if (both) scores(1, i);
      if ((i & 1) || i == n - 1) commit_if(smem_u32(&k_empty[(i >> 1) & 1]), on);
    };
    if (n > 0 && wait(&q_full[0], 0, 0x73Cu) && (!both || wait(&q_full[1], 0, 0x73Du)))
      next_scores(0);
    for (int i = 0; i < n && ok; ++i) {
      if (i + 1 < n) next_scores(i + 1);
      if ((i & 1) == 0) wait(&v_full[(i >> 1) & 1], (i >> 2) & 1, 0x732u);
      if (!wait(&p_ready[i & 1], (i >> 1) & 1, 0x733u)) break;
      tc_fence_after();
      values(0, i);
      if (both) {
        if (!wait(&p_ready[2 + (i & 1)], (i >> 1) & 1, 0x735u)) break;
        tc_fence_after();
        values(1, i);
      }
      if ((i & 1) || i == n - 1) commit_if(smem_u32(&v_empty[(i >> 1) & 1]), on);
    }
    if (!ok) {
      // products in flight end before the tensor memory is freed
      commit_if(smem_u32(&drain[0]), on);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(smem_u32(&drain[0]), 0) && globaltimer() - t0 < 100000000ull) {
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ---------------- converters: keys (warps 8-11), values (13-15) ----------------
    const bool is_k = warp < 12;
    const uint8_t* codes = is_k ? a.c.k : a.c.v;
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    const uint32_t dst0 = sbase + (is_k ? L::kK : L::kV);
    // A tile's eight groups of 16 tokens, each in one page, go round the warps: key
    // warp w has groups 2 w and 2 w + 1, value warp w groups w, w + 3 and w + 6.  A
    // lane's 16 codes are chunk lane / 8 of a half row of token lane % 8, so that
    // eight lanes store one 16-byte unit of eight different rows: no bank conflict.
    constexpr int GL = D / 32;                   // loads of a lane for a group
    constexpr int HV = D / 64;                   // half rows
    const int ch = lane >> 3, w = is_k ? warp & 3 : warp - 13;
    const int g0 = is_k ? 2 * w : w, gs = is_k ? 1 : 3, ng = is_k || w == 2 ? 2 : 3;
    const int page = a.c.page, nblk = page / a.c.bt;
    auto pages = [&](int t0, int (&pg)[3]) {
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        const int t = t0 + 16 * (g0 + h * gs);
        pg[h] = -1;
        if (h < ng && t < part.hi && t + 16 > all.lo) {
          pg[h] = (int)kv::page_of(a.b, a.c, b, t);
          if (pg[h] < 0 && lane == 0) record_status(a.status, kStatusBadInput, 0x722u);
        }
      }
    };
    auto load = [&](uint4 (&x)[3][GL], int t0, const int (&pg)[3]) {
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        const int tg = t0 + 16 * (g0 + h * gs);
        const uint8_t* p =
            codes + (((int64_t)pg[h] * a.c.H + hk) * page + tg % page + (lane & 7)) * D + 16 * ch;
#pragma unroll
        for (int e = 0; e < GL; ++e) {           // 8 tokens x 64 codes each
          const int t = tg + (lane & 7) + 8 * (e / HV);
          x[h][e] = make_uint4(0u, 0u, 0u, 0u);
          if (pg[h] >= 0 && t >= all.lo && t < part.hi)
            x[h][e] = ld_codes16(p + 8 * (e / HV) * D + 64 * (e % HV));
        }
      }
    };
    auto store = [&](const uint4 (&x)[3][GL], uint32_t dst) {
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        if (h >= ng) break;
#pragma unroll
        for (int e = 0; e < GL; ++e) {
          uint32_t f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            codes_to_f16<DT>(word_of(x[h][e], i), f[2 * i], f[2 * i + 1]);
          const uint32_t base = dst + (uint32_t)(e % HV) * L::kHalf;
          const int row_ = 16 * (g0 + h * gs) + (lane & 7) + 8 * (e / HV);
          st_shared16(base + sw128(row_, 2 * ch), f[0], f[1], f[2], f[3]);
          st_shared16(base + sw128(row_, 2 * ch + 1), f[4], f[5], f[6], f[7]);
        }
      }
    };
    // scales of token t0 + 32 w + lane (UNI: of its group, whole groups are on)
    float ks = 0.f, vs = 1.f;
    bool on = false;
    auto scales = [&](int t0, const int (&pg)[3]) {
      const int t = t0 + 32 * w + lane, p = lane < 16 ? pg[0] : pg[1];
      on = p >= 0 && (UNI || (t >= all.lo && t < part.hi));
      ks = 0.f;
      vs = 1.f;
      if (on) {
        const int64_t blk = ((int64_t)p * a.c.H + hk) * nblk + (t % page) / a.c.bt;
        ks = a.c.ks[blk];
        vs = a.c.vs[blk];
      }
    };
    uint4 x[3][GL];
    int pg[3];
    if (nt > 0) {
      pages(part.lo, pg);
      load(x, part.lo, pg);
      if (is_k) scales(part.lo, pg);
    }
    for (int j = 0; j < nt; ++j) {
      if (!wait_bar(&empty[j & 1], ((j >> 1) & 1) ^ 1, abort_flag, a.status, 0x736u))
        break;
      if (is_k) {
        float* sc = reinterpret_cast<float*>(smem + L::kSc + (uint32_t)(j & 3) * L::kScSlot);
        vs = value_scale(vs);
        const float cs = ks * (fabsf(a.scale) * kLog2e);
        const float lv = on ? lg2(vs) : -INFINITY, iv = on ? __fdividef(1.f, vs) : 0.f;
        if constexpr (UNI) {
          if ((lane & 15) == 0)
            reinterpret_cast<float4*>(sc)[2 * w + (lane >> 4)] = make_float4(cs, lv, iv, 0.f);
        } else {
          sc[32 * w + lane] = cs;
          sc[BN + 32 * w + lane] = lv;
          sc[2 * BN + 32 * w + lane] = iv;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sc_full[j & 3]));
      }
      const int t1 = part.lo + (j + 1) * BN;
      if (j + 1 < nt) pages(t1, pg);              // the next tile's pages, then its codes
      store(x, dst0 + (uint32_t)(j & 1) * L::kTile);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&full[j & 1]));
      if (j + 1 < nt) {
        load(x, t1, pg);
        if (is_k) scales(t1, pg);
      }
    }
  } else if (warp < 8) {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs) : "memory");
    const int t = warp >> 2;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ot = tmem + quad + L::kO + t * D;
    const bool idle = t == 1 && !two;
    // queries: a thread per row, scaled by a power of two, fp16, swizzled
    const int row = R0 + tid;
    const bool row_on = row < n_rows;
    float rd = 1.f;
    if (!idle) {
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
      if (a.scale < 0.f) up = -up;          // scores then only take the scale's magnitude
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
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_full[t]));
    }
    int row_lo = 0, row_hi = 0, in_lo, in_hi, unused;
    if (row_on) row_range(a, s, row / g, row_lo, row_hi);
    // tokens that every row of this row tile sees
    const int i0 = min(s.n - 1, (R0 + t * BM) / g), i1 = min(s.n - 1, (R0 + t * BM + BM - 1) / g);
    row_range(a, s, i1, in_lo, unused);
    row_range(a, s, i0, unused, in_hi);
    float mo = -INFINITY, l = 0.f;
    bool ok = true;
    for (int i = 0; i < nb && !idle; ++i) {
      const int t0 = part.lo + i * SN, j = i >> 1;       // block i of tile j
      const uint32_t st = tmem + quad + L::kS + 2 * SN * t + SN * (i & 1);
      ok = ((i & 1) ||
            wait_bar(&sc_full[j & 3], (j >> 2) & 1, abort_flag, a.status, 0x738u)) &&
           wait_bar(&s_full[2 * t + (i & 1)], j & 1, abort_flag, a.status, 0x739u);
      if (!ok) break;
      tc_fence_after();
      // UNI: the block's four groups (alike with 64); otherwise its 64 entries of each of
      // three arrays
      const float4* sc4 =
          reinterpret_cast<const float4*>(smem + L::kSc + (uint32_t)(j & 3) * L::kScSlot) +
          (UNI ? 4 : SN / 4) * (i & 1);
      const bool masked = t0 < in_lo || t0 + SN > in_hi;
      float4 one;                          // UNI == SN: the block's scales
      if constexpr (UNI == SN) {
        group_scales(sc4 + (t0 < all.lo ? min(3, (all.lo - t0) >> 4) : 0), rd, one.x, one.y, one.z);
      }
      const int a0 = row_lo - t0, a1 = row_hi - t0;
      // all scores at once: a load's latency is near that of a whole row
      uint32_t y[SN];
#pragma unroll
      for (int q = 0; q < SN / 32; ++q) tmem_ld32(st + 32 * q, y + 32 * q);
      tmem_ld_wait();
      if constexpr (!UNI) {
#pragma unroll
        for (int e4 = 0; e4 < SN / 4; ++e4) {
          float c[4], v[4];
          ld_shared4(sc4 + e4, c);
          ld_shared4(sc4 + BN / 4 + e4, v);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[4 * e4 + e] = __float_as_uint(token_y(y[4 * e4 + e], c[e], rd, v[e]));
        }
      }
      if (masked) {                        // -inf outside the row's range
#pragma unroll
        for (int i = 0; i < SN; ++i)
          if (i < a0 || i >= a1) y[i] = 0xFF800000u;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < SN / 16; ++q) {
        float m0 = max3(y[16 * q], y[16 * q + 1], y[16 * q + 2]);
        float m1 = max3(y[16 * q + 3], y[16 * q + 4], y[16 * q + 5]);
#pragma unroll
        for (int i = 6; i < 14; i += 4) {
          m0 = max3(__float_as_uint(m0), y[16 * q + i], y[16 * q + i + 1]);
          m1 = max3(__float_as_uint(m1), y[16 * q + i + 2], y[16 * q + i + 3]);
        }
        m0 = max3(__float_as_uint(m0), y[16 * q + 14], y[16 * q + 15]);
        if constexpr (UNI == 16) {
          float c, lv, iv;
          group_scales(sc4 + q, rd, c, lv, iv);
          mx = fmaxf(mx, fmaf(c, fmaxf(m0, m1), lv));
        } else {
          mx = max3(__float_as_uint(mx), __float_as_uint(m0), __float_as_uint(m1));
        }
      }
      if constexpr (UNI == SN) mx = fmaf(one.x, mx, one.y);
      const bool up = mx > mo + kTop;      // true for the first keys seen
      if (__any_sync(0xffffffffu, up)) {
        const float d = up ? mo - (mx - kBelow) : 0.f, f = ex2(d);   // 0 for the first keys seen
        if (up) mo = mx - kBelow;
        l = times_ex2(l, d);
        if (i > 0) {
          if (!wait_bar(&o_done[t], (i - 1) & 1, abort_flag, a.status, 0x73Au)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t r[16];
            tmem_ld16(ot + 16 * q, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st16(ot + 16 * q, r);
          }
        }
      }
      const float neg = -finite(mo);
      uint64_t sums[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < SN / 32; ++h) {
        uint32_t p[16];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t* w = y + 32 * h + 16 * u;
          if constexpr (UNI) {
            float c, lv, iv;
            if constexpr (UNI == SN) {
              c = one.x;
              lv = one.y;
              iv = one.z;
            } else {
              group_scales(sc4 + 2 * h + u, rd, c, lv, iv);
            }
            const uint64_t c2 = pack2(c, c), b2 = pack2(lv + neg, lv + neg);
            uint64_t& sum = sums[u];
            if (UNI != SN) sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint64_t d = fma2((uint64_t)w[2 * i + 1] << 32 | w[2 * i], c2, b2);
              const float p0 = ex2(lo2(d)), p1 = ex2(hi2(d));
              sum = add2(sum, pack2(p0, p1));
              p[8 * u + i] = pack_f16(p0, p1);
            }
            if (UNI != SN) l = fmaf(lo2(sum) + hi2(sum), iv, l);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float iv[4], x[4];
              ld_shared4(sc4 + BN / 2 + 8 * h + 4 * u + i, iv);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[e] = ex2(__uint_as_float(w[4 * i + e]) + neg);
                l = fmaf(x[e], iv[e], l);
              }
              p[8 * u + 2 * i] = pack_f16(x[0], x[1]);
              p[8 * u + 2 * i + 1] = pack_f16(x[2], x[3]);
            }
          }
        }
        tmem_st16(st + 16 * h, p);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if constexpr (UNI == SN) {
        const uint64_t sum = add2(sums[0], sums[1]);
        l = fmaf(lo2(sum) + hi2(sum), one.z, l);
      }
      if (lane == 0) mbar_arrive(smem_u32(&p_ready[2 * t + (i & 1)]));
    }
    if (nt > 0 && !idle && ok)
      ok = wait_bar(&o_last[t], 0, abort_flag, a.status, 0x73Bu);
    if (ok && !idle) {
      tc_fence_after();
      // O goes out 32 columns at a time by way of this row tile's queries, which no
      // product reads any more: a lane stores its row's 16-byte units, eight lanes
      // then write one row's 128 bytes side by side.
      const bool whole = parts.splits == 1;
      const float f = whole ? (l == 0.f ? 0.f : __fdiv_rn(1.f, l)) : 1.f;
      const bool vec = ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)(2 * a.ldo) |
                         (uintptr_t)(2 * a.ho)) & 7) == 0;
      const uint32_t stage = sbase + L::kQ + (uint32_t)t * L::kTile + (uint32_t)(warp & 3) * 4096u;
      const int unit = lane & 7, first = R0 + 32 * warp + (lane >> 3);
      int64_t at[8];                       // of rows first + 4 i, or -1
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rw = first + 4 * i;
        const int64_t tok = s.row0 + rw / g, head = hk * g + rw % g;
        at[i] = rw >= n_rows ? -1
                : whole      ? tok * a.ldo + head * a.ho
                             : ((tok * a.Hq + head) * parts.splits + split) * D;
      }
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t r[32];
        if (nt > 0) {
          tmem_ld32(ot + 32 * q, r);
          tmem_ld_wait();
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = l == 0.f ? 0.f : __uint_as_float(r[4 * u + e]) * f;
          st_shared16(stage + sw128(lane, u), __float_as_uint(x[0]), __float_as_uint(x[1]),
                      __float_as_uint(x[2]), __float_as_uint(x[3]));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(
              smem + (stage - sbase) + sw128(4 * i + (lane >> 3), unit));
          if (at[i] < 0) continue;
          const int64_t d = at[i] + 32 * q + 4 * unit;
          if (!whole) {
            *reinterpret_cast<float4*>(parts.o + d) = x;
          } else if (vec) {
            uint2 w;
            w.x = (uint32_t)float_to_bf16_bits(x.x) | (uint32_t)float_to_bf16_bits(x.y) << 16;
            w.y = (uint32_t)float_to_bf16_bits(x.z) | (uint32_t)float_to_bf16_bits(x.w) << 16;
            *reinterpret_cast<uint2*>(a.out + d) = w;
          } else {
            a.out[d] = float_to_bf16_bits(x.x);
            a.out[d + 1] = float_to_bf16_bits(x.y);
            a.out[d + 2] = float_to_bf16_bits(x.z);
            a.out[d + 3] = float_to_bf16_bits(x.w);
          }
        }
        __syncwarp();
      }
      if (row_on) {
        const int64_t tok = s.row0 + row / g, head = hk * g + row % g;
        if (!whole)
          *reinterpret_cast<float2*>(parts.stat +
                                     2 * ((tok * a.Hq + head) * parts.splits + split)) =
              make_float2(l, mo);
        else if (a.lse)
          a.lse[tok * a.Hq + head] =
              l == 0.f ? -INFINITY : (mo + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DT, int D, int UNI>
cudaError_t launch_t(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  auto kern = attn_tc_kernel<DT, D, UNI>;
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
  const int64_t grid = attn_grid({tiles, a.b.B, p.splits, a.c.H});
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

template <int DT>
cudaError_t launch_dt(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  const int uni = a.c.bt % SN == 0 ? SN : a.c.bt % 16 == 0 ? 16 : 0;
  if (a.c.D == 64)
    return uni == SN ? launch_t<DT, 64, SN>(a, p, st)
           : uni     ? launch_t<DT, 64, 16>(a, p, st)
                     : launch_t<DT, 64, 0>(a, p, st);
  return uni == SN ? launch_t<DT, 128, SN>(a, p, st)
         : uni     ? launch_t<DT, 128, 16>(a, p, st)
                   : launch_t<DT, 128, 0>(a, p, st);
}

}  // namespace

int64_t attn_tc_tiles(int64_t max_q, int64_t group) {
  return (max_q * group + 2 * BM - 1) / (2 * BM);
}

bool attn_tc_takes(int64_t D, int64_t page) { return (D == 64 || D == 128) && page % 16 == 0; }

// One CTA runs on an SM, so a call takes as many rounds of CTAs as units / 148,
// rounded up; splitting the keys evens the rounds out.  In units of a key tile
// (2.7 us measured): a CTA's start and end are about two, and the partial rows of a
// split, 1 KB a row written and read, units * 256 KB at 6.5 TB/s.
int attn_tc_chunk(int64_t B, int64_t Hkv, int64_t max_q, int64_t group, int64_t span) {
  const int64_t units = std::max<int64_t>(1, B * Hkv * attn_tc_tiles(max_q, group));
  const int64_t tiles = std::max<int64_t>(1, (span + BN - 1) / BN);
  int64_t best = 1;
  double least = 0.0;
  for (int64_t p = 1; p <= 64 && (p == 1 || tiles / p >= 4); ++p) {
    const int64_t per = (tiles + p - 1) / p;
    const double cost = (double)((units * p + 147) / 148) * (double)(per + 2) +
                        (p > 1 ? 1.0 + 0.0144 * (double)(units * p) : 0.0);
    if (p == 1 || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best == 1 ? 1 << 30 : (int)((tiles + best - 1) / best * BN);
}

cudaError_t launch_attn_tc(const AttnArgs& a, const AttnParts& p, cudaStream_t st) {
  return a.c.dtype == kInt8 ? launch_dt<kInt8>(a, p, st) : launch_dt<kFp8>(a, p, st);
}

}  // namespace bq
