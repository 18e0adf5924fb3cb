// kv_common.cuh -- device helpers shared by the cache write and the attention:
// which sequence a row or a unit of work belongs to, and the checks of what
// only the device can see (offsets, lengths, page numbers).
#pragma once

#include "bq_common.cuh"
#include "layer_ops.h"

namespace bq {
namespace kv {

// Largest b in [0, B) with key(b) <= x, for a nondecreasing key(); 0 if none.
// Called by whole warps: the lanes count side by side, one or two memory
// latencies instead of log2 B.
template <class F>
__device__ __forceinline__ int last_at_most(int B, int64_t x, F key) {
  if (B <= 1024) {
    int n = 0;
    for (int i = threadIdx.x & 31; i < B; i += 32) n += key(i) <= x ? 1 : 0;
    return max(0, __reduce_add_sync(0xffffffffu, n) - 1);
  }
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (key(mid) <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The sequence whose rows row t may belong to.
__device__ __forceinline__ int seq_of(const KvBatch& kb, int64_t t) {
  return last_at_most(kb.B, t, [&](int i) { return (int64_t)kb.off[i]; });
}

// Rows and length of sequence b; false if they cannot be used (then nothing
// of the sequence is read or written).
struct Seq {
  int row0, n, len;
};

__device__ __forceinline__ bool load_seq(const KvBatch& kb, int page, int b, Seq& s) {
  s.row0 = kb.off[b];
  const int end = kb.off[b + 1];
  s.n = end - s.row0;
  s.len = kb.lens[b];
  return s.row0 >= 0 && end >= s.row0 && (int64_t)end <= kb.T && s.len >= 0 &&
         (int64_t)s.len <= (int64_t)kb.table_cols * page;
}

// Page of token t of sequence b, or -1 if the table holds no page of the cache there.
__device__ __forceinline__ int64_t page_of(const KvBatch& kb, const KvCacheView& c, int b, int t) {
  const int32_t p = kb.table[(int64_t)b * kb.ld_table + t / c.page];
  return p >= 0 && (int64_t)p < c.n_pages ? (int64_t)p : -1;
}

// Units of work of the cache write: a unit is one block of bt tokens that the
// call adds tokens to.  Sequence b owns the unit numbers from
// floor(off[b] / bt) + 2 b on: its n tokens touch at most floor(n / bt) + 2
// blocks (n > 0), and floor((o + n) / bt) - floor(o / bt) >= floor(n / bt).
__device__ __forceinline__ int64_t first_unit(const KvBatch& kb, int bt, int b) {
  return (int64_t)(kb.off[b] / bt) + 2 * (int64_t)b;
}

inline int64_t unit_bound(int64_t T, int64_t B, int64_t bt) { return T / bt + 2 * B; }

}  // namespace kv
}  // namespace bq
