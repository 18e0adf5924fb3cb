// attn.h -- what the attention kernels share on the host side: the split of
// the keys over CTAs and its workspace, and the kernels' launchers.
#pragma once

#include <initializer_list>

#include "layer_ops.h"

namespace bq {

// Partial results of a row (token t, query head h), one per split: fp32 O[D] in
// units of 2^mo, and {l, mo}: mo is the split's reference for the row's y = z +
// lg2 vs (z the scores in log2 units, vs the value scales), l = sum 2^(z - mo).  A
// split that saw no key of the row has l = 0 and writes no O; one that holds no
// key that the row may see need not exist.
struct AttnParts {
  float* o;        // [T * Hq][splits][D]
  float* stat;     // [T * Hq][splits][2]
  int splits;      // 1: no partials, the kernel writes the result itself
  int chunk;       // keys of a split
};

inline size_t attn_part_bytes(int64_t rows, int splits, int64_t D) {
  if (splits <= 1) return 0;
  const size_t one = (size_t)splits * (size_t)(D + 2) * sizeof(float);
  if ((size_t)rows > kAttnMaxWorkspace / one) return kAttnMaxWorkspace + 1;
  return (size_t)rows * one + 16;
}

// A grid's CTAs from its factors; INT32_MAX + 1, which no launch takes, for more.
inline int64_t attn_grid(std::initializer_list<int64_t> factors) {
  int64_t n = 1;
  for (int64_t f : factors) {
    if (f > 0 && n > INT32_MAX / f) return (int64_t)INT32_MAX + 1;
    n *= f;
  }
  return n;
}

cudaError_t launch_attn_merge(const AttnArgs& a, const AttnParts& p, cudaStream_t st);

// Few rows per sequence and key head (decoding): attn_decode.cu.
bool attn_decode_takes(int64_t D, int64_t page);
int attn_decode_chunk(int64_t B, int64_t Hkv, int64_t rows, int64_t span);
cudaError_t launch_attn_decode(const AttnArgs& a, const AttnParts& p, cudaStream_t st);

// Many rows (prompts): attn_tc.cu.
bool attn_tc_takes(int64_t D, int64_t page);
int64_t attn_tc_tiles(int64_t max_q, int64_t group);
int attn_tc_chunk(int64_t B, int64_t Hkv, int64_t max_q, int64_t group, int64_t span);
cudaError_t launch_attn_tc(const AttnArgs& a, const AttnParts& p, cudaStream_t st);

}  // namespace bq
