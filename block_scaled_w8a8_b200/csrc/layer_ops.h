// layer_ops.h -- host-side launcher declarations of the operators between two
// block-scaled linears of a decoder layer: RMS norm with an 8-bit output,
// rotary positions, the paged 8-bit cache of keys and values and the
// attention over it.  Launchers only enqueue; api.cu checks the arguments.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bq {

// dtype of NormArgs::dtype beyond kInt8 / kFp8: MXFP8 (E8M0 scale atoms).
constexpr int kMxFp8 = 2;

struct NormArgs {
  const uint16_t* x; int64_t ldx;
  const uint16_t* res; int64_t ldr;      // or nullptr
  const uint16_t* w; float w_off, eps;
  int64_t M, K, group;                   // group: 32 for MXFP8
  int dtype;                             // kInt8, kFp8 or kMxFp8
  uint8_t* q; int64_t ldq;
  float* s;                              // [ceil(K/group)][M]; MXFP8: unused
  uint8_t* sf;                           // MXFP8 scale atoms
  uint16_t* res_out; int64_t ldro;       // or nullptr
  uint16_t* h; int64_t ldh;              // or nullptr
};

// Widest row the norm takes: a row of bf16 values in shared memory.
constexpr int64_t kNormMaxK = 98304;

cudaError_t launch_rmsnorm_quant(const NormArgs& a, cudaStream_t st);

struct RopeArgs {
  const uint16_t* x; int64_t ldt, ldh;   // token and head strides (elements)
  uint16_t* out; int64_t ldot, ldoh;
  const int32_t* pos;
  const double* turns;                   // [rot / 2] turns per position
  int64_t T, H, D, rot;
  int interleaved;
  float mscale;
};

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st);

// A paged cache: codes [n_pages][H][page][D], scales [n_pages][H][page / bt].
struct KvCacheView {
  uint8_t* k; uint8_t* v;
  float* ks; float* vs;
  int64_t n_pages;
  int H, page, D, bt;
  int dtype;
};

// The sequences of one call: rows [off[b], off[b+1]) of the token arrays are
// the last tokens of sequence b, whose length (they included) is lens[b];
// token t of it lives in page table[b * ld_table + t / page].
struct KvBatch {
  const int32_t* off; const int32_t* lens; const int32_t* table;
  int64_t ld_table;
  int table_cols, B;
  int64_t T;
};

struct AppendArgs {
  KvCacheView c;
  KvBatch b;
  const uint16_t* k; int64_t ldk, hk;    // token and head strides (elements)
  const uint16_t* v; int64_t ldv, hv;
  unsigned* status;
};

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st);

struct AttnArgs {
  KvCacheView c;
  KvBatch b;
  const uint16_t* q; int64_t ldq, hq;    // token and head strides (elements)
  uint16_t* out; int64_t ldo, ho;
  float* lse;                            // [T][Hq] or nullptr
  int Hq;
  int max_q, max_kv;                     // bounds on every sequence's rows and length
  float scale;
  int causal;
  int window;                            // keys a row sees, 0 = all before it
  unsigned* status;
};

// Rows (tokens x heads of its group) of a sequence and key head that the kernels number.
constexpr int64_t kAttnMaxRows = 1 << 30;
constexpr size_t kAttnMaxWorkspace = (size_t)1 << 60;

// Above kAttnMaxWorkspace if it would be larger than that.
size_t attn_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            int64_t max_q, int64_t max_kv, int64_t page, int64_t bt);
cudaError_t launch_kv_attention(const AttnArgs& a, void* ws, cudaStream_t st);

}  // namespace bq
