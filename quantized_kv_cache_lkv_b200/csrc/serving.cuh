// serving.cuh -- argument blocks and launchers of the page plan, the rotary
// tables and the norm + rotation + append (internal to liblkv).
#pragma once
#include "lkv_kernels.cuh"

namespace lkv {

constexpr int kPlanMaxBatch = 16384;  // two prefix sums of every sequence in shared memory

struct PlanArgs {
  int B, pps, num_pages, n_cap, free_cap;
  const int32_t *lens, *n_new, *free_pages, *free_count;
  int32_t *table, *new_lens, *cu, *positions, *token_seq;
  int64_t* slots;
  int32_t *free_left, *status;
  bool wide;  // positions, token_seq and slots are 16-byte aligned
};

struct RopeTableArgs {
  int kind, half, rows;
  double base, factor, low, high, orig, attn;
  float* table;  // [rows][half][2]
};

struct RopeAppendArgs {
  int n_cap, Hq, Hkv, num_pages, page_tokens, G, kb, vb, rot;
  const int32_t* n_tokens;  // nullable
  const int32_t* positions;
  const int64_t* slots;
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements from token to token
  const uint16_t *q_weight, *k_weight;     // nullable
  float eps, one;                          // one = 1.0f, as in QuantizeArgs
  bool reciprocal;                         // quantizer multiplies by reciprocals
  const float* table;
  int table_rows;
  uint16_t* q_out;
  uint8_t *k_codes, *v_codes;
  float *k_sz, *v_sz;
  int iters;                               // row batches of one warp's item
  bool split;                              // keys and values as items of their own
  int ahead;                               // tokens from an item to the one it prefetches (0: none)
};

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s);
cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t s);
cudaError_t launch_rope_append(const RopeAppendArgs& a, int D, bool interleaved, cudaStream_t s);

}  // namespace lkv
