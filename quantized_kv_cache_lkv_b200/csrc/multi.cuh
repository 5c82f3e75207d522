// multi.cuh -- argument block and launcher of the multi-token decode
// (internal to liblkv).
#pragma once
#include "lkv_kernels.cuh"

namespace lkv {
namespace multi {

constexpr int kMaxWarps = 16;
constexpr int kMaxBatch = 8192;   // the tile prefix of every sequence sits in shared memory
constexpr int kMaxQueries = 64;   // new tokens of one sequence
constexpr int kMaxStages = 4;
constexpr int kMaxGrid = 1024;    // CTAs (one per SM)

// Query rows of a unit come in n-tiles of 8; the accumulators of NT n-tiles
// take 32 NT registers a thread, which sets the warps of a CTA.
constexpr int kWarpsFor(int nt) { return nt == 1 ? 16 : 12; }

struct MultiArgs {
  int B, Hq, Hkv, T_cap, G, r, max_q, n_rows, kb, vb;
  const int32_t* lens;
  const int32_t* cu_q;      // nullable: one new token per sequence
  const uint16_t* q;
  const uint8_t *kc, *vc;
  const float *ksz, *vsz;
  float scale, softcap;     // softcap 0: none
  int window;               // 0: none
  const float* slopes;      // nullable
  const int32_t* prefix;    // nullable
  const int32_t* starts;    // nullable
  float *out, *lse;         // lse nullable
  const int32_t* table;     // nullable: contiguous cache
  int pps, num_pages;
  // workspace
  int* status;
  const unsigned long long* timeout_ns;
  int* arrive;              // [kMaxGrid]: CTAs done with the unit that begins in a CTA and ends in a later one
  int units_max;            // units of a sequence at most
  float* pieces;            // [grid][warps][2] pieces
  float* cpieces;           // [grid][2] pieces
  // shared memory and ring
  int tt, stages, stage_bytes, off_ksz, off_vc, off_vsz, off_tr, off_first, off_ring;
};

// Launch shape and workspace of one call.
struct MultiPlan {
  int nt, warps, grid;
  size_t smem, ws_arrive, ws_pieces, ws_cpieces, ws_total;
};

// Fills the plan and the layout fields of a; false when the shape is not handled.
bool plan_multi(MultiArgs& a, int D, MultiPlan& p);
cudaError_t launch_multi(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s);

}  // namespace multi
}  // namespace lkv
