// multi.cuh -- argument block, launch shapes and launcher of the multi-token
// decode (internal to liblkv).
#pragma once
#include "lkv_kernels.cuh"

namespace lkv {
namespace multi {

constexpr int kMaxBatch = 4096;   // the tile prefix of every sequence sits in shared memory
constexpr int kMaxQueries = 64;   // new tokens of one sequence
constexpr int kMaxGrid = 1024;    // CTAs (one per SM)
constexpr int kSmemMax = 227 * 1024 - 2048;  // 2 KB for what is allocated statically

// 32-bit constants that a K group of a token brings (see multi_impl.cuh).
constexpr int centre_words(int kb) { return kb == 16 ? 0 : kb == 6 ? 4 : kb == 4 ? 2 : 1; }

// Shared memory of one instantiation: per warp a ring of stages (one tile
// each: K codes, K pairs, V codes, V pairs) and scratch.
struct Shape {
  int warps, tt, stages, stage, off_ksz, off_vc, off_vsz, scratch;
};

// Query rows of a unit come in n-tiles of 8; the accumulators of NT n-tiles
// take 32 NT registers a thread, which sets the warps of a CTA: 12 or 8 (16 with
// 128 registers each issue 1.5 times the instructions: 98 us against 78 at
// K6V4, B16, T8192).  Two
// stages per warp at least.  Tiles of 32 tokens (fewer, larger copies, and the
// work per tile shared by more tokens) if they fit beside all the warps, else
// 16 tokens, then fewer warps: wide rows need few warps to keep up with their
// bytes.
constexpr Shape shape_of(int D, int kb, int vb, int G, int nt) {
  const int ng = D / G;
  Shape s{};
  for (int warps = nt == 1 ? 12 : 8; warps >= 4; warps -= 4)
    for (int tt = 32; tt >= 16; tt /= 2) {
      const int sz = tt * ng * 8;
      s.warps = warps;
      s.tt = tt;
      s.off_ksz = tt * D * kb / 8;
      s.off_vc = s.off_ksz + (kb < 16 ? sz : 0);
      s.off_vsz = s.off_vc + tt * D * vb / 8;
      s.stage = (s.off_vsz + (vb < 16 ? sz : 0) + 127) / 128 * 128;
      s.scratch = (tt * 8 * nt * 4 + tt * ng * centre_words(kb) * 4 + 127) / 128 * 128;
      const int room = kSmemMax - (kMaxBatch + 1) * 4 - warps * s.scratch;
      s.stages = room / (warps * s.stage);
      if (s.stages > 4) s.stages = 4;
      if (s.stages >= 2) return s;
    }
  return s;
}

constexpr size_t smem_of(const Shape& s, int B) {
  return (size_t)s.warps * (s.stages * s.stage + s.scratch) + (size_t)(B + 1) * 4;
}

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
  float* pieces;            // [grid][warps] pieces
  float* cpieces;           // [grid][2] pieces
};

// Launch shape and workspace of one call.
struct MultiPlan {
  int nt, grid, units_max;  // units_max: of one sequence
  Shape sh;
  size_t ws_arrive, ws_pieces, ws_cpieces, ws_total;
};

void plan_multi(const MultiArgs& a, int D, MultiPlan& p);

// Dispatch on (V width, D, G, n-tiles) for one K width.
cudaError_t launch_multi_k2(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s);
cudaError_t launch_multi_k4(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s);
cudaError_t launch_multi_k6(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s);
cudaError_t launch_multi_k8(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s);
cudaError_t launch_multi_k16(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s);

}  // namespace multi
}  // namespace lkv
