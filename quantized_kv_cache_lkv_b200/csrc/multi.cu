// multi.cu -- launch shapes of the multi-token decode (kernel: multi_impl.cuh).
#include "multi_impl.cuh"

namespace lkv {
namespace multi {

namespace {
size_t up(size_t x, size_t to) { return (x + to - 1) / to * to; }
constexpr size_t kSmemMax = 227 * 1024 - 1024;  // 1 KB for the statically allocated part
constexpr size_t kHeader = 256;                 // workspace: status, wait limit
}  // namespace

bool plan_multi(MultiArgs& a, int D, MultiPlan& p) {
  const int rows = a.max_q * a.r;
  p.nt = rows <= 8 ? 1 : 2;
  p.grid = num_sms() < kMaxGrid ? num_sms() : kMaxGrid;
  a.units_max = a.Hkv * ((rows + 8 * p.nt - 1) / (8 * p.nt));
  const int ng = D / a.G;
  auto layout = [&](int tt) {
    const int k = tt * D * a.kb / 8, v = tt * D * a.vb / 8, sz = tt * ng * 8;
    a.tt = tt;
    a.off_ksz = k;
    a.off_vc = a.off_ksz + (a.kb < 16 ? sz : 0);
    a.off_vsz = a.off_vc + v;
    // 16 bytes more: the last run of a row may be cut out of two words
    a.stage_bytes = (int)up((size_t)a.off_vsz + (a.vb < 16 ? sz : 0) + 16, 128);
  };
  // Two stages per warp at least.  Tiles of 32 tokens (fewer, larger copies)
  // if they fit beside all the warps, else 16, then fewer warps: wide rows
  // need few warps to keep up with their bytes.
  const int all = kWarpsFor(p.nt);
  bool fits = false;
  for (int warps = all; warps >= 4 && !fits; warps -= 4)
    for (int tt = 32; tt >= 16 && !fits; tt /= 2) {
      layout(tt);
      p.warps = warps;
      a.off_tr = kMaxWarps * kMaxStages * 8;
      a.off_first = a.off_tr + warps * 512 * p.nt;
      a.off_ring = (int)up((size_t)a.off_first + (size_t)(a.B + 1) * 4, 128);
      const size_t room = a.off_ring < (int)kSmemMax ? kSmemMax - a.off_ring : 0;
      a.stages = (int)(room / ((size_t)warps * a.stage_bytes));
      if (a.stages > kMaxStages) a.stages = kMaxStages;
      fits = a.stages >= 2;
    }
  if (!fits) return false;
  p.smem = (size_t)a.off_ring + (size_t)p.warps * a.stages * a.stage_bytes;
  const size_t piece = (size_t)8 * p.nt * (D + 2) * 4;
  p.ws_arrive = kHeader;
  // at a fixed place: the counters are zero between calls, whatever the sizes
  p.ws_pieces = p.ws_arrive + kMaxGrid * 4;
  p.ws_cpieces = up(p.ws_pieces + (size_t)p.grid * p.warps * 2 * piece, 256);
  p.ws_total = up(p.ws_cpieces + (size_t)p.grid * 2 * piece, 256);
  return true;
}

template <int D, int NT, bool G32>
static cudaError_t launch_t(const MultiArgs& a, const MultiPlan& p, cudaStream_t s) {
  auto kern = multi_kernel<D, NT, G32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, 32 * p.warps, p.smem, s>>>(a);
  return cudaGetLastError();
}

template <int D, int NT>
static cudaError_t launch_g(const MultiArgs& a, const MultiPlan& p, cudaStream_t s) {
  return a.G == 32 ? launch_t<D, NT, true>(a, p, s) : launch_t<D, NT, false>(a, p, s);
}

cudaError_t launch_multi(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s) {
  if (D == 64) return p.nt == 1 ? launch_g<64, 1>(a, p, s) : launch_g<64, 2>(a, p, s);
  return p.nt == 1 ? launch_g<128, 1>(a, p, s) : launch_g<128, 2>(a, p, s);
}

}  // namespace multi
}  // namespace lkv
