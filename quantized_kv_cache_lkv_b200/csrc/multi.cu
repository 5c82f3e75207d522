// multi.cu -- launch plan of the multi-token decode (kernel: multi_impl.cuh).
#include "multi.cuh"

namespace lkv {
namespace multi {

void plan_multi(const MultiArgs& a, int D, MultiPlan& p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int rows = a.max_q * a.r;
  p.nt = rows <= 8 ? 1 : 2;
  p.sh = shape_of(D, a.kb, a.vb, a.kb == 16 && a.vb == 16 ? 64 : a.G, p.nt);
  p.grid = num_sms() < kMaxGrid ? num_sms() : kMaxGrid;
  p.units_max = a.Hkv * ((rows + 8 * p.nt - 1) / (8 * p.nt));
  const size_t piece = (size_t)8 * p.nt * (D + 2) * 4;
  p.ws_arrive = 256;  // behind the status word and the wait limit
  // at a fixed place: the counters are zero between calls, whatever the sizes
  p.ws_pieces = p.ws_arrive + kMaxGrid * 4;
  p.ws_cpieces = up(p.ws_pieces + (size_t)p.grid * p.sh.warps * piece);
  p.ws_total = up(p.ws_cpieces + (size_t)p.grid * 2 * piece);
}

}  // namespace multi
}  // namespace lkv
