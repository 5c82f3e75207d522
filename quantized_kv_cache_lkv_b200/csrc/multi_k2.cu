// multi_k2.cu -- the multi-token decode over 2-bit K.
#include "multi_launch.cuh"

namespace lkv {
namespace multi {
cudaError_t launch_multi_k2(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s) { return launch_k<2>(a, D, p, s); }
}  // namespace multi
}  // namespace lkv
