// multi_k4.cu -- the multi-token decode over 4-bit K.
#include "multi_launch.cuh"

namespace lkv {
namespace multi {
cudaError_t launch_multi_k4(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s) { return launch_k<4>(a, D, p, s); }
}  // namespace multi
}  // namespace lkv
