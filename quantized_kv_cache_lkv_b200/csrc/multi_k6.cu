// multi_k6.cu -- the multi-token decode over 6-bit K.
#include "multi_launch.cuh"

namespace lkv {
namespace multi {
cudaError_t launch_multi_k6(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s) { return launch_k<6>(a, D, p, s); }
}  // namespace multi
}  // namespace lkv
