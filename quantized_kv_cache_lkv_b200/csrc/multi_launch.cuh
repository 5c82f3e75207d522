// multi_launch.cuh -- dispatch of one K width of the multi-token decode.
#pragma once
#include "multi_impl.cuh"

namespace lkv {
namespace multi {

template <int D, int KB, int VB, int G, int NT>
cudaError_t launch_c(const MultiArgs& a, const MultiPlan& p, cudaStream_t s) {
  using C = Cfg<D, KB, VB, G, NT>;
  static_assert(C::STAGES >= 2, "a ring of two stages");
  // the limit belongs to the kernel and not to the call: what the largest batch needs, so that calls of other batches from
  // other threads do not lower it between this line and the launch
  const cudaError_t e =
      cudaFuncSetAttribute(multi_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(p.sh, kMaxBatch));
  if (e != cudaSuccess) return e;
  multi_kernel<C><<<p.grid, 32 * C::WARPS, smem_of(p.sh, a.B), s>>>(a);
  return cudaGetLastError();
}

template <int D, int KB, int VB, int G>
cudaError_t launch_n(const MultiArgs& a, const MultiPlan& p, cudaStream_t s) {
  return p.nt == 1 ? launch_c<D, KB, VB, G, 1>(a, p, s) : launch_c<D, KB, VB, G, 2>(a, p, s);
}

template <int KB, int VB>
cudaError_t launch_d(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s) {
  // at 16 bits for both there are no groups
  if constexpr (KB == 16 && VB == 16) return D == 64 ? launch_n<64, KB, VB, 64>(a, p, s) : launch_n<128, KB, VB, 64>(a, p, s);
  if (D == 64) return a.G == 32 ? launch_n<64, KB, VB, 32>(a, p, s) : launch_n<64, KB, VB, 64>(a, p, s);
  if (a.G == 32) return launch_n<128, KB, VB, 32>(a, p, s);
  return a.G == 64 ? launch_n<128, KB, VB, 64>(a, p, s) : launch_n<128, KB, VB, 128>(a, p, s);
}

template <int KB>
cudaError_t launch_k(const MultiArgs& a, int D, const MultiPlan& p, cudaStream_t s) {
  switch (a.vb) {
    case 2: return launch_d<KB, 2>(a, D, p, s);
    case 4: return launch_d<KB, 4>(a, D, p, s);
    case 6: return launch_d<KB, 6>(a, D, p, s);
    case 8: return launch_d<KB, 8>(a, D, p, s);
    case 16: return launch_d<KB, 16>(a, D, p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace multi
}  // namespace lkv
