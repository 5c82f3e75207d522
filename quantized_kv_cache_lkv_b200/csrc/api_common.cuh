// api_common.cuh -- host-side checks shared by the extern "C" entry points.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/lkv.h"
#include <cuda_runtime.h>

namespace lkv {

constexpr size_t kAlign = 256;
constexpr size_t kHeaderBytes = 256;  // status, wait limit, done counter, skip-count accumulators

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// 16 is the passthrough width: the row holds the bf16 values, with no (scale, zero)
inline bool bits_ok(int b) { return b == 2 || b == 4 || b == 6 || b == 8 || b == 16; }
inline bool dim_ok(int D) { return D == 64 || D == 128; }
inline bool group_ok(int G, int D) { return (G == 32 || G == 64 || G == 128) && G <= D && D % G == 0; }
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }
// A pointer that must be valid when its tensor is non-empty.
inline bool ptr_ok(const void* p, bool nonempty) { return !nonempty || (p != nullptr && aligned16(p)); }

inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? LKV_OK : LKV_ERR_CUDA; }

inline int check_cache_shape(int B, int Hkv, int T_cap, int D, int G) {
  if (B < 0 || Hkv <= 0 || T_cap < 0) return LKV_ERR_INVALID_ARG;
  if (!dim_ok(D) || !group_ok(G, D)) return LKV_ERR_UNSUPPORTED;
  if (((long long)T_cap * (D / G)) % 2 != 0) return LKV_ERR_UNSUPPORTED;
  return LKV_OK;
}

// Whether [a, a + na) and [b, b + nb) share a byte (a null or empty tensor shares none).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace lkv
