// rope_table.cu -- cos and sin tables of the rotary positions
// (lkv_rope_table).
//
// Row p, pair i: attn * (cos, sin)(p f_i).  An angle p f_i of a far position
// has few bits of fraction left in fp32, so the angles are taken in fp64, and
// to keep the fp64 work small each block evaluates sincos only at its first
// row, at one slab of rows and at one row, and reaches the others by the
// addition theorem:
//   (cos, sin)(x + y) = (cos x cos y - sin x sin y, sin x cos y + cos x sin y),
// four fp64 operations a value pair, at most 15 + 31 steps from an evaluated angle
// (error below 2e-14, rounded once to fp32).  Bound by the table's write and the
// fp64 to fp32 conversions: 131071 rows of 48 pairs in 9.6 us (5.2 TB/s).
#include <algorithm>
#include <cmath>

#include "api_common.cuh"
#include "serving.cuh"

namespace lkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;  // rot_dim <= 128

// The frequency of each pair, made on the host (a few fp64 functions in a row
// would be half of a small table's time on the device).
struct Frequencies {
  double f[kMaxHalf];
};

Frequencies frequencies(const RopeTableArgs& a) {
  const double two_pi = 6.283185307179586476925286766559, rot = 2.0 * a.half, log_base = std::log(a.base);
  // the ramp's ends, by dimension
  double lo = 0.0, hi = 0.0;
  if (a.kind == LKV_ROPE_RAMP) {
    lo = std::max(std::floor(rot * std::log(a.orig / (a.high * two_pi)) / (2.0 * log_base)), 0.0);
    hi = std::min(std::ceil(rot * std::log(a.orig / (a.low * two_pi)) / (2.0 * log_base)), rot - 1.0);
  }
  Frequencies fr{};
  for (int i = 0; i < a.half; ++i) {
    const double f = std::exp(-log_base * i / a.half);
    double mix = 1.0;  // share of the unscaled frequency
    if (a.kind == LKV_ROPE_LINEAR) mix = 0.0;
    if (a.kind == LKV_ROPE_SMOOTH) mix = std::min(std::max((a.orig * f / two_pi - a.low) / (a.high - a.low), 0.0), 1.0);
    if (a.kind == LKV_ROPE_RAMP) mix = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
    fr.f[i] = mix == 1.0 ? f : (1.0 - mix) * (f / a.factor) + mix * f;
  }
  return fr;
}

__device__ __forceinline__ double2 turn(double2 x, double2 y) {
  return make_double2(x.x * y.x - x.y * y.y, x.y * y.x + x.x * y.y);
}

// kRun: rows of one thread.  131071 rows of 48 pairs: 9.6 us with 32, 10.4 with
// 16; 8192 rows of 64 pairs, where blocks are few: 4.2 against 3.2.
template <int kRun>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(float* table, double attn, int half, int rows, int slabs,
                                                              const __grid_constant__ Frequencies fr) {
  __shared__ double2 s_base[kMaxHalf], s_slab[kMaxHalf], s_one[kMaxHalf];
  const int tid = threadIdx.x;
  const long long p0 = (long long)blockIdx.x * slabs * kRun;
  // one evaluation a thread: three angles of each pair
  if (tid < 3 * half) {
    const int i = tid % half, which = tid / half;
    const double f = fr.f[i];
    double2 v;
    sincos(f * (which == 0 ? (double)p0 : which == 1 ? (double)kRun : 1.0), &v.y, &v.x);
    if (which == 0) s_base[i] = make_double2(v.x * attn, v.y * attn);
    else if (which == 1) s_slab[i] = v;
    else s_one[i] = v;
  }
  __syncthreads();
  // two adjacent pairs of a thread: 16-byte stores
  const int quads = half / 2, i = 2 * (tid % quads), slab = tid / quads;
  if (slab >= slabs) return;
  double2 v = s_base[i], w = s_base[i + 1];
  for (int k = 0; k < slab; ++k) { v = turn(v, s_slab[i]); w = turn(w, s_slab[i + 1]); }
  const double2 v1 = s_one[i], w1 = s_one[i + 1];
  long long p = p0 + (long long)slab * kRun;
  const long long end = p + kRun < rows ? p + kRun : rows;
  float4* dst = reinterpret_cast<float4*>(table) + (p * half + i) / 2;
#pragma unroll 4
  for (; p < end; ++p, dst += quads) {
    *dst = make_float4((float)v.x, (float)v.y, (float)w.x, (float)w.y);
    v = turn(v, v1);
    w = turn(w, w1);
  }
}

}  // namespace

template <int kRun>
static cudaError_t launch_run(const RopeTableArgs& a, cudaStream_t s) {
  const int slabs = std::min(kThreads / (a.half / 2), 16);
  const long long rows = (long long)slabs * kRun;
  const long long blocks = (a.rows + rows - 1) / rows;
  rope_table_kernel<kRun><<<(unsigned)blocks, kThreads, 0, s>>>(a.table, a.attn, a.half, a.rows, slabs, frequencies(a));
  return cudaGetLastError();
}

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  // long runs once they still give every SM a few blocks
  return (long long)a.rows * a.half >= (long long)num_sms() * 4 * kThreads * 2 * 16 ? launch_run<32>(a, s) : launch_run<16>(a, s);
}

}  // namespace lkv
