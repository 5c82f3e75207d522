// rope_append.cu -- RMS norm of each query and key head, rotary positions and
// the quantized append, in one pass over the new tokens (lkv_rope_append_kv).
//
// For a head x of D channels, every fp32 operation rounded on its own:
//   ss = sum x_i^2 in the pairwise order of adjacent values,
//   n_i = (x_i * (1 / sqrt(ss / D + eps))) * w_i,
//   pairs (a, b) of the first rot channels turn by the token's table row:
//   (a c - b s, b c + a s); q and k are rounded once to bf16, and K and V go
//   through the quantizer of lkv_quantize_kv.
// The fixed order and the separate roundings (this file is built without
// multiply-add contraction) make codes and q bit-exact against the formula.
//
// Bound by bytes for prompts (22.5 KB a token with 32 query and 8 KV heads of
// 128) and by latency for decode steps.  A warp takes one token and a run of
// its heads, D/16 lanes a head, so the token's table row is read into
// registers once per run.  Query rows need no channel order for the output,
// so in the half layout lane j takes the 8 channels from 8j and the 8 from
// rot/2 + 8j: whole pairs, no exchange between lanes.  Key rows are quantized
// in groups of adjacent channels, so there a lane keeps its 16 adjacent ones
// and reads their partners too (one row in six at 32 / 8 heads).
#include <algorithm>

#include "serving.cuh"

namespace lkv {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ uint4 ld8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

__device__ __forceinline__ void widen8(const uint4& u, float* x) {
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint4 narrow8(const float* x) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// 1 / sqrt(mean of squares + eps) of a row: the lane's 16 adjacent channels in
// two words of 8, then the row's lanes.
template <int D>
__device__ __forceinline__ float row_rstd(const uint4& u0, const uint4& u1, float eps, unsigned mask) {
  float x[16];
  widen8(u0, x);
  widen8(u1, x + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = x[i] * x[i];
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = x[2 * i] + x[2 * i + 1];
  float t = x[0];
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) t = t + __shfl_xor_sync(mask, t, off);
  return __fdiv_rn(1.0f, __fsqrt_rn(t * (1.0f / D) + eps));
}

__device__ __forceinline__ void norm8(float* x, float r, const float* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (x[i] * r) * w[i];
}

// Where a lane's two runs of 8 channels lie in a query row.
struct Runs {
  int a, b;     // first channels
  bool turn;    // the pairs (a + i, b + i) (half layout) or the adjacent ones inside both runs turn
};

template <bool INTER>
__device__ __forceinline__ Runs query_runs(int j, int rot) {
  if (INTER) return {16 * j, 16 * j + 8, 16 * j < rot};
  const int half = rot / 2;
  if (8 * j < half) return {8 * j, half + 8 * j, true};
  return {16 * j, 16 * j + 8, false};
}

template <int D, int BITS>
__device__ __forceinline__ void quantize_row16(const uint32_t (&w)[8], uint8_t* codes, float* sz, int j, int lpg,
                                               unsigned mask, float one, bool reciprocal) {
  if constexpr (BITS == 16) {
    *reinterpret_cast<uint4*>(codes + j * 32) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(codes + j * 32 + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    LaneWords<BITS> lw;
    float scale, zero;
    quantize16<BITS>(w, lpg, mask, one, lw, scale, zero, reciprocal);
    store_lane_words<BITS>(codes + j * (2 * BITS), lw);
    if (j % lpg == 0) *reinterpret_cast<float2*>(sz + 2 * (j / lpg)) = make_float2(scale, zero);
  }
}

template <int D>
__device__ __forceinline__ void store_row(const RopeAppendArgs& a, int bits, const uint32_t (&w)[8], uint8_t* base,
                                          float* sz_base, long long row, int j, unsigned mask) {
  uint8_t* codes = base + row * (D * bits / 8);
  float* sz = sz_base + row * (D / a.G) * 2;
  const int lpg = a.G / kDimsPerLane;
  switch (bits) {
    case 2: quantize_row16<D, 2>(w, codes, sz, j, lpg, mask, a.one, a.reciprocal); break;
    case 4: quantize_row16<D, 4>(w, codes, sz, j, lpg, mask, a.one, a.reciprocal); break;
    case 6: quantize_row16<D, 6>(w, codes, sz, j, lpg, mask, a.one, a.reciprocal); break;
    case 8: quantize_row16<D, 8>(w, codes, sz, j, lpg, mask, a.one, a.reciprocal); break;
    default: quantize_row16<D, 16>(w, codes, sz, j, lpg, mask, a.one, a.reciprocal); break;
  }
}

// Cache row of KV head g for a slot, or -1.
__device__ __forceinline__ long long slot_row(const RopeAppendArgs& a, long long slot, int g) {
  if (slot < 0) return -1;
  const long long page = slot / a.page_tokens;
  if (page >= a.num_pages) return -1;
  return (page * a.Hkv + g) * a.page_tokens + slot % a.page_tokens;
}

// Query heads [h0, h1) of token t.
template <int D, bool INTER>
__device__ void query_rows(const RopeAppendArgs& a, int t, int pos, int h0, int h1) {
  constexpr int LPR = D / kDimsPerLane, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR;
  const unsigned mask = row_lane_mask<LPR>(lane);
  const Runs run = query_runs<INTER>(j, a.rot);
  const bool norm = a.q_weight != nullptr;
  float wa[8], wb[8], cs[16];
  if (norm) { widen8(ld8(a.q_weight + run.a), wa); widen8(ld8(a.q_weight + run.b), wb); }
  if (run.turn) {  // 8 pairs from 8 j: (cos, sin) side by side
    const float4* src = reinterpret_cast<const float4*>(a.table + ((long long)pos * (a.rot / 2) + 8 * j) * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(src + i);
      cs[4 * i] = v.x; cs[4 * i + 1] = v.y; cs[4 * i + 2] = v.z; cs[4 * i + 3] = v.w;
    }
  }
  const uint16_t* src = a.q + t * a.q_stride;
  uint16_t* dst = a.q_out + (long long)t * a.Hq * D;
  const bool square = norm && !INTER;  // the sum wants adjacent channels, the pairs others
  uint4 ua, ub, s0, s1;
  auto fetch = [&](int h) {
    if (h >= h1) return;
    const uint16_t* row = src + (long long)h * D;
    ua = ld8(row + run.a);
    ub = ld8(row + run.b);
    if (square) { s0 = ld8(row + 16 * j); s1 = ld8(row + 16 * j + 8); }
  };
  fetch(h0 + sub);
  for (int h = h0 + sub; h - sub < h1; h += RPW) {
    const uint4 va = ua, vb = ub, q0 = square ? s0 : ua, q1 = square ? s1 : ub;
    fetch(h + RPW);
    if (h >= h1) continue;  // the lanes of a row agree
    float x[8], y[8];
    widen8(va, x);
    widen8(vb, y);
    if (norm) {
      const float r = row_rstd<D>(q0, q1, a.eps, mask);
      norm8(x, r, wa);
      norm8(y, r, wb);
    }
    if (run.turn) {
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = x[2 * i], q = x[2 * i + 1], c = cs[2 * i], s = cs[2 * i + 1];
          x[2 * i] = p * c - q * s;
          x[2 * i + 1] = q * c + p * s;
          const float p2 = y[2 * i], q2 = y[2 * i + 1], c2 = cs[8 + 2 * i], s2 = cs[8 + 2 * i + 1];
          y[2 * i] = p2 * c2 - q2 * s2;
          y[2 * i + 1] = q2 * c2 + p2 * s2;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x[i], q = y[i], c = cs[2 * i], s = cs[2 * i + 1];
          x[i] = p * c - q * s;
          y[i] = q * c + p * s;
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + (long long)h * D + run.a) = narrow8(x);
    *reinterpret_cast<uint4*>(dst + (long long)h * D + run.b) = narrow8(y);
  }
}

// Key heads g0 .. of token t, one batch of 32 / (D / 16) rows.
template <int D, bool INTER>
__device__ void key_rows(const RopeAppendArgs& a, int t, int pos, long long slot, int g0) {
  constexpr int LPR = D / kDimsPerLane;
  const int lane = threadIdx.x & 31, j = lane % LPR, g = g0 + lane / LPR;
  const unsigned mask = row_lane_mask<LPR>(lane);
  if (g >= a.Hkv) return;
  const long long row = slot_row(a, slot, g);
  if (row < 0) return;
  const uint16_t* src = a.k + t * a.k_stride + (long long)g * D;
  const uint4 u0 = ld8(src + 16 * j), u1 = ld8(src + 16 * j + 8);
  float x[16];
  widen8(u0, x);
  widen8(u1, x + 8);
  float r = 1.0f;
  if (a.k_weight != nullptr) {
    r = row_rstd<D>(u0, u1, a.eps, mask);
    float w[8];
    widen8(ld8(a.k_weight + 16 * j), w);
    norm8(x, r, w);
    widen8(ld8(a.k_weight + 16 * j + 8), w);
    norm8(x + 8, r, w);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // runs of 8 channels
    const int c0 = 16 * j + 8 * e;
    float* z = x + 8 * e;
    if (c0 >= a.rot) continue;
    if constexpr (INTER) {
      const float4* src4 = reinterpret_cast<const float4*>(a.table + (long long)pos * a.rot + c0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = __ldg(src4 + i);
        const float p = z[4 * i], q = z[4 * i + 1], p2 = z[4 * i + 2], q2 = z[4 * i + 3];
        z[4 * i] = p * v.x - q * v.y;
        z[4 * i + 1] = q * v.x + p * v.y;
        z[4 * i + 2] = p2 * v.z - q2 * v.w;
        z[4 * i + 3] = q2 * v.z + p2 * v.w;
      }
    } else {
      const int half = a.rot / 2;
      const bool low = c0 < half;
      const int other = low ? c0 + half : c0 - half, pair = low ? c0 : c0 - half;
      float o[8];
      widen8(ld8(src + other), o);
      if (a.k_weight != nullptr) {
        float w[8];
        widen8(ld8(a.k_weight + other), w);
        norm8(o, r, w);
      }
      const float4* src4 = reinterpret_cast<const float4*>(a.table + ((long long)pos * half + pair) * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(src4 + i);
        const float p = z[2 * i], q = z[2 * i + 1], po = o[2 * i], qo = o[2 * i + 1];
        // the first of a pair: a c - b s; the second: b c + a s
        z[2 * i] = low ? p * v.x - po * v.y : p * v.x + po * v.y;
        z[2 * i + 1] = low ? q * v.z - qo * v.w : q * v.z + qo * v.w;
      }
    }
  }
  const uint4 n0 = narrow8(x), n1 = narrow8(x + 8);
  const uint32_t w[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
  store_row<D>(a, a.kb, w, a.k_codes, a.k_sz, row, j, mask);
}

template <int D>
__device__ void value_rows(const RopeAppendArgs& a, int t, long long slot, int g0) {
  constexpr int LPR = D / kDimsPerLane;
  const int lane = threadIdx.x & 31, j = lane % LPR, g = g0 + lane / LPR;
  const unsigned mask = row_lane_mask<LPR>(lane);
  if (g >= a.Hkv) return;
  const long long row = slot_row(a, slot, g);
  if (row < 0) return;
  const uint16_t* src = a.v + t * a.v_stride + (long long)g * D;
  const uint4 u0 = ld8(src + 16 * j), u1 = ld8(src + 16 * j + 8);
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  store_row<D>(a, a.vb, w, a.v_codes, a.v_sz, row, j, mask);
}

// One warp: one token and one of its items -- query runs, then key batches,
// then value batches.
template <int D, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) rope_append_kernel(RopeAppendArgs a, int q_items, int kv_items) {
  constexpr int RPW = 32 / (D / kDimsPerLane);
  const int items = q_items + 2 * kv_items;
  const long long id = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const long long t = id / items;
  const int item = (int)(id % items);
  if (t >= a.n_cap) return;
  const int n = a.n_tokens ? clamp_len(__ldg(a.n_tokens), a.n_cap) : a.n_cap;
  const int pos = a.rot > 0 ? __ldg(a.positions + t) : 0;
  if (t >= n) return;
  if (a.rot > 0 && (pos < 0 || pos >= a.table_rows)) return;  // no such angle: the token is left out
  if (item < q_items) {
    const int h0 = item * RPW * a.iters;
    query_rows<D, INTER>(a, (int)t, pos, h0, min(a.Hq, h0 + RPW * a.iters));
  } else {
    const long long slot = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
    if (item < q_items + kv_items) key_rows<D, INTER>(a, (int)t, pos, slot, (item - q_items) * RPW);
    else value_rows<D>(a, (int)t, slot, (item - q_items - kv_items) * RPW);
  }
}

template <int D, bool INTER>
cudaError_t launch_t(RopeAppendArgs a, cudaStream_t s) {
  constexpr int RPW = 32 / (D / kDimsPerLane);
  // one batch of rows a warp while that leaves SMs idle, else runs of four
  const long long batches = (long long)a.n_cap * ((a.Hq + RPW - 1) / RPW);
  a.iters = batches >= (long long)num_sms() * 64 ? 4 : 1;
  const int q_items = (a.Hq + RPW * a.iters - 1) / (RPW * a.iters), kv_items = (a.Hkv + RPW - 1) / RPW;
  const long long blocks = ((long long)a.n_cap * (q_items + 2 * kv_items) + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  rope_append_kernel<D, INTER><<<(unsigned)blocks, 32 * kWarps, 0, s>>>(a, q_items, kv_items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, int D, bool interleaved, cudaStream_t s) {
  if (D == 64) return interleaved ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
  return interleaved ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
}

}  // namespace lkv
