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
// in groups of adjacent channels: they are rotated like queries and change
// order through shared memory (16384 tokens: 86 us, and 92 where lanes kept
// their 16 adjacent channels and read and normed the partners too).  16384
// tokens of 32 / 8 heads into a K6V4 cache: 84 us for 369 MB (4.4 TB/s); 16
// tokens: 3.2 us, and 9.8 at a capacity of 16384 (27.5 while the rows behind the
// count were prefetched too).
#include <algorithm>

#include "serving.cuh"

namespace lkv {

namespace {

constexpr int kWarps = 4;
// 72 registers (16384 tokens of 32 / 8 heads: 5 blocks 95 us, 6 86, 7 85, 8 88);
// where only some channels turn 80 (64 of 128: 6 blocks 95 us, 7 99)
constexpr int blocks_per_sm(bool whole) { return whole ? 7 : 6; }
constexpr int kRun = 4;  // query batches of a warp in large calls (2: 103 us, 8: 92 us)

__device__ __forceinline__ uint4 ld8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// 8 adjacent channels for packed fp32 arithmetic: e holds the even ones (0, 2),
// (4, 6), o the odd ones (1, 3), (5, 7) -- the low and high halves of two
// words, so that sums of adjacent values and pairs are whole-register
// operations.
struct Eight {
  float2 e[2], o[2];
};

__device__ __forceinline__ Eight widen8(const uint4& u) {
  return {{make_float2(bf16_lo(u.x), bf16_lo(u.y)), make_float2(bf16_lo(u.z), bf16_lo(u.w))},
          {make_float2(bf16_hi(u.x), bf16_hi(u.y)), make_float2(bf16_hi(u.z), bf16_hi(u.w))}};
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint4 narrow8(const Eight& v) {
  return make_uint4(pack2(v.e[0].x, v.o[0].x), pack2(v.e[0].y, v.o[0].y), pack2(v.e[1].x, v.o[1].x), pack2(v.e[1].y, v.o[1].y));
}

// Sum of squares of 8 channels, pairwise, adjacent values first.
__device__ __forceinline__ float squares8(const Eight& v) {
  const float2 a = exact_add2(exact_mul2(v.e[0], v.e[0]), exact_mul2(v.o[0], v.o[0]));
  const float2 b = exact_add2(exact_mul2(v.e[1], v.e[1]), exact_mul2(v.o[1], v.o[1]));
  return (a.x + a.y) + (b.x + b.y);
}

__device__ __forceinline__ float rstd_of(float ss, float inv_d, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(ss * inv_d + eps));
}

// 1 / sqrt(mean of squares + eps) of a row: the lane's 16 adjacent channels,
// then the row's lanes.
template <int D>
__device__ __forceinline__ float row_rstd(const Eight& v0, const Eight& v1, float eps, unsigned mask) {
  float t = squares8(v0) + squares8(v1);
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) t = t + __shfl_xor_sync(mask, t, off);
  return rstd_of(t, 1.0f / D, eps);
}

// The same when lane j holds the 8 channels from 8 j and the 8 from D/2 + 8 j.
template <int D>
__device__ __forceinline__ float row_rstd_halves(const Eight& v0, const Eight& v1, float eps, unsigned mask) {
  float2 t = make_float2(squares8(v0), squares8(v1));
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1)
    t = exact_add2(t, make_float2(__shfl_xor_sync(mask, t.x, off), __shfl_xor_sync(mask, t.y, off)));
  return rstd_of(t.x + t.y, 1.0f / D, eps);
}

__device__ __forceinline__ void norm8(Eight& v, float r, const Eight& w) {
  const float2 rr = f2(r);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v.e[i] = exact_mul2(exact_mul2(v.e[i], rr), w.e[i]);
    v.o[i] = exact_mul2(exact_mul2(v.o[i], rr), w.o[i]);
  }
}

// p + q for two rounded products.  A packed multiply that feeds a packed add
// would be contracted by the code generator, so the sum is p * 1 + q with a 1
// it does not know.
__device__ __forceinline__ float2 sum_of_products(float2 p, float2 q, float one) { return exact_fma2(p, f2(one), q); }

// (a, b) -> (a c - b s, b c + a s), with ns = -s.
__device__ __forceinline__ void turn2(float2& a, float2& b, float2 c, float2 s, float2 ns, float one) {
  const float2 x = sum_of_products(exact_mul2(a, c), exact_mul2(b, ns), one);
  const float2 y = sum_of_products(exact_mul2(b, c), exact_mul2(a, s), one);
  a = x;
  b = y;
}

// (cos, sin) of 8 pairs, for channels in the order of Eight.
struct Turns {
  Eight c, s;
};

__device__ __forceinline__ Turns load_turns(const float* table) {  // 8 pairs (cos, sin) side by side
  const float4* p = reinterpret_cast<const float4*>(table);
  const float4 a = __ldg(p), b = __ldg(p + 1), c = __ldg(p + 2), d = __ldg(p + 3);
  return {{{make_float2(a.x, b.x), make_float2(c.x, d.x)}, {make_float2(a.z, b.z), make_float2(c.z, d.z)}},
          {{make_float2(a.y, b.y), make_float2(c.y, d.y)}, {make_float2(a.w, b.w), make_float2(c.w, d.w)}}};
}

__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Pairs (x_i, y_i), i = 0 .. 7.
__device__ __forceinline__ void turn_halves(Eight& x, Eight& y, const Turns& t, float one) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    turn2(x.e[i], y.e[i], t.c.e[i], t.s.e[i], neg2(t.s.e[i]), one);
    turn2(x.o[i], y.o[i], t.c.o[i], t.s.o[i], neg2(t.s.o[i]), one);
  }
}

// Adjacent pairs inside 8 channels; cs: (cos, sin) of the 4 pairs.
__device__ __forceinline__ void turn_adjacent(Eight& v, const float4& p, const float4& q, float one) {
  const float2 c0 = make_float2(p.x, p.z), s0 = make_float2(p.y, p.w), c1 = make_float2(q.x, q.z), s1 = make_float2(q.y, q.w);
  turn2(v.e[0], v.o[0], c0, s0, neg2(s0), one);
  turn2(v.e[1], v.o[1], c1, s1, neg2(s1), one);
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

// Run k of a row (channels from 8 k): the lane that holds it in the half
// layout's order, as its first or second.
struct Holder {
  int lane;
  bool second;
};
__device__ __forceinline__ Holder holder_of(int k, int rot, int row_lane0) {
  const int hr = rot / 16;
  return {row_lane0 + (k < hr ? k : k < 2 * hr ? k - hr : k / 2), k < hr ? false : k < 2 * hr ? true : (k & 1) != 0};
}

// row_rstd when a lane's runs are any two of the row; h: who holds runs 2 j and 2 j + 1.
template <int D>
__device__ __forceinline__ float row_rstd_runs(const Eight& v0, const Eight& v1, const Holder (&h)[2], float eps, unsigned mask) {
  const float s0 = squares8(v0), s1 = squares8(v1);
  float p[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float x = __shfl_sync(mask, s0, h[i].lane), y = __shfl_sync(mask, s1, h[i].lane);
    p[i] = h[i].second ? y : x;
  }
  float t = p[0] + p[1];
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) t = t + __shfl_xor_sync(mask, t, off);
  return rstd_of(t, 1.0f / D, eps);
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

// Query heads [h0, h1) of token t.  WHOLE: half layout with every channel turning.
template <int D, bool INTER, bool WHOLE>
__device__ __forceinline__ void query_rows(const RopeAppendArgs& a, int t, int pos, int h0, int h1) {
  constexpr int LPR = D / kDimsPerLane, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR;
  const unsigned mask = row_lane_mask<LPR>(lane);
  const Runs run = WHOLE ? Runs{8 * j, D / 2 + 8 * j, true} : query_runs<INTER>(j, a.rot);
  const bool norm = a.q_weight != nullptr;
  const Holder hold[2] = {holder_of(2 * j, a.rot, lane - j), holder_of(2 * j + 1, a.rot, lane - j)};
  const uint16_t* src = a.q + t * a.q_stride;
  uint16_t* dst = a.q_out + (long long)t * a.Hq * D;
  uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
  auto fetch = [&](int h) {
    if (h >= h1) return;
    const uint16_t* row = src + (long long)h * D;
    ua = ld8(row + run.a);
    ub = ld8(row + run.b);
  };
  fetch(h0 + sub);
  Eight wa, wb;
  if (norm) { wa = widen8(ld8(a.q_weight + run.a)); wb = widen8(ld8(a.q_weight + run.b)); }
  Turns cs;
  float4 near[4];
  if (run.turn) {  // 8 pairs from 8 j
    const float* at = a.table + ((long long)pos * (WHOLE ? D / 2 : a.rot / 2) + 8 * j) * 2;
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) near[i] = __ldg(reinterpret_cast<const float4*>(at) + i);
    } else {
      cs = load_turns(at);
    }
  }
  for (int h = h0 + sub; h - sub < h1; h += RPW) {
    Eight x = widen8(ua), y = widen8(ub);
    fetch(h + RPW);
    if (h >= h1) continue;  // the lanes of a row agree
    if (norm) {
      const float r = WHOLE ? row_rstd_halves<D>(x, y, a.eps, mask)
                      : INTER ? row_rstd<D>(x, y, a.eps, mask) : row_rstd_runs<D>(x, y, hold, a.eps, mask);
      norm8(x, r, wa);
      norm8(y, r, wb);
    }
    if (run.turn) {
      if constexpr (INTER) {
        turn_adjacent(x, near[0], near[1], a.one);
        turn_adjacent(y, near[2], near[3], a.one);
      } else {
        turn_halves(x, y, cs, a.one);
      }
    }
    *reinterpret_cast<uint4*>(dst + (long long)h * D + run.a) = narrow8(x);
    *reinterpret_cast<uint4*>(dst + (long long)h * D + run.b) = narrow8(y);
  }
}

// Key and value heads g0 .. of token t, one batch of 32 / (D / 16) rows.
// All loads of the rows come before the first use, the slot's among them.
// In the half layout keys turn in the lanes' query runs and go through shared
// memory into the quantizer's order.
template <int D, bool INTER, bool WHOLE>
__device__ __forceinline__ void key_value_rows(const RopeAppendArgs& a, int t, int pos, int g0, bool keys, bool values) {
  constexpr int LPR = D / kDimsPerLane;
  const int lane = threadIdx.x & 31, j = lane % LPR, g = g0 + lane / LPR;
  const unsigned mask = row_lane_mask<LPR>(lane);
  if (g >= a.Hkv) return;
  const Runs run = WHOLE ? Runs{8 * j, D / 2 + 8 * j, true} : query_runs<INTER>(j, a.rot);
  const bool norm = a.k_weight != nullptr;
  const uint16_t* src = a.k + t * a.k_stride + (long long)g * D;
  const uint16_t* vsrc = a.v + t * a.v_stride + (long long)g * D + 16 * j;
  const uint4 k0 = ld8(src + run.a), k1 = ld8(src + run.b);
  uint4 v0 = k0, v1 = k1;
  if (values) { v0 = ld8(vsrc); v1 = ld8(vsrc + 8); }
  const long long row = slot_row(a, __ldg(reinterpret_cast<const long long*>(a.slots) + t), g);
  if (row < 0) return;  // the lanes of a row agree
  if (values) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    store_row<D>(a, a.vb, w, a.v_codes, a.v_sz, row, j, mask);
  }
  if (!keys) return;
  Eight x = widen8(k0), y = widen8(k1);
  if (norm) {
    const Holder hold[2] = {holder_of(2 * j, a.rot, lane - j), holder_of(2 * j + 1, a.rot, lane - j)};
    const float r = WHOLE ? row_rstd_halves<D>(x, y, a.eps, mask)
                    : INTER ? row_rstd<D>(x, y, a.eps, mask) : row_rstd_runs<D>(x, y, hold, a.eps, mask);
    norm8(x, r, widen8(ld8(a.k_weight + run.a)));
    norm8(y, r, widen8(ld8(a.k_weight + run.b)));
  }
  if (run.turn) {  // 8 pairs from 8 j
    const float* at = a.table + ((long long)pos * (WHOLE ? D / 2 : a.rot / 2) + 8 * j) * 2;
    if constexpr (INTER) {
      const float4* p = reinterpret_cast<const float4*>(at);
      turn_adjacent(x, __ldg(p), __ldg(p + 1), a.one);
      turn_adjacent(y, __ldg(p + 2), __ldg(p + 3), a.one);
    } else {
      turn_halves(x, y, load_turns(at), a.one);
    }
  }
  uint4 n0 = narrow8(x), n1 = narrow8(y);
  if constexpr (!INTER) {
    __shared__ uint4 s_run[kWarps][64];  // the rows' runs of 8 channels in order
    uint4* of_row = s_run[threadIdx.x / 32] + lane / LPR * 2 * LPR;
    of_row[run.a / 8] = n0;
    of_row[run.b / 8] = n1;
    __syncwarp(mask);
    n0 = of_row[2 * j];
    n1 = of_row[2 * j + 1];
  }
  const uint32_t w[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
  store_row<D>(a, a.kb, w, a.k_codes, a.k_sz, row, j, mask);
}

// The 128-byte lines of `bytes` bytes from p, one per lane, on their way into L2.
__device__ __forceinline__ void prefetch_lines(const void* p, int bytes, int lane) {
  if (lane >= 0 && lane * 128 < bytes) prefetch_l2(static_cast<const char*>(p) + lane * 128);
}

// One warp: one token and one of its items -- query runs, then key and value
// batches.
template <int D, bool INTER, bool WHOLE>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(WHOLE)) rope_append_kernel(RopeAppendArgs a, int q_items, int kv_items) {
  constexpr int RPW = 32 / (D / kDimsPerLane);
  const int items = q_items + kv_items;
  const long long id = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
  const long long t = id / items;
  const int item = (int)(id % items);
  if (t >= a.n_cap) return;
  const int lane = threadIdx.x & 31;
  const bool query = item < q_items;
  const int h0 = item * RPW * a.iters, h1 = min(a.Hq, h0 + RPW * a.iters);
  const int kv = a.split ? (item - q_items) / 2 : item - q_items, g0 = kv * RPW, g1 = min(a.Hkv, g0 + RPW);
  const int n = a.n_tokens ? clamp_len(__ldg(a.n_tokens), a.n_cap) : a.n_cap;
  const int pos = a.rot > 0 ? __ldg(a.positions + t) : 0;  // with the count, not behind it: one wait in a small call
  if (t >= n) return;
  if (a.ahead > 0 && t + a.ahead < n) {
    // the same item of a token that no resident warp has reached yet
    const long long u = t + a.ahead;
    if (query) {
      prefetch_lines(a.q + u * a.q_stride + h0 * D, (h1 - h0) * D * 2, lane);
    } else {
      prefetch_lines(a.k + u * a.k_stride + g0 * D, (g1 - g0) * D * 2, lane < 16 ? lane : -1);
      prefetch_lines(a.v + u * a.v_stride + g0 * D, (g1 - g0) * D * 2, lane - 16);
    }
  }
  if (a.rot > 0 && (pos < 0 || pos >= a.table_rows)) return;  // no such angle: the token is left out
  if (query) {
    query_rows<D, INTER, WHOLE>(a, (int)t, pos, h0, h1);
  } else {
    const bool second = a.split && ((item - q_items) & 1);
    key_value_rows<D, INTER, WHOLE>(a, (int)t, pos, g0, !second, !a.split || second);
  }
}

template <int D, bool INTER, bool WHOLE>
cudaError_t launch_t(RopeAppendArgs a, cudaStream_t s) {
  constexpr int RPW = 32 / (D / kDimsPerLane);
  // one batch of rows a warp while that leaves SMs idle, else runs of four and keys with values: by the capacity, as the
  // host does not know the count
  const long long batches = (long long)a.n_cap * ((a.Hq + RPW - 1) / RPW);
  const bool many = batches >= (long long)num_sms() * 64;
  a.iters = many ? kRun : 1;
  a.split = !many;
  const int q_items = (a.Hq + RPW * a.iters - 1) / (RPW * a.iters), kv_items = (a.Hkv + RPW - 1) / RPW * (many ? 1 : 2);
  // tokens that the resident warps hold at a time
  a.ahead = many ? (int)((long long)num_sms() * blocks_per_sm(WHOLE) * kWarps / (q_items + kv_items)) + 1 : 0;
  const long long blocks = ((long long)a.n_cap * (q_items + kv_items) + kWarps - 1) / kWarps;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  rope_append_kernel<D, INTER, WHOLE><<<(unsigned)blocks, 32 * kWarps, 0, s>>>(a, q_items, kv_items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, int D, bool interleaved, cudaStream_t s) {
  const bool whole = !interleaved && a.rot == D;
  if (D == 64) {
    if (interleaved) return launch_t<64, true, false>(a, s);
    return whole ? launch_t<64, false, true>(a, s) : launch_t<64, false, false>(a, s);
  }
  if (interleaved) return launch_t<128, true, false>(a, s);
  return whole ? launch_t<128, false, true>(a, s) : launch_t<128, false, false>(a, s);
}

}  // namespace lkv
