// multi_impl.cuh -- attention of one or a few new tokens per sequence over
// the packed cache (lkv_decode_attention_multi and its paged form): capped,
// biased and masked scores, one pass with a running softmax.
//
// The mathematics, per query row (new token i, head h of KV head g):
//   x_t = softmax_scale * q . khat_t, capped by a tanh, biased by distance,
//   out = sum_t e_t vhat_t / sum_t e_t,  e_t = exp(x_t - m),  m a running bound
// over the visible t.  With khat = scale * code + zero per group of channels,
//   q . khat_t = sum_g scale_tg (q_g . code_tg) + zero_tg (sum of q_g)
//   out        = sum_t (e_t scale_tg) code_tg + sum_t e_t zero_tg
// so both products run on integer codes, exact in 16-bit floating point.  They
// are centred, code - 2^(bits-1) with zero + 2^(bits-1) scale: with codes from 0 up
// the two terms are large and cancel (8-bit K: rel-L2 1.2e-5 instead of 1e-6).
//
// What bounds it: the packed rows, read once (K6V4, D 128, G 64: 192 bytes a
// row, 8.3 clocks of one SM at the copy bandwidth), and close behind the
// instructions that turn codes into MMA operands.  So:
//   - tokens are the M rows of mma.m16n8k16 in the K product and its K rows in
//     the V product, and the query rows (heads of the group x new tokens) its
//     N = 8 columns: with 1 to 8 query rows nothing but columns is padded;
//   - K codes become fp16 integers (mma_k.cuh) against q scaled by a power of
//     two: exact products.  V codes become bf16 integers against e * scale
//     split in two bf16 terms (hi + lo leaves at most 2^-18 of the product);
//   - the channel-to-row and token-to-slot orders of the MMAs are free, so
//     every lane reads whole runs of codes of one token from shared memory,
//     and the codes of two tokens are paired by one byte permute per half
//     word, before they are unpacked;
//   - the running maximum moves only when it would grow by more than 2^8
//     (e stays far inside fp32), so rescaling is rare.
//
// Work split: the tiles (kTile tokens or half of it) of all units -- a unit
// is one (sequence, KV head, block of 8 NT query rows) -- lie end to end, and
// every warp of the grid takes an equal run of them with a ring of its own in
// shared memory: no barrier until the end.  A unit inside one warp's run is
// written straight out.  Units cut by run ends leave (max, sum, partial
// output) pieces in the workspace; the CTA joins those of its warps, and for a
// unit cut between CTAs the last one to arrive joins the CTAs' pieces, always
// in order, so results do not depend on timing.
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "lkv_kernels.cuh"
#include "mma_k.cuh"
#include "multi.cuh"

namespace lkv {
namespace multi {

using fused::hmma16816;
using fused::hmma16816_bf16;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;  // the running bound moves when a score passes it by 2^8

__device__ __forceinline__ float ex2(float x) {  // 2^x; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ the sequence side
// What a sequence asks for: query rows, and which tiles some of them see.
struct Seq {
  int T, c0, n;        // cached tokens, first query row, new tokens
  int pre, lo;         // tokens before pre are visible; so are those from lo on (up to the query)
  int start;           // document start
  int np, t_lo, cnt;   // prefix tiles, first tile past them, tiles of a unit
  int units;           // Hkv * row blocks
};

template <int NT>
__device__ __forceinline__ Seq load_seq(const MultiArgs& a, int b) {
  Seq s;
  s.T = clamp_len(__ldg(a.lens + b), a.T_cap);
  int c0 = b, c1 = b + 1;
  if (a.cu_q != nullptr) {
    c0 = clamp_len(__ldg(a.cu_q + b), a.n_rows);
    c1 = clamp_len(__ldg(a.cu_q + b + 1), a.n_rows);
  }
  s.c0 = c0;
  s.n = min(max(c1 - c0, 0), a.max_q);
  s.pre = a.prefix ? min(max(__ldg(a.prefix + b), 0), s.T) : 0;
  s.start = a.starts ? max(__ldg(a.starts + b), 0) : 0;
  int lo = s.start;
  if (a.window > 0) lo = max(lo, s.T - s.n - a.window + 1);
  s.lo = min(lo, s.T);
  const int hi_t = (s.T + a.tt - 1) / a.tt, pre_t = (s.pre + a.tt - 1) / a.tt;
  s.t_lo = s.lo / a.tt;
  s.np = min(pre_t, s.t_lo);
  s.cnt = max(1, s.np + max(0, hi_t - s.t_lo));  // a row that sees nothing still owns a tile: its zeros are written
  s.units = a.Hkv * ((s.n * a.r + 8 * NT - 1) / (8 * NT));
  return s;
}

// ------------------------------------------------------------------ V codes
// A lane holds CH consecutive codes of a token (CH * VB bits, right aligned
// in N words).
template <int VB, int CH>
struct VRun {
  static constexpr int bits = VB * CH;
  static constexpr int N = (bits + 31) / 32;
};

// Lane g's run of block blk of one row (p: the row's first byte in shared
// memory).  Runs of 24 and 48 bits are cut out of two words.
template <int VB, int CH>
__device__ __forceinline__ void load_run(const uint8_t* p, int blk, int g, uint32_t (&w)[VRun<VB, CH>::N]) {
  constexpr int bytes = VB * CH / 8;
  const uint8_t* q = p + blk * 8 * bytes;
  if constexpr (bytes == 1) {
    w[0] = q[g];
  } else if constexpr (bytes == 2) {
    w[0] = reinterpret_cast<const uint16_t*>(q)[g];
  } else if constexpr (bytes == 3) {
    const int off = 3 * g;
    const uint32_t* x = reinterpret_cast<const uint32_t*>(q + (off & ~3));
    // bits past the first word are needed only where the run starts late in it
    const uint32_t hi = (off & 3) >= 2 ? x[1] : 0u;
    w[0] = __funnelshift_r(x[0], hi, (off & 3) * 8);
  } else if constexpr (bytes == 4) {
    w[0] = reinterpret_cast<const uint32_t*>(q)[g];
  } else if constexpr (bytes == 6) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(q + ((6 * g) & ~3));
    const uint32_t lo = x[0], hi = x[1];
    const int sh = (g & 1) * 16;
    w[0] = __funnelshift_r(lo, hi, sh);
    w[1] = hi >> sh;
  } else if constexpr (bytes == 8) {
    const uint2 v = reinterpret_cast<const uint2*>(q)[g];
    w[0] = v.x; w[1] = v.y;
  } else {
    static_assert(bytes == 16, "run of 16 bytes");
    const uint4 v = reinterpret_cast<const uint4*>(q)[g];
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
}

__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Centred codes of two tokens (runs x, y) as bf16 pairs (x in the low half),
// exact: out[c] for c = 0 .. CH-1.  Up to 6 bits a code is placed under the
// pattern 0x4300 (128, unit spacing) and 128 + 2^(VB-1) subtracted; 8 bits go
// through fp32 the same way; 16 bits are the values themselves.
template <int VB, int CH>
__device__ __forceinline__ void pair_codes(const uint32_t (&x)[VRun<VB, CH>::N], const uint32_t (&y)[VRun<VB, CH>::N],
                                           uint32_t (&out)[CH]) {
  if constexpr (VB == 16) {
#pragma unroll
    for (int c = 0; c < CH; ++c) out[c] = __byte_perm(x[c / 2], y[c / 2], (c & 1) ? 0x7632 : 0x5410);
  } else if constexpr (VB == 8) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t sel = 0x7650u + (c & 3);  // bytes {code, 0, 0, 0x4B}
      const float2 f = make_float2(__uint_as_float(__byte_perm(x[c / 4], 0x4B000000u, sel)),
                                   __uint_as_float(__byte_perm(y[c / 4], 0x4B000000u, sel)));
      const float2 d = __fadd2_rn(f, make_float2(-8388736.0f, -8388736.0f));
      out[c] = pack_bf16(d.x, d.y);
    }
  } else {
    constexpr int cw = VB == 2 ? 8 : VB == 4 ? 4 : 2;  // codes of one 16-bit window
    constexpr uint32_t mask = ((1u << VB) - 1u) * 0x00010001u;
#pragma unroll
    for (int c0 = 0; c0 < CH; c0 += cw) {
      const int bit = c0 * VB, wi = bit / 32, sh = bit % 32;
      uint32_t z;
      if (sh % 16 == 0) {
        z = __byte_perm(x[wi], y[wi], sh ? 0x7632 : 0x5410);
      } else {
        const int wn = wi + 1 < VRun<VB, CH>::N ? wi + 1 : wi;
        z = __byte_perm(__funnelshift_r(x[wi], x[wn], sh), __funnelshift_r(y[wi], y[wn], sh), 0x5410);
      }
#pragma unroll
      for (int c = 0; c < cw && c0 + c < CH; ++c)
        out[c0 + c] = bsub2(((z >> (c * VB)) & mask) | 0x43004300u, 0x43004300u + (1u << (VB - 1)) * 0x00010001u);
    }
  }
}

// ------------------------------------------------------------------ K codes
// Register J of a lane's 16 codes: two centred codes as exact fp16 values
// (c - 2^(KB-1)) * 2^off, by the extraction plan of mma_k.cuh.
template <int KB, int J, int SW>
__device__ __forceinline__ uint32_t k_reg(const uint32_t (&w)[SW]) {
  if constexpr (KB == 16) {
    return w[J];
  } else {
    using R = fused::RegChannels<KB, J>;
    constexpr uint32_t mid = ((1u << (KB - 1)) << R::lo_off) | ((1u << (KB - 1)) << (16 + R::hi_off));
    return fused::hsub2_u32(fused::a_reg_bits<KB, J, SW>(w), fused::kF16Magic2 + mid);
  }
}

// The value of the middle code of a (scale, zero) pair.
template <int BITS>
__device__ __forceinline__ float centre(float scale, float zero) {
  return fmaf((float)(1 << (BITS - 1)), scale, zero);
}

// ------------------------------------------------------------------ one warp's state
template <int D, int NT, bool G32>
struct Work {
  static constexpr int BLK = D / 64;                 // 64-channel blocks
  static constexpr int MT = D / 16;                  // m-tiles of the output
  static constexpr int NG = G32 ? D / 32 : D / 64;   // (scale, zero) slots; G = 128 reads slot 0 for both blocks
  static constexpr int KG = G32 ? 2 : 1;             // K groups inside a 64-channel block
  float o[MT][NT][4];
  float zacc[NT][NG];   // sum of e * zero, this lane's tokens, row g
  float m[NT], l[NT];   // running bound (base 2) and sum of e (this lane's tokens), row g
  uint32_t qf[NT][BLK][8];
  float ka[NT][2];            // factor of the code product, columns 2 tig and 2 tig + 1
  float kz[NT][NG][2];        // the same times the sum of q over the group: the factor of zero
  int p[NT], lo[NT];          // row g: position of its token, first visible token behind the prefix
  float slope[NT];
  bool on[NT];
  // unit
  int b, ui, g, rb, T, c0, n, pre, p_min, lo_max;
};

// q of the unit's rows as B fragments, and the factors of the affine part.
template <int D, int NT, bool G32>
__device__ __forceinline__ void load_unit(const MultiArgs& a, const Seq& s, int b, int ui, Work<D, NT, G32>& w) {
  using W = Work<D, NT, G32>;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int rbs = s.units / a.Hkv;
  w.b = b; w.ui = ui; w.g = ui / rbs; w.rb = ui % rbs;
  w.T = s.T; w.c0 = s.c0; w.n = s.n; w.pre = s.pre;
  const int r0 = w.rb * 8 * NT, r1 = min(r0 + 8 * NT, s.n * a.r);
  // bounds that hold for every row of the block: a tile between them needs no mask
  const int i0 = r0 / a.r, i1 = (r1 - 1) / a.r;
  w.p_min = s.T - s.n + i0;
  w.lo_max = max(s.start, a.window > 0 ? s.T - s.n + i1 - a.window + 1 : 0);
#pragma unroll
  for (int mt = 0; mt < W::MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[mt][nt][i] = 0.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = r0 + nt * 8 + gid;
    const int i = row / a.r, h = w.g * a.r + row % a.r;
    w.on[nt] = row < r1;
    w.p[nt] = s.T - s.n + i;
    w.lo[nt] = max(s.start, a.window > 0 ? w.p[nt] - a.window + 1 : 0);
    w.slope[nt] = w.on[nt] && a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.0f;
    w.m[nt] = -INFINITY;
    w.l[nt] = 0.0f;
    uint32_t raw[W::BLK][8];
#pragma unroll
    for (int blk = 0; blk < W::BLK; ++blk) {
      uint4 u = make_uint4(0, 0, 0, 0), v = u;
      if (w.on[nt]) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((long long)(s.c0 + i) * a.Hq + h) * D + blk * 64 + tig * 16);
        u = __ldg(src); v = __ldg(src + 1);
      }
      raw[blk][0] = u.x; raw[blk][1] = u.y; raw[blk][2] = u.z; raw[blk][3] = u.w;
      raw[blk][4] = v.x; raw[blk][5] = v.y; raw[blk][6] = v.z; raw[blk][7] = v.w;
    }
    // sums of q over each group, and its largest magnitude
    float big = 0.0f, sum[W::NG];
#pragma unroll
    for (int gi = 0; gi < W::NG; ++gi) { sum[gi] = 0.0f; w.zacc[nt][gi] = 0.0f; }
#pragma unroll
    for (int blk = 0; blk < W::BLK; ++blk) {
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = bf16_lo(raw[blk][j]), y = bf16_hi(raw[blk][j]);
        t += x + y;
        big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
      }
      t += __shfl_xor_sync(kFull, t, 1);
      if constexpr (G32) {
        const float other = __shfl_xor_sync(kFull, t, 2);
        sum[2 * blk] = tig < 2 ? t : other;
        sum[2 * blk + 1] = tig < 2 ? other : t;
      } else {
        t += __shfl_xor_sync(kFull, t, 2);
        sum[blk] = t;
      }
    }
    big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
    big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
    float unit = a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e;
    float back = unit;
    if (a.kb == 16) {
#pragma unroll
      for (int blk = 0; blk < W::BLK; ++blk)
#pragma unroll
        for (int j = 0; j < 8; ++j) w.qf[nt][blk][j] = raw[blk][j];
    } else {
      // a power of two brings the row's largest |q| into [2^14, 2^15): the fp16 values are exact
      int e = 14 + 127 - (int)(__float_as_uint(big) >> 23);
      e = big == 0.0f ? 0 : max(-126, min(126, e));
      const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
      back = unit * down;
#pragma unroll
      for (int blk = 0; blk < W::BLK; ++blk) {
        __half qh[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          qh[2 * j] = __float2half_rn(bf16_lo(raw[blk][j]) * up);
          qh[2 * j + 1] = __float2half_rn(bf16_hi(raw[blk][j]) * up);
        }
        switch (a.kb) {
          case 2: fused::bfrag_one<2, 64, 0>(qh, 0, true, w.qf[nt][blk]); break;
          case 4: fused::bfrag_one<4, 64, 0>(qh, 0, true, w.qf[nt][blk]); break;
          case 6: fused::bfrag_one<6, 64, 0>(qh, 0, true, w.qf[nt][blk]); break;
          default: fused::bfrag_one<8, 64, 0>(qh, 0, true, w.qf[nt][blk]); break;
        }
      }
    }
    // the K product leaves columns 2 tig and 2 tig + 1 in this lane
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int src = 4 * (2 * tig + j);
      w.ka[nt][j] = __shfl_sync(kFull, back, src);
#pragma unroll
      for (int gi = 0; gi < W::NG; ++gi) w.kz[nt][gi][j] = unit * __shfl_sync(kFull, sum[gi], src);
    }
  }
}

// ------------------------------------------------------------------ scores of 16 tokens
// acc[blk * KG + half][nt] += K codes (rows = tokens t0 + gid, t0 + gid + 8) x q.
template <int KB, int D, int NT, bool G32>
__device__ __forceinline__ void k_product(const uint8_t* kc, const Work<D, NT, G32>& w,
                                          float (&acc)[Work<D, NT, G32>::BLK * Work<D, NT, G32>::KG][NT][4]) {
  using W = Work<D, NT, G32>;
  constexpr int RB = D * KB / 8, SW = KB / 2;  // row bytes, words of a lane's 16 codes
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int blk = 0; blk < W::BLK; ++blk) {
    uint32_t x[SW], y[SW];
    const uint8_t* p = kc + gid * RB + blk * 8 * KB + tig * 2 * KB;
    if constexpr (SW % 4 == 0) {
#pragma unroll
      for (int i = 0; i < SW; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + 4 * i), v = *reinterpret_cast<const uint4*>(p + 8 * RB + 4 * i);
        x[i] = u.x; x[i + 1] = u.y; x[i + 2] = u.z; x[i + 3] = u.w;
        y[i] = v.x; y[i + 1] = v.y; y[i + 2] = v.z; y[i + 3] = v.w;
      }
    } else if constexpr (SW == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(p), v = *reinterpret_cast<const uint2*>(p + 8 * RB);
      x[0] = u.x; x[1] = u.y; y[0] = v.x; y[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        x[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
        y[i] = *reinterpret_cast<const uint32_t*>(p + 8 * RB + 4 * i);
      }
    }
    auto step = [&](auto ks_c) {
      constexpr int ks = decltype(ks_c)::value;
      const uint32_t a0 = k_reg<KB, 2 * ks, SW>(x), a1 = k_reg<KB, 2 * ks, SW>(y);
      const uint32_t a2 = k_reg<KB, 2 * ks + 1, SW>(x), a3 = k_reg<KB, 2 * ks + 1, SW>(y);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t b0 = w.qf[nt][blk][2 * ks], b1 = w.qf[nt][blk][2 * ks + 1];
        if constexpr (KB == 16) {
          hmma16816_bf16(acc[blk * W::KG][nt], a0, a1, a2, a3, b0, b1);
        } else if constexpr (!G32) {
          hmma16816(acc[blk][nt], a0, a1, a2, a3, b0, b1);
        } else {
          // lanes tig < 2 hold the block's first group of 32 channels, the others its second
          hmma16816(acc[2 * blk][nt], a0, a1, a2, a3, tig < 2 ? b0 : 0u, tig < 2 ? b1 : 0u);
          hmma16816(acc[2 * blk + 1][nt], a0, a1, a2, a3, tig < 2 ? 0u : b0, tig < 2 ? 0u : b1);
        }
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
}

// out += sum over the 16 tokens of (e * scale) code: rows = channels, slots
// 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9 = tokens tig, tig + 4, tig + 8, tig + 12.
// dead: bit j set when no row of the unit sees token tig + 4 j (its 16-bit
// values may be anything and are taken as zero; codes are finite as they are).
template <int VB, int D, int NT, bool G32>
__device__ __forceinline__ void v_product(const uint8_t* vc, const float* vsz, int ng, Work<D, NT, G32>& w,
                                          const float (&e)[NT][4], const unsigned (&seen)[NT], unsigned dead) {
  using W = Work<D, NT, G32>;
  constexpr int RB = D * VB / 8;
  constexpr int CH = (G32 && VB != 16) ? 4 : 8;  // codes of a lane's run; a run stays inside one group
  constexpr int NB = D / (8 * CH), TPB = CH / 2; // runs of a row per lane, m-tiles of a run
  constexpr int N = VRun<VB, CH>::N;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int per = D / (8 * CH) / (VB == 16 ? 1 : ng);  // runs of one group
  uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    const bool fresh = VB == 16 ? blk == 0 : blk % per == 0;
    if (fresh) {
      float sc[4], ze[4];
      if constexpr (VB != 16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 t = *reinterpret_cast<const float2*>(vsz + ((tig + 4 * j) * ng + blk / per) * 2);
          sc[j] = t.x; ze[j] = centre<VB>(t.x, t.y);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (VB == 16) {
            x[j] = e[nt][j];
          } else {
            // a row that does not see the token must not meet its (scale, zero): they may be anything
            const bool ok = seen[nt] >> j & 1;
            x[j] = ok ? e[nt][j] * sc[j] : 0.0f;
            if (ok) w.zacc[nt][blk / (NB / W::NG)] += e[nt][j] * ze[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          hi[nt][j] = pack_bf16(x[2 * j], x[2 * j + 1]);
          lo[nt][j] = pack_bf16(x[2 * j] - bf16_lo(hi[nt][j]), x[2 * j + 1] - bf16_hi(hi[nt][j]));
        }
      }
    }
    uint32_t run[4][N];
#pragma unroll
    for (int j = 0; j < 4; ++j) load_run<VB, CH>(vc + (tig + 4 * j) * RB, blk, gid, run[j]);
    if constexpr (VB == 16) {
      if (dead) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) run[j][i] = dead >> j & 1 ? 0u : run[j][i];
      }
    }
    uint32_t u[CH], v[CH];
    pair_codes<VB, CH>(run[0], run[1], u);
    pair_codes<VB, CH>(run[2], run[3], v);
#pragma unroll
    for (int mi = 0; mi < TPB; ++mi)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        hmma16816_bf16(w.o[blk * TPB + mi][nt], u[2 * mi], u[2 * mi + 1], v[2 * mi], v[2 * mi + 1], hi[nt][0], hi[nt][1]);
        hmma16816_bf16(w.o[blk * TPB + mi][nt], u[2 * mi], u[2 * mi + 1], v[2 * mi], v[2 * mi + 1], lo[nt][0], lo[nt][1]);
      }
  }
}

// Channel of output register (mt, half) for lane gid: runs of CH channels.
template <int D, bool G32>
__device__ __forceinline__ int out_channel(int mt, int half, int gid, bool wide) {
  if (G32 && !wide) return (mt / 2) * 32 + gid * 4 + (mt % 2) * 2 + half;
  return (mt / 4) * 64 + gid * 8 + (mt % 4) * 2 + half;
}

// 16 tokens from position t0 (n of them staged): scores, running softmax, output.
template <int D, int NT, bool G32>
__device__ __forceinline__ void step16(const MultiArgs& a, Work<D, NT, G32>& w, const uint8_t* kc, const float* ksz,
                                       const uint8_t* vc, const float* vsz, float* tr, int t0, int ng) {
  using W = Work<D, NT, G32>;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  float acc[W::BLK * W::KG][NT][4];
#pragma unroll
  for (int i = 0; i < W::BLK * W::KG; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][nt][j] = 0.0f;
  switch (a.kb) {
    case 2: k_product<2, D, NT, G32>(kc, w, acc); break;
    case 4: k_product<4, D, NT, G32>(kc, w, acc); break;
    case 6: k_product<6, D, NT, G32>(kc, w, acc); break;
    case 8: k_product<8, D, NT, G32>(kc, w, acc); break;
    default: k_product<16, D, NT, G32>(kc, w, acc); break;
  }
  // fold (scale, zero): rows gid and gid + 8, columns 2 tig and 2 tig + 1
  float s[NT][4];
  if (a.kb == 16) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float t = acc[0][nt][j];
        if constexpr (W::BLK == 2) t += acc[W::KG][nt][j];
        s[nt][j] = t * w.ka[nt][j & 1];
      }
  } else {
    float sc[2][W::NG], ze[2][W::NG];
    const float mid = (float)(1 << (a.kb - 1));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int gi = 0; gi < W::NG; ++gi) {
        const float2 t = *reinterpret_cast<const float2*>(ksz + ((gid + 8 * i) * ng + gi * ng / W::NG) * 2);
        sc[i][gi] = t.x; ze[i][gi] = fmaf(mid, t.x, t.y);
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float t = sc[j >> 1][0] * acc[0][nt][j];
#pragma unroll
        for (int gi = 1; gi < W::NG; ++gi) t = fmaf(sc[j >> 1][gi], acc[gi][nt][j], t);
        float z = ze[j >> 1][0] * w.kz[nt][0][j & 1];
#pragma unroll
        for (int gi = 1; gi < W::NG; ++gi) z = fmaf(ze[j >> 1][gi], w.kz[nt][gi][j & 1], z);
        s[nt][j] = fmaf(t, w.ka[nt][j & 1], z);
      }
  }
  // transpose through shared memory: lane (gid, tig) takes row gid, tokens tig + 4 j
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    *reinterpret_cast<float2*>(tr + nt * 128 + gid * 8 + 2 * tig) = make_float2(s[nt][0], s[nt][1]);
    *reinterpret_cast<float2*>(tr + nt * 128 + (gid + 8) * 8 + 2 * tig) = make_float2(s[nt][2], s[nt][3]);
  }
  __syncwarp();
  float e[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) e[nt][j] = tr[nt * 128 + (tig + 4 * j) * 8 + gid];
  __syncwarp();
  if (a.softcap > 0.0f) {
    const float c = a.softcap * kLog2e;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[nt][j] = c * tanhf(e[nt][j]);
  }
  if (a.slopes != nullptr) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[nt][j] = fmaf(w.slope[nt], (float)(t0 + tig + 4 * j - w.p[nt]), e[nt][j]);
  }
  const bool whole = t0 + 15 < w.T && ((t0 >= w.lo_max && t0 + 15 <= w.p_min) || t0 + 15 < w.pre);
  unsigned seen[NT], dead = 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) seen[nt] = w.on[nt] ? 15u : 0u;
  if (!whole) {
    unsigned any = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = t0 + tig + 4 * j;
        const bool ok = w.on[nt] && t < w.T && (t < w.pre || (t >= w.lo[nt] && t <= w.p[nt]));
        if (!ok) seen[nt] &= ~(1u << j);
        if (ok) any |= 1u << j;
      }
    // seen by any row of the unit: over the lanes of the same tig
    any |= __shfl_xor_sync(kFull, any, 4);
    any |= __shfl_xor_sync(kFull, any, 8);
    any |= __shfl_xor_sync(kFull, any, 16);
    dead = ~any & 15u;
  }
  float mx[NT];
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!(seen[nt] >> j & 1)) e[nt][j] = -INFINITY;
    float t = fmaxf(fmaxf(e[nt][0], e[nt][1]), fmaxf(e[nt][2], e[nt][3]));
    t = fmaxf(t, __shfl_xor_sync(kFull, t, 1));
    t = fmaxf(t, __shfl_xor_sync(kFull, t, 2));
    mx[nt] = t;
    grow |= t > w.m[nt] + kLazy;  // from -inf: any finite score
  }
  if (__any_sync(kFull, grow)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m = fmaxf(w.m[nt], mx[nt]);
      const float al = m == -INFINITY ? 1.0f : ex2(w.m[nt] - m);
      w.m[nt] = m;
      w.l[nt] *= al;
#pragma unroll
      for (int gi = 0; gi < W::NG; ++gi) w.zacc[nt][gi] *= al;
      const float a0 = __shfl_sync(kFull, al, 8 * tig), a1 = __shfl_sync(kFull, al, 8 * tig + 4);
#pragma unroll
      for (int mt = 0; mt < W::MT; ++mt) {
        w.o[mt][nt][0] *= a0; w.o[mt][nt][1] *= a1;
        w.o[mt][nt][2] *= a0; w.o[mt][nt][3] *= a1;
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float m = w.m[nt] == -INFINITY ? 0.0f : w.m[nt];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[nt][j] = ex2(e[nt][j] - m);
    w.l[nt] += (e[nt][0] + e[nt][1]) + (e[nt][2] + e[nt][3]);
  }
  switch (a.vb) {
    case 2: v_product<2, D, NT, G32>(vc, vsz, ng, w, e, seen, dead); break;
    case 4: v_product<4, D, NT, G32>(vc, vsz, ng, w, e, seen, dead); break;
    case 6: v_product<6, D, NT, G32>(vc, vsz, ng, w, e, seen, dead); break;
    case 8: v_product<8, D, NT, G32>(vc, vsz, ng, w, e, seen, dead); break;
    default: v_product<16, D, NT, G32>(vc, vsz, ng, w, e, seen, dead); break;
  }
}

// ------------------------------------------------------------------ writing a unit or a piece
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY; }

// A piece: (max, sum) of 8 NT rows, then their partial outputs.
template <int D, int NT>
constexpr int piece_floats() { return 8 * NT * (D + 2); }

template <int D, int NT, bool G32>
__device__ __forceinline__ void flush(const MultiArgs& a, Work<D, NT, G32>& w, float* piece) {
  using W = Work<D, NT, G32>;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const bool wide = a.vb == 16;
  const int rows = min(8 * NT, w.n * a.r - w.rb * 8 * NT);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float l = w.l[nt];
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
#pragma unroll
    for (int gi = 0; gi < W::NG; ++gi) {
      float z = w.zacc[nt][gi];
      z += __shfl_xor_sync(kFull, z, 1);
      z += __shfl_xor_sync(kFull, z, 2);
      w.zacc[nt][gi] = z;
    }
    const int mine = nt * 8 + gid;
    if (tig == 0 && mine < rows) {
      if (piece != nullptr) {
        *reinterpret_cast<float2*>(piece + 2 * mine) = make_float2(w.m[nt], l);
      } else if (a.lse != nullptr) {
        const int row = w.rb * 8 * NT + mine;
        a.lse[(long long)(w.c0 + row / a.r) * a.Hq + w.g * a.r + row % a.r] = lse_of(w.m[nt], l);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int src = 4 * (2 * tig + j), col = nt * 8 + 2 * tig + j;
      const float lc = __shfl_sync(kFull, l, src);
      float z[W::NG];
#pragma unroll
      for (int gi = 0; gi < W::NG; ++gi) z[gi] = __shfl_sync(kFull, w.zacc[nt][gi], src);
      const float f = piece != nullptr ? 1.0f : (lc > 0.0f ? 1.0f / lc : 0.0f);
      if (col < rows) {
        float* dst;
        if (piece != nullptr) {
          dst = piece + 16 * NT + col * D;
        } else {
          const int row = w.rb * 8 * NT + col;
          dst = a.out + ((long long)(w.c0 + row / a.r) * a.Hq + w.g * a.r + row % a.r) * D;
        }
#pragma unroll
        for (int mt = 0; mt < W::MT; mt += 2) {
          // at G = 128 both 64-channel blocks share slot 0
          const float zz = G32 ? z[mt / 2] : (D / a.G < W::NG ? z[0] : z[mt / 4]);
          if (G32 && wide) {  // 16-bit runs span both 32-channel slots, which hold no zeros
            *reinterpret_cast<float4*>(dst + out_channel<D, G32>(mt, 0, gid, true)) =
                make_float4(w.o[mt][nt][j] * f, w.o[mt][nt][2 + j] * f, w.o[mt + 1][nt][j] * f, w.o[mt + 1][nt][2 + j] * f);
          } else {
            *reinterpret_cast<float4*>(dst + out_channel<D, G32>(mt, 0, gid, wide)) =
                make_float4((w.o[mt][nt][j] + zz) * f, (w.o[mt][nt][2 + j] + zz) * f, (w.o[mt + 1][nt][j] + zz) * f,
                            (w.o[mt + 1][nt][2 + j] + zz) * f);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
// A cut unit: its tiles [u0, u1) in the list, and whose it is.
struct Cut {
  int u0, u1, b, ui;
};

// The tile that a warp looks at next.
struct Cursor {
  Seq s;
  int b, ui, ti;
};

template <int NT>
__device__ __forceinline__ void seek(const MultiArgs& a, const int* first, int x, Cursor& c) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  c.b = lo;
  c.s = load_seq<NT>(a, lo);
  const int rem = x - first[lo];
  c.ui = rem / c.s.cnt;
  c.ti = rem % c.s.cnt;
}

template <int NT>
__device__ __forceinline__ void advance(const MultiArgs& a, const int* first, Cursor& c) {
  if (++c.ti < c.s.cnt) return;
  c.ti = 0;
  if (++c.ui < c.s.units) return;
  c.ui = 0;
  do ++c.b; while (c.b < a.B && first[c.b + 1] == first[c.b]);  // past sequences without new tokens
  if (c.b < a.B) c.s = load_seq<NT>(a, c.b);
}

__device__ __forceinline__ int tile_pos(const Seq& s, int ti, int tt) { return (ti < s.np ? ti : s.t_lo + ti - s.np) * tt; }

// Start the copies of a tile into a stage; the bytes complete on bar.
__device__ __forceinline__ void fetch_tile(const MultiArgs& a, const Cursor& c, int rbs, uint8_t* stage, uint64_t* bar,
                                           int krb, int vrb, int ng, uint64_t policy) {
  const int t0 = tile_pos(c.s, c.ti, a.tt);
  int n = min(a.tt, c.s.T - t0);
  if (n <= 0) return;
  if (ng & 1) n += n & 1;  // (scale, zero) rows of 8 bytes go in pairs; the capacity is even then
  const int g = c.ui / rbs;
  long long row;
  if (a.table == nullptr) {
    row = ((long long)c.b * a.Hkv + g) * a.T_cap + t0;
  } else {
    int page = __ldg(a.table + (long long)c.b * a.pps + t0 / kPageTokens);
    if (page < 0 || page >= a.num_pages) {
      atomicMax(a.status, kStatusInvalidArg);
      page = 0;
    }
    row = ((long long)page * a.Hkv + g) * kPageTokens + t0 % kPageTokens;
  }
  const uint32_t kbytes = n * krb, vbytes = n * vrb, sz = n * ng * 8;
  mbar_arrive_expect_tx(bar, kbytes + vbytes + (a.kb < 16 ? sz : 0) + (a.vb < 16 ? sz : 0));
  bulk_g2s(stage, a.kc + row * krb, kbytes, bar, policy);
  if (a.kb < 16) bulk_g2s(stage + a.off_ksz, a.ksz + row * ng * 2, sz, bar, policy);
  bulk_g2s(stage + a.off_vc, a.vc + row * vrb, vbytes, bar, policy);
  if (a.vb < 16) bulk_g2s(stage + a.off_vsz, a.vsz + row * ng * 2, sz, bar, policy);
}

// Join the pieces of a cut unit, one (row, 4 channels) element per thread and
// step; piece k of [k0, k1) is at pieces + (2 k + slot) * PF, slot 1 when the
// unit starts behind the k-th run's begin.  Writes the unit's output, or the
// joined piece `to`.
template <int D, int NT, typename Begin>
__device__ __forceinline__ void join_element(const MultiArgs& a, const Cut& u, const Seq& s, int el, const float* pieces,
                                             int k0, int k1, Begin begin, float* to) {
  constexpr int PF = piece_floats<D, NT>();
  const int row_in = el / (D / 4), d4 = el % (D / 4);
  const int rbs = s.units / a.Hkv, g = u.ui / rbs, rb = u.ui % rbs;
  const int row = rb * 8 * NT + row_in;
  if (row >= s.n * a.r) return;
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k = k0; k < k1; ++k) {
    if (begin(k) == begin(k + 1)) continue;  // an empty run has no piece
    const float* p = pieces + (long long)(2 * k + (u.u0 > begin(k) ? 1 : 0)) * PF;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + 2 * row_in));
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + 16 * NT + row_in * D) + d4);
    const float m = fmaxf(M, ml.x);
    if (m == -INFINITY) continue;
    const float f = ex2(M - m), f2 = ex2(ml.x - m);
    L = L * f + ml.y * f2;
    o.x = o.x * f + v.x * f2; o.y = o.y * f + v.y * f2;
    o.z = o.z * f + v.z * f2; o.w = o.w * f + v.w * f2;
    M = m;
  }
  if (to != nullptr) {
    if (d4 == 0) *reinterpret_cast<float2*>(to + 2 * row_in) = make_float2(M, L);
    reinterpret_cast<float4*>(to + 16 * NT + row_in * D)[d4] = o;
  } else {
    const long long at = (long long)(s.c0 + row / a.r) * a.Hq + g * a.r + row % a.r;
    const float f = L > 0.0f ? 1.0f / L : 0.0f;
    reinterpret_cast<float4*>(a.out + at * D)[d4] = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    if (d4 == 0 && a.lse != nullptr) a.lse[at] = lse_of(M, L);
  }
}

template <int D, int NT, bool G32>
__global__ void __launch_bounds__(32 * kWarpsFor(NT), 1) multi_kernel(MultiArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x / 32;
  constexpr int PF = piece_floats<D, NT>();
  const int ng = D / a.G;
  const int krb = D * a.kb / 8, vrb = D * a.vb / 8;

  __shared__ int s_wsum[32];
  __shared__ Cut s_cut[kMaxWarps + 1];
  __shared__ int s_ncut;
  __shared__ int s_last[2];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  float* tr = reinterpret_cast<float*>(smem + a.off_tr) + warp * 128 * NT;
  int* first = reinterpret_cast<int*>(smem + a.off_first);
  uint8_t* ring = smem + a.off_ring + (size_t)warp * a.stages * a.stage_bytes;
  uint64_t* bar = bars + warp * a.stages;

  // tiles before each sequence
  {
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq<NT>(a, b);
      mine += s.units * s.cnt;
      first[b] = s.units * s.cnt;
      if (blockIdx.x == 0) {
        const int t = __ldg(a.lens + b);
        bool bad = t < 0 || t > a.T_cap;
        if (a.cu_q != nullptr) {
          const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1);
          bad |= c0 < 0 || c1 < c0 || c1 > a.n_rows || c1 - c0 > a.max_q;
        }
        if (bad) atomicMax(a.status, kStatusInvalidArg);
      }
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) s_wsum[warp] = incl;
    if (lane < a.stages) mbar_init(bar + lane, 1);
    fence_mbar_init();
    __syncthreads();
    int run = incl - mine;
    for (int w = 0; w < warp; ++w) run += s_wsum[w];
    for (int b = b0; b < b1; ++b) { const int c = first[b]; first[b] = run; run += c; }
    if (tid == (int)blockDim.x - 1) first[a.B] = run;
    __syncthreads();
  }
  const int total = first[a.B];
  if (total == 0) return;
  // as many CTAs as give every warp a tile: fewer cuts, and no join between CTAs for small calls
  const int C = min((int)gridDim.x, (total + W - 1) / W);
  const int cta = blockIdx.x;
  if (cta >= C) return;
  auto cta_begin = [&](int c) { return (int)((long long)total * c / C); };
  const int x0 = cta_begin(cta), x1 = cta_begin(cta + 1);
  auto warp_begin = [&](int w) { return x0 + (int)((long long)(x1 - x0) * w / W); };

  {
    const int w0 = warp_begin(warp), w1 = warp_begin(warp + 1);
    float* pieces = a.pieces + (long long)(cta * W + warp) * 2 * PF;
    const uint64_t limit = *a.timeout_ns ? *a.timeout_ns : 2000000000ull;
    const uint64_t policy = policy_evict_first();
    bool dead = false;
    if (w0 < w1) {
      Cursor c, f;  // the tile being used and the tile being fetched
      seek<NT>(a, first, w0, c);
      f = c;
      int fx = w0;
      for (int i = 0; i < a.stages && fx < w1; ++i, ++fx) {
        if (lane == 0) fetch_tile(a, f, f.s.units / a.Hkv, ring + i * a.stage_bytes, bar + i, krb, vrb, ng, policy);
        advance<NT>(a, first, f);
      }
      Work<D, NT, G32> w;
      load_unit<D, NT, G32>(a, c.s, c.b, c.ui, w);
      int st = 0;
      uint32_t parity = 0;  // bit i: phase of stage i
      for (int x = w0; x < w1; ++x) {
        const int t0 = tile_pos(c.s, c.ti, a.tt);
        const int n = min(a.tt, c.s.T - t0);
        uint8_t* stage = ring + st * a.stage_bytes;
        if (n > 0) {
          if (!dead && !mbar_wait(bar + st, parity >> st & 1, limit)) {
            if (lane == 0) atomicMax(a.status, kStatusTimeout);
            dead = true;
          }
          dead = __any_sync(kFull, dead);
          parity ^= 1u << st;
          if (!dead) {
            const float* ksz = reinterpret_cast<const float*>(stage + a.off_ksz);
            const float* vsz = reinterpret_cast<const float*>(stage + a.off_vsz);
            for (int k = 0; k < n; k += 16)
              step16<D, NT, G32>(a, w, stage + k * krb, ksz + k * ng * 2, stage + a.off_vc + k * vrb, vsz + k * ng * 2, tr,
                                 t0 + k, ng);
          }
        }
        __syncwarp();
        if (fx < w1) {
          if (lane == 0 && !dead) {
            fence_proxy_async_smem();
            fetch_tile(a, f, f.s.units / a.Hkv, stage, bar + st, krb, vrb, ng, policy);
          }
          advance<NT>(a, first, f);
          ++fx;
        }
        st = st + 1 == a.stages ? 0 : st + 1;
        const bool end = c.ti + 1 == c.s.cnt;
        if (end || x + 1 == w1) {
          const int u0 = x - c.ti;  // the unit's first tile
          const bool all = end && u0 >= w0;
          flush<D, NT, G32>(a, w, all ? nullptr : pieces + (u0 > w0 ? PF : 0));
        }
        if (x + 1 < w1) {
          advance<NT>(a, first, c);
          if (end) load_unit<D, NT, G32>(a, c.s, c.b, c.ui, w);
        }
      }
      // after a wait that gave up: let the copies still in flight land before the shared memory goes
      if (dead)
        for (int i = 0; i < a.stages; ++i) mbar_wait(bar + i, parity >> i & 1, 1000000ull);
    }
  }
  __syncthreads();

  // ---- units cut by a run end: one thread per boundary finds its unit
  if (warp == 0) {
    Cut u{0, 0, 0, 0};
    bool cut = false;
    if (lane <= W) {
      const int x = lane < W ? warp_begin(lane) : x1;
      if (x < total) {
        Cursor c;
        seek<NT>(a, first, x, c);
        u.u0 = x - c.ti; u.u1 = u.u0 + c.s.cnt; u.b = c.b; u.ui = c.ui;
        cut = u.u0 < x;
      }
    }
    // boundaries rise, so equal units stand side by side (among those that cut)
    unsigned cuts = __ballot_sync(kFull, cut);
    const unsigned below = cuts & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : 0;
    const int pu = __shfl_sync(kFull, u.u0, prev);
    const bool lead = cut && (!below || pu != u.u0);
    const unsigned leads = __ballot_sync(kFull, lead);
    if (lead) s_cut[__popc(leads & ((1u << lane) - 1u))] = u;
    if (lane == 0) { s_ncut = __popc(leads); s_last[0] = s_last[1] = 0; }
  }
  __syncthreads();
  const int ncut = s_ncut;
  constexpr int EL = 8 * NT * D / 4;
  const float* mine = a.pieces + (long long)cta * W * 2 * PF;
  float* cpieces = a.cpieces;
  bool shared_any = false;
  for (int i = 0; i < ncut; ++i) {
    const Cut u = s_cut[i];
    const bool shared = u.u0 < x0 || u.u1 > x1;
    shared_any |= shared;
  }
  for (int el = tid; el < ncut * EL; el += blockDim.x) {
    const Cut u = s_cut[el / EL];
    const Seq s = load_seq<NT>(a, u.b);
    const bool shared = u.u0 < x0 || u.u1 > x1;
    int k0 = 0, k1 = W;
    while (k0 < W && warp_begin(k0 + 1) <= u.u0) ++k0;
    while (k1 > k0 && warp_begin(k1 - 1) >= u.u1) --k1;
    float* to = shared ? cpieces + (long long)(2 * cta + (u.u0 > x0 ? 1 : 0)) * PF : nullptr;
    join_element<D, NT>(a, u, s, el % EL, mine, k0, k1, warp_begin, to);
  }
  if (!shared_any) return;

  // ---- units cut between CTAs: the last to arrive joins the CTAs' pieces
  __threadfence();
  __syncthreads();
  auto cta_of = [&](int x) { return (int)((((long long)x + 1) * C - 1) / total); };
  if (tid < 2) {
    const int i = tid == 0 ? 0 : ncut - 1;
    const Cut u = s_cut[i];
    const bool shared = (u.u0 < x0 || u.u1 > x1) && (tid == 0 || i != 0);
    if (shared) {
      const int want = cta_of(u.u1 - 1) - cta_of(u.u0) + 1;
      int* arrive = a.arrive + cta_of(u.u0);  // a CTA begins at most one unit that it does not end
      __threadfence();
      const int got = atomicAdd(arrive, 1) + 1;
      if (got == want) {
        *arrive = 0;  // ready for the next call
        __threadfence();
        s_last[tid] = 1;
      }
    }
  }
  __syncthreads();
  for (int t = 0; t < 2; ++t) {
    if (!s_last[t]) continue;
    const Cut u = s_cut[t == 0 ? 0 : ncut - 1];
    const Seq s = load_seq<NT>(a, u.b);
    for (int el = tid; el < EL; el += blockDim.x)
      join_element<D, NT>(a, u, s, el, cpieces, cta_of(u.u0), cta_of(u.u1 - 1) + 1, cta_begin, nullptr);
  }
}

}  // namespace multi
}  // namespace lkv
