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
// so both products run on integer codes, exact in fp16.  The codes are
// centred -- any integer may move from the codes into zero -- because with
// codes from 0 up the two terms are large and cancel.  V takes the middle code.
// K takes the code nearest to the value 0: its outlier channels stretch the
// range of a group, and the middle can lie far from most of its values.
//
// What bounds it: the packed rows, read once (K6V4, D 128, G 64: 192 bytes a
// row, 8.3 clocks of one SM at the copy bandwidth), and the instructions that
// turn codes into MMA operands, which take longer than the bytes.  So:
//   - tokens are the M rows of mma.m16n8k16 in the K product and its K rows in
//     the V product, and the query rows (heads of the group x new tokens) its
//     N = 8 columns: with 1 to 8 query rows nothing but columns is padded;
//   - K codes become fp16 integers against q scaled by a power of two
//     (mma_k.cuh): exact products.  V codes become fp16 integers against
//     e * scale split in two fp16 terms (22 bits), in a unit of its own for each
//     query row and channel group: a power of two that keeps e * scale below
//     2^15 and moves only when one passes that.  It follows the products and not
//     the scales, since a token of large scale may have no weight, and a small
//     group may stand beside a large one.  At the 16-bit width both products are
//     bf16, e split in three terms;
//   - the channel-to-row and token-to-slot orders of the MMAs are free, so
//     every lane reads whole runs of codes of one token from shared memory,
//     and the codes of two tokens are paired by one byte permute per half
//     word, before they are unpacked;
//   - what depends on a token alone -- centring, the zeroing of what nobody
//     sees -- is done once, by the lane of that token, in the tile's (scale, zero)
//     rows in shared memory;
//   - the reference exponent is an integer and moves only when a score passes
//     it by 2^8, so rescaling is rare and exact.
//
// Work split: the tiles (32 tokens, 16 where rows are wide) of all units -- a
// unit is one (sequence, KV head, block of 8 NT query rows) -- lie end to end,
// and every warp of the grid takes an equal run of them with a ring of its own
// in shared memory: no barrier until the end.  A unit inside one warp's run is
// written straight out.  Units cut by run ends leave (exponent, sum, partial
// output) pieces in the workspace; the CTA joins those of its warps, and for a
// unit cut between CTAs the last one to arrive joins the CTAs' pieces, always
// in order, so results do not depend on timing.
//
// Measured on a B200, device time: K6V4, B16 x 8192, 32 / 8 heads, capped and
// paged: 73 us for 201.7 MB (2.8 TB/s); 16 query rows over 131072 tokens: 121 us
// (113 before the units followed the products: 7% more instructions); 8-bit, G 32,
// 64 ragged sequences behind a window of 1024: 59 us for 167 MB.
#pragma once
#include <type_traits>

#include "lkv_kernels.cuh"
#include "mma_k.cuh"
#include "multi.cuh"

namespace lkv {
namespace multi {

using fused::hsub2_u32;
using fused::kF16Magic2;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;      // the reference moves when a score passes it by 2^8
// Units of e * scale in fp16: a row whose products may reach 2^15 (fp16 ends at
// 65504) has them moved.  The bound is the row's largest e times the tile's
// largest scale.  Where the tile's scales lie within 2^kNarrow, the largest
// product is at least 2^-(kNarrow + 2) of it, good enough to place a unit by: one
// power moves all groups of the row and the bound comes to 2^kPlace, that of the
// smallest group to 2^(kPlace - kSpread) or more.  Elsewhere the largest product of
// each group is found and comes to 2^kPlace itself.  What fp16 drops, 2^-25, is
// then 2^-25 of a group's largest product at worst and 2^-33 as a rule.
constexpr int kOverExp = 15, kPlace = 8;
constexpr unsigned kNarrow = 3, kSpread = 3, kLeast = 127 - 90;  // the last: from 2^-90 the units are normal numbers
constexpr float kOver = (float)(1 << kOverExp);
constexpr int kUnitMax = 126;  // its inverse is a normal number

__device__ __forceinline__ float ex2(float x) {  // 2^x; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// mma.m16n8k16, fp32 accumulators (fragment layout: mma_k.cuh).  Pure functions
// of their operands, so that independent products may be interleaved.
__device__ __forceinline__ void hmma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void hmma16816_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero: c need not be cleared.
__device__ __forceinline__ void hmma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void hmma16816_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The exponent of a positive normal number.
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// 2^n for an integer-valued n; 0 below the normal range.
__device__ __forceinline__ float pow2i(float n) {
  return n < -126.0f ? 0.0f : __uint_as_float((uint32_t)((int)fminf(n, 127.0f) + 127) << 23);
}

// tanh from its continued fraction x / (1 + x^2 / (3 + x^2 / (5 + ...))), cut
// after the 13: relative error below 2e-7 up to |x| = 2.  Beyond, from the
// exponential, where 2 / (1 + e^2x) is small and its error smaller still.
__device__ __forceinline__ float tanh_near(float x) {
  const float y = x * x;
  const float num = fmaf(fmaf(y + 378.0f, y, 17325.0f), y, 135135.0f);
  const float den = fmaf(fmaf(fmaf(28.0f, y, 3150.0f), y, 62370.0f), y, 135135.0f);
  return x * num * rcp(den);
}
__device__ __forceinline__ float tanh_far(float x) {
  const float t = 1.0f - 2.0f * rcp(1.0f + ex2(2.0f * kLog2e * fabsf(x)));
  return copysignf(t, x);
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

template <int NT, int TT>
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
  const int hi_t = (s.T + TT - 1) / TT, pre_t = (s.pre + TT - 1) / TT;
  s.t_lo = s.lo / TT;
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

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 unpack_f16(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Code c of a run stays at this bit of its half word (no shift below 10 bits of
// mantissa): its MMA operand carries the factor 2^off, taken out at the end.
template <int VB>
constexpr int code_off(int c) {
  return VB == 2 ? 2 * (c & 3) : VB == 4 ? 4 * (c & 1) : 0;
}

// Centred codes of two tokens (runs x, y) as fp16 pairs (x in the low half),
// exact: out[c] = (code_c - 2^(VB-1)) * 2^off for c = 0 .. CH-1.  A code is
// placed under the pattern 0x6400 (1024, unit spacing) and the pattern and the
// middle subtracted at once; 16 bits are the bf16 values themselves.
template <int VB, int CH>
__device__ __forceinline__ void pair_codes(const uint32_t (&x)[VRun<VB, CH>::N], const uint32_t (&y)[VRun<VB, CH>::N],
                                           uint32_t (&out)[CH]) {
  if constexpr (VB == 16) {
#pragma unroll
    for (int c = 0; c < CH; ++c) out[c] = __byte_perm(x[c / 2], y[c / 2], (c & 1) ? 0x7632 : 0x5410);
  } else if constexpr (VB == 8) {
#pragma unroll
    for (int c = 0; c < CH; c += 2) {
      const uint32_t z = __byte_perm(x[c / 4], y[c / 4], (c & 2) ? 0x7362 : 0x5140);  // {x, y, x', y'}
      out[c] = hsub2_u32(__byte_perm(z, 0x64646464u, 0x4140), kF16Magic2 + 0x00800080u);
      out[c + 1] = hsub2_u32(__byte_perm(z, 0x64646464u, 0x4342), kF16Magic2 + 0x00800080u);
    }
  } else {
    constexpr int cw = VB == 2 ? 8 : VB == 4 ? 4 : 2;  // codes of one 16-bit window
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
      for (int c = 0; c < cw && c0 + c < CH; ++c) {
        const int off = code_off<VB>(c);
        const uint32_t mask = (((1u << VB) - 1u) << off) * 0x00010001u, mid = ((1u << (VB - 1)) << off) * 0x00010001u;
        out[c0 + c] = hsub2_u32(((z >> (c * VB - off)) & mask) | kF16Magic2, kF16Magic2 + mid);
      }
    }
  }
}

// ------------------------------------------------------------------ one warp's state
template <int D_, int KB_, int VB_, int G_, int NT_>
struct Cfg {
  static constexpr int D = D_, KB = KB_, VB = VB_, G = G_, NT = NT_;
  static constexpr int WARPS = shape_of(D_, KB_, VB_, G_, NT_).warps;
  static constexpr int STAGES = shape_of(D_, KB_, VB_, G_, NT_).stages, STAGE = shape_of(D_, KB_, VB_, G_, NT_).stage;
  static constexpr int OFF_KSZ = shape_of(D_, KB_, VB_, G_, NT_).off_ksz, OFF_VC = shape_of(D_, KB_, VB_, G_, NT_).off_vc;
  static constexpr int OFF_VSZ = shape_of(D_, KB_, VB_, G_, NT_).off_vsz, SCRATCH = shape_of(D_, KB_, VB_, G_, NT_).scratch;
  static constexpr int TT = shape_of(D_, KB_, VB_, G_, NT_).tt, TS = TT / 16;  // tokens of a tile, MMA tiles of it
  static constexpr int BLK = D / 64;                // 64-channel blocks
  static constexpr int MT = D / 16;                 // m-tiles of the output
  static constexpr int NG = D / G;                  // groups
  static constexpr int AC = KB == 16 ? 1 : NG;      // accumulators of a score: one per group
  static constexpr int KRB = D * KB / 8, VRB = D * VB / 8;
  // codes of a lane's V run: a run stays inside one group
  static constexpr int CH = (G == 32 && VB != 16) ? 4 : 8;
  static constexpr int RUNS = D / (8 * CH), TPB = CH / 2;  // runs of a row per lane, m-tiles of a run
  static constexpr int GRUNS = VB == 16 ? RUNS : RUNS / NG;  // runs of one group
};

template <typename C>
struct Work {
  float o[C::MT][C::NT][4];
  float zacc[C::NT][C::NG];   // sum of e * zero, this lane's tokens, row gid
  float ref[C::NT], l[C::NT]; // reference exponent (an integer) and sum of e (this lane's tokens), row gid
  bool live[C::NT];           // the row has seen a token
  float refc[C::NT][2];       // references of columns 2 tig and 2 tig + 1 (0 when scores are capped)
  float u[C::NT][C::NG];      // o of row gid is the output times 2^-ref times this, a power of two (quantized V)
  int orow[C::NT];            // row gid's place in out: row * Hq + head
  uint32_t qf[C::NT][C::BLK][8];
  float ka[C::NT][2];              // factor of the code product, columns 2 tig and 2 tig + 1
  float kz[C::NT][C::NG][2];       // the same times the sum of q over the group: the factor of zero
  int p[C::NT], lo[C::NT];         // row gid: position of its token, first visible token behind the prefix
  float slope[C::NT];
  bool on[C::NT];
  int g, rb, T, c0, n, pre, p_min, p_max, lo_min, lo_max;  // the unit
};

// q of the unit's rows as B fragments, and the factors of the affine part.
template <typename C>
__device__ __forceinline__ void load_unit(const MultiArgs& a, const Seq& s, int ui, Work<C>& w) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int rbs = s.units / a.Hkv;
  w.g = ui / rbs; w.rb = ui % rbs;
  w.T = s.T; w.c0 = s.c0; w.n = s.n; w.pre = s.pre;
  const int r0 = w.rb * 8 * C::NT, r1 = min(r0 + 8 * C::NT, s.n * a.r);
  // what every row of the block sees, and what any row sees
  const int i0 = r0 / a.r, i1 = (r1 - 1) / a.r;
  w.p_min = s.T - s.n + i0;  // below T
  w.p_max = s.T - s.n + i1;
  w.lo_min = max(s.start, a.window > 0 ? w.p_min - a.window + 1 : 0);
  w.lo_max = max(s.start, a.window > 0 ? w.p_max - a.window + 1 : 0);
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[mt][nt][i] = 0.0f;
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    const int row = r0 + nt * 8 + gid;
    const int i = row / a.r, h = w.g * a.r + row % a.r;
    w.on[nt] = row < r1;
    w.p[nt] = s.T - s.n + i;
    w.orow[nt] = (s.c0 + i) * a.Hq + h;
    w.lo[nt] = max(s.start, a.window > 0 ? w.p[nt] - a.window + 1 : 0);
    w.slope[nt] = w.on[nt] && a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.0f;
    w.ref[nt] = w.l[nt] = w.refc[nt][0] = w.refc[nt][1] = 0.0f;
    w.live[nt] = false;
    uint32_t raw[C::BLK][8];
#pragma unroll
    for (int blk = 0; blk < C::BLK; ++blk) {
      uint4 u = make_uint4(0, 0, 0, 0), v = u;
      if (w.on[nt]) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((long long)(s.c0 + i) * a.Hq + h) * C::D + blk * 64 + tig * 16);
        u = __ldg(src); v = __ldg(src + 1);
      }
      raw[blk][0] = u.x; raw[blk][1] = u.y; raw[blk][2] = u.z; raw[blk][3] = u.w;
      raw[blk][4] = v.x; raw[blk][5] = v.y; raw[blk][6] = v.z; raw[blk][7] = v.w;
    }
    // sums of q over each group, and its largest magnitude
    float big = 0.0f, sum[C::NG];
#pragma unroll
    for (int gi = 0; gi < C::NG; ++gi) {
      sum[gi] = w.zacc[nt][gi] = 0.0f;
      w.u[nt][gi] = pow2i((float)kUnitMax);
    }
#pragma unroll
    for (int blk = 0; blk < C::BLK; ++blk) {
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = bf16_lo(raw[blk][j]), y = bf16_hi(raw[blk][j]);
        t += x + y;
        big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
      }
      t += __shfl_xor_sync(kFull, t, 1);
      const float other = __shfl_xor_sync(kFull, t, 2);
      if constexpr (C::G == 32) {
        sum[2 * blk] = tig < 2 ? t : other;
        sum[2 * blk + 1] = tig < 2 ? other : t;
      } else {
        sum[blk * C::NG / C::BLK] += t + other;
      }
    }
    big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
    big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
    const float unit = a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e;
    float back = unit;
    if constexpr (C::KB == 16) {
#pragma unroll
      for (int blk = 0; blk < C::BLK; ++blk)
#pragma unroll
        for (int j = 0; j < 8; ++j) w.qf[nt][blk][j] = raw[blk][j];
    } else {
      // a power of two brings the row's largest |q| into [2^14, 2^15): the fp16 values are exact
      int e = 14 + 127 - (int)(__float_as_uint(big) >> 23);
      e = big == 0.0f ? 0 : max(-126, min(126, e));
      const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
      back = unit * down;
#pragma unroll
      for (int blk = 0; blk < C::BLK; ++blk) {
        __half qh[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          qh[2 * j] = __float2half_rn(bf16_lo(raw[blk][j]) * up);
          qh[2 * j + 1] = __float2half_rn(bf16_hi(raw[blk][j]) * up);
        }
        fused::bfrag_one<C::KB, 64, 0>(qh, 0, true, w.qf[nt][blk]);
      }
    }
    // the K product leaves columns 2 tig and 2 tig + 1 in this lane
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int src = 4 * (2 * tig + j);
      w.ka[nt][j] = __shfl_sync(kFull, back, src);
#pragma unroll
      for (int gi = 0; gi < C::NG; ++gi) w.kz[nt][gi][j] = unit * __shfl_sync(kFull, sum[gi], src);
    }
  }
}

// ------------------------------------------------------------------ what a token brings
// Per warp: transposed scores, and the constants that take each token's K
// centre out of the codes.
template <typename C>
struct Scratch {
  static constexpr int kScores = C::TT * 8 * C::NT;  // floats
  static constexpr int kBytes = kScores * 4 + C::TT * C::NG * centre_words(C::KB) * 4;
};

// The fp16 pattern of two codes at bits (lo, hi) of their half words holds
// 1024 + c 2^off; less 1024 + centre 2^off it is the centred code.  Which of a
// token's constants that is: at 6 and 4 bits one for each pair of offsets in
// the plan of mma_k.cuh, else the centre itself.
template <int KB>
constexpr int centre_index(int lo) {
  return KB == 6 ? (lo == 0 ? 0 : lo == 1 ? 1 : lo == 4 ? 2 : 3) : KB == 4 ? (lo == 0 ? 0 : 1) : 0;
}
constexpr uint32_t centre_mul(int lo, int hi) { return (1u << lo) | (1u << (16 + hi)); }

constexpr float kRound = 12582912.0f;       // 1.5 * 2^23: adding it rounds to an integer in the low bits
constexpr uint32_t kRoundBits = 0x4B400000u;

// The lane of a token readies its (scale, zero) rows: K's zero becomes the
// value of the code nearest 0 (the code itself goes to cen), V's that of the
// middle code.  What no row sees becomes 0 in V.  big: the largest V scale of
// each group, as bits.
template <typename C>
__device__ __forceinline__ void ready_tokens(const Work<C>& w, uint8_t* stage, uint32_t* cen, int t0, bool whole,
                                             unsigned (&big)[C::NG]) {
  const int lane = threadIdx.x & 31;
  const bool mine = C::TT == 32 || lane < C::TT;
  const int t = t0 + lane;
  const bool alive = whole || (t < w.T && (t < w.pre || (t >= w.lo_min && t <= w.p_max)));
  if constexpr (C::KB < 16) {
    float* ksz = reinterpret_cast<float*>(stage + C::OFF_KSZ) + lane * C::NG * 2;
    if (mine) {
#pragma unroll
      for (int gi = 0; gi < C::NG; ++gi) {
        const float2 v = *reinterpret_cast<const float2*>(ksz + 2 * gi);
        const float c = fminf(fmaxf(-v.y * rcp(v.x), 0.0f), (float)((1 << C::KB) - 1)) + kRound;
        constexpr int CW = centre_words(C::KB);
        uint32_t* to = cen + (lane * C::NG + gi) * CW;
        const uint32_t n = __float_as_uint(c) - kRoundBits;
        if constexpr (C::KB == 6) {
          *reinterpret_cast<uint4*>(to) = make_uint4(n * centre_mul(0, 2) + kF16Magic2, n * centre_mul(1, 3) + kF16Magic2,
                                                     n * centre_mul(4, 0) + kF16Magic2, n * centre_mul(2, 4) + kF16Magic2);
        } else if constexpr (C::KB == 4) {
          *reinterpret_cast<uint2*>(to) = make_uint2(n * centre_mul(0, 0) + kF16Magic2, n * centre_mul(4, 4) + kF16Magic2);
        } else {
          to[0] = n;
        }
        ksz[2 * gi + 1] = fmaf(c - kRound, v.x, v.y);
      }
    }
  }
  if constexpr (C::VB < 16) {
    float2* vsz = reinterpret_cast<float2*>(stage + C::OFF_VSZ) + lane * C::NG;
    float2 v[C::NG];
#pragma unroll
    for (int gi = 0; gi < C::NG; ++gi) {
      v[gi] = make_float2(0.0f, 0.0f);
      if (mine && alive) v[gi] = vsz[gi];
    }
#pragma unroll
    for (int gi = 0; gi < C::NG; ++gi) {
      big[gi] = __reduce_max_sync(kFull, __float_as_uint(fabsf(v[gi].x)));
      v[gi].y = fmaf((float)(1 << (C::VB - 1)), v[gi].x, v[gi].y);
    }
    if (mine) {
#pragma unroll
      for (int gi = 0; gi < C::NG; ++gi) vsz[gi] = v[gi];
    }
  } else if (!whole) {
    unsigned gone = __ballot_sync(kFull, mine && !alive);
    while (gone) {
      const int r = __ffs(gone) - 1;
      gone &= gone - 1;
      uint8_t* row = stage + C::OFF_VC + r * C::VRB;
#pragma unroll
      for (int i = 0; i < C::VRB / 128; ++i) reinterpret_cast<uint32_t*>(row)[lane + 32 * i] = 0u;
    }
  }
  __syncwarp();
}

// The (scale, zero) pairs of a token's NG groups.
template <int NG>
__device__ __forceinline__ void load_pairs(const float* p, float2 (&sz)[NG]) {
  if constexpr (NG == 1) {
    sz[0] = *reinterpret_cast<const float2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < NG; i += 2) {
      const float4 v = *reinterpret_cast<const float4*>(p + 2 * i);
      sz[i] = make_float2(v.x, v.y);
      sz[i + 1] = make_float2(v.z, v.w);
    }
  }
}

// ------------------------------------------------------------------ scores
// Register J of a lane's 16 codes: two codes less the centre as exact fp16
// values times 2^off, by the extraction plan of mma_k.cuh; at 16 bits the two
// bf16 values.
template <int KB, int J>
__device__ __forceinline__ uint32_t k_reg(const uint32_t (&word)[KB / 2], const uint32_t (&cen)[4]) {
  if constexpr (KB == 16) {
    return word[J];
  } else {
    using R = fused::RegChannels<KB, J>;
    constexpr int i = centre_index<KB>(R::lo_off);
    static_assert(KB != 6 || centre_mul(R::lo_off, R::hi_off) == (i == 0 ? centre_mul(0, 2) : i == 1 ? centre_mul(1, 3) : i == 2 ? centre_mul(4, 0) : centre_mul(2, 4)),
                  "a constant for each pair of offsets");
    static_assert(KB != 4 || centre_mul(R::lo_off, R::hi_off) == (i == 0 ? centre_mul(0, 0) : centre_mul(4, 4)), "and at 4 bits");
    uint32_t k = cen[i];
    if constexpr (centre_words(KB) == 1) k = k * centre_mul(R::lo_off, R::hi_off) + kF16Magic2;
    return hsub2_u32(fused::a_reg_bits<KB, J, KB / 2>(word), k);
  }
}

// acc[group][nt] = K codes (rows = tokens 16 ts + gid, + 8) x q.
template <typename C>
__device__ __forceinline__ void k_product(const uint8_t* kc, const uint32_t* cen, const Work<C>& w, int ts,
                                          float (&acc)[C::AC][C::NT][4]) {
  constexpr int KB = C::KB, RB = C::KRB, SW = KB / 2;  // row bytes, words of a lane's 16 codes
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const uint8_t* base = kc + (16 * ts + gid) * RB + tig * 2 * KB;
#pragma unroll
  for (int blk = 0; blk < C::BLK; ++blk) {
    uint32_t x[SW], y[SW];
    const uint8_t* p = base + blk * 8 * KB;
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
    uint32_t cx[4] = {0, 0, 0, 0}, cy[4] = {0, 0, 0, 0};
    if constexpr (KB < 16) {
      // the lane's codes lie in one group: its half of the block at G = 32
      constexpr int CW = centre_words(KB);
      const int gi = C::G == 32 ? 2 * blk + (tig >> 1) : blk * C::NG / C::BLK;
      const uint32_t *px = cen + ((16 * ts + gid) * C::NG + gi) * CW, *py = px + 8 * C::NG * CW;
      if constexpr (CW == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(px), v = *reinterpret_cast<const uint4*>(py);
        cx[0] = u.x; cx[1] = u.y; cx[2] = u.z; cx[3] = u.w;
        cy[0] = v.x; cy[1] = v.y; cy[2] = v.z; cy[3] = v.w;
      } else if constexpr (CW == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(px), v = *reinterpret_cast<const uint2*>(py);
        cx[0] = u.x; cx[1] = u.y; cy[0] = v.x; cy[1] = v.y;
      } else {
        cx[0] = *px; cy[0] = *py;
      }
    }
    auto step = [&](auto ks_c) {
      constexpr int ks = decltype(ks_c)::value;
      const uint32_t a0 = k_reg<KB, 2 * ks>(x, cx), a1 = k_reg<KB, 2 * ks>(y, cy);
      const uint32_t a2 = k_reg<KB, 2 * ks + 1>(x, cx), a3 = k_reg<KB, 2 * ks + 1>(y, cy);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        const uint32_t b0 = w.qf[nt][blk][2 * ks], b1 = w.qf[nt][blk][2 * ks + 1];
        // a group's first product starts its accumulator
        constexpr int per = KB == 16 ? C::BLK : C::G == 32 ? 1 : C::BLK / C::NG;  // blocks of an accumulator
        const bool start = ks == 0 && blk % per == 0;
        if constexpr (KB == 16) {
          if (start) hmma16816_bf16_first(acc[0][nt], a0, a1, a2, a3, b0, b1);
          else hmma16816_bf16(acc[0][nt], a0, a1, a2, a3, b0, b1);
        } else if constexpr (C::G != 32) {
          if (start) hmma16816_first(acc[blk * C::NG / C::BLK][nt], a0, a1, a2, a3, b0, b1);
          else hmma16816(acc[blk * C::NG / C::BLK][nt], a0, a1, a2, a3, b0, b1);
        } else {
          // lanes tig < 2 hold the block's first group of 32 channels, the others its second
          const uint32_t l0 = tig < 2 ? b0 : 0u, l1 = tig < 2 ? b1 : 0u, h0 = tig < 2 ? 0u : b0, h1 = tig < 2 ? 0u : b1;
          if (start) {
            hmma16816_first(acc[2 * blk][nt], a0, a1, a2, a3, l0, l1);
            hmma16816_first(acc[2 * blk + 1][nt], a0, a1, a2, a3, h0, h1);
          } else {
            hmma16816(acc[2 * blk][nt], a0, a1, a2, a3, l0, l1);
            hmma16816(acc[2 * blk + 1][nt], a0, a1, a2, a3, h0, h1);
          }
        }
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
}

// ------------------------------------------------------------------ output
// Sets each row's and group's unit by its largest product in the tile; x: the
// exponents of e.  A unit rises by at most 2^by[nt], what the row's reference has
// risen by.
template <typename C>
__device__ __forceinline__ void set_units(Work<C>& w, const float* vsz, const float (&x)[C::TS][C::NT][4], const float (&by)[C::NT]) {
  constexpr int PER = C::MT / C::NG;  // m-tiles of a group
  const int tig = threadIdx.x & 3;
#pragma unroll
  for (int gi = 0; gi < C::NG; ++gi)
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      float t = 0.0f;
#pragma unroll
      for (int ts = 0; ts < C::TS; ++ts)
#pragma unroll
        for (int j = 0; j < 4; ++j) t = fmaxf(t, fabsf(ex2(x[ts][nt][j]) * vsz[((16 * ts + tig + 4 * j) * C::NG + gi) * 2]));
      t = fmaxf(t, __shfl_xor_sync(kFull, t, 1));
      t = fmaxf(t, __shfl_xor_sync(kFull, t, 2));
      const float at = (float)exponent_of(w.u[nt][gi]);
      float to = fminf(at + by[nt], (float)kUnitMax);
      if (t * pow2i(to) >= kOver) to = (float)(kPlace - exponent_of(t));
      w.u[nt][gi] = pow2i(to);
      const float f = pow2i(to - at - by[nt]);
      const float f0 = __shfl_sync(kFull, f, 8 * tig), f1 = __shfl_sync(kFull, f, 8 * tig + 4);
#pragma unroll
      for (int mt = 0; mt < PER; ++mt) {
        float(&o)[4] = w.o[gi * PER + mt][nt];
        o[0] *= f0; o[1] *= f1;
        o[2] *= f0; o[3] *= f1;
      }
    }
}

// o += sum over 16 tokens of (e * scale) code: rows = channels, slots 2 tig,
// 2 tig + 1, 2 tig + 8, 2 tig + 9 = tokens tig, tig + 4, tig + 8, tig + 12.
template <typename C>
__device__ __forceinline__ void v_product(const uint8_t* vc, const float* vsz, Work<C>& w, int ts, const float (&e)[C::NT][4]) {
  constexpr int VB = C::VB, CH = C::CH, N = VRun<VB, CH>::N;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const uint8_t* base = vc + (16 * ts + tig) * C::VRB;
  const float* szb = vsz + (16 * ts + tig) * C::NG * 2;
  constexpr int TERMS = VB == 16 ? 3 : 2;
  uint32_t pw[C::NT][TERMS][2];
  float2 sz[4][C::NG];
  if constexpr (VB < 16 && C::NG <= 2) {  // four groups at once would take 32 registers
#pragma unroll
    for (int j = 0; j < 4; ++j) load_pairs<C::NG>(szb + 4 * j * C::NG * 2, sz[j]);
  }
#pragma unroll
  for (int run = 0; run < C::RUNS; ++run) {
    if (run % C::GRUNS == 0) {
      const int gi = run / C::GRUNS;
      if constexpr (VB < 16 && C::NG > 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sz[j][gi] = *reinterpret_cast<const float2*>(szb + (4 * j * C::NG + gi) * 2);
      }
      if constexpr (VB == 16) {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = e[nt][2 * j], y = e[nt][2 * j + 1];
            const uint32_t h = pack_bf16(x, y);
            const float xr = x - bf16_lo(h), yr = y - bf16_hi(h);
            const uint32_t m = pack_bf16(xr, yr);
            pw[nt][0][j] = h;
            pw[nt][1][j] = m;
            pw[nt][2][j] = pack_bf16(xr - bf16_lo(m), yr - bf16_hi(m));
          }
      } else {
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // the product first: beside a tiny scale the unit alone would take e out of fp32
            const float2 xy = exact_mul2(make_float2(e[nt][2 * j] * sz[2 * j][gi].x, e[nt][2 * j + 1] * sz[2 * j + 1][gi].x), f2(w.u[nt][gi]));
            const float x = xy.x, y = xy.y;
            w.zacc[nt][gi] = fmaf(e[nt][2 * j], sz[2 * j][gi].y, fmaf(e[nt][2 * j + 1], sz[2 * j + 1][gi].y, w.zacc[nt][gi]));
            const uint32_t h = pack_f16(x, y);
            const float2 f = unpack_f16(h);
            pw[nt][0][j] = h;
            pw[nt][1][j] = pack_f16(x - f.x, y - f.y);
          }
      }
    }
    uint32_t r[4][N];
#pragma unroll
    for (int j = 0; j < 4; ++j) load_run<VB, CH>(base + 4 * j * C::VRB, run, gid, r[j]);
    uint32_t u[CH], v[CH];
    pair_codes<VB, CH>(r[0], r[1], u);
    pair_codes<VB, CH>(r[2], r[3], v);
#pragma unroll
    for (int term = 0; term < TERMS; ++term)
#pragma unroll
      for (int mi = 0; mi < C::TPB; ++mi)
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          float(&o)[4] = w.o[run * C::TPB + mi][nt];
          if constexpr (VB == 16) {
            hmma16816_bf16(o, u[2 * mi], u[2 * mi + 1], v[2 * mi], v[2 * mi + 1], pw[nt][term][0], pw[nt][term][1]);
          } else {
            hmma16816(o, u[2 * mi], u[2 * mi + 1], v[2 * mi], v[2 * mi + 1], pw[nt][term][0], pw[nt][term][1]);
          }
        }
  }
}

// One staged tile from position t0: scores, running softmax, output.
template <typename C>
__device__ __forceinline__ void tile_step(const MultiArgs& a, Work<C>& w, uint8_t* stage, float* tr, int t0) {
  constexpr int TS = C::TS, TT = C::TT, NT = C::NT, NG = C::NG;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  uint32_t* cen = reinterpret_cast<uint32_t*>(tr + Scratch<C>::kScores);
  const float* ksz = reinterpret_cast<const float*>(stage + C::OFF_KSZ);
  const float* vsz = reinterpret_cast<const float*>(stage + C::OFF_VSZ);
  const int t1 = t0 + C::TT - 1;
  const bool whole = (t0 >= w.lo_max && t1 <= w.p_min) || t1 < w.pre;  // p_min and pre lie before T
  unsigned big[NG];
  ready_tokens<C>(w, stage, cen, t0, whole, big);
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) {
    float acc[C::AC][NT][4];
    k_product<C>(stage, cen, w, ts, acc);
    // fold (scale, zero): rows gid and gid + 8, columns 2 tig and 2 tig + 1.  The
    // reference goes in before the one large rounding, so the scores that
    // matter, those near it, are rounded at their small distance from it.
    float s[NT][4];
    if constexpr (C::KB == 16) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] = fmaf(acc[0][nt][j], w.ka[nt][j & 1], -w.refc[nt][j & 1]);
    } else {
      float2 sz[2][NG];
#pragma unroll
      for (int i = 0; i < 2; ++i) load_pairs<NG>(ksz + (16 * ts + gid + 8 * i) * NG * 2, sz[i]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float t = sz[j >> 1][0].x * acc[0][nt][j], z = -w.refc[nt][j & 1];
#pragma unroll
          for (int gi = 1; gi < NG; ++gi) t = fmaf(sz[j >> 1][gi].x, acc[gi][nt][j], t);
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) z = fmaf(sz[j >> 1][gi].y, w.kz[nt][gi][j & 1], z);
          s[nt][j] = fmaf(t, w.ka[nt][j & 1], z);
        }
    }
    // transpose through shared memory: lane (gid, tig) takes row gid, tokens tig + 4 j
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float* dst = tr + (ts * NT + nt) * 128 + gid * 8 + 2 * tig;
      *reinterpret_cast<float2*>(dst) = make_float2(s[nt][0], s[nt][1]);
      *reinterpret_cast<float2*>(dst + 64) = make_float2(s[nt][2], s[nt][3]);
    }
  }
  __syncwarp();
  float e[TS][NT][4];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) e[ts][nt][j] = tr[(ts * NT + nt) * 128 + (tig + 4 * j) * 8 + gid];
  if (a.softcap > 0.0f) {
    const float c = a.softcap * kLog2e;
    bool far = false;
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) far |= fabsf(e[ts][nt][j]) > 2.0f;
    if (__any_sync(kFull, far)) {
#pragma unroll
      for (int ts = 0; ts < TS; ++ts)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = e[ts][nt][j];
            e[ts][nt][j] = fmaf(c, fabsf(x) > 2.0f ? tanh_far(x) : tanh_near(x), -w.ref[nt]);
          }
    } else {
#pragma unroll
      for (int ts = 0; ts < TS; ++ts)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) e[ts][nt][j] = fmaf(c, tanh_near(e[ts][nt][j]), -w.ref[nt]);
    }
  }
  if (a.slopes != nullptr) {
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          e[ts][nt][j] = fmaf(w.slope[nt], (float)(t0 + 16 * ts + tig + 4 * j - w.p[nt]), e[ts][nt][j]);
  }
  if (!whole) {
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + 16 * ts + tig + 4 * j;
          if (!(t < w.T && (t < w.pre || (t >= w.lo[nt] && t <= w.p[nt])))) e[ts][nt][j] = -INFINITY;
        }
  }
  float mx[NT];
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float t = -INFINITY;
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
      t = fmaxf(t, fmaxf(fmaxf(e[ts][nt][0], e[ts][nt][1]), fmaxf(e[ts][nt][2], e[ts][nt][3])));
    t = fmaxf(t, __shfl_xor_sync(kFull, t, 1));
    t = fmaxf(t, __shfl_xor_sync(kFull, t, 2));
    mx[nt] = t;
    grow |= t > (w.live[nt] ? kLazy : -INFINITY);
    if constexpr (C::VB < 16) {
      // a bound of the row's products: exponents of its largest e, of the tile's largest scale and of the unit.  A moving
      // reference does not change it (e falls as the unit rises)
      unsigned k = 0;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) k = max(k, big[gi] + __float_as_uint(w.u[nt][gi]));
      grow |= __float2int_ru(t) > kOverExp + 2 * 127 - 1 - (int)(k >> 23);
    }
  }
  const bool slow = __any_sync(kFull, grow);
  if (slow) {
    // one power for all groups of a row will do while the tile's scales lie close together
    bool easy = true;
    if constexpr (C::VB < 16) {
      const int t = t0 + lane;
      if ((TT == 32 || lane < TT) && (whole || (t < w.T && (t < w.pre || (t >= w.lo_min && t <= w.p_max))))) {
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) easy &= __float_as_uint(fabsf(vsz[(lane * NG + gi) * 2])) + (kNarrow << 23) >= big[gi];
      }
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) easy &= big[gi] >= kLeast << 23;
    }
    float f[NT], d[NT], up[NT];  // factor of o, and what the units rise by: all as one, or at most
    bool exact = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool any = mx[nt] > -INFINITY;
      const float most = any ? ceilf(mx[nt] + w.ref[nt]) : w.ref[nt];
      const float ref = w.live[nt] ? fmaxf(w.ref[nt], most) : most;
      const float by = ref - w.ref[nt], al = pow2i(-by);
      f[nt] = al;
      if constexpr (C::VB < 16) {
        // o keeps its value where the units take the factor up: what is small beside the old reference may matter now
        // (past 2^400 nothing is left of it, and larger powers would round)
        up[nt] = d[nt] = w.live[nt] ? fminf(by, 400.0f) : 0.0f;
        unsigned k0 = 0xFFFFFFFFu, k1 = 0;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          k0 = min(k0, big[gi] + __float_as_uint(w.u[nt][gi]));
          k1 = max(k1, big[gi] + __float_as_uint(w.u[nt][gi]));
        }
        const float over = ceilf(mx[nt] - by) + d[nt] + (float)((int)(k1 >> 23) - (2 * 127 - 1) - kPlace);  // of the bound
        if (over > 0.0f) {
          d[nt] -= over;
          easy &= k1 - k0 <= kSpread << 23;
        }
        f[nt] = pow2i(d[nt] - by);
      }
      w.live[nt] |= any;
      w.ref[nt] = ref;
      w.l[nt] *= al;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) w.zacc[nt][gi] *= al;
#pragma unroll
      for (int ts = 0; ts < TS; ++ts)
#pragma unroll
        for (int j = 0; j < 4; ++j) e[ts][nt][j] -= by;
      const float r0 = __shfl_sync(kFull, ref, 8 * tig), r1 = __shfl_sync(kFull, ref, 8 * tig + 4);
      if (a.softcap <= 0.0f) { w.refc[nt][0] = r0; w.refc[nt][1] = r1; }
    }
    if constexpr (C::VB < 16) exact = !__all_sync(kFull, easy);
    if (!exact) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (C::VB < 16) {
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) w.u[nt][gi] = __uint_as_float(__float_as_uint(w.u[nt][gi]) + ((unsigned)(int)d[nt] << 23));
        }
        const float a0 = __shfl_sync(kFull, f[nt], 8 * tig), a1 = __shfl_sync(kFull, f[nt], 8 * tig + 4);
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          w.o[mt][nt][0] *= a0; w.o[mt][nt][1] *= a1;
          w.o[mt][nt][2] *= a0; w.o[mt][nt][3] *= a1;
        }
      }
    } else {
      if constexpr (C::VB < 16) set_units<C>(w, vsz, e, up);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
#pragma unroll
      for (int j = 0; j < 4; ++j) e[ts][nt][j] = ex2(e[ts][nt][j]);
      w.l[nt] += (e[ts][nt][0] + e[ts][nt][1]) + (e[ts][nt][2] + e[ts][nt][3]);
    }
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) v_product<C>(stage + C::OFF_VC, vsz, w, ts, e[ts]);
}

// ------------------------------------------------------------------ writing a unit or a piece
// A sum of 0 is a row that sees nothing; one that is not a number has scores that are none, which count for no reference.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : isnan(l) ? l : (m + log2f(l)) * kLn2;
}

// A piece: (reference, sum) of 8 NT rows, then their partial outputs.
template <int D, int NT>
constexpr int piece_floats() { return 8 * NT * (D + 2); }

// Channel of output register (mt, half) for lane gid: runs of CH channels.
template <typename C>
__device__ __forceinline__ int out_channel(int mt, int half, int gid) {
  return (mt / C::TPB) * 8 * C::CH + gid * C::CH + (mt % C::TPB) * 2 + half;
}

template <typename C>
__device__ __forceinline__ void flush(const MultiArgs& a, Work<C>& w, float* piece) {
  constexpr int NT = C::NT, NG = C::NG;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int rows = min(8 * NT, w.n * a.r - w.rb * 8 * NT);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float l = w.l[nt];
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    const float m = w.live[nt] ? w.ref[nt] : -INFINITY;
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      float z = w.zacc[nt][gi];
      z += __shfl_xor_sync(kFull, z, 1);
      z += __shfl_xor_sync(kFull, z, 2);
      w.zacc[nt][gi] = z;
    }
    const int mine = nt * 8 + gid;
    if (tig == 0 && mine < rows) {
      if (piece != nullptr) {
        *reinterpret_cast<float2*>(piece + 2 * mine) = make_float2(m, l);
      } else if (a.lse != nullptr) {
        a.lse[w.orow[nt]] = lse_of(m, l);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int src = 4 * (2 * tig + j), col = nt * 8 + 2 * tig + j;
      const float lc = __shfl_sync(kFull, l, src);
      const int orow = __shfl_sync(kFull, w.orow[nt], src);
      float z[NG], unit[NG];
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) {
        z[gi] = __shfl_sync(kFull, w.zacc[nt][gi], src);
        unit[gi] = pow2i((float)-exponent_of(__shfl_sync(kFull, w.u[nt][gi], src)));
      }
      const float f = piece != nullptr ? 1.0f : (lc > 0.0f ? 1.0f / lc : 0.0f);
      if (col < rows) {
        float* dst = piece != nullptr ? piece + 16 * NT + col * C::D : a.out + (long long)orow * C::D;
#pragma unroll
        for (int mt = 0; mt < C::MT; mt += 2) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = ((mt + i / 2) % C::TPB) * 2 + (i & 1);  // the code's place in its run
            const int gi = mt / C::TPB / C::GRUNS;
            const float x = w.o[mt + i / 2][nt][2 * (i & 1) + j];
            y[i] = (C::VB == 16 ? x : fmaf(x * (1.0f / (float)(1 << code_off<C::VB>(c))), unit[gi], z[gi])) * f;
          }
          *reinterpret_cast<float4*>(dst + out_channel<C>(mt, 0, gid)) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
// A cut unit: its tiles [u0, u1) in the list, the rows it stands for, the
// runs that hold its pieces, and for one cut between CTAs the CTAs that do
// (first piece in slot).
struct Cut {
  int u0, u1, c0, g, row0, rows, k0, k1, ck0, ck1, slot;
};

// Where tile x of the list lies: sequence, unit of it, tile of that.
struct Place {
  Seq s;
  int b, ui, ti;
};

template <int NT, int TT>
__device__ __forceinline__ Place seek(const MultiArgs& a, const int* first, int x) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  Place p;
  p.b = lo;
  p.s = load_seq<NT, TT>(a, lo);
  const int rem = x - first[lo];
  p.ui = rem / p.s.cnt;
  p.ti = rem - p.ui * p.s.cnt;
  return p;
}

// The tile that a warp fetches next.
struct Feed {
  int b, ui, left;             // tiles left in the unit, this one among them
  int t0, T, edge, to;         // its first token; behind the prefix tiles, at edge, comes to
  int cnt, units, rbs, begin;  // rbs: row blocks of a KV head; begin: first token of a unit
  long long base;              // contiguous: the head's first row; paged: the sequence's first table entry
  long long page_row;          // paged: the head's first row of the page at hand, less that page's first token
  int page;                    // its place in the table, -1: none yet
  bool fresh;                  // the warp's first tile of the unit
};

__device__ __forceinline__ void feed_base(const MultiArgs& a, Feed& f) {
  f.base = a.table == nullptr ? ((long long)f.b * a.Hkv + f.ui / f.rbs) * a.T_cap : (long long)f.b * a.pps;
  f.page = -1;
}

template <int NT, int TT>
__device__ __forceinline__ void feed_from(const MultiArgs& a, const Place& p, Feed& f) {
  f.b = p.b; f.ui = p.ui; f.left = p.s.cnt - p.ti;
  f.T = p.s.T; f.edge = p.s.np * TT; f.to = p.s.t_lo * TT;
  f.cnt = p.s.cnt; f.units = p.s.units; f.rbs = p.s.units / a.Hkv;
  f.begin = p.s.np > 0 ? 0 : f.to;
  f.t0 = p.ti < p.s.np ? p.ti * TT : f.to + (p.ti - p.s.np) * TT;
  f.fresh = true;
  feed_base(a, f);
}

template <int NT, int TT>
__device__ __forceinline__ void feed_next(const MultiArgs& a, const int* first, Feed& f) {
  f.fresh = false;
  if (--f.left > 0) {
    f.t0 += TT;
    if (f.t0 == f.edge) f.t0 = f.to;
    return;
  }
  if (f.ui + 1 < f.units) {
    ++f.ui;
    f.left = f.cnt;
    f.t0 = f.begin;
    f.fresh = true;
    feed_base(a, f);
  } else {
    int b = f.b;
    do ++b; while (b < a.B && first[b + 1] == first[b]);  // past sequences without new tokens
    if (b < a.B) feed_from<NT, TT>(a, Place{load_seq<NT, TT>(a, b), b, 0, 0}, f);
  }
}

// What a stage holds: first token, staged tokens (0: nothing to see, no copy),
// sequence and unit.
constexpr int kFresh = 1 << 8, kEnd = 1 << 9;

// Start the copies of a tile into a stage, one lane each; the bytes complete on bar.
template <typename C>
__device__ __forceinline__ void fetch_tile(const MultiArgs& a, Feed& f, uint8_t* stage, int4* what, uint64_t* bar,
                                           const uint8_t* src, int row_bytes, int off) {
  const int lane = threadIdx.x & 31;
  int n = max(0, min(C::TT, f.T - f.t0));
  if (lane == 0) *what = make_int4(f.t0, n | (f.fresh ? kFresh : 0) | (f.left == 1 ? kEnd : 0), f.b, f.ui);
  if (n > 0) {
    // (scale, zero) rows of 8 bytes go in pairs; the capacity is even then
    if constexpr ((C::NG & 1) && (C::KB < 16 || C::VB < 16)) n += n & 1;
    long long row = f.base + f.t0;
    if (a.table != nullptr) {
      if (f.t0 / kPageTokens != f.page) {
        f.page = f.t0 / kPageTokens;
        int page = __ldg(a.table + f.base + f.page);
        if (page < 0 || page >= a.num_pages) {
          if (lane == 0) atomicMax(a.status, kStatusInvalidArg);
          page = 0;
        }
        f.page_row = (((long long)page * a.Hkv + f.ui / f.rbs) - f.page) * kPageTokens;
      }
      row = f.page_row + f.t0;
    }
    constexpr int all = C::KRB + C::VRB + (C::KB < 16 ? C::NG * 8 : 0) + (C::VB < 16 ? C::NG * 8 : 0);
    if (lane == 0) mbar_arrive_expect_tx(bar, n * all);
    __syncwarp();
    if (lane < 4 && row_bytes > 0) bulk_g2s(stage + off, src + row * row_bytes, n * row_bytes, bar, policy_evict_first());
  }
}

// Pieces of other CTAs are read past L1.
template <bool L2, typename T>
__device__ __forceinline__ T ld(const T* p) {
  if constexpr (L2) return __ldcg(p);
  else return *p;
}

// Row `row` of the pieces p0 .. p1 - 1 joined (at(k) is where piece k lies), by
// any number of threads on their own: the row's reference and sum, and four
// channels (the i-th float4 of a piece's output).  Eight pieces are in flight
// at a time, their references and sums with them: every thread of a row makes
// the weights 2^(ref_k - max) again, which costs less than a first pass and a
// barrier (71 us with those, 66 without: 16-bit documents, 16 query rows).
template <int NT, bool L2, typename At>
__device__ __forceinline__ void join_pieces(int p0, int p1, const At& at, int row, int i, float2& ml, float4& o) {
  float m = -INFINITY, l = 0.0f;
  o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k0 = p0; k0 < p1; k0 += 8) {
    float2 w[8];
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = make_float2(-INFINITY, 0.0f);
      v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (k0 + j < p1) {
        const float* p = at(k0 + j);
        w[j] = ld<L2>(reinterpret_cast<const float2*>(p) + row);
        v[j] = ld<L2>(reinterpret_cast<const float4*>(p + 16 * NT) + i);
      }
    }
    float t = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaxf(t, w[j].x);
    const float back = m == t ? 1.0f : pow2i(m - t);  // references are integers: exact
    l *= back;
    o.x *= back; o.y *= back; o.z *= back; o.w *= back;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = w[j].x == -INFINITY ? 0.0f : pow2i(w[j].x - t);
      l = fmaf(w[j].y, f, l);
      o.x = fmaf(v[j].x, f, o.x); o.y = fmaf(v[j].y, f, o.y);
      o.z = fmaf(v[j].z, f, o.z); o.w = fmaf(v[j].w, f, o.w);
    }
    m = t;
  }
  ml = make_float2(m, l);
}

// Publishes what the block wrote before its barrier, and shows what other blocks published before.
__device__ __forceinline__ int add_acq_rel(int* p, int x) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(x) : "memory");
  return old;
}

template <typename C>
__global__ void __launch_bounds__(32 * C::WARPS, 1) multi_kernel(MultiArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int D = C::D, NT = C::NT, TT = C::TT, W = C::WARPS, ST = C::STAGES;
  constexpr int PF = piece_floats<D, NT>();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  __shared__ int s_wsum[32];
  __shared__ Cut s_cut[W + 1];
  __shared__ int s_ncut, s_begin[W + 1];
  __shared__ int s_last[2];
  __shared__ uint64_t s_bar[W * ST];
  __shared__ int4 s_what[W * ST];
  static_assert(Scratch<C>::kBytes <= C::SCRATCH, "a warp's scratch fits");
  uint8_t* ring = smem + (size_t)warp * ST * C::STAGE;
  float* tr = reinterpret_cast<float*>(smem + W * ST * C::STAGE + warp * C::SCRATCH);
  int* first = reinterpret_cast<int*>(smem + W * (ST * C::STAGE + C::SCRATCH));
  uint64_t* bar = s_bar + warp * ST;
  int4* what = s_what + warp * ST;

  // tiles before each sequence
  {
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq<NT, TT>(a, b);
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
    if (lane < ST) mbar_init(bar + lane, 1);
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
  const int ctas = min((int)gridDim.x, (total + W - 1) / W);
  const int cta = blockIdx.x;
  if (cta >= ctas) return;
  // equal runs: the first `rem` of them one longer
  const int q0 = total / ctas, rem0 = total - q0 * ctas;
  auto cta_begin = [&](int c) { return c * q0 + min(c, rem0); };
  const int x0 = cta_begin(cta), x1 = cta_begin(cta + 1);
  const int q1 = (x1 - x0) / W, rem1 = (x1 - x0) - q1 * W;
  auto warp_begin = [&](int w) { return x0 + w * q1 + min(w, rem1); };

  // Units cut by a run end: one lane per boundary finds its unit.  By one warp, while its first copies are under way.
  auto cta_of = [&](int x) { return x < rem0 * (q0 + 1) ? x / (q0 + 1) : rem0 + (x - rem0 * (q0 + 1)) / q0; };
  auto find_cuts = [&]() {
    if (lane <= W) s_begin[lane] = lane < W ? warp_begin(lane) : x1;
    Cut u{};
    bool cut = false;
    if (lane <= W) {
      const int x = lane < W ? warp_begin(lane) : x1;
      if (x < total) {
        const Place p = seek<NT, TT>(a, first, x);
        u.u0 = x - p.ti;
        u.u1 = u.u0 + p.s.cnt;
        const int rbs = p.s.units / a.Hkv;
        u.g = p.ui / rbs;
        u.row0 = (p.ui - u.g * rbs) * 8 * NT;
        u.rows = min(8 * NT, p.s.n * a.r - u.row0);
        u.c0 = p.s.c0;
        cut = u.u0 < x;
      }
    }
    // boundaries rise, so equal units stand side by side (among those that cut)
    const unsigned cuts = __ballot_sync(kFull, cut);
    const unsigned below = cuts & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : 0;
    const int pu = __shfl_sync(kFull, u.u0, prev);
    const bool lead = cut && (!below || pu != u.u0);
    const unsigned leads = __ballot_sync(kFull, lead);
    if (lead) {
      // its pieces: the runs that reach past its begin and start before its end
      u.k0 = 0;
      u.k1 = W;
      while (warp_begin(u.k0 + 1) <= u.u0) ++u.k0;
      while (warp_begin(u.k1 - 1) >= u.u1) --u.k1;
      if (u.u0 < x0 || u.u1 > x1) {
        u.ck0 = cta_of(u.u0);
        u.ck1 = cta_of(u.u1 - 1) + 1;
        u.slot = u.u0 > cta_begin(u.ck0) ? 1 : 0;
      }
      s_cut[__popc(leads & ((1u << lane) - 1u))] = u;
    }
    if (lane == 0) { s_ncut = __popc(leads); s_last[0] = s_last[1] = 0; }
  };

  float* const early = a.pieces + (long long)cta * W * PF;  // pieces of units that end inside a run, one per warp
  static_assert(PF * 4 <= ST * C::STAGE, "a run's last piece fits its ring");
  {
    const int w0 = warp_begin(warp), w1 = warp_begin(warp + 1);
    if (w0 < w1) {
      const uint64_t limit = *a.timeout_ns ? *a.timeout_ns : 2000000000ull;
      // lanes 0 .. 3 copy K codes, K pairs, V codes, V pairs
      const uint8_t* src = lane == 0 ? a.kc : lane == 1 ? reinterpret_cast<const uint8_t*>(a.ksz)
                           : lane == 2 ? a.vc : reinterpret_cast<const uint8_t*>(a.vsz);
      const int row_bytes = lane == 0 ? C::KRB : lane == 1 ? (C::KB < 16 ? C::NG * 8 : 0)
                            : lane == 2 ? C::VRB : (C::VB < 16 ? C::NG * 8 : 0);
      const int off = lane == 0 ? 0 : lane == 1 ? C::OFF_KSZ : lane == 2 ? C::OFF_VC : C::OFF_VSZ;
      const Place p = seek<NT, TT>(a, first, w0);
      bool here = p.ti == 0;  // the unit at hand begins in this run
      Feed f;
      feed_from<NT, TT>(a, p, f);
      int fx = w0;
      for (int i = 0; i < ST && fx < w1; ++i, ++fx) {
        if (i > 0) feed_next<NT, TT>(a, first, f);
        fetch_tile<C>(a, f, ring + i * C::STAGE, what + i, bar + i, src, row_bytes, off);
      }
      __syncwarp();
      if (warp == W - 1) find_cuts();
      Work<C> w;
      bool dead = false;
      int st = 0;
      uint32_t parity = 0;  // bit i: phase of stage i
      for (int x = w0; x < w1; ++x) {
        const int4 d = what[st];
        uint8_t* stage = ring + st * C::STAGE;
        if (d.y & kFresh) {
          load_unit<C>(a, load_seq<NT, TT>(a, d.z), d.w, w);
          here = here || x > w0;
        }
        if (d.y & 0xFF) {
          if (!dead && !mbar_wait(bar + st, parity >> st & 1, limit)) {
            if (lane == 0) atomicMax(a.status, kStatusTimeout);
            dead = true;
          }
          dead = __any_sync(kFull, dead);
          parity ^= 1u << st;
          if (!dead) tile_step<C>(a, w, stage, tr, d.x);
          fence_proxy_async_smem();  // the stage's reads and writes come before the copies that refill it
        }
        __syncwarp();
        if (fx < w1 && !dead) {
          feed_next<NT, TT>(a, first, f);
          fetch_tile<C>(a, f, stage, what + st, bar + st, src, row_bytes, off);
          ++fx;
        }
        st = st + 1 == ST ? 0 : st + 1;
        if ((d.y & kEnd) || x + 1 == w1 || dead) {
          float* to = (d.y & kEnd) && here ? nullptr : x + 1 == w1 || dead ? reinterpret_cast<float*>(ring) : early + warp * PF;
          flush<C>(a, w, to);
        }
        if (dead) break;
        __syncwarp();
      }
      // after a wait that gave up: let the copies still in flight land before the shared memory goes
      if (dead)
        for (int i = 0; i < ST; ++i) mbar_wait(bar + i, parity >> i & 1, 1000000ull);
    } else {
      if (warp == W - 1) find_cuts();
      // a run without tiles (fewer tiles than warps) leaves an empty piece
      float* piece = reinterpret_cast<float*>(ring);
      for (int i = lane; i < PF; i += 32) piece[i] = i < 16 * NT && !(i & 1) ? -INFINITY : 0.0f;
    }
  }
  __syncthreads();
  const int ncut = s_ncut;
  if (ncut == 0) return;
  const int b0 = s_begin[0], b1 = s_begin[W];  // x0 and x1: not kept in registers across the loop, which has none to spare
  constexpr int ROWS = 8 * NT, EL = ROWS * D / 4;
  auto is_shared = [&](const Cut& u) { return u.u0 < b0 || u.u1 > b1; };
  auto out_row = [&](const Cut& u, int row) {
    const int i = (u.row0 + row) / a.r;
    return (long long)(u.c0 + i) * a.Hq + u.g * a.r + (u.row0 + row) - i * a.r;
  };
  auto write_row = [&](const Cut& u, int row, float2 ml) {
    if (a.lse != nullptr) a.lse[out_row(u, row)] = lse_of(ml.x, ml.y);
  };
  auto write_out = [&](const Cut& u, int row, int d4, float2 ml, float4 o) {
    const float f = ml.y > 0.0f ? 1.0f / ml.y : 0.0f;
    reinterpret_cast<float4*>(a.out + out_row(u, row) * D)[d4] = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  };
  // a run's last piece lies in its ring, the piece of a unit that ends earlier in the workspace
  auto piece_of = [&](const Cut& u, int k) -> const float* {
    if (k == u.k1 - 1 && u.u1 < s_begin[k + 1]) return early + k * PF;
    return reinterpret_cast<const float*>(smem + (size_t)k * ST * C::STAGE);
  };
  float* const to0 = a.cpieces + (long long)2 * cta * PF;
  for (int el = tid; el < ncut * EL; el += 32 * W) {
    const int i = el / EL, at = el % EL, row = at / (D / 4);
    const Cut& u = s_cut[i];
    if (row >= u.rows) continue;
    float2 ml;
    float4 o;
    join_pieces<NT, false>(u.k0, u.k1, [&](int k) { return piece_of(u, k); }, row, at, ml, o);
    float* const to = to0 + (u.u0 > b0 ? PF : 0);
    if (is_shared(u)) {
      if (at % (D / 4) == 0) reinterpret_cast<float2*>(to)[row] = ml;
      reinterpret_cast<float4*>(to + 16 * NT)[at] = o;
    } else {
      if (at % (D / 4) == 0) write_row(u, row, ml);
      write_out(u, row, at % (D / 4), ml, o);
    }
  }
  // a unit that began in an earlier CTA can only be the first, one that ends in a later the last
  if (!is_shared(s_cut[0]) && !is_shared(s_cut[ncut - 1])) return;

  // ---- units cut between CTAs: the last to arrive joins the CTAs' pieces
  __syncthreads();
  if (tid < 2) {
    const int i = tid == 0 ? 0 : ncut - 1;
    const Cut& u = s_cut[i];
    if (is_shared(u) && (tid == 0 || i != 0)) {
      int* arrive = a.arrive + u.ck0;  // a CTA begins at most one unit that it does not end
      if (add_acq_rel(arrive, 1) + 1 == u.ck1 - u.ck0) {
        *arrive = 0;  // ready for the next call
        s_last[tid] = 1;
      }
    }
  }
  __syncthreads();
  for (int t = 0; t < 2; ++t) {
    if (!s_last[t]) continue;  // the same for every thread
    const Cut& u = s_cut[t == 0 ? 0 : ncut - 1];
    auto at = [&](int k) -> const float* { return a.cpieces + (long long)(2 * k + (k == u.ck0 ? u.slot : 0)) * PF; };
    for (int i = tid; i < u.rows * (D / 4); i += 32 * W) {
      const int row = i / (D / 4);
      float2 ml;
      float4 o;
      join_pieces<NT, true>(u.ck0, u.ck1, at, row, i, ml, o);
      if (i % (D / 4) == 0) write_row(u, row, ml);
      write_out(u, row, i % (D / 4), ml, o);
    }
  }
}

}  // namespace multi
}  // namespace lkv
