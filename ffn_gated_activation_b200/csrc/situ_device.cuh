// Device code shared by the library's translation units: vector loads and
// stores, storage types, the SiTU-GLU element arithmetic, the block-scaled
// (MXFP8, NVFP4) stores, bounded mbarrier waits, bulk copies and clusters.
// Everything has internal linkage.
#pragma once

#include <cuda.h>  // CUtensorMap
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "situ_glu.h"

namespace {

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;  // log2(e)
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxThreads = 256;  // CTA size ceiling
constexpr int kVecBytes = 16;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Hardware tanh (MUFU).  Its relative error (about 2^-11) is far below half a
// bf16 ulp (2^-9 relative), so it is used only where the result is rounded to
// bf16 and nothing is accumulated from it: the up branch of the bf16 forward.
__device__ __forceinline__ float tanh_approx(float x) {
  float y;
  asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max() that propagates NaN (a NaN input must give a NaN output).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Read-only streaming load (no L1 allocation) and evict-first store: every
// byte is touched once.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "l"(p));
  return r;
}

__device__ __forceinline__ void st_stream(void* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// 32-byte forms (sm_100): two adjacent 16-byte vectors in one instruction.
// The address must be 32-byte aligned.
struct U8 {
  uint4 a, b;
};

__device__ __forceinline__ U8 ld_stream32(const void* p) {
  U8 r;
  asm("ld.global.nc.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w)
      : "l"(p));
  return r;
}

__device__ __forceinline__ void st_stream32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.cs.v8.u32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Packed fp32 pairs: sm_100 executes one f32x2 add/mul/fma per issue slot.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 splat(float a) { return make_float2(a, a); }

__device__ __forceinline__ float2 ex2_neg2(float2 y) {  // (2^-y.x, 2^-y.y)
  return make_float2(ex2_approx(-y.x), ex2_approx(-y.y));
}
__device__ __forceinline__ float2 rcp2(float2 a) { return make_float2(rcp_approx(a.x), rcp_approx(a.y)); }

// A pair of input elements as fp32 bit patterns (bf16 widened exactly).
struct Bits2 {
  uint32_t lo, hi;
};

__device__ __forceinline__ float2 as_f2(Bits2 b) { return make_float2(__uint_as_float(b.lo), __uint_as_float(b.hi)); }
__device__ __forceinline__ float2 abs_f2(Bits2 b) {
  return make_float2(__uint_as_float(b.lo & 0x7fffffffu), __uint_as_float(b.hi & 0x7fffffffu));
}
// x with its sign bit flipped where the sign bit of `s` is set.
__device__ __forceinline__ float xor_sign(float x, uint32_t s) {
  return __uint_as_float(__float_as_uint(x) ^ (s & 0x80000000u));
}
__device__ __forceinline__ float2 xor_sign2(float2 x, Bits2 s) { return make_float2(xor_sign(x.x, s.lo), xor_sign(x.y, s.hi)); }
// s negative ? a : b, element-wise on the sign bit of s.
__device__ __forceinline__ float2 select_neg2(Bits2 s, float2 a, float2 b) {
  const uint32_t m0 = static_cast<uint32_t>(static_cast<int32_t>(s.lo) >> 31);
  const uint32_t m1 = static_cast<uint32_t>(static_cast<int32_t>(s.hi) >> 31);
  return make_float2(__uint_as_float((__float_as_uint(a.x) & m0) | (__float_as_uint(b.x) & ~m0)),
                     __uint_as_float((__float_as_uint(a.y) & m1) | (__float_as_uint(b.y) & ~m1)));
}

// Storage types.  A 16-byte vector holds 8 bf16 or 4 fp32 values, i.e. 4 or 2
// pairs.  Pair p of a vector is (element 2p, element 2p + 1).
struct Bf16 {
  static constexpr int kPairs = 4;
  __device__ __forceinline__ static Bits2 pair(const uint4& v, int p) {
    const uint32_t w = p == 0 ? v.x : p == 1 ? v.y : p == 2 ? v.z : v.w;
    return {w << 16, w & 0xffff0000u};
  }
  __device__ __forceinline__ static uint32_t pack(float2 f) {
    uint32_t r;  // cvt packs its first source into the high half
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
    return r;
  }
  __device__ __forceinline__ static void put(uint4& v, int p, float2 f) {
    const uint32_t w = pack(f);
    if (p == 0) v.x = w; else if (p == 1) v.y = w; else if (p == 2) v.z = w; else v.w = w;
  }
};

struct F32 {
  static constexpr int kPairs = 2;
  __device__ __forceinline__ static Bits2 pair(const uint4& v, int p) {
    return p == 0 ? Bits2{v.x, v.y} : Bits2{v.z, v.w};
  }
  __device__ __forceinline__ static void put(uint4& v, int p, float2 f) {
    if (p == 0) {
      v.x = __float_as_uint(f.x);
      v.y = __float_as_uint(f.y);
    } else {
      v.z = __float_as_uint(f.x);
      v.w = __float_as_uint(f.y);
    }
  }
};

// 1 - 2^-y, given E = 2^-y from the MUFU.  Where |y| is small, 1 - E cancels;
// there the Taylor series of 1 - exp(-x) in x = y ln 2 is used, written in y:
//   sum_k (-1)^(k+1) (ln 2)^k y^k / k!.
// bf16 outputs: terms to y^4 for |x| < 1/16 (truncation below 2^-22 relative;
// 1 - E above it within about 2^-19).  fp32 outputs: terms to y^6 for
// |x| < 1/4 (truncation below 2^-24; 1 - E above it within about 2^-21).
// Valid for either sign of y.
template <typename S>
struct Series;

template <>
struct Series<Bf16> {
  static constexpr float kYmax = 0.0625f / kLn2;
  __device__ __forceinline__ static float2 eval(float2 y) {
    const float c1 = kLn2, c2 = -kLn2 * kLn2 / 2.0f, c3 = kLn2 * kLn2 * kLn2 / 6.0f,
                c4 = -kLn2 * kLn2 * kLn2 * kLn2 / 24.0f;
    float2 p = fma2(y, splat(c4), splat(c3));
    p = fma2(p, y, splat(c2));
    p = fma2(p, y, splat(c1));
    return mul2(p, y);
  }
};

template <>
struct Series<F32> {
  static constexpr float kYmax = 0.25f / kLn2;
  __device__ __forceinline__ static float2 eval(float2 y) {
    const float l = kLn2;
    const float c1 = l, c2 = -l * l / 2.0f, c3 = l * l * l / 6.0f, c4 = -l * l * l * l / 24.0f,
                c5 = l * l * l * l * l / 120.0f, c6 = -l * l * l * l * l * l / 720.0f;
    float2 p = fma2(y, splat(c6), splat(c5));
    p = fma2(p, y, splat(c4));
    p = fma2(p, y, splat(c3));
    p = fma2(p, y, splat(c2));
    p = fma2(p, y, splat(c1));
    return mul2(p, y);
  }
};

// The bf16 backward's up branch feeds T_u only as a relative factor (dG within
// 2^-8, d_w as a sum of terms with independent rounding), so terms to y^3 for
// |x| < 1/32 suffice there (truncation below 2^-19.6; 1 - E above it within
// about 2^-18).
struct SeriesBf16Up {
  static constexpr float kYmax = 0.03125f / kLn2;
  __device__ __forceinline__ static float2 eval(float2 y) {
    const float c1 = kLn2, c2 = -kLn2 * kLn2 / 2.0f, c3 = kLn2 * kLn2 * kLn2 / 6.0f;
    float2 p = fma2(y, splat(c3), splat(c2));
    p = fma2(p, y, splat(c1));
    return mul2(p, y);
  }
};

// Series used for the backward's up branch, per storage type.
template <typename S>
struct UpSeries {
  using type = Series<S>;
};
template <>
struct UpSeries<Bf16> {
  using type = SeriesBf16Up;
};

template <typename S, typename P = Series<S>>
__device__ __forceinline__ float2 one_minus_exp2_neg(float2 y, float2 E) {
  const float2 series = P::eval(y);
  const float2 direct = fma2(E, splat(-1.0f), splat(1.0f));
  return make_float2(fabsf(y.x) < P::kYmax ? series.x : direct.x, fabsf(y.y) < P::kYmax ? series.y : direct.y);
}

// How the two gate exponentials relate for the given beta.
enum GateMode : int {
  kGateGeneric = 0,  // two independent exponentials
  kGateSquare = 1,   // beta = 4: E_s = E_t^2
  kGateEqual = 2,    // beta = 2: E_s = E_t
  kGateRoot = 3,     // beta = 1: E_t = E_s^2
};

struct Coeffs {
  float beta;    // gate beta
  float lb;      // linear beta (1 without one)
  float inv_lb;  // 1 / linear beta
  float kt;      // 2 log2(e) / beta:    E_t = 2^-(|g| kt)
  float ku;      // 2 log2(e) / beta_L:  E_u = 2^-(|u| ku)
  float bb;      // beta * beta_L (beta without a linear beta)
};

// Exponentials of the gate: E_t = 2^-y with y = |g| kt (or g kt, signed form)
// and E_s = exp(-|g|) (exp(-g)).  `y` must already hold the scaled argument.
template <int GATE>
__device__ __forceinline__ void gate_exps(float2 y, float2& Et, float2& Es) {
  if (GATE == kGateSquare) {
    Et = ex2_neg2(y);
    Es = mul2(Et, Et);
  } else if (GATE == kGateEqual) {
    Et = ex2_neg2(y);
    Es = Et;
  } else if (GATE == kGateRoot) {  // kt = 2 log2(e): E_s = 2^-(y/2), E_t = E_s^2
    Es = ex2_neg2(mul2(y, splat(0.5f)));
    Et = mul2(Es, Es);
  } else {
    Et = ex2_neg2(y);
    Es = make_float2(0.0f, 0.0f);  // set by the caller from its own argument
  }
}

// ---- forward, bf16 storage ------------------------------------------------
// Signed form: with H = exp(-2g/beta) and Hs = exp(-g) (g of either sign),
//   tanh(g/beta) = (1 - H) / (1 + H),  sigmoid(g) = 1 / (1 + Hs),
//   T_g = beta (1 - H) / ((1 + H)(1 + Hs)),
// so neither a sign select nor |g| is needed.  The exponent argument is
// clamped at 2^126 (a NaN passes through); when (1 + H)(1 + Hs) overflows the
// reciprocal is 0 and T_g flushes to 0, which happens only where
// |T_g| < 4 exp(-59) -- below the bf16 output's absolute resolution of the
// tolerance.  The up branch uses the MUFU tanh (see tanh_approx).
template <int GATE, bool HAS_LB>
__device__ __forceinline__ float2 fwd_pair_bf16(Bits2 gb, Bits2 ub, float2 wbb, const Coeffs& c) {
  const float2 g = as_f2(gb);
  float2 y = mul2(g, splat(c.kt));
  y = make_float2(max_nan(y.x, -126.0f), max_nan(y.y, -126.0f));
  float2 H, Hs;
  gate_exps<GATE>(y, H, Hs);
  if (GATE == kGateGeneric) {
    float2 ys = mul2(g, splat(kLog2e));
    Hs = ex2_neg2(make_float2(max_nan(ys.x, -126.0f), max_nan(ys.y, -126.0f)));
  }
  const float2 em = one_minus_exp2_neg<Bf16>(y, H);
  const float2 den = mul2(add2(splat(1.0f), H), add2(splat(1.0f), Hs));
  float2 t;  // T_u / beta_L (or U)
  if (HAS_LB) {
    const float2 a = mul2(as_f2(ub), splat(c.inv_lb));
    t = make_float2(tanh_approx(a.x), tanh_approx(a.y));
  } else {
    t = as_f2(ub);
  }
  // em / den = T_g / beta lies in [-1, 1]: form it first so that a huge |1 - H|
  // meets its zero reciprocal before it can meet a large U.
  return mul2(mul2(em, rcp2(den)), mul2(t, wbb));
}

// ---- |g| form (fp32 forward and every backward) ---------------------------
// E_t = exp(-2|g|/beta) <= 1 and E_s = exp(-|g|) <= 1, so no intermediate can
// overflow; the sign of g enters through selects and sign flips.
struct GateAbs {
  float2 Et, Es, emt;  // emt = 1 - Et, accurate
};

template <int GATE, typename S>
__device__ __forceinline__ GateAbs gate_abs(Bits2 gb, const Coeffs& c) {
  const float2 ag = abs_f2(gb);
  const float2 y = mul2(ag, splat(c.kt));
  GateAbs r;
  gate_exps<GATE>(y, r.Et, r.Es);
  if (GATE == kGateGeneric) r.Es = ex2_neg2(mul2(ag, splat(kLog2e)));
  r.emt = one_minus_exp2_neg<S>(y, r.Et);
  return r;
}

template <typename S, typename P = Series<S>>
__device__ __forceinline__ float2 up_emu(Bits2 ub, const Coeffs& c, float2& Eu) {
  const float2 y = mul2(abs_f2(ub), splat(c.ku));
  Eu = ex2_neg2(y);
  return one_minus_exp2_neg<S, P>(y, Eu);
}

// fp32 forward of a pair.  Y = w beta beta_L s_g s_u (1 - E_t) sig (1 - E_u)
// / ((1 + E_t)(1 + E_s)(1 + E_u)), sig = 1 (g >= 0) or E_s (g < 0).
template <int GATE, bool HAS_LB, typename S>
__device__ __forceinline__ float2 fwd_pair_abs(Bits2 gb, Bits2 ub, float2 wbb, const Coeffs& c) {
  const GateAbs e = gate_abs<GATE, S>(gb, c);
  const float2 sig = select_neg2(gb, e.Es, splat(1.0f));
  float2 num = mul2(e.emt, sig);
  float2 den = mul2(add2(splat(1.0f), e.Et), add2(splat(1.0f), e.Es));
  if (HAS_LB) {
    float2 Eu;
    const float2 emu = up_emu<S>(ub, c, Eu);
    num = mul2(num, emu);
    den = mul2(den, add2(splat(1.0f), Eu));
    // sign of the product: s_g s_u
    const Bits2 s = {gb.lo ^ ub.lo, gb.hi ^ ub.hi};
    return xor_sign2(mul2(num, mul2(rcp2(den), wbb)), s);
  }
  num = mul2(num, abs_f2(ub));
  const Bits2 s = {gb.lo ^ ub.lo, gb.hi ^ ub.hi};
  return xor_sign2(mul2(num, mul2(rcp2(den), wbb)), s);
}

// Whether the backward of a pair takes the signed gate form: beta = 4, bf16
// dG and dU, and a caller whose every output derived from them tolerates the
// clamp below (CLAMPED): the native-output kernels and the per-column-weight
// backward, whose bf16 gradients carry an absolute tolerance far above the
// clamped values and whose weight gradients are sums.  Outputs that keep
// relative accuracy for tiny values -- block-scaled codes, whose scale
// follows the block, and per-element weight gradients -- take the |g| form
// (the block-scaled backward takes the signed form without the clamp where a
// warp vote shows it idle).  Measured on B200: 5 % less time for the bf16
// backward, 5-6 % for the per-column one.
template <int GATE, typename S, bool CLAMPED>
struct SignedBwd {
  static constexpr bool value = CLAMPED && GATE == kGateSquare && std::is_same<S, Bf16>::value;
};

// Backward of a pair.  With A = (1 + E_t)(1 + E_s), B = 1 + E_u (1 without a
// linear beta), sig as above and
//   tq  = (beta/4) tanh(g/beta) (1 + E_t)              (= (beta/4) s_g (1 - E_t))
//   T_g  = 4 tq sig / A  (tgA = tq sig A = T_g A^2 / 4)
//   T_g' = 4 [E_t sig (1 + E_s) + tq (1 + E_t) E_s] / A^2
//          (the sech^2(g/beta) sigmoid and beta tanh sigmoid (1 - sigmoid) terms)
//   T_u  = beta_L su / B,  su = s_u (1 - E_u),   T_u' = 4 E_u / B^2
// one reciprocal R = 1 / (A B)^2 serves every quotient.  The per-row factors
// are folded into two constants: k.x = 4 beta_L w (dG) and k.y = 16 w (dU);
// the d_w terms are accumulated without their factor 4 beta_L, which the
// caller applies once per row.  Returns dG, dU; adds go T_g T_u / (4 beta_L)
// to acc.
// The signed backward's clamp applied to packed bf16 gate values: g >= -27.75
// (a bf16 number; y = g kt >= -20.02 for beta = 4), NaN kept, one
// instruction per pair of elements.
__device__ __forceinline__ uint4 clamp_gate_bf16x8(uint4 v) {
  const uint32_t lo = 0xC1DEC1DEu;  // -27.75 in both halves
  asm("max.NaN.bf16x2 %0, %0, %4;\n\tmax.NaN.bf16x2 %1, %1, %4;\n\t"
      "max.NaN.bf16x2 %2, %2, %4;\n\tmax.NaN.bf16x2 %3, %3, %4;"
      : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
      : "r"(lo));
  return v;
}

template <int GATE, bool HAS_LB, typename S, bool CLAMPED = false, bool PRECLAMPED = false>
__device__ __forceinline__ void bwd_pair(Bits2 gb, Bits2 ub, float2 go, float2 kdg, float2 kdu, const Coeffs& c,
                                         float2& dg, float2& du, float2& acc) {
  float2 A, tgA, ng;
  if constexpr (SignedBwd<GATE, S, CLAMPED>::value) {
    // Signed form (beta = 4, bf16 outputs), as in the bf16 forward: with
    // H = exp(-g/2) and Hs = H^2 = exp(-g) for g of either sign,
    //   T_g  = 4 (1 - H) / A,                 A = (1 + H)(1 + Hs),
    //   T_g' = 4 [H (1 + Hs) + (1 - H)(1 + H) Hs] / A^2,
    // so no |g|, sign flip or select is needed.  The exponent argument is
    // clamped at 20 (g >= -27.7: H <= 2^20, A <= 2^60, (A B)^2 <= 2^122), where
    // |T_g| < 4e-12 and |T_g'| < 1e-11: far below a bf16 output's absolute
    // resolution of the tolerance.  PRECLAMPED: the caller clamped the packed
    // bf16 gate values at -27.75 instead (y >= -20.02, (A B)^2 <= 2^122.1).
    float2 y = mul2(as_f2(gb), splat(c.kt));
    if constexpr (!PRECLAMPED) y = make_float2(max_nan(y.x, -20.0f), max_nan(y.y, -20.0f));
    const float2 H = ex2_neg2(y), Hs = mul2(H, H);
    // 1 - H: below |x| = 1/32 from the series to x^3 (truncation under
    // 2^-19.6), above it 1 - H (MUFU error under 2^-17 relative there): both
    // far below what a bf16 output and a per-row sum of terms need.
    const float2 em = one_minus_exp2_neg<S, SeriesBf16Up>(y, H);
    const float2 opH = add2(splat(1.0f), H), opHs = add2(splat(1.0f), Hs);
    A = mul2(opH, opHs);
    tgA = mul2(em, A);                                // T_g A^2 / 4
    ng = fma2(H, opHs, mul2(mul2(em, opH), Hs));      // T_g' A^2 / 4
  } else {
    const GateAbs e = gate_abs<GATE, S>(gb, c);
    const float2 sig = select_neg2(gb, e.Es, splat(1.0f));
    const float2 opt = add2(splat(1.0f), e.Et), ops = add2(splat(1.0f), e.Es);
    A = mul2(opt, ops);
    float2 tq = xor_sign2(e.emt, gb);
    if (GATE != kGateSquare) tq = mul2(tq, splat(0.25f * c.beta));  // beta = 4: the factor is 1
    tgA = mul2(mul2(tq, sig), A);                                    // T_g A^2 / 4
    ng = fma2(mul2(e.Et, sig), ops, mul2(mul2(tq, opt), e.Es));      // T_g' A^2 / 4
  }
  if (HAS_LB) {
    float2 Eu;
    const float2 su = xor_sign2(up_emu<S, typename UpSeries<S>::type>(ub, c, Eu), ub);  // T_u B / beta_L
    const float2 B = add2(splat(1.0f), Eu);
    const float2 AB = mul2(A, B);
    const float2 gR = mul2(go, rcp2(mul2(AB, AB)));  // go / (A B)^2
    const float2 sB = mul2(su, B);
    const float2 gRt = mul2(gR, tgA);
    dg = mul2(mul2(gR, kdg), mul2(sB, ng));  // go w T_u T_g'
    du = mul2(gRt, mul2(Eu, kdu));           // go w T_g T_u'
    acc = fma2(gRt, sB, acc);                // go T_g T_u / (4 beta_L)
  } else {
    const float2 u = as_f2(ub);
    const float2 gR = mul2(go, rcp2(mul2(A, A)));  // go / A^2
    const float2 gRt = mul2(gR, tgA);
    dg = mul2(mul2(gR, kdg), mul2(u, ng));
    du = mul2(gRt, kdu);
    acc = fma2(gRt, u, acc);
  }
}

// Per-row constants of the backward: k.x = 4 beta_L w (dG); k.y = 16 w (dU:
// 4 from T_g, 4 from T_u' = 4 E_u / B^2), or 4 w without a linear beta
// (T_u' = 1); and the d_w scale 4 beta_L (beta_L = 1 without a linear beta).
template <bool HAS_LB>
__device__ __forceinline__ float2 bwd_row_consts(float w, const Coeffs& c) {
  return make_float2(4.0f * c.lb * w, (HAS_LB ? 16.0f : 4.0f) * w);
}
__device__ __forceinline__ float bwd_dw_scale(const Coeffs& c) { return 4.0f * c.lb; }

// Routing weight of a row.
struct RwArgs {
  const void* rw;
  int64_t stride;
  int mode;  // situ_rw_mode_t
  int bf16;  // storage dtype is bf16
};

__device__ __forceinline__ float load_rw(const RwArgs& a, int64_t row) {
  if (a.mode == SITU_RW_NONE) return 1.0f;
  const int64_t idx = a.mode == SITU_RW_ROW ? row * a.stride : 0;
  if (a.bf16) {
    const uint16_t h = __ldg(reinterpret_cast<const unsigned short*>(a.rw) + idx);
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  }
  return __ldg(reinterpret_cast<const float*>(a.rw) + idx);
}

// Sum over the CTA, in an order fixed by blockDim alone.  The result is valid
// in thread 0.  `slot` must alternate between two buffers from one call to
// the next so that a single barrier per call suffices.
__device__ __forceinline__ float block_sum(float v, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slot[warp] = v;
  __syncthreads();
  float total = 0.0f;
  if (warp == 0) {
    total = lane < static_cast<int>(blockDim.x >> 5) ? slot[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  return total;
}

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 r;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

__device__ __forceinline__ void st_stream8(void* p, const uint2& v) {
  asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ float2 bf16x2_to_f2(uint32_t q) {
  return make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
}

// ---------------------------------------------------------------------------
// MXFP8 outputs (OCP Microscaling Formats v1.0)
// ---------------------------------------------------------------------------
// Y (forward) or d_gate_up (backward) leave the kernel as FP8 E4M3 codes with
// one E8M0 scale per 32 consecutive elements of a row, the format of the
// MXFP8 recipe the SiTU-GLU integration was tested with (Megatron-LM PR #6673,
// "Test results").  A block is the 32 / kElems adjacent lanes that own its
// vectors (4 for bf16 inputs, 8 for fp32); its largest magnitude is combined
// with lane shuffles, so the fp32 values are quantised straight from
// registers.  Shared exponent e, stored as the byte e + 127:
//   SITU_MX_RULE_OCP:  floor(log2 amax) - 8 (the exponent of E4M3's largest
//                      normal), elements clamped to +-448;
//   SITU_MX_RULE_CEIL: the smallest e with amax <= 448 2^e (nothing clamps);
// both at least -127.  Both exponents come from the bits of amax, exactly.
// A block holding a NaN or an infinity gets scale byte 255 (NaN) and NaN codes.

constexpr int kMxBlock = 32;

struct MxOut {
  char* data;            // E4M3 codes, [tokens, cols]
  int64_t data_pitch;    // bytes
  uint8_t* scale;        // E8M0 bytes, [tokens, cols / 32]
  int64_t scale_pitch;   // bytes
  int rule;              // situ_mx_rule_t
};

__device__ __forceinline__ void st_stream_u32(void* p, uint32_t v) {
  asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Four E4M3 codes (nearest even, clamped to +-448, NaN to NaN) of a.x, a.y,
// b.x, b.y, in that byte order.  cvt...e4m3x2 puts its first source in the
// upper byte of the 16-bit result.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Where a thread's vector j of a row goes: its codes at byte kElems j of the
// row, its block's scale byte at j / (32 / kElems) (written by the block's
// first lane).  Computed once per thread.
template <typename S>
struct MxSlot {
  int code_off;
  int scale_off;
  bool lead;
  __device__ __forceinline__ explicit MxSlot(int j) {
    constexpr int kElems = 2 * S::kPairs, kLanes = kMxBlock / kElems;
    code_off = j * kElems;
    scale_off = j / kLanes;
    lead = (j % kLanes) == 0;
  }
};

// Quantise the kPairs pairs y of one vector of a row.  Every lane of the warp
// calls this (the block maximum is shuffled); lanes with `active` set store
// their codes and the first lane of each block the scale byte -- or, with
// SCALE_ALL_LANES, every lane of the block the same byte, which drops a branch
// (measured faster in the backward, slower in the forward).  A block is
// active or inactive as a whole (rows are multiples of 32 elements).
template <typename S, bool ACTIVE_ALWAYS = false, bool SCALE_ALL_LANES = false>
__device__ __forceinline__ void mx_store_vec(const float2 (&y)[S::kPairs], bool active, char* data_row,
                                             uint8_t* scale_row, const MxSlot<S>& slot, int rule) {
  constexpr int kElems = 2 * S::kPairs;
  constexpr int kLanes = kMxBlock / kElems;
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < S::kPairs; ++p) amax = max_nan(amax, max_nan(fabsf(y[p].x), fabsf(y[p].y)));
  if (!ACTIVE_ALWAYS && !active) amax = 0.0f;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const uint32_t ab = __float_as_uint(amax);
  const int ef = static_cast<int>(ab >> 23);  // amax >= 0 (or NaN with the sign bit clear)
  // e + 127 = (ef - 127) - 8 + 127, plus one under the no-clamp rule when the
  // significand of amax exceeds 1.75 (448 = 1.75 2^8); zero and subnormal
  // blocks land on the smallest scale; ef = 255 (NaN, inf) gives the NaN scale.
  int sb = ef - 8 + ((rule == SITU_MX_RULE_CEIL && (ab & 0x7fffffu) > 0x600000u) ? 1 : 0);
  sb = sb < 0 ? 0 : sb;
  const bool nan_blk = ef >= 255;
  sb = nan_blk ? 255 : sb;
  // 2^-e as a normal float (biased exponent 254 - sb in [7, 254] for sb <= 247);
  // a NaN block scales by NaN, so that its codes come out NaN.
  const float inv = nan_blk ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(254 - sb) << 23);
  uint32_t q[S::kPairs / 2];
#pragma unroll
  for (int k = 0; k < S::kPairs / 2; ++k) q[k] = e4m3x4(mul2(y[2 * k], splat(inv)), mul2(y[2 * k + 1], splat(inv)));
  if (!ACTIVE_ALWAYS && !active) return;
  char* p = data_row + slot.code_off;
  if constexpr (kElems == 8)
    st_stream8(p, make_uint2(q[0], q[1]));
  else
    st_stream_u32(p, q[0]);
  if (SCALE_ALL_LANES || slot.lead) scale_row[slot.scale_off] = static_cast<uint8_t>(sb);
}

// ---- NVFP4 (E2M1 codes, an E4M3 scale per 16 elements, a per-tensor scale)
// NVIDIA's NVFP4 format, the other block-scaled recipe the SiTU-GLU path was
// tested with (Megatron-LM PR #6673, "Test results").  With A the tensor's
// largest magnitude, S_enc = 448 * 6 / A (1 when A is 0 or not finite); block
// b of 16 elements stores s_b = E4M3(amax_b * S_enc / 6) and each element the
// E2M1 code of y * (S_enc / s_b) (nearest even, clamped to +-6); decoding is
// q * s_b / S_enc.  Codes are packed two per byte, element 2k in the low
// nibble.  A block holding NaN or infinity gets scale code 0x7F.

struct Nvfp4Out {
  char* data;            // packed E2M1 codes, [tokens, cols / 2] bytes
  int64_t data_pitch;    // bytes
  uint8_t* scale;        // E4M3 block scales, [tokens, cols / 16]
  int64_t scale_pitch;   // bytes
  const float* amax;     // device: the tensor's largest finite magnitude (read by the quantising pass)
  float* amax_out;       // the same word, written by the amax pass (host-side use)
};

// An NVFP4 output of the backward: where its codes go, and whether the
// caller gives the tensor maximum.
struct Nvfp4Bwd {
  Nvfp4Out out;
  int amax_given;
};

// Two E2M1 codes of (lo, hi) in one byte, lo in the low nibble (cvt packs its
// first source into the high nibble); four such bytes per register.
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x4(const float2 (&v)[2]) {
  uint16_t r;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "mov.b16 %0, {b0, b1};\n\t}"
      : "=h"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y));
  return r;
}

__device__ __forceinline__ float nvfp4_tensor_scale(float amax) {
  return (amax > 0.0f && amax <= 3.402823466e38f) ? 2688.0f / amax : 1.0f;  // 448 * 6 / A
}

// Quantise the kPairs pairs y of vector j of a row into NVFP4.  Every lane of
// the warp calls this (the block maximum is shuffled over the 16 / kElems
// lanes of a block); lanes with `active` set store their codes and the first
// lane of each block (SCALE_ALL_LANES: every lane of it) its scale code.
template <typename S, bool ACTIVE_ALWAYS = false, bool SCALE_ALL_LANES = false>
__device__ __forceinline__ void nvfp4_store_vec(const float2 (&y)[S::kPairs], bool active, char* data_row,
                                                uint8_t* scale_row, int j, float s_enc) {
  constexpr int kElems = 2 * S::kPairs;
  constexpr int kLanes = 16 / kElems;
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < S::kPairs; ++p) amax = max_nan(amax, max_nan(fabsf(y[p].x), fabsf(y[p].y)));
  if (!ACTIVE_ALWAYS && !active) amax = 0.0f;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const bool special = __float_as_uint(amax) >= 0x7f800000u;
  const uint8_t sc = special ? static_cast<uint8_t>(0x7f)
                             : static_cast<uint8_t>(__nv_cvt_float_to_fp8(amax * s_enc / 6.0f, __NV_SATFINITE, __NV_E4M3));
  const float sb = special ? 0.0f : __half2float(__half(__nv_cvt_fp8_to_halfraw(sc, __NV_E4M3)));
  // S_enc / s_b to 2 ulp (s_b is at most 448): an extra rounding of a few
  // 2^-24 that can only move an element sitting on an E2M1 midpoint
  const float r = sb > 0.0f ? __fdividef(s_enc, sb) : 0.0f;
  float2 q[S::kPairs];
#pragma unroll
  for (int p = 0; p < S::kPairs; ++p) q[p] = mul2(y[p], splat(r));
  if (!ACTIVE_ALWAYS && !active) return;
  if constexpr (S::kPairs == 4) {
    st_stream_u32(data_row + j * 4, e2m1x8(q));
  } else {
    const uint16_t v = static_cast<uint16_t>(e2m1x4(q));
    asm volatile("st.global.cs.u16 [%0], %1;" ::"l"(data_row + j * 2), "h"(v) : "memory");
  }
  if (SCALE_ALL_LANES || j % kLanes == 0) scale_row[j / kLanes] = sc;
}

// ---------------------------------------------------------------------------
// Bounded mbarrier waits, bulk copies and clusters
// ---------------------------------------------------------------------------

constexpr unsigned long long kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kStatusWaitExpired = 1;

// Status word of this translation unit's kernels (situ_glu_device_status reads
// every unit's).
[[maybe_unused]] __device__ int g_device_status = 0;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long global_timer_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Wait for the phase of parity `parity` to complete; false once `limit_ns`
// (the kernels': kWaitLimitNs) has passed.
__device__ __forceinline__ bool mbar_wait_for(uint64_t* b, uint32_t parity, unsigned long long limit_ns) {
  if (mbar_try_wait(b, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(b, parity))
    if (global_timer_ns() - t0 > limit_ns) return false;
  return true;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity) {
  return mbar_wait_for(b, parity, kWaitLimitNs);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// Thread-block clusters: this CTA's rank, its cluster's index and count
// (1-D grids), and cluster-scope addressing and synchronisation.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_index() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_count() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
  return r;
}
// The shared::cluster address of the same shared-memory location in CTA `rank`.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint4 lds16(const unsigned char* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void consumer_bar(int n) { asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory"); }

}  // namespace
