// arnq_glu.cuh -- gated activation + per-row dynamic quantization:
//
//   in = act(g) * u * smooth,   g = x[:, :n], u = x[:, n:]
//   act(g) = g / (1 + exp(-z)),  z = g (SiLU) or
//            z = 2 sqrt(2/pi) (g + 0.044715 g^3)   (GELU, tanh form: 0.5 (1 + tanh(z/2)) is the sigmoid of z)
//   scale = row_max(|in|) / Q,  code = round(in / scale)
//
// Binary32 error of a value, in units of |in| 2^-24: the exponential's argument
// is off by at most 1.5 |z| (the product with log2 e and that constant's
// rounding), for GELU 6 |z| (those of z too), which the sigmoid passes on for
// z < 0 and weakens to at most 0.28 of it for z > 0; the exponential's own 4
// (2 ulp), that for the reciprocal 2 and the three roundings of 1 + e and the
// products add 9.  Altogether 9 + s max(-z, 0), s = 2 or 6, with a margin of one
// for z > 0, for z >= kLow.  Below that, where the sigmoid nears the end of
// binary32's range, a value is at most 1.5e-33 |u smooth|: with |u smooth| <=
// 1e8 it and its error are far below what a row's maximum of at least kTiny
// (1e-18) can tell from zero; a row with a larger factor there is computed in
// fp64.
// The binary32 values are 2^64 times the true ones (the sigmoid is formed so, at
// no cost): gate * sigmoid then never falls below the normal range, where it would
// lose bits that a large up value lifts, and a gate beyond 2^64 overflows and sends
// its row to fp64.  up * smooth may fall below it in bf16 and lose up to 2^-150; times
// less than 2^128 that is 2^-22 at most, a quarter of 2^-24 of a maximum of at least
// kTiny (18.4 so scaled), and goes into the bounds' spare unit.
#pragma once

#include "arnq_rowquant.cuh"

namespace arnq {

constexpr float kLow = -80.f;
constexpr float kValueScale = 18446744073709551616.f;  // 2^64

enum : int { ACT_SILU = 0, ACT_GELU_TANH = 1 };

struct GluParams {
  RowOut out;
  const uint16_t *x;       // [rows, 2n]
  const uint16_t *smooth;  // [n] or nullptr
};

// 1 / (1 + exp(-z)) in fp64 to some 1e-14, for decisions that sit many orders
// of magnitude above that: exp(-z) = 2^k exp(r), |r| <= ln2 / 2 (ln2 taken
// off in two parts, the first of 32 bits so that k times it is exact: Cody and
// Waite's reduction), by its Taylor
// series to r^12 (the next term is below 2e-16), paired up to shorten the
// chain (Estrin's scheme); the reciprocal from the binary32 one by Newton
// steps.  Beyond +-700 the sigmoid is 1 or too small for any output.
__device__ __forceinline__ double sigmoid64(double z) {
  const double y = fmin(fmax(-z, -700.0), 700.0);
  const double kf = rint(y * 1.4426950408889634);
  const double r = __fma_rn(kf, -1.9082149292705877e-10, __fma_rn(kf, -0.6931471803691238, y));
  const double r2 = r * r, r4 = r2 * r2;
  const double a0 = 1.0 + r, a1 = __fma_rn(r, 1.0 / 6, 0.5), a2 = __fma_rn(r, 1.0 / 120, 1.0 / 24),
               a3 = __fma_rn(r, 1.0 / 5040, 1.0 / 720), a4 = __fma_rn(r, 1.0 / 362880, 1.0 / 40320),
               a5 = __fma_rn(r, 1.0 / 39916800, 1.0 / 3628800);
  const double b0 = __fma_rn(r2, a1, a0), b1 = __fma_rn(r2, a3, a2),
               b2 = __fma_rn(r2, __fma_rn(r2, 1.0 / 479001600, a5), a4);
  const double e = __fma_rn(r4, __fma_rn(r4, b2, b1), b0);
  const double d = 1.0 + e * __longlong_as_double(static_cast<long long>(static_cast<int>(kf) + 1023) << 52);
  if (d > 1e37) return div_ieee(1.0, d);
  double q = static_cast<double>(__fdividef(1.f, __double2float_rn(d)));
  q = __fma_rn(__fma_rn(-d, q, 1.0), q, q);
  return __fma_rn(__fma_rn(-d, q, 1.0), q, q);
}
// one value in fp64 (a gate of minus infinity: infinity times zero)
template <class T, int ACT>
__device__ __noinline__ double glu64(const uint16_t *gate, const uint16_t *up, const uint16_t *smooth) {
  const double g = static_cast<double>(Cvt<T>::f1(*gate));
  const double t = static_cast<double>(Cvt<T>::f1(*up));
  double in;
  if (g == 0.0 || t == 0.0) {
    in = __dmul_rn(g, t);  // (0 times an infinity or NaN is NaN, here and below)
  } else if (g < -1e300) {
    in = __longlong_as_double(0x7FF8000000000000ll);
  } else {
    double z = g;
    if (ACT == ACT_GELU_TANH) z = 1.5957691216057308 * (g + 0.044715 * g * g * g);
    in = g * sigmoid64(z) * t;
  }
  return smooth ? in * static_cast<double>(Cvt<T>::f1(*smooth)) : in;
}

template <class T_, int ACT, int QT_, int MODE_, int UPT_>
struct GluOp {
  typedef T_ T;
  typedef GluParams Params;
  static constexpr int QT = QT_, UPT = UPT_, kInputs = 2;
  static constexpr bool kReadsSlots = true;
  static constexpr float kLeast = kTiny * kValueScale;
  static constexpr int MODE = MODE_;
  static constexpr bool STAGED = is_wide(MODE_) && UPT_ > 0;
  static constexpr int kMaxThreads = UPT == 4 ? 512 : 1024, kMinCtas = UPT == 4 ? 2 : 1;
  struct Keep {
    float low;  // the unit's smallest z, at most 0
  };
  const Params &p;
  __device__ __forceinline__ explicit GluOp(const Params &q) : p(q) {}
  __device__ __forceinline__ void setup(RowSmem &, int, int, int) {}
  __device__ __forceinline__ const uint16_t *gate_of(int64_t row) const {
    return p.x + row * (2 * static_cast<int64_t>(p.out.n));
  }
  __device__ __forceinline__ void stage(int64_t row, int u, uint4 *slot, int stride) const {
    const bool there = MODE == WIDE || 8 * u < p.out.n;
    const uint16_t *r = gate_of(row) + (there ? 8 * u : 0);
    if (MODE == WIDE) {
      copy16_async(slot, r);
      copy16_async(slot + stride, r + p.out.n);
    } else {
      copy16_async(slot, r, there);
      copy16_async(slot + stride, r + p.out.n, there);
    }
  }
  template <class E, class N>
  __device__ __forceinline__ void prepare(RowSmem &, int64_t, Keep *, const uint4 *, int, E &&, int, N &&) {}

  static __device__ __forceinline__ float2 arg2(float2 g) {
    if (ACT == ACT_SILU) return g;
    // 2 sqrt(2/pi) = 1.5957691..., times 0.044715 = 0.0713548...
    const float2 c = make_float2(0.07135481282839f, 0.07135481282839f),
                 d = make_float2(1.59576912160573f, 1.59576912160573f);
    return __fmul2_rn(g, __ffma2_rn(__fmul2_rn(c, g), g, d));
  }
  static __device__ __forceinline__ float exp2_approx(float y) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    return e;
  }
  __device__ __forceinline__ bool value(int64_t row, int u, Keep &keep, const uint4 *slot, int stride,
                                        float2 v[4]) const {
    float2 g[4], t[4];
    if (STAGED) {
      unpack<T>(slot[0], g);
      unpack<T>(slot[stride], t);
    } else {
      unpack<T>(load_unit<MODE>(gate_of(row), u, p.out.n), g);
      unpack<T>(load_unit<MODE>(gate_of(row) + p.out.n, u, p.out.n), t);
    }
    if (p.smooth) {
      float2 s[4];
      unpack<T>(load_unit<MODE>(p.smooth, u, p.out.n), s);
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = __fmul2_rn(t[k], s[k]);  // exact in the normal range
    }
    float low = 0.f;
    const float2 l = make_float2(-1.44269504088896f, -1.44269504088896f),
                 unit = make_float2(1.f / kValueScale, 1.f / kValueScale);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // g * sigmoid(z) * u * smooth times 2^64, exp(-z) = 2^(-z log2 e)
      const float2 z = arg2(g[k]);
      asm("min.f32 %0, %1, %2, %3;" : "=f"(low) : "f"(z.x), "f"(z.y), "f"(low));
      const float2 y = __fmul2_rn(z, l);
      const float2 e = __ffma2_rn(make_float2(exp2_approx(y.x), exp2_approx(y.y)), unit, unit);
      v[k] = __fmul2_rn(__fmul2_rn(g[k], make_float2(rcp_approx(e.x), rcp_approx(e.y))), t[k]);
    }
    keep.low = low;
    // a sigmoid that nears or leaves binary32's range matters only beside a
    // huge factor
    return !(low < kLow) || abs_max8(t) <= 1e8f;
  }
  __device__ __forceinline__ double value64(int64_t row, int c) const {
    const uint16_t *g = gate_of(row) + c;
    return glu64<T, ACT>(g, g + p.out.n, p.smooth ? p.smooth + c : nullptr);
  }
  __device__ __forceinline__ bool zero_row(int64_t row, int tid, int nt) const {
    uint32_t bits = 0u;
    for (int u = tid; u < p.out.units; u += nt) {
      const uint4 g = load_unit<MODE>(gate_of(row), u, p.out.n), t = load_unit<MODE>(gate_of(row) + p.out.n, u, p.out.n);
      bits |= g.x | g.y | g.z | g.w | t.x | t.y | t.z | t.w;
    }
    return (bits & 0x7FFF7FFFu) == 0u;
  }
  __device__ __forceinline__ void save(double *) const {}
  __device__ __forceinline__ void restore(int64_t, const double *) const {}
  // units that may hold the maximum: 2^-13 covers the error for every z >= kLow
  __device__ __forceinline__ float slack(float M) const { return M * 1.220703125e-4f; }
  static constexpr float kUnit24 = 5.9604644775390625e-8f;  // 2^-24
  static constexpr float kSlope = ACT == ACT_SILU ? 2.f : 6.f;
  // the row's maximum is taken to have z >= -2 (coarse() counts on it)
  __device__ __forceinline__ bool sure(int64_t row, int u, const float2 v[4], float thr) const {
    bool ok = true;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (fabsf(elem(v, j)) >= thr) {
        const float g = Cvt<T>::f1(gate_of(row)[column<MODE>(u, j)]);
        ok = ok && arg2(make_float2(g, g)).x >= -2.f;
      }
    return ok;
  }
  // a value's 9 + slope max(-z, 0), the scale's (the same at z = -2) and 5 for
  // the scale's and the quotient's roundings
  __device__ __forceinline__ float coarse(const Keep &keep, float) const {
    constexpr float q = (QT == 1 ? 7.01f : 127.01f) * kUnit24;
    return __fmaf_rn(fminf(-keep.low, -kLow), q * kSlope, q * (24.f + 2.f * kSlope));
  }
};

}  // namespace arnq
