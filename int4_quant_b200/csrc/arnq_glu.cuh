// arnq_glu.cuh -- gated activation + per-row dynamic quantization:
//
//   in = act(g) * u * smooth,   g = x[:, :n], u = x[:, n:]
//   act(g) = g / (1 + exp(-z)),  z = g (SiLU) or
//            z = 2 sqrt(2/pi) (g + 0.044715 g^3)   (GELU, tanh form: 0.5 (1 + tanh(z/2)) is the sigmoid of z)
//   scale = row_max(|in|) / Q,  code = round(in / scale)
//
// Binary32 error of a value, in units of |in| 2^-24: the exponential's
// argument is off by at most 6 |z| (roundings of z and of the product with
// log2 e, the constants'), which the sigmoid passes on for z < 0 and weakens
// to at most 0.28 * 6 for z > 0; the exponential (4), the division (4) and
// the remaining roundings (3) add 11.  The quotient by the scale adds 3.
// Altogether |error| <= |in| 2^-24 (20 + 8 max(-z, 0)) with a margin.  Values
// with z < kLow, whose sigmoid nears the end of binary32's range, are
// computed in fp64.
#pragma once

#include "arnq_rowquant.cuh"

namespace arnq {

constexpr float kLow = -80.f;

enum : int { ACT_SILU = 0, ACT_GELU_TANH = 1 };

struct GluParams {
  RowOut out;
  const uint16_t *x;       // [rows, 2n]
  const uint16_t *smooth;  // [n] or nullptr
};

template <class T_, int ACT, int QT_, bool VEC_, int UPT_>
struct GluOp {
  typedef T_ T;
  typedef GluParams Params;
  static constexpr int QT = QT_, UPT = UPT_;
  static constexpr bool VEC = VEC_;
  static constexpr int kMaxThreads = UPT == 4 ? 512 : 1024, kMinCtas = 1;
  struct Raw {
    uint4 g, u;
  };
  const Params &p;
  __device__ __forceinline__ explicit GluOp(const Params &q) : p(q) {}
  __device__ __forceinline__ void setup(RowSmem &, int, int, int) {}
  __device__ __forceinline__ Raw fetch(int64_t row, int u) const {
    const uint16_t *r = p.x + row * (2 * static_cast<int64_t>(p.out.n));
    Raw w;
    w.g = load_unit<VEC, UPT != 0>(r, u, p.out.n);
    w.u = load_unit<VEC, UPT != 0>(r + p.out.n, u, p.out.n);
    return w;
  }
  __device__ __forceinline__ Raw refetch(int64_t row, int u) const { return fetch(row, u); }
  template <class E>
  __device__ __forceinline__ void prepare(RowSmem &, int64_t, Raw *, E &&, int) {}

  static __device__ __forceinline__ float arg(float g) {
    if (ACT == ACT_SILU) return g;
    // 2 sqrt(2/pi) = 1.5957691..., times 0.044715 = 0.0713548...
    return g * __fmaf_rn(0.07135481282839f * g, g, 1.59576912160573f);
  }
  // g * sigmoid(z): exp(-z) = 2^(-z log2 e)
  static __device__ __forceinline__ float act(float g, float z) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504088896f * z));
    return __fdividef(g, 1.f + e);
  }
  __device__ __forceinline__ void value(const Raw &w, int u, float2 v[4]) const {
    float2 g[4], t[4];
    unpack<T>(w.g, g);
    unpack<T>(w.u, t);
    float low = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float zx = arg(g[k].x), zy = arg(g[k].y);
      low = fminf(low, fminf(zx, zy));
      v[k] = __fmul2_rn(make_float2(act(g[k].x, zx), act(g[k].y, zy)), t[k]);
    }
    if (p.smooth) {
      float2 s[4];
      unpack<T>(load_unit<VEC, false>(p.smooth, u, p.out.n), s);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(v[k], s[k]);
    }
    if (low < kLow) {  // sigmoids near or below the end of binary32's range
      const int cnt = min(8, p.out.n - 8 * u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= cnt || !(arg(elem(g, j)) < kLow)) continue;
        const float f = __double2float_rn(value64(w, u, j));
        if (j & 1) v[j >> 1].y = f;
        else v[j >> 1].x = f;
      }
    }
  }
  __device__ __forceinline__ double value64(const Raw &w, int u, int j) const {
    const double g = static_cast<double>(Cvt<T>::f1(get16(w.g, j)));
    const double t = static_cast<double>(Cvt<T>::f1(get16(w.u, j)));
    if (g == 0.0 || t == 0.0) return __dmul_rn(g, t);  // (0 times an infinity or NaN is NaN)
    double z = g;
    if (ACT == ACT_GELU_TANH) z = 1.5957691216057308 * (g + 0.044715 * g * g * g);
    const double a = g / (1.0 + exp(-z));
    double in = a * t;
    if (p.smooth) in *= static_cast<double>(Cvt<T>::f1(p.smooth[8 * u + j]));
    return in;
  }
  // candidates for the maximum: 2^-13 covers the error for every z >= kLow
  __device__ __forceinline__ float slack(float M) const { return M * 1.220703125e-4f; }
  __device__ __forceinline__ float tolerance(const Raw &w, int j, float t, float) const {
    const float z = arg(Cvt<T>::f1(get16(w.g, j)));
    return fabsf(t) * __fmaf_rn(fmaxf(-z, 0.f), 4.76837158203125e-7f, 1.1920928955078125e-6f);
  }
};

}  // namespace arnq
