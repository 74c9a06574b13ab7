// arnq_norms.cuh -- the norms around a block's residual, then per-row dynamic
// quantization:
//
//   p  = h / sqrt(mean(h^2) + eps_post) * gamma_post
//   x' = RN16(x + alpha * gate * p)            (written as xOut)
//   in = (x' / sqrt(mean(x'^2) + eps) * gamma + beta) * smooth
//   scale = row_max(|in|) / Q, code = round(in / scale); or, without codes, `in` as
//   binary32 gives it (four roundings at most), rounded to 16 bits
//
// x' is decided like the codes: the binary32 sum v = x + h*G*(alpha/Rms(h)),
// G = gamma_post*gate (exact: two 16-bit values), carries an error of a few
// 2^-24 of its terms (kFactorError, kSumError below); where both ends of that
// interval do not round to the same 16-bit value the element is recomputed in
// fp64 (1e-4 of the elements in bf16, 1e-3 in fp16).
#pragma once

#include "arnq_rowquant.cuh"

namespace arnq {

// h * (gamma_post * gate) is exact in binary32 for bf16: 8 + 16 bits
template <class T> constexpr bool kExactProducts = false;
template <> constexpr bool kExactProducts<Bf16> = true;

struct NormsParams {
  RowOut out;
  const uint16_t *h, *x, *gamma_post, *gate, *gamma, *beta, *smooth;
  uint16_t *x_out;        // may be x; may be nullptr
  int32_t rows_per_gate;  // rows that share a row of gate; rows: one gate row for all
  float alpha, eps_post, eps;
  double inv_n;           // 1 / n
};

// 1/Rms of a row in fp64, and in binary32 times `alpha`; ss >= 0 or NaN.
struct Rms {
  double inv64;  // alpha / Rms
  float inv;     // the same rounded
  bool cold;     // outside the range where the binary32 path is bounded
};
// A sum of squares that overflowed or (with no eps to speak of) underflowed.
__device__ __forceinline__ bool ss_out_of_range(double ss, float eps) {
  return !(ss <= 1e37) || !(ss >= 1e-30 || eps >= 1e-12f);
}
__device__ __forceinline__ Rms make_rms(double ss, double inv_n, float eps, float alpha, bool cold) {
  Rms r;
  const double ms = __fma_rn(ss, inv_n, static_cast<double>(eps));
  if (cold || !(ms >= 1e-30)) {
    // a zero Rms normalises a row of zeros: its values stay zero
    const double rms = sqrt_ieee(ms);
    r.inv64 = rms == 0.0 ? 0.0 : div_ieee(static_cast<double>(alpha), rms);
    cold = true;
  } else {
    r.inv64 = __dmul_rn(static_cast<double>(alpha), rsqrt64(ms));
  }
  r.inv = __double2float_rn(r.inv64);
  // a factor near the ends of binary32's range has no useful rounding bound
  const float a = fabsf(r.inv);
  r.cold = cold || !(a <= 1e30f && (a >= 1e-30f || r.inv64 == 0.0));
  return r;
}

// x' of one element in fp64, rounded once
template <class T>
__device__ __forceinline__ uint16_t x64(uint16_t h, uint16_t x, const uint16_t *gamma_post,
                                        const uint16_t *gate, double inv) {
  double t = __dmul_rn(__dmul_rn(static_cast<double>(Cvt<T>::f1(h)), inv),
                       static_cast<double>(Cvt<T>::f1(*gamma_post)));
  if (gate) t = __dmul_rn(t, static_cast<double>(Cvt<T>::f1(*gate)));
  return round16<T>(__dadd_rn(static_cast<double>(Cvt<T>::f1(x)), t));
}
// The elements of unit u whose halves differ between lo and hi (the bound's two
// ends), from the unit's inputs h and x.
template <class T, int MODE>
__device__ __noinline__ uint4 settle_x(uint4 lo, uint4 hi, uint4 h, uint4 x, const uint16_t *gamma_post,
                                       const uint16_t *gate, double inv, int u, int n) {
  unsigned m = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t d = word_of(lo, k) ^ word_of(hi, k);
    m |= (d & 0xFFFFu ? 1u << (2 * k) : 0u) | (d >> 16 ? 2u << (2 * k) : 0u);
  }
#pragma unroll 1
  for (; m; m &= m - 1u) {
    const int j = __ffs(m) - 1, c = column<MODE>(u, j);
    set16(lo, j, c < n ? x64<T>(get16(h, j), get16(x, j), gamma_post + c, gate ? gate + c : nullptr, inv)
                       : static_cast<uint16_t>(0));
  }
  return lo;
}
// This thread's part of a row's sum of squares in fp64 throughout: of row a or,
// where x' was not stored, of x' made from h, x.
template <class T>
__device__ __noinline__ double sumsq_cold(const uint16_t *a, const uint16_t *h, const uint16_t *x,
                                          const uint16_t *gamma_post, const uint16_t *gate, double inv,
                                          int n) {
  double s = 0.0;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    const uint16_t w = a ? a[c] : x64<T>(h[c], x[c], gamma_post + c, gate ? gate + c : nullptr, inv);
    const double v = static_cast<double>(Cvt<T>::f1(w));
    s = __fma_rn(v, v, s);
  }
  return s;
}

template <class T_, int QT_, int MODE_, int UPT_>
struct NormsOp {
  typedef T_ T;
  typedef NormsParams Params;
  static constexpr int QT = QT_, UPT = UPT_, kInputs = 2;
  static constexpr bool kReadsSlots = false;  // after prepare()
  // The binary32 values of `in` are 2^64 times the true ones in bf16, whose x' / Rms
  // may otherwise fall below the normal range and lose bits (2^-150) that a large
  // gamma * smooth lifts.  So scaled they lose 2^-22 at most (times less than 2^128),
  // a quarter of 2^-24 of a maximum of at least kLeast, within the bounds below, which
  // count four roundings where there are three.  (fp16 values leave no range.)
  static constexpr float kValueScale = kExactProducts<T> ? 18446744073709551616.f : 1.f;
  static constexpr float kLeast = kTiny * kValueScale;
  static constexpr int MODE = MODE_;
  static constexpr bool STAGED = is_wide(MODE_) && UPT_ > 0;
  static constexpr int kMaxThreads = UPT == 4 ? (QT == kQNone ? 288 : 384) : 1024,
                       kMinCtas = UPT == 4 ? (QT == kQNone ? 3 : 2) : 1;
  struct Keep {
    float2 f[4];  // the unit's h, then its x'
  };
  // Error of v = x + (h G) f in units of 2^-24: the factor f one of |h G f|, the
  // product h G none in bf16 (8 + 16 bits) and one in fp16 (11 + 22), the
  // fused multiply-add one of |v|; and the bound's own roundings (v +- e).
  static constexpr float kFactorError = (kExactProducts<T> ? 1.25f : 2.25f) * 5.9604644775390625e-8f;
  static constexpr float kSumError = 2.25f * 5.9604644775390625e-8f;
  // What G = gamma_post * gate loses below the normal range, at most 2^-150, times
  // sqrt(ARNQ_MAX_N) < 363, with a factor of two for this constant's own rounding
  // and the bound's (fp16: G is exact); the sum itself loses up to 2^-150 there.
  static constexpr float kGateLoss = kExactProducts<T> ? 363.f * 1.401298464324817e-45f : 0.f;
  static constexpr float kLeastError = 4.f * 1.401298464324817e-45f;
  const Params &p;
  float bmax;  // max |beta * smooth|, times kValueScale
  const uint16_t *gate_row;
  Rms post, pre;
  bool zero;  // x' is zero throughout
  __device__ __forceinline__ explicit NormsOp(const Params &q)
      : p(q), bmax(0.f), gate_row(nullptr), zero(false) {}

  __device__ __forceinline__ void setup(RowSmem &sm, int tid, int nt, int nwarps) {
    if (!p.beta) return;
    float b = 0.f;
    for (int u = tid; u < p.out.units; u += nt) {
      float2 v[4];
      unpack<T>(load_unit<MODE>(p.beta, u, p.out.n), v);
      times(v, p.smooth, u);
      b = abs_top8(v, b);
    }
    bmax = block_max(b, sm.top[1], nwarps) * kValueScale;
    __syncthreads();  // the slots are used again at once
  }
  __device__ __forceinline__ void times(float2 v[4], const uint16_t *by, int u) const {
    if (!by) return;
    float2 s[4];
    unpack<T>(load_unit<MODE>(by, u, p.out.n), s);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(v[k], s[k]);
  }
  __device__ __forceinline__ void find_gate(int64_t row) {
    gate_row = p.gate ? p.gate + static_cast<int64_t>(static_cast<uint32_t>(row) /
                                                      static_cast<uint32_t>(p.rows_per_gate)) *
                                     p.out.n
                      : nullptr;
  }
  __device__ __forceinline__ void stage(int64_t row, int u, uint4 *slot, int stride) const {
    const bool there = MODE == WIDE || 8 * u < p.out.n;
    const int64_t off = row * p.out.n + (there ? 8 * u : 0);
    if (MODE == WIDE) {
      copy16_async(slot, p.h + off);
      copy16_async(slot + stride, p.x + off);
    } else {
      copy16_async(slot, p.h + off, there);
      copy16_async(slot + stride, p.x + off, there);
    }
  }
  __device__ __forceinline__ uint4 get_h(int64_t row, int u, const uint4 *slot) const {
    return STAGED ? slot[0] : load_unit<MODE>(p.h + row * p.out.n, u, p.out.n);
  }
  __device__ __forceinline__ uint4 get_x(int64_t row, int u, const uint4 *slot, int stride) const {
    return STAGED ? slot[stride] : load_unit<MODE>(p.x + row * p.out.n, u, p.out.n);
  }
  // long rows: x' of a unit after the row's first phases, read back or made again
  __device__ __forceinline__ void x_again(int64_t row, int u, Keep &keep) const {
    if (p.x_out) {
      unpack<T>(load_unit<MODE>(p.x_out + row * p.out.n, u, p.out.n), keep.f);
    } else {
      unpack<T>(get_h(row, u, nullptr), keep.f);
      make_x(row, u, keep, nullptr, 0);
    }
  }

  // keep: the unit's h, turned into its x', which is returned packed too
  __device__ __forceinline__ uint4 make_x(int64_t row, int u, Keep &keep, const uint4 *slot, int stride) const {
    float2 x[4], G[4];
    const uint4 xw = get_x(row, u, slot, stride);
    unpack<T>(xw, x);
    unpack<T>(load_unit<MODE>(p.gamma_post, u, p.out.n), G);
    times(G, gate_row, u);
    const float2 f = make_float2(post.inv, post.inv);
    float2 v[4];
    float tmax = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 hg = __fmul2_rn(keep.f[k], G[k]);
      v[k] = __ffma2_rn(hg, f, x[k]);
      tmax = abs_max3_nan(hg.x, hg.y, tmax);
    }
    // the unit's largest |h G| serves its eight elements; products below the
    // normal range lose up to 2^-149 each, and what G lost is multiplied by h,
    // which is at most sqrt(n) Rms(h); a cold row has no binary32 bound:
    // everything in fp64
    const float floor_e = post.cold ? __int_as_float(0x7F800000)
                                    : __fmaf_rn(fabsf(post.inv), 1.1754944e-38f,
                                                __fmaf_rn(fabsf(p.alpha), kGateLoss, kLeastError));
    const float e = __fmaf_rn(tmax, fabsf(post.inv) * kFactorError, floor_e);
    uint32_t lo[4], hi[4], differ = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 bound = make_float2(__fmaf_rn(fabsf(v[k].x), kSumError, e), __fmaf_rn(fabsf(v[k].y), kSumError, e));
      const float2 a = __ffma2_rn(bound, make_float2(-1.f, -1.f), v[k]), b = __fadd2_rn(v[k], bound);
      lo[k] = Cvt<T>::pack(a.x, a.y);
      hi[k] = Cvt<T>::pack(b.x, b.y);
      differ |= lo[k] ^ hi[k];
    }
    uint4 r = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    // a product overflowed (0 times it would be NaN) or is NaN, or the row is cold
    // (v may be NaN where 0 met a factor that overflowed, and lo equal hi)
    const bool beyond = !(tmax <= kHuge) || post.cold;
    if (differ || beyond) {
      const uint4 hw = get_h(row, u, slot);
      if (!beyond && ((hw.x | hw.y | hw.z | hw.w) & 0x7FFF7FFFu) == 0u)  // (padding) v is x itself
        r = make_uint4(Cvt<T>::pack(v[0].x, v[0].y), Cvt<T>::pack(v[1].x, v[1].y), Cvt<T>::pack(v[2].x, v[2].y),
                       Cvt<T>::pack(v[3].x, v[3].y));
      else
        r = settle_x<T, MODE>(r, beyond ? make_uint4(~lo[0], ~lo[1], ~lo[2], ~lo[3]) : make_uint4(hi[0], hi[1], hi[2], hi[3]),
                              hw, xw, p.gamma_post, gate_row, post.inv64, u, p.out.n);
    }
    unpack<T>(r, keep.f);
    return r;
  }

  template <class E, class N>
  __device__ __forceinline__ void prepare(RowSmem &sm, int64_t row, Keep *keep, const uint4 *slot, int nt,
                                          E &&each, int nwarps, N &&next) {
    const int stride = UPT * nt;
    find_gate(row);
    // ---- Rms of h
    double ss = 0.0;
    each([&](int u, int i) {
      unpack<T>(get_h(row, u, slot + i * nt), keep[i].f);
      ss += sumsq(keep[i].f);
    });
    ss = block_sum(ss, sm.sum[0], nwarps);
    bool cold = ss_out_of_range(ss, p.eps_post);
    if (cold) {  // the same for every thread
      ss = sumsq_cold<T>(p.h + row * p.out.n, nullptr, nullptr, nullptr, nullptr, 0.0, p.out.n);
      ss = block_sum(ss, sm.sum[2], nwarps);
    }
    post = make_rms(ss, p.inv_n, p.eps_post, p.alpha, cold);
    // ---- x' and its Rms
    ss = 0.0;
    each([&](int u, int i) {
      if (UPT == 0) unpack<T>(get_h(row, u, nullptr), keep[0].f);
      const uint4 x = make_x(row, u, keep[i], slot + i * nt, stride);
      ss += sumsq(keep[i].f);
      if (p.x_out) store_unit<MODE>(p.x_out + row * p.out.n, u, p.out.n, x);
    });
    asm volatile("" : "+d"(ss));  // the slots have been read once ss is there
    next();
    ss = block_sum(ss, sm.sum[1], nwarps);
    cold = ss_out_of_range(ss, p.eps);
    if (cold) {
      const int64_t off = row * p.out.n;
      __syncwarp();  // x' was stored by other threads: of the warp, or in front of block_sum's barrier
      ss = sumsq_cold<T>(p.x_out ? p.x_out + off : nullptr, p.h + off, p.x + off, p.gamma_post, gate_row,
                         post.inv64, p.out.n);
      ss = block_sum(ss, sm.sum[2], nwarps);
    }
    zero = ss == 0.0;
    pre = make_rms(ss, p.inv_n, p.eps, 1.f, cold);
    if (kValueScale != 1.f) {
      pre.cold = pre.cold || !(pre.inv <= 1e30f / kValueScale);
      pre.inv *= kValueScale;
    }
  }

  __device__ __forceinline__ bool value(int64_t row, int u, Keep &keep, const uint4 *, int, float2 v[4]) const {
    if (UPT == 0) x_again(row, u, keep);
    float2 G[4], B[4];
    unpack<T>(load_unit<MODE>(p.gamma, u, p.out.n), G);
    times(G, p.smooth, u);
    const float2 r = make_float2(pre.inv, pre.inv), up = make_float2(kValueScale, kValueScale),
                 down = make_float2(1.f / kValueScale, 1.f / kValueScale);
    if (p.beta) {
      unpack<T>(load_unit<MODE>(p.beta, u, p.out.n), B);
      times(B, p.smooth, u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (kValueScale != 1.f) B[k] = __fmul2_rn(B[k], up);
        v[k] = __ffma2_rn(__fmul2_rn(keep.f[k], r), G[k], B[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(__fmul2_rn(keep.f[k], r), G[k]);
    }
    if (QT == kQNone && kValueScale != 1.f) {  // (the values themselves are wanted)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(v[k], down);
    }
    return !pre.cold;
  }
  __device__ __forceinline__ double value64(int64_t row, int c) const {
    const int64_t at = row * p.out.n + c;
    const uint16_t x = p.x_out ? p.x_out[at]
                               : x64<T>(p.h[at], p.x[at], p.gamma_post + c, gate_row ? gate_row + c : nullptr,
                                        post.inv64);
    double y = __dmul_rn(__dmul_rn(static_cast<double>(Cvt<T>::f1(x)), pre.inv64),
                         static_cast<double>(Cvt<T>::f1(p.gamma[c])));
    if (p.beta) y = __dadd_rn(y, static_cast<double>(Cvt<T>::f1(p.beta[c])));
    if (p.smooth) y = __dmul_rn(y, static_cast<double>(Cvt<T>::f1(p.smooth[c])));
    return y;
  }
  __device__ __forceinline__ bool zero_row(int64_t, int, int) const { return zero && !p.beta; }
  __device__ __forceinline__ void save(double *stat) const {
    stat[0] = post.inv64;
    stat[1] = pre.inv64;
  }
  __device__ __forceinline__ void restore(int64_t row, const double *stat) {
    post.inv64 = stat[0];
    pre.inv64 = stat[1];
    find_gate(row);
  }
  // |in - in64| <= (M + 2 bmax) 4 2^-24: one rounding each of the factor, the
  // two products and the addition
  __device__ __forceinline__ float slack(float M) const {
    return __fmaf_rn(2.f, bmax, M) * 2.384185791015625e-7f;
  }
  __device__ __forceinline__ bool sure(int64_t, int, const float2[4], float) const { return true; }
  // over the scale: that, the scale's own (4, the same) and 5 for the scale's and
  // the quotient's roundings; one more for the bound's
  __device__ __forceinline__ float coarse(const Keep &, float inv) const {
    return __fmaf_rn(2.f * bmax, inv, QT == 1 ? 7.f : 127.f) * (14.f * 5.9604644775390625e-8f);
  }
};

}  // namespace arnq
