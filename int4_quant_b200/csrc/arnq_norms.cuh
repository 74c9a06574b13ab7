// arnq_norms.cuh -- the norms around a block's residual, then per-row dynamic
// quantization:
//
//   p  = h / sqrt(mean(h^2) + eps_post) * gamma_post
//   x' = RN16(x + alpha * gate * p)            (written as xOut)
//   in = (x' / sqrt(mean(x'^2) + eps) * gamma + beta) * smooth
//   scale = row_max(|in|) / Q, code = round(in / scale); or RN16(in), no codes
//
// x' is decided like the codes: the binary32 sum v = x + h*G*(alpha/Rms(h)),
// G = gamma_post*gate (exact: two 16-bit values), carries an error e of at
// most |h*G*alpha/Rms| 2^-22 + |v| 2^-23 (two roundings of the factor, one of
// the fused multiply-add, with a margin of two); where v - e and v + e round
// to different 16-bit values the element is recomputed in fp64.
#pragma once

#include "arnq_rowquant.cuh"

namespace arnq {

struct NormsParams {
  RowOut out;
  const uint16_t *h, *x, *gamma_post, *gate, *gamma, *beta, *smooth;
  uint16_t *x_out;        // may be x; may be nullptr
  int32_t rows_per_gate;  // rows that share a row of gate; rows: one gate row for all
  float alpha, eps_post, eps;
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
    const double rms = __dsqrt_rn(ms);
    r.inv64 = rms == 0.0 ? 0.0 : __ddiv_rn(static_cast<double>(alpha), rms);
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

template <class T_, int QT_, bool VEC_, int UPT_>
struct NormsOp {
  typedef T_ T;
  typedef NormsParams Params;
  static constexpr int QT = QT_, UPT = UPT_;
  static constexpr bool VEC = VEC_;
  static constexpr int kMaxThreads = UPT == 4 ? 512 : 1024, kMinCtas = 1;
  struct Raw {
    uint4 h, x;  // after prepare(): x holds x'
  };
  const Params &p;
  float bmax;      // max |beta * smooth|
  double inv_n;
  const uint16_t *gate_row;
  Rms post, pre;
  __device__ __forceinline__ explicit NormsOp(const Params &q) : p(q), bmax(0.f), gate_row(nullptr) {
    inv_n = __ddiv_rn(1.0, static_cast<double>(q.out.n));
  }

  __device__ __forceinline__ void setup(RowSmem &sm, int tid, int nt, int nwarps) {
    if (!p.beta) return;
    unsigned b = 0u;
    for (int u = tid; u < p.out.units; u += nt) {
      float2 v[4];
      unpack<T>(load_unit<VEC, false>(p.beta, u, p.out.n), v);
      times(v, p.smooth, u);
      b = max(b, abs_bits8(v));
    }
    bmax = block_max(b, sm.top, nwarps);
    __syncthreads();  // the slots are used again at once
  }
  __device__ __forceinline__ void times(float2 v[4], const uint16_t *by, int u) const {
    if (!by) return;
    float2 s[4];
    unpack<T>(load_unit<VEC, false>(by, u, p.out.n), s);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(v[k], s[k]);
  }

  __device__ __forceinline__ Raw fetch(int64_t row, int u) const {
    const int64_t off = row * p.out.n;
    Raw w;
    w.h = load_unit<VEC, UPT != 0>(p.h + off, u, p.out.n);
    w.x = load_unit<VEC, UPT != 0>(p.x + off, u, p.out.n);
    return w;
  }
  // long rows: x' of a unit after the row's first phases, read back or made again
  __device__ __forceinline__ Raw refetch(int64_t row, int u) const {
    Raw w;
    if (p.x_out) {
      w.x = load_unit<VEC, false>(p.x_out + row * p.out.n, u, p.out.n);
    } else {
      w = fetch(row, u);
      w.x = make_x(row, w, u);
    }
    return w;
  }

  // x' of one element in fp64, from the inputs in memory
  __device__ __forceinline__ uint16_t x64(int64_t row, int c) const {
    const int64_t at = row * p.out.n + c;
    double t = __dmul_rn(__dmul_rn(static_cast<double>(Cvt<T>::f1(p.h[at])), post.inv64),
                         static_cast<double>(Cvt<T>::f1(p.gamma_post[c])));
    if (gate_row) t = __dmul_rn(t, static_cast<double>(Cvt<T>::f1(gate_row[c])));
    return round16<T>(__dadd_rn(static_cast<double>(Cvt<T>::f1(p.x[at])), t));
  }
  __device__ __forceinline__ uint4 make_x(int64_t row, const Raw &w, int u) const {
    float2 h[4], x[4], G[4];
    unpack<T>(w.h, h);
    unpack<T>(w.x, x);
    unpack<T>(load_unit<VEC, false>(p.gamma_post, u, p.out.n), G);
    times(G, gate_row, u);
    const float2 f = make_float2(post.inv, post.inv);
    const float fe = fabsf(post.inv) * 2.384185791015625e-7f;  // 2^-22
    // products below the normal range lose up to 2^-149 each; a cold row has
    // no binary32 bound: everything in fp64
    const float floor_e = post.cold ? __int_as_float(0x7F800000) : fabsf(post.inv) * 1.1754944e-38f;
    uint32_t lo[4], hi[4], differ = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 hg = __fmul2_rn(h[k], G[k]);
      const float2 v = __ffma2_rn(hg, f, x[k]);
      const float2 e = make_float2(
          __fmaf_rn(fabsf(hg.x), fe, __fmaf_rn(fabsf(v.x), 1.1920928955078125e-7f, floor_e)),
          __fmaf_rn(fabsf(hg.y), fe, __fmaf_rn(fabsf(v.y), 1.1920928955078125e-7f, floor_e)));
      lo[k] = Cvt<T>::pack(v.x - e.x, v.y - e.y);
      hi[k] = Cvt<T>::pack(v.x + e.x, v.y + e.y);
      differ |= lo[k] ^ hi[k];
    }
    uint4 r = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (differ) {
      const uint4 d = make_uint4(lo[0] ^ hi[0], lo[1] ^ hi[1], lo[2] ^ hi[2], lo[3] ^ hi[3]);
      const int cnt = min(8, p.out.n - 8 * u);
      for (int j = 0; j < cnt; ++j)
        if (get16(d, j)) set16(r, j, x64(row, 8 * u + j));
      if (!VEC)
        for (int j = cnt; j < 8; ++j) set16(r, j, 0);
    }
    return r;
  }

  template <class E>
  __device__ __forceinline__ void prepare(RowSmem &sm, int64_t row, Raw *raw, E &&each, int nwarps) {
    gate_row = p.gate ? p.gate + static_cast<int64_t>(static_cast<uint32_t>(row) /
                                                      static_cast<uint32_t>(p.rows_per_gate)) *
                                     p.out.n
                      : nullptr;
    // ---- Rms of h
    double ss = 0.0;
    each([&](int u, int i) {
      if (UPT == 0) raw[0].h = load_unit<VEC, false>(p.h + row * p.out.n, u, p.out.n);
      ss += sumsq<T>(raw[i].h);
    });
    ss = block_sum(ss, sm.sum[0], nwarps);
    bool cold = ss_out_of_range(ss, p.eps_post);
    if (cold) {  // the same for every thread
      ss = 0.0;
      each([&](int u, int i) {
        if (UPT == 0) raw[0].h = load_unit<VEC, false>(p.h + row * p.out.n, u, p.out.n);
        ss += sumsq64<T>(raw[i].h);
      });
      ss = block_sum(ss, sm.sum[2], nwarps);
    }
    post = make_rms(ss, inv_n, p.eps_post, p.alpha, cold);
    // ---- x' and its Rms
    ss = 0.0;
    each([&](int u, int i) {
      if (UPT == 0) raw[0] = fetch(row, u);
      raw[i].x = make_x(row, raw[i], u);
      ss += sumsq<T>(raw[i].x);
      if (p.x_out) store_unit<VEC>(p.x_out + row * p.out.n, u, p.out.n, raw[i].x);
    });
    ss = block_sum(ss, sm.sum[1], nwarps);
    cold = ss_out_of_range(ss, p.eps);
    if (cold) {
      ss = 0.0;
      each([&](int u, int i) {
        if (UPT == 0) raw[0] = refetch(row, u);
        ss += sumsq64<T>(raw[i].x);
      });
      ss = block_sum(ss, sm.sum[2], nwarps);
    }
    pre = make_rms(ss, inv_n, p.eps, 1.f, cold);
  }

  __device__ __forceinline__ void value(const Raw &w, int u, float2 v[4]) const {
    float2 x[4], G[4], B[4];
    unpack<T>(w.x, x);
    unpack<T>(load_unit<VEC, false>(p.gamma, u, p.out.n), G);
    times(G, p.smooth, u);
    const float2 r = make_float2(pre.inv, pre.inv);
    if (p.beta) {
      unpack<T>(load_unit<VEC, false>(p.beta, u, p.out.n), B);
      times(B, p.smooth, u);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __ffma2_rn(__fmul2_rn(x[k], r), G[k], B[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(__fmul2_rn(x[k], r), G[k]);
    }
    if (pre.cold) {  // no binary32 bound: a maximum that sends the row to fp64
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = 8 * u + j < p.out.n ? __double2float_rn(value64(w, u, j)) : 0.f;
        if (j & 1) v[j >> 1].y = f;
        else v[j >> 1].x = f;
      }
    }
  }
  __device__ __forceinline__ double value64(const Raw &w, int u, int j) const {
    const int c = 8 * u + j;
    double y = __dmul_rn(__dmul_rn(static_cast<double>(Cvt<T>::f1(get16(w.x, j))), pre.inv64),
                         static_cast<double>(Cvt<T>::f1(p.gamma[c])));
    if (p.beta) y = __dadd_rn(y, static_cast<double>(Cvt<T>::f1(p.beta[c])));
    if (p.smooth) y = __dmul_rn(y, static_cast<double>(Cvt<T>::f1(p.smooth[c])));
    return y;
  }
  // |in - in64| <= |x' inv G| 2^-22 + |in| 2^-24 <= (M + 2 bmax) 2^-21
  __device__ __forceinline__ float slack(float M) const {
    return __fmaf_rn(2.f, bmax, M) * 4.76837158203125e-7f;
  }
  // (Q + 2 bmax / scale) 2^-20: the same over the scale, and its reciprocal's error
  __device__ __forceinline__ float tolerance(const Raw &, int, float, float inv) const {
    return __fmaf_rn(2.f * bmax, inv, QT == 1 ? 7.f : 127.f) * 9.5367431640625e-7f;
  }
};

}  // namespace arnq
