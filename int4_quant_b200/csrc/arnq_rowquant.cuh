// arnq_rowquant.cuh -- the kernel shared by the operators that compute a row
// of values and quantize it: rows are dealt out to CTAs, a row's units of
// eight elements to the CTA's threads.
//
// An operator (`Op`) supplies the row's values: in binary32 (value()), with a
// bound on their error, and any single one in fp64 (value64()).  The kernel
// finds the row maximum, the scale RN32(max|in| / Q) and the codes
// RNE(in / scale) that the fp64 values give:
//   - the binary32 maximum M is within the error bound of the true one, so
//     the true maximum is among the elements whose binary32 value comes that
//     close to M: their fp64 values are reduced (an integer maximum of their
//     bit patterns, the same in any order), usually one element a row;
//   - a code is decided in binary32 unless the quotient lies within its error
//     of a half-way point; then by the fp64 value (code_exact).
// Rows whose maximum is below kTiny, above kHuge or not finite are computed
// in fp64 throughout.  A row holding a NaN gets scale NaN, one holding an
// infinity scale infinity (NaN if both), both with codes 0; an all-zero row
// gets scale 0 and codes 0.
//
// Memory-bound: each input is read once (the next row's loads are issued
// before the current row's arithmetic) and each output written once.
// No tensor cores: nothing here is a contraction.
#pragma once

#include "arnq_kernels.cuh"

namespace arnq {

constexpr float kTiny = 1e-25f, kHuge = 1e37f;
constexpr int kQNone = 2;  // no codes: the values themselves in 16 bits

// ------------------------------------------------------------ units of eight

__device__ __forceinline__ uint32_t word_of(const uint4 &w, int i) {
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}
__device__ __forceinline__ uint16_t get16(const uint4 &w, int j) {
  return static_cast<uint16_t>(word_of(w, j >> 1) >> ((j & 1) * 16));
}
__device__ __forceinline__ void set16(uint4 &w, int j, uint16_t v) {
  const uint32_t sh = (j & 1) * 16, keep = ~(0xFFFFu << sh), put = static_cast<uint32_t>(v) << sh;
  if ((j >> 1) == 0) w.x = (w.x & keep) | put;
  if ((j >> 1) == 1) w.y = (w.y & keep) | put;
  if ((j >> 1) == 2) w.z = (w.z & keep) | put;
  if ((j >> 1) == 3) w.w = (w.w & keep) | put;
}

// Elements 8u .. 8u+7 of a row of n starting at `row`; zeros past its end.
// VEC: the row is 16-byte aligned and n a multiple of 8.
template <bool VEC, bool STREAM>
__device__ __forceinline__ uint4 load_unit(const uint16_t *row, int u, int n) {
  if (VEC) return STREAM ? ld_stream16(row + 8 * static_cast<int64_t>(u))
                         : *reinterpret_cast<const uint4 *>(row + 8 * static_cast<int64_t>(u));
  uint32_t w[4];
  const int c = 8 * u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = c + 2 * i < n ? row[c + 2 * i] : 0u;
    const uint32_t hi = c + 2 * i + 1 < n ? row[c + 2 * i + 1] : 0u;
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool VEC>
__device__ __forceinline__ void store_unit(uint16_t *row, int u, int n, const uint4 &w) {
  if (VEC) {
    *reinterpret_cast<uint4 *>(row + 8 * static_cast<int64_t>(u)) = w;
    return;
  }
  const int c = 8 * u;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < n) row[c + j] = get16(w, j);
}

template <class T>
__device__ __forceinline__ void unpack(const uint4 &w, float2 f[4]) {
  f[0] = Cvt<T>::f2(w.x);
  f[1] = Cvt<T>::f2(w.y);
  f[2] = Cvt<T>::f2(w.z);
  f[3] = Cvt<T>::f2(w.w);
}

// fp64 -> 16 bits in one rounding: to binary32 rounded to odd (the truncated
// value's last bit set when inexact), which keeps on which side of a 16-bit
// half-way point the value lies, then to nearest even.
template <class T>
__device__ __forceinline__ uint16_t round16(double v) {
  const float z = __double2float_rz(v);
  const uint32_t odd = static_cast<double>(z) == v || v != v ? 0u : 1u;
  return static_cast<uint16_t>(Cvt<T>::pack(__uint_as_float(__float_as_uint(z) | odd), 0.f));
}

// Sum of squares of a unit in fp64.  Each square is exact in binary32 (but for
// overflow and underflow), which is cheaper than squaring in fp64; adding
// them in binary32, even four at a time, was seen to move a rounding of x'.
template <class T>
__device__ __forceinline__ double sumsq(const uint4 &w) {
  float2 f[4];
  unpack<T>(w, f);
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 q = __fmul2_rn(f[k], f[k]);
    s += static_cast<double>(q.x);
    s += static_cast<double>(q.y);
  }
  return s;
}
template <class T>
__device__ __forceinline__ double sumsq64(const uint4 &w) {
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double v = static_cast<double>(Cvt<T>::f1(get16(w, j)));
    s = __fma_rn(v, v, s);
  }
  return s;
}

// ------------------------------------------------------------ block reductions

// Slots of one kind of reduction.  Two reductions of the same kind are always
// separated by a barrier of another kind.
struct RowSmem {
  double sum[3][32];
  unsigned top[32];
  unsigned long long cand[2];  // fp64 maxima of a row, by row parity
};

// Sum over the CTA (every warp takes part); one barrier.
__device__ __forceinline__ double block_sum(double v, double *slots, int nwarps) {
  v = warp_sum_d(v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  double s = lane < nwarps ? slots[lane] : 0.0;
  for (int o = 16; o > 0; o >>= 1)
    if (o < nwarps) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return __shfl_sync(0xFFFFFFFFu, s, 0);
}
// Maximum of non-negative floats over the CTA by their bit patterns, which
// put a NaN above everything; one barrier.
__device__ __forceinline__ float block_max(unsigned bits, unsigned *slots, int nwarps) {
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = bits;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, lane < nwarps ? slots[lane] : 0u));
}

// m / Q rounded once to fp64, for Q = 127 or 7: a quotient from the rounded
// reciprocal, corrected by its exact remainder (Markstein's theorem: the
// correction rounds correctly when the reciprocal is correctly rounded).
template <int Q>
__device__ __forceinline__ double div_q(double m) {
  constexpr double r = 1.0 / Q;
  const double q = __dmul_rn(m, r);
  return __fma_rn(__fma_rn(-static_cast<double>(Q), q, m), r, q);
}

__device__ __forceinline__ float abs_max8(const float2 v[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
  return m;
}
// the largest bit pattern of |v|: NaN counts as the largest
__device__ __forceinline__ unsigned abs_bits8(const float2 v[4]) {
  unsigned m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, __float_as_uint(v[i].x) & 0x7FFFFFFFu);
    m = max(m, __float_as_uint(v[i].y) & 0x7FFFFFFFu);
  }
  return m;
}
__device__ __forceinline__ float elem(const float2 v[4], int j) {
  return j & 1 ? v[j >> 1].y : v[j >> 1].x;
}

// Output side of a launch, common to the operators.
struct RowOut {
  uint8_t *y;
  float *scale;
  int64_t rows;
  int32_t n;
  int32_t units;  // ceil(n / 8)
};

// ------------------------------------------------------------ the kernel

// Op: struct with
//   Params, T, VEC, UPT (units per thread held in registers; 0: rows longer
//   than that are read again in every phase), QT (ARNQ code type 0 INT8,
//   1 INT4, kQNone)
//   Raw, fetch(row, u) -> Raw       a unit's inputs
//   begin(row), prepare(...)        the row's statistics
//   value(raw, u, v)                a unit's binary32 values
//   value64(raw, u, j)              one value in fp64
//   slack(M)                        bound on |value - value64| over the row
//   tolerance(raw, j, t, inv)       bound on the error of the quotient t
template <class Op>
__global__ void __launch_bounds__(Op::kMaxThreads, Op::kMinCtas) rowquant_kernel(typename Op::Params p) {
  constexpr int UPT = Op::UPT, NU = UPT > 0 ? UPT : 1;
  constexpr bool VEC = Op::VEC;
  constexpr int Q = Op::QT == 1 ? 7 : 127;
  __shared__ RowSmem sm;
  const int tid = threadIdx.x, nt = blockDim.x, nwarps = nt >> 5;
  const RowOut &out = p.out;
  const int n = out.n, units = out.units;

  // programmatic dependent launch: nothing in memory is touched before the
  // preceding work on the stream is complete
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Op op(p);
  op.setup(sm, tid, nt, nwarps);
  if (tid < 2) sm.cand[tid] = 0ull;

  typename Op::Raw raw[NU], next[NU];
  auto each = [&](auto &&f) {
    if (UPT > 0) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = tid + i * nt;
        if (u < units) f(u, i);
      }
    } else {
      for (int u = tid; u < units; u += nt) f(u, 0);
    }
  };
  int64_t row = blockIdx.x;
  if (UPT > 0 && row < out.rows) each([&](int u, int i) { next[i] = op.fetch(row, u); });

  int parity = 0;
  for (; row < out.rows; row += gridDim.x, parity ^= 1) {
    if (UPT > 0) {
#pragma unroll
      for (int i = 0; i < NU; ++i) raw[i] = next[i];
      const int64_t nr = row + gridDim.x;
      if (nr < out.rows) each([&](int u, int i) { next[i] = op.fetch(nr, u); });
    }
    op.prepare(sm, row, raw, each, nwarps);
    float2 v[NU][4];
    auto take = [&](int u, int i) {  // long rows: a unit's values, made again
      if (UPT == 0) {
        raw[0] = op.refetch(row, u);
        op.value(raw[0], u, v[0]);
      }
    };

    if (Op::QT == kQNone) {
      uint16_t *yr = reinterpret_cast<uint16_t *>(out.y) + row * n;
      each([&](int u, int i) {
        if (UPT > 0) op.value(raw[i], u, v[i]);
        take(u, i);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = Cvt<typename Op::T>::pack(v[i][k].x, v[i][k].y);
        store_unit<VEC>(yr, u, n, make_uint4(w[0], w[1], w[2], w[3]));
      });
      continue;
    }

    // ---- row maximum in binary32
    unsigned bits = 0u;
    each([&](int u, int i) {
      if (UPT > 0) op.value(raw[i], u, v[i]);
      take(u, i);
      bits = max(bits, abs_bits8(v[i]));
    });
    const float M = block_max(bits, sm.top, nwarps);
    const bool wide = !(M >= kTiny && M <= kHuge);  // the whole row in fp64
    if (tid == 0) sm.cand[parity ^ 1] = 0ull;       // the next row's

    // ---- fp64 maximum over the elements that may hold it
    const float thr = M - 2.f * op.slack(M);
    each([&](int u, int i) {
      if (UPT == 0) take(u, i);
      if (!wide && abs_max8(v[i]) < thr) return;
      const int cnt = min(8, n - 8 * u);
      for (int j = 0; j < cnt; ++j) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) a = j == k ? fabsf(elem(v[i], k)) : a;
        if (!wide && a < thr) continue;
        atomicMax(&sm.cand[parity], static_cast<unsigned long long>(
                                        __double_as_longlong(fabs(op.value64(raw[i], u, j)))));
      }
    });
    __syncthreads();
    const double top = __longlong_as_double(static_cast<long long>(sm.cand[parity]));
    const double dq = wide ? __ddiv_rn(top, static_cast<double>(Q)) : div_q<Q>(top);
    const float sc = __double2float_rn(dq);
    if (tid == 0) out.scale[row] = sc;
    const bool finite = sc > 0.f && sc <= 3.402823466e38f;  // else every code is 0
    const float inv = __frcp_rn(sc);

    // ---- codes
    const int64_t code_bytes = Op::QT == 1 ? n / 2 : n;
    uint8_t *yr = out.y + row * code_bytes;
    each([&](int u, int i) {
      if (UPT == 0) take(u, i);
      uint32_t q[8];
      unsigned near = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = elem(v[i], j) * inv;
        const float r = t + kMagic;
        q[j] = __float_as_uint(r);
        const float d = t - (r - kMagic);
        if (fabsf(fabsf(d) - 0.5f) <= op.tolerance(raw[i], j, t, inv)) near |= 1u << j;
      }
      if (wide) near = finite ? 0xFFu : 0u;
      const int cnt = min(8, n - 8 * u);
      if (!VEC) near &= (1u << cnt) - 1u;
      // bytes (INT8) or nibbles (INT4) of the eight codes, column 0 lowest
      uint64_t w = 0;
      if (Op::QT == 0) {
        const uint32_t lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
        const uint32_t hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
        w = static_cast<uint64_t>(hi) << 32 | lo;
      } else {
        uint32_t x = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) x |= (q[j] & 0xFu) << (4 * j);
        w = x;
      }
      if (wide) w = 0;
      while (near) {
        const int j = __ffs(near) - 1;
        near &= near - 1u;
        const double in = op.value64(raw[i], u, j);
        int code;
        if (wide) code = in == in ? code_of(in, sc, Q) : 0;
        else code = code_exact(in, sc, __double2float_rn(in) * inv, Q);
        const int width = Op::QT == 1 ? 4 : 8;
        const uint64_t mask = ((1ull << width) - 1ull) << (width * j);
        w = (w & ~mask) | ((static_cast<uint64_t>(static_cast<uint32_t>(code)) << (width * j)) & mask);
      }
      if (VEC) {
        if (Op::QT == 0) reinterpret_cast<uint2 *>(yr)[u] = make_uint2(static_cast<uint32_t>(w), static_cast<uint32_t>(w >> 32));
        else reinterpret_cast<uint32_t *>(yr)[u] = static_cast<uint32_t>(w);
      } else if (Op::QT == 0) {
        for (int j = 0; j < cnt; ++j) yr[8 * u + j] = static_cast<uint8_t>(w >> (8 * j));
      } else {
        for (int j = 0; j < cnt / 2; ++j) yr[4 * u + j] = static_cast<uint8_t>(w >> (8 * j));
      }
    });
  }
  // the next kernel on the stream may start its set-up (it waits for this
  // grid's completion before touching memory)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace arnq
