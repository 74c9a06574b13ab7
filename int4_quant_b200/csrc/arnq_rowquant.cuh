// arnq_rowquant.cuh -- the kernel shared by the operators that compute a row
// of values and quantize it: rows are dealt out to CTAs, a row's units of
// eight elements to the CTA's threads.
//
// An operator (`Op`) supplies the row's values: in binary32 (value()), with a
// bound on their error, and any single one in fp64 (value64()).  The kernel
// finds the row maximum, the scale RN32(max|in| / Q) and the codes
// RNE(in / scale) that the fp64 values give:
//   - the binary32 maximum M is within the error bound of the true one, so
//     the true maximum is in a unit whose binary32 values come that close to
//     M: the fp64 values of those units are reduced (an integer maximum of
//     their bit patterns, the same in any order), usually one unit a row;
//   - a code is decided in binary32 unless the quotient lies within its error
//     of a half-way point; the codes of units with such a one are decided by
//     their fp64 values (code_exact).
// The fp64 work is done by warps together, eight lanes to a unit, in code kept
// out of the row's main path, which has to stay in the instruction cache (in
// line in every unit it cost 217 us instead of 150 on the norms of 8192 x 4096).
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

constexpr float kTiny = 1e-18f, kHuge = 1e37f;
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
__device__ __forceinline__ double sumsq(const float2 f[4]) {
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 q = __fmul2_rn(f[k], f[k]);
    s += static_cast<double>(q.x);
    s += static_cast<double>(q.y);
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

// Sum over the CTA (every warp takes part); one barrier, none for one warp.
__device__ __forceinline__ double block_sum(double v, double *slots, int nwarps) {
  v = warp_sum_d(v);
  if (nwarps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  if (nwarps <= 4) {
    double s = slots[0] + slots[1];
    for (int i = 2; i < nwarps; ++i) s += slots[i];
    return s;
  }
  double s = lane < nwarps ? slots[lane] : 0.0;
  for (int o = 16; o > 0; o >>= 1)
    if (o < nwarps) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return __shfl_sync(0xFFFFFFFFu, s, 0);
}
// Maximum of non-negative floats over the CTA by their bit patterns, which
// put a NaN above everything; one barrier.
__device__ __forceinline__ float block_max(float v, unsigned *slots, int nwarps) {
  const unsigned bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[threadIdx.x >> 5] = bits;
  __syncthreads();
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, lane < nwarps ? slots[lane] : 0u));
}

// IEEE division and square root, out of line: used by rare rows
static __device__ __noinline__ double div_ieee(double a, double b) { return __ddiv_rn(a, b); }
static __device__ __noinline__ double sqrt_ieee(double a) { return __dsqrt_rn(a); }

// m / Q rounded once to fp64, for Q = 127 or 7: a quotient from the rounded
// reciprocal, corrected by its exact remainder (Markstein's theorem: the
// correction rounds correctly when the reciprocal is correctly rounded).
template <int Q>
__device__ __forceinline__ double div_q(double m) {
  constexpr double r = 1.0 / Q;
  const double q = __dmul_rn(m, r);
  return __fma_rn(__fma_rn(-static_cast<double>(Q), q, m), r, q);
}

// max(|a|, |b|, |c|) in one instruction; abs_max3 ignores NaN, abs_max3_nan
// returns it
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float abs_max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float abs_max8(const float2 v[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = abs_max3(v[i].x, v[i].y, m);
  return m;
}
// |v|'s largest bit pattern, NaN counting as the largest, with `m` so far
__device__ __forceinline__ float abs_top8(const float2 v[4], float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = abs_max3_nan(v[i].x, v[i].y, m);
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

// ------------------------------------------------------------ staging

// The next row's inputs wait in shared memory, copied by each thread for
// itself (16 bytes at a time, asynchronously): slot (tensor, i) of thread tid
// holds unit tid + i*nt of that tensor.  A thread reads only what it copied,
// so its own wait is all the synchronisation there is.
__device__ __forceinline__ void copy16_async(uint4 *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// ------------------------------------------------------------ the kernel

// The fp64 values of the units flagged by the lanes of a warp: eight lanes a
// unit, four units a round.  flags: bit i for the lane's unit first + i*step;
// use(u, c, in): in = value64(row, c) of column c = 8u + lane % 8 (0 behind the
// row's end), called by every lane; u < 0 for lanes without a unit.
template <int NU, class Op, class Use>
__device__ __forceinline__ void flagged_units(const Op &op, int64_t row, unsigned flags, int first, int step,
                                              int n, const uint4 *at, Use &&use) {
  const int lane = threadIdx.x & 31, group = lane >> 3;
#pragma unroll 1
  for (int i = 0; i < NU; ++i) {
    unsigned who = __ballot_sync(0xFFFFFFFFu, (flags >> i) & 1u);
    while (who) {
      unsigned mine = who;
      for (int g = 0; g < group; ++g) mine &= mine - 1u;
      for (int g = 0; g < 4; ++g) who &= who - 1u;
      const int u = mine ? first - lane + (__ffs(mine) - 1) + i * step : -1;
      const int c = 8 * u + (lane & 7);
      use(u, c, u >= 0 && c < n ? op.value64(row, c, at) : 0.0);
    }
  }
}

// Op: struct with
//   Params, T, VEC (16-byte units), UPT (units per thread held in registers;
//   0: rows longer than that are read again in every phase), FULL (units fill
//   the threads exactly: no unit is checked, which lets a thread's units
//   overlap), QT (code type: 0 INT8, 1 INT4, kQNone), STAGED (inputs staged as above), kInputs
//   (tensors staged), Keep (what a unit keeps besides its values)
//   stage(row, u, slot, stride)     issues the copies of a unit
//   prepare(...)                    the row's statistics
//   value(row, u, keep, ..., v)     a unit's binary32 values; returns false
//                                   where they have no error bound
//   value64(row, c, at)             one value in fp64, from memory (or the
//                                   row's slots at `at`, if not null)
//   kReadsSlots                     value() reads the slots too, not prepare()
//                                   alone: the next row is staged later
//   slack(M)                        bound on |value - value64| over the row
//   coarse(keep, inv)               bound on the error of a unit's quotients
template <class Op>
__global__ void __launch_bounds__(Op::kMaxThreads, Op::kMinCtas) rowquant_kernel(const __grid_constant__ typename Op::Params p) {
  constexpr int UPT = Op::UPT, NU = UPT > 0 ? UPT : 1;
  constexpr bool VEC = Op::VEC;
  constexpr int Q = Op::QT == 1 ? 7 : 127;
  __shared__ RowSmem sm;
  extern __shared__ uint4 slots[];
  const int tid = threadIdx.x, nt = blockDim.x, nwarps = nt >> 5;
  const RowOut &out = p.out;
  const int n = out.n, units = out.units;

  // programmatic dependent launch: nothing in memory is touched before the
  // preceding work on the stream is complete
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Op op(p);
  auto each = [&](auto &&f) {
    if (UPT > 0) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = tid + i * nt;
        if (Op::FULL || u < units) f(u, i);
      }
    } else {
      for (int u = tid; u < units; u += nt) f(u, 0);
    }
  };
  // f(u, i) sets the lane's flag of a unit; then the flagged units in fp64
  // (`at`: the row's staged inputs where they are still there)
  auto each_flagged = [&](int64_t row, const uint4 *at, auto &&f, auto &&use) {
    if (UPT > 0) {
      unsigned flags = 0u;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = tid + i * nt;
        if ((Op::FULL || u < units) && f(u, i)) flags |= 1u << i;
      }
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, flags != 0u)) flagged_units<NU>(op, row, flags, tid, nt, n, at, use);
    } else {
      for (int u0 = tid & ~31; u0 < units; u0 += nt) {  // whole warps
        const int u = u0 + (tid & 31);
        const unsigned flags = u < units && f(u, 0) ? 1u : 0u;
        __syncwarp();
        flagged_units<1>(op, row, flags, u, 0, n, at, use);
      }
    }
  };
  int64_t row = blockIdx.x;
  auto stage = [&](int64_t r) {
    if (Op::STAGED) {
      if (r < out.rows)
        each([&](int u, int i) { op.stage(r, u, slots + i * nt + tid, UPT * nt); });
      copies_commit();
    }
  };
  stage(row);
  op.setup(sm, tid, nt, nwarps);
  if (tid < 2) sm.cand[tid] = 0ull;

  int parity = 0;
  for (; row < out.rows; row += gridDim.x, parity ^= 1) {
    typename Op::Keep keep[NU];
    float2 v[NU][4];
    if (Op::STAGED) copies_wait();
    op.prepare(sm, row, keep, slots + tid, nt, each, nwarps);
    if (!Op::kReadsSlots) stage(row + gridDim.x);  // prepare() has read them, behind a barrier

    if (Op::QT == kQNone) {
      uint16_t *yr = reinterpret_cast<uint16_t *>(out.y) + row * n;
      each_flagged(
          row, nullptr,
          [&](int u, int i) {
            const bool ok = op.value(row, u, keep[i], slots + i * nt + tid, UPT * nt, v[i]);
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = Cvt<typename Op::T>::pack(v[i][k].x, v[i][k].y);
            store_unit<VEC>(yr, u, n, make_uint4(w[0], w[1], w[2], w[3]));
            return !ok;
          },
          [&](int u, int c, double in) {
            if (u >= 0 && c < n) yr[c] = round16<typename Op::T>(in);
          });
      continue;
    }

    // ---- row maximum in binary32
    float top32 = 0.f;
    each([&](int u, int i) {
      if (!op.value(row, u, keep[i], slots + i * nt + tid, UPT * nt, v[i])) top32 = __int_as_float(0x7F800000);
      top32 = abs_top8(v[i], top32);
    });
    const float M = block_max(top32, sm.top, nwarps);
    const bool wide = !(M >= kTiny && M <= kHuge);  // the whole row in fp64
    if (tid == 0) sm.cand[parity ^ 1] = 0ull;       // the next row's

    // ---- fp64 maximum over the units that may hold it
    const float thr = M - 2.f * op.slack(M);
    if (__any_sync(0xFFFFFFFFu, wide || top32 >= thr)) {
      unsigned long long best = 0ull;
      each_flagged(
          row, Op::STAGED && Op::kReadsSlots ? slots : nullptr,
          [&](int u, int i) {
            if (UPT == 0) op.value(row, u, keep[i], slots, 0, v[i]);
            return wide || abs_max8(v[i]) >= thr;
          },
          [&](int, int, double in) {
            best = max(best, static_cast<unsigned long long>(__double_as_longlong(fabs(in))));
          });
      if (best) atomicMax(&sm.cand[parity], best);
    }
    __syncthreads();
    if (Op::kReadsSlots) stage(row + gridDim.x);
    const double top = __longlong_as_double(static_cast<long long>(sm.cand[parity]));
    const float sc = __double2float_rn(wide ? div_ieee(top, static_cast<double>(Q)) : div_q<Q>(top));
    if (tid == 0) out.scale[row] = sc;
    const bool finite = sc > 0.f && sc <= 3.402823466e38f;  // else every code is 0
    const float inv = __fdividef(1.f, sc);

    // ---- codes
    const int64_t code_bytes = Op::QT == 1 ? n / 2 : n;
    uint8_t *yr = out.y + row * code_bytes;
    each_flagged(
        row, nullptr,
        [&](int u, int i) {
          if (UPT == 0) op.value(row, u, keep[i], slots, 0, v[i]);
          // t = value/scale; adding kMagic rounds it to a whole number whose
          // low bits are the code; what was rounded off tells how near a
          // half-way point it was
          uint32_t q[8];
          float off = 0.f;
          const float2 inv2 = make_float2(inv, inv), mag = make_float2(kMagic, kMagic),
                       neg = make_float2(-kMagic, -kMagic), minus = make_float2(-1.f, -1.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 t = __fmul2_rn(v[i][k], inv2);
            const float2 r = __fadd2_rn(t, mag);
            const float2 d = __ffma2_rn(__fadd2_rn(r, neg), minus, t);
            off = abs_max3(d.x, d.y, off);
            q[2 * k] = __float_as_uint(r.x);
            q[2 * k + 1] = __float_as_uint(r.y);
          }
          uint32_t lo, hi;  // eight codes, column 0 lowest
          if (Op::QT == 0) {
            lo = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
            hi = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
          } else {
            const uint32_t even = __byte_perm(__byte_perm(q[0], q[2], 0x0040), __byte_perm(q[4], q[6], 0x0040), 0x5410);
            const uint32_t odd = __byte_perm(__byte_perm(q[1], q[3], 0x0040), __byte_perm(q[5], q[7], 0x0040), 0x5410);
            lo = (even & 0x0F0F0F0Fu) | ((odd << 4) & 0xF0F0F0F0u);
            hi = 0u;
          }
          if (VEC) {
            if (Op::QT == 0) reinterpret_cast<uint2 *>(yr)[u] = make_uint2(lo, hi);
            else reinterpret_cast<uint32_t *>(yr)[u] = lo;
          } else {
            const int cnt = min(8, n - 8 * u), bytes = Op::QT == 0 ? cnt : cnt / 2;
            uint8_t *to = yr + static_cast<int64_t>(u) * (Op::QT == 0 ? 8 : 4);
#pragma unroll
            for (int j = 0; j < (Op::QT == 0 ? 8 : 4); ++j)
              if (j < bytes) to[j] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
          }
          return wide || off >= 0.5f - op.coarse(keep[i], inv);
        },
        [&](int u, int c, double in) {
          int code = 0;
          if (finite && in == in)
            code = wide ? code_of_t(div_ieee(in, static_cast<double>(sc)), Q)
                        : code_exact(in, sc, __double2float_rn(in) * inv, Q);
          if (Op::QT == 0) {
            if (u >= 0 && c < n) yr[c] = static_cast<uint8_t>(code);
          } else {
            const int up = __shfl_down_sync(0xFFFFFFFFu, code, 1);
            if (u >= 0 && c < n && (c & 1) == 0) yr[c >> 1] = static_cast<uint8_t>((code & 0xF) | (up << 4));
          }
        });
  }
  // the next kernel on the stream may start its set-up (it waits for this
  // grid's completion before touching memory)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace arnq
