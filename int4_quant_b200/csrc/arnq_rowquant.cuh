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
// Neither holds a row up: its codes are written with the binary32 scale, whose
// distance from the exact one the bound covers, and the units left to decide
// are listed in a record.  After sixteen rows, or its last, the CTA settles its
// records, eight lanes a row for the exact scales, then eight lanes a listed
// unit for its codes.  (Decided within each row, out of line, they cost latency that
// every warp of the row waits for: the gated activation of 4096 x 16384 went from 114
// to 78 us when the records came.  In line in every unit the loop left the
// instruction cache: norms of 8192 x 4096 217 us, 127 out of line.  Both at earlier
// steps; now 82 and 77 us.)
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

// A unit is eight elements of a row, held as eight 16-bit halves.  Which ones:
//   WIDE   8u + j: one 16-byte access (n a multiple of 8, everything aligned)
//   TAIL   the same for threads that hold more units than the row has: those
//          behind its end are masked where they are loaded and stored
//   PAIRS  element pairs 64 apart, the warp's lanes side by side: four 4-byte
//          (or eight 2-byte) accesses of whole runs (n even)
//   ONES   elements 32 apart, the lanes side by side (n odd)
enum : int { WIDE = 0, PAIRS = 1, ONES = 2, TAIL = 3 };
constexpr bool is_wide(int mode) { return mode == WIDE || mode == TAIL; }
template <int MODE>
__device__ __forceinline__ int column(int u, int j) {
  if (is_wide(MODE)) return 8 * u + j;
  const int base = (u >> 5) * 256, lane = u & 31;
  return MODE == PAIRS ? base + (j >> 1) * 64 + 2 * lane + (j & 1) : base + j * 32 + lane;
}
__host__ __device__ inline int units_of(int mode, int n) {
  return is_wide(mode) ? n / 8 : (n + 255) / 256 * 32;
}

// Unit u of a row of n; zeros past the row's end.
template <int MODE>
__device__ __forceinline__ uint4 load_unit(const uint16_t *row, int u, int n) {
  if (MODE == TAIL && 8 * u >= n) return make_uint4(0u, 0u, 0u, 0u);
  if (is_wide(MODE)) return *reinterpret_cast<const uint4 *>(row + 8 * static_cast<int64_t>(u));
  const int c = column<MODE>(u, 0);
  const uint16_t *p = row + c;
  uint32_t r[4];
  if ((u >> 5) * 256 + 256 <= n) {  // (the warp's 256 elements all exist)
    const bool words = MODE == PAIRS && (reinterpret_cast<uintptr_t>(row) & 3) == 0;
    if (words) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const uint32_t *>(p + 64 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = p[64 * i] | static_cast<uint32_t>(p[64 * i + (MODE == PAIRS ? 1 : 32)]) << 16;
    }
  } else if (MODE == PAIRS) {
    const bool words = (reinterpret_cast<uintptr_t>(row) & 3) == 0;  // the same for the whole tensor
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = 0u;
      if (c + 64 * i < n)
        r[i] = words ? *reinterpret_cast<const uint32_t *>(p + 64 * i)
                     : p[64 * i] | static_cast<uint32_t>(p[64 * i + 1]) << 16;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = c + 64 * i < n ? p[64 * i] : 0u, hi = c + 64 * i + 32 < n ? p[64 * i + 32] : 0u;
      r[i] = lo | hi << 16;
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int MODE>
__device__ __forceinline__ void store_unit(uint16_t *row, int u, int n, const uint4 &w) {
  if (is_wide(MODE)) {
    if (MODE == TAIL && 8 * u >= n) return;
    *reinterpret_cast<uint4 *>(row + 8 * static_cast<int64_t>(u)) = w;
    return;
  }
  const int c = column<MODE>(u, 0);
  uint16_t *p = row + c;
  if (MODE == PAIRS && (reinterpret_cast<uintptr_t>(row) & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 64 * i < n) *reinterpret_cast<uint32_t *>(p + 64 * i) = word_of(w, i);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = column<MODE>(u, j) - c;
    if (c + d < n) p[d] = get16(w, j);
  }
}

// Eight codes (bytes, or nibbles in lo) of unit u of the code row.
template <int MODE, int QT>
__device__ __forceinline__ void store_codes(uint8_t *row, int u, int n, uint32_t lo, uint32_t hi) {
  if (is_wide(MODE)) {
    if (MODE == TAIL && 8 * u >= n) return;
    if (QT == 0) reinterpret_cast<uint2 *>(row)[u] = make_uint2(lo, hi);
    else reinterpret_cast<uint32_t *>(row)[u] = lo;
    return;
  }
  if (QT == 1) {  // (PAIRS) a byte a pair
    const int c = column<MODE>(u, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 64 * i < n) row[(c + 64 * i) >> 1] = static_cast<uint8_t>(lo >> (8 * i));
    return;
  }
  const int c = column<MODE>(u, 0);
  if (MODE == PAIRS && (reinterpret_cast<uintptr_t>(row) & 1) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 64 * i < n)
        *reinterpret_cast<uint16_t *>(row + c + 64 * i) = static_cast<uint16_t>((i < 2 ? lo : hi) >> (16 * (i & 1)));
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = column<MODE>(u, j) - c;
    if (c + d < n) row[c + d] = static_cast<uint8_t>((j < 4 ? lo : hi) >> (8 * (j & 3)));
  }
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

// Sum of squares of a unit in fp64 (two chains).  Adding the squares in
// binary32, even four at a time, was seen to move a rounding of x'.
__device__ __forceinline__ double sumsq(const float2 f[4]) {
  double s = 0.0, t = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const double a = static_cast<double>(f[k].x), b = static_cast<double>(f[k].y);
    s = __fma_rn(a, a, s);
    t = __fma_rn(b, b, t);
  }
  return s + t;
}

// ------------------------------------------------------------ block reductions

// What a row leaves to decide in fp64.
constexpr int kRecords = 16;
constexpr int kListCap = 48;  // units with codes near a half-way point
constexpr int kMaxCap = 12;   // units that may hold the maximum
struct RowRecord {
  double stat[2];  // what the operator needs for the row's fp64 values
  int64_t row;
  float scale;
  int32_t units, tops;        // listed so far (beyond a list's room: the whole row is redone)
  uint16_t unit[kListCap], top[kMaxCap];
};

// Slots of one kind of reduction.  Two reductions of the same kind are always
// separated by a barrier of another kind.
struct RowSmem {
  double sum[3][32];
  unsigned top[2][32];       // by row parity
  unsigned long long cand;   // fp64 maximum of a row that is in fp64 throughout
  RowRecord rec[kRecords];
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
  int32_t units;  // of a row
};

// ------------------------------------------------------------ staging

// The next row's inputs wait in shared memory, copied by each thread for
// itself (16 bytes at a time, asynchronously): slot (tensor, i) of thread tid
// holds unit tid + i*nt of that tensor.  A thread reads only what it copied,
// so its own wait is all the synchronisation there is.
// there: false for a unit behind the row's end (zeros; the address is not read)
__device__ __forceinline__ void copy16_async(uint4 *dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_async(uint4 *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// ------------------------------------------------------------ the kernel

__device__ __forceinline__ float rcp_approx(float y) {
  float e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  return e;
}

// Column c's code into row yr (nothing for c >= n), by eight lanes, of which an
// even one and the next have neighbouring columns (INT4); all eight call it.
template <int QT>
__device__ __forceinline__ void put_code(uint8_t *yr, int c, int n, int code) {
  if (QT == 0) {
    if (c < n) yr[c] = static_cast<uint8_t>(code);
  } else {
    const int up = __shfl_down_sync(0xFFu << (threadIdx.x & 24), code, 1, 8);
    if (c < n && (c & 1) == 0) yr[c >> 1] = static_cast<uint8_t>((code & 0xF) | (up << 4));
  }
}

// Settles `count` records: eight lanes a row find its scale, then the units
// listed in all of them are decided, eight lanes a unit.
template <class Op>
__device__ __forceinline__ void settle_rows(Op &op, RowRecord *recs, int count, const RowOut &out) {
  constexpr int Q = Op::QT == 1 ? 7 : 127;
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3, groups = blockDim.x >> 3, n = out.n;
  const unsigned mask = 0xFFu << (threadIdx.x & 24);
  __syncthreads();  // the rows' codes, x' and records are written
#pragma unroll 1
  for (int r = group; r < count; r += groups) {
    RowRecord &rec = recs[r];
    op.restore(rec.row, rec.stat);
    const bool all = rec.tops > kMaxCap;
    const int tops = all ? (n + 7) / 8 : rec.tops;
    double top = 0.0;
#pragma unroll 1
    for (int i = 0; i < tops; ++i) {
      const int c = all ? 8 * i + lane : column<Op::MODE>(rec.top[i], lane);
      if (c < n) top = fmax(top, fabs(op.value64(rec.row, c)));
    }
    top = group_max_d(top, mask, 8);
    if (lane == 0) {
      rec.scale = __double2float_rn(div_q<Q>(top));
      out.scale[rec.row] = rec.scale;
    }
  }
  __syncthreads();
  int r = 0, before = 0;  // the record that holds item i, and the items of those before it
#pragma unroll 1
  for (int i = group;; i += groups) {
    int here = 0;
    for (; r < count; ++r) {
      here = recs[r].units > kListCap ? (n + 7) / 8 : recs[r].units;
      if (i < before + here) break;
      before += here;
    }
    if (r >= count) break;
    const RowRecord &rec = recs[r];
    op.restore(rec.row, rec.stat);
    const int c = rec.units > kListCap ? 8 * (i - before) + lane : column<Op::MODE>(rec.unit[i - before], lane);
    const float sc = rec.scale;
    const double in = c < n ? op.value64(rec.row, c) : 0.0;
    __syncwarp(mask);
    put_code<Op::QT>(out.y + rec.row * (Op::QT == 1 ? n / 2 : n), c, n,
                     code_exact(in, sc, __double2float_rn(in) * rcp_approx(sc), Q));
  }
  __syncthreads();
  if (threadIdx.x < count) recs[threadIdx.x].units = recs[threadIdx.x].tops = 0;
}

// Op: struct with
//   Params, T, MODE (the units' shape), UPT (units per thread held in registers,
//   exactly: units behind the row's end are masked, not branched around, so
//   that a thread's units overlap; 0: rows longer than that are read again in
//   every phase), QT (code type: 0 INT8, 1 INT4, kQNone), STAGED (inputs
//   staged as above), kInputs (tensors staged), Keep (what a unit keeps
//   besides its values)
//   stage(row, u, slot, stride)     issues the copies of a unit
//   prepare(..., next)              the row's statistics; calls next() when the
//                                   thread's slots have been read, unless
//                                   kReadsSlots
//   value(row, u, keep, ..., v)     a unit's binary32 values, all of a row times the
//                                   same constant (codes do not depend on it);
//                                   returns false where they have no error bound
//   kLeast                          kTiny times that constant
//   value64(row, c)                 one value in fp64, from memory
//   kReadsSlots                     value() reads the slots, not prepare()
//   zero_row(row, tid, nt)          whether this thread's part of the row's
//                                   inputs is zero, and so the row's values
//   slack(M)                        bound on value()'s error over the row
//   sure(row, u, v, thr)            whether the values >= thr of a unit are as
//                                   near their fp64 values as coarse() takes the
//                                   row's maximum to be; else the whole row is
//                                   decided in fp64
//   coarse(keep, inv)               bound on the error of a unit's quotients, that
//                                   of the binary32 scale included
//   save(stat), restore(row, stat)  what value64() needs of the row
template <class Op>
__global__ void __launch_bounds__(Op::kMaxThreads, Op::kMinCtas) rowquant_kernel(const __grid_constant__ typename Op::Params p) {
  constexpr int UPT = Op::UPT, NU = UPT > 0 ? UPT : 1;
  constexpr int MODE = Op::MODE;
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
        f(tid + i * nt, i);
      }
    } else {
      for (int u = tid; u < units; u += nt) f(u, 0);
    }
  };
  // use(c, value64(row, c)) for every column, by whole warps (c >= n: none)
  auto each_column64 = [&](int64_t r, auto &&use) {
#pragma unroll 1
    for (int c0 = tid & ~31; c0 < n; c0 += nt) {
      const int c = c0 + (tid & 31);
      use(c, c < n ? op.value64(r, c) : 0.0);
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
  if (tid < kRecords) sm.rec[tid].units = sm.rec[tid].tops = 0;

  int parity = 0, records = 0;
  for (; row < out.rows; row += gridDim.x, parity ^= 1) {
    typename Op::Keep keep[NU];
    float2 v[NU][4];
    if (Op::STAGED) copies_wait();
    op.prepare(sm, row, keep, slots + tid, nt, each, nwarps, [&]() { stage(row + gridDim.x); });

    if (Op::QT == kQNone) {
      uint16_t *yr = reinterpret_cast<uint16_t *>(out.y) + row * n;
      bool sure = true;
      each([&](int u, int i) {
        sure = op.value(row, u, keep[i], slots + i * nt + tid, UPT * nt, v[i]) && sure;
        sure = sure && abs_top8(v[i], 0.f) <= kHuge;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = Cvt<typename Op::T>::pack(v[i][k].x, v[i][k].y);
        store_unit<MODE>(yr, u, n, make_uint4(w[0], w[1], w[2], w[3]));
      });
      if (__syncthreads_or(!sure))
        each_column64(row, [&](int c, double in) {
          if (c < n) yr[c] = round16<typename Op::T>(in);
        });
      continue;
    }

    // ---- row maximum in binary32
    float top32 = 0.f;
    each([&](int u, int i) {
      if (!op.value(row, u, keep[i], slots + i * nt + tid, UPT * nt, v[i])) top32 = __int_as_float(0x7F800000);
      top32 = abs_top8(v[i], top32);
    });
    const float M = block_max(top32, sm.top[parity], nwarps);
    if (Op::kReadsSlots) stage(row + gridDim.x);  // value() has read them, behind the barrier
    RowRecord &rec = sm.rec[records];
    const int64_t code_bytes = Op::QT == 1 ? n / 2 : n;
    uint8_t *yr = out.y + row * code_bytes;
    const bool wide = !(M >= Op::kLeast && M <= kHuge);
    if (M == 0.f && __syncthreads_and(op.zero_row(row, tid, nt))) {
      // ---- a row of zeros (padding)
      if (tid == 0) out.scale[row] = 0.f;
      each([&](int u, int) { store_codes<MODE, Op::QT>(yr, u, n, 0u, 0u); });
      continue;
    }
    if (wide) {
      // ---- the whole row in fp64
      if (tid == 0) sm.cand = 0ull;
      __syncthreads();
      unsigned long long best = 0ull;
      each_column64(row, [&](int, double in) {
        best = max(best, static_cast<unsigned long long>(__double_as_longlong(fabs(in))));
      });
      if (best) atomicMax(&sm.cand, best);
      __syncthreads();
      const float sc = __double2float_rn(
          div_ieee(__longlong_as_double(static_cast<long long>(sm.cand)), static_cast<double>(Q)));
      const bool finite = sc > 0.f && sc <= 3.402823466e38f;  // else every code is 0
      if (tid == 0) out.scale[row] = sc;
      each_column64(row, [&](int c, double in) {
        put_code<Op::QT>(yr, c, n,
                         finite && in == in ? code_of_t(div_ieee(in, static_cast<double>(sc)), Q) : 0);
      });
      continue;
    }

    // ---- units that may hold the maximum, listed
    if (top32 >= M - 2.f * op.slack(M)) {
      each([&](int u, int i) {
        if (UPT == 0) op.value(row, u, keep[i], slots, 0, v[i]);
        if (abs_max8(v[i]) < M - 2.f * op.slack(M)) return;
        const bool sure = op.sure(row, u, v[i], M - 2.f * op.slack(M));
        const int at = atomicAdd(&rec.tops, sure ? 1 : kMaxCap + 1);
        if (at < kMaxCap) rec.top[at] = static_cast<uint16_t>(u);
        // a scale that coarse() does not cover: every code is decided in fp64
        if (!sure) atomicAdd(&rec.units, kListCap + 1);
      });
    }
    if (tid == 0) {
      op.save(rec.stat);
      rec.row = row;
    }

    // ---- codes, with the binary32 scale
    const float inv = rcp_approx(M * (1.f / Q));
    each([&](int u, int i) {
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
      store_codes<MODE, Op::QT>(yr, u, n, lo, hi);
      if (off >= 0.5f - op.coarse(keep[i], inv)) {
        const int at = atomicAdd(&rec.units, 1);
        if (at < kListCap) rec.unit[at] = static_cast<uint16_t>(u);
      }
    });
    if (++records == kRecords) {
      settle_rows(op, sm.rec, records, out);
      records = 0;
    }
  }
  if (Op::QT != kQNone) settle_rows(op, sm.rec, records, out);
  // the next kernel on the stream may start its set-up (it waits for this
  // grid's completion before touching memory)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace arnq
