// arnq_rowquant_host.h -- launch of rowquant_kernel: which units per thread,
// how many threads and CTAs.
#pragma once

#include <cmath>

#include "arnq_host.h"
#include "arnq_rowquant.cuh"

namespace arnq {

// shape and code-type checks shared by the operators; qdt may be
// ARNQ_NO_CODES where `values` allows it
inline arnq_status check_rows(int64_t rows, int64_t n, int dt, int qdt, bool values) {
  if (dt != ARNQ_BF16 && dt != ARNQ_FP16) return ARNQ_ERR_DTYPE;
  if (qdt != ARNQ_INT8 && qdt != ARNQ_INT4 && qdt != ARNQ_INT4_INT32 &&
      !(values && qdt == ARNQ_NO_CODES))
    return ARNQ_ERR_DTYPE;
  if (rows < 0 || n < 0 || rows > INT32_MAX || n > ARNQ_MAX_N) return ARNQ_ERR_SHAPE;
  if (rows == 0 || n == 0) return ARNQ_ERR_EMPTY;
  if (qdt == ARNQ_INT4 && n % 2 != 0) return ARNQ_ERR_SHAPE;
  if (qdt == ARNQ_INT4_INT32 && n % 8 != 0) return ARNQ_ERR_SHAPE;
  return ARNQ_OK;
}

// QT of the kernels (an eight-codes-a-word INT4 row has the bytes of a packed one)
inline int kernel_qt(int qdt) {
  return qdt == ARNQ_NO_CODES ? kQNone : qdt == ARNQ_INT8 ? 0 : 1;
}

// Units of eight per thread (0: the row is read again in every phase) and
// threads for a row of `units`.  Four units a thread where rows outnumber the
// SMs and max4 such threads hold the row (a row's fixed cost, reductions and barriers, is then shared by few
// threads); with fewer rows the row's latency counts: the most threads.
inline void row_threads(int units, bool wide, bool many, int max4, int *upt, int *threads) {
  if (many && units <= 4 * max4) *upt = units <= 32 ? 1 : 4;
  else if (units <= 1024) *upt = 1;
  else if (wide && units <= 2048) *upt = 2;
  else *upt = units <= 4 * max4 ? 4 : 0;
  const int per = *upt == 0 ? 2 : *upt;
  int t = static_cast<int>(div_up(div_up(units, per), 32) * 32);
  if (t > 1024) t = 1024;
  *threads = t;
}

template <class Op>
arnq_status launch_rows(typename Op::Params p, int threads, cudaStream_t stream) {
  const void *fn = reinterpret_cast<const void *>(rowquant_kernel<Op>);
  int dev = 0, sms = 0, per_sm = 0;
  arnq_status st = current_device(&dev, &sms);
  if (st != ARNQ_OK) return st;
  const int smem = Op::STAGED ? Op::kInputs * Op::UPT * threads * 16 : 0;
  st = resident_ctas(fn, dev, threads, smem, &per_sm);
  if (st != ARNQ_OK) return st;
  const int64_t slots = static_cast<int64_t>(per_sm) * sms;
  return launch_dependent(fn, dim3(static_cast<unsigned>(p.out.rows < slots ? p.out.rows : slots)),
                          threads, smem, 1, stream, &p);
}

}  // namespace arnq
