// arnq_glu.cu -- arnq_glu_dynamic_quant: argument checks and launch.
#include "arnq_glu.cuh"
#include "arnq_rowquant_host.h"

namespace {
using namespace arnq;

template <class T, int ACT, int QT, int MODE>
arnq_status by_upt(const GluParams &p, int upt, int threads, cudaStream_t s) {
  if (upt == 1) return launch_rows<GluOp<T, ACT, QT, MODE, 1>>(p, threads, s);
  if constexpr (is_wide(MODE))
    if (upt == 2) return launch_rows<GluOp<T, ACT, QT, MODE, 2>>(p, threads, s);
  if (upt == 4) return launch_rows<GluOp<T, ACT, QT, MODE, 4>>(p, threads, s);
  if constexpr (MODE != TAIL) return launch_rows<GluOp<T, ACT, QT, MODE, 0>>(p, threads, s);
  return ARNQ_ERR_PLAN;  // (not reached: rows read again are WIDE)
}
template <class T, int ACT, int QT>
arnq_status by_mode(const GluParams &p, int mode, int upt, int threads, cudaStream_t s) {
  if (mode == WIDE) return by_upt<T, ACT, QT, WIDE>(p, upt, threads, s);
  if (mode == TAIL) return by_upt<T, ACT, QT, TAIL>(p, upt, threads, s);
  if constexpr (QT != 1)
    if (mode == ONES) return by_upt<T, ACT, QT, ONES>(p, upt, threads, s);
  return by_upt<T, ACT, QT, PAIRS>(p, upt, threads, s);
}
template <class T, int ACT>
arnq_status by_codes(const GluParams &p, int qt, int mode, int upt, int threads, cudaStream_t s) {
  return qt == 0 ? by_mode<T, ACT, 0>(p, mode, upt, threads, s)
                 : by_mode<T, ACT, 1>(p, mode, upt, threads, s);
}
template <class T>
arnq_status by_act(const GluParams &p, int act, int qt, int mode, int upt, int threads,
                   cudaStream_t s) {
  return act == ARNQ_SILU ? by_codes<T, ACT_SILU>(p, qt, mode, upt, threads, s)
                          : by_codes<T, ACT_GELU_TANH>(p, qt, mode, upt, threads, s);
}
}  // namespace

extern "C" arnq_status arnq_glu_dynamic_quant(const void *x, const void *smooth, int64_t rows,
                                              int64_t n, arnq_dtype dt, arnq_activation act,
                                              arnq_qdtype qdt, void *y, float *scale,
                                              void *stream) {
  arnq_status st = check_rows(rows, n, dt, qdt, false);
  if (st != ARNQ_OK) return st;
  if (act != ARNQ_SILU && act != ARNQ_GELU_TANH) return ARNQ_ERR_ARG;
  if (!x || !y || !scale) return ARNQ_ERR_NULL_PTR;
  if (!is_aligned(x, 2) || !is_aligned(smooth, 2) || !is_aligned(scale, 4)) return ARNQ_ERR_ALIGN;
  if (qdt == ARNQ_INT4_INT32 && !is_aligned(y, 4)) return ARNQ_ERR_ALIGN;
  GluParams p;
  p.out.y = static_cast<uint8_t *>(y);
  p.out.scale = scale;
  p.out.rows = rows;
  p.out.n = static_cast<int32_t>(n);
  p.x = static_cast<const uint16_t *>(x);
  p.smooth = static_cast<const uint16_t *>(smooth);
  const int qt = kernel_qt(qdt);
  const bool vec = n % 8 == 0 && is_aligned(x, 16) && is_aligned(smooth, 16) &&
                   is_aligned(y, qt == 0 ? 8 : 4);
  int dev = 0, sms = 0, upt = 0, threads = 0;
  st = current_device(&dev, &sms);
  if (st != ARNQ_OK) return st;
  int mode = vec ? WIDE : n % 2 == 0 ? PAIRS : ONES;
  p.out.units = units_of(mode, p.out.n);
  row_threads(p.out.units, mode == WIDE, rows > sms, 512, &upt, &threads);
  if (upt > 0 && p.out.units != upt * threads) {  // threads hold units behind the row's end
    if (mode == WIDE) mode = TAIL;
    p.out.units = upt * threads;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dt == ARNQ_BF16 ? by_act<Bf16>(p, act, qt, mode, upt, threads, s)
                         : by_act<Fp16>(p, act, qt, mode, upt, threads, s);
}
