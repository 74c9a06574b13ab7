// arnq_norms.cu -- arnq_post_norm_add_rms_norm_dynamic_quant: argument checks
// and launch.
#include "arnq_norms.cuh"
#include "arnq_rowquant_host.h"

namespace {
using namespace arnq;

template <class T, int QT, int MODE>
arnq_status by_upt(const NormsParams &p, int upt, int threads, cudaStream_t s) {
  if (upt == 1) return launch_rows<NormsOp<T, QT, MODE, 1>>(p, threads, s);
  if constexpr (is_wide(MODE))
    if (upt == 2) return launch_rows<NormsOp<T, QT, MODE, 2>>(p, threads, s);
  if (upt == 4) return launch_rows<NormsOp<T, QT, MODE, 4>>(p, threads, s);
  if constexpr (MODE != TAIL) return launch_rows<NormsOp<T, QT, MODE, 0>>(p, threads, s);
  return ARNQ_ERR_PLAN;  // (not reached: rows read again are WIDE)
}
template <class T, int QT>
arnq_status by_mode(const NormsParams &p, int mode, int upt, int threads, cudaStream_t s) {
  if (mode == WIDE) return by_upt<T, QT, WIDE>(p, upt, threads, s);
  if (mode == TAIL) return by_upt<T, QT, TAIL>(p, upt, threads, s);
  if constexpr (QT != 1)
    if (mode == ONES) return by_upt<T, QT, ONES>(p, upt, threads, s);
  return by_upt<T, QT, PAIRS>(p, upt, threads, s);
}
template <class T>
arnq_status by_codes(const NormsParams &p, int qt, int mode, int upt, int threads, cudaStream_t s) {
  if (qt == 0) return by_mode<T, 0>(p, mode, upt, threads, s);
  if (qt == 1) return by_mode<T, 1>(p, mode, upt, threads, s);
  return by_mode<T, kQNone>(p, mode, upt, threads, s);
}
}  // namespace

extern "C" arnq_status arnq_post_norm_add_rms_norm_dynamic_quant(
    const void *h, const void *x, const void *gamma_post, const void *gate, int64_t gate_rows,
    float residual_scale, const void *gamma, const void *beta, const void *smooth, int64_t rows,
    int64_t n, arnq_dtype dt, float eps_post, float eps, arnq_qdtype qdt, void *y, float *scale,
    void *x_out, void *stream) {
  arnq_status st = check_rows(rows, n, dt, qdt, true);
  if (st != ARNQ_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !(eps_post >= 0.f) || !std::isfinite(eps_post))
    return ARNQ_ERR_EPS;
  if (!std::isfinite(residual_scale)) return ARNQ_ERR_ARG;
  if ((gate != nullptr) != (gate_rows != 0) || gate_rows < 0 || gate_rows > rows ||
      (gate_rows > 0 && rows % gate_rows != 0))
    return ARNQ_ERR_ARG;
  const int qt = kernel_qt(qdt);
  if (!h || !x || !gamma_post || !gamma || !y || (qt != kQNone && !scale)) return ARNQ_ERR_NULL_PTR;
  const void *t16[] = {h, x, gamma_post, gate, gamma, beta, smooth, x_out};
  bool vec = n % 8 == 0;
  for (const void *q : t16) {
    if (!is_aligned(q, 2)) return ARNQ_ERR_ALIGN;
    vec = vec && is_aligned(q, 16);
  }
  if (qt != kQNone && !is_aligned(scale, 4)) return ARNQ_ERR_ALIGN;
  if (qdt == ARNQ_INT4_INT32 && !is_aligned(y, 4)) return ARNQ_ERR_ALIGN;
  if (qt == kQNone && !is_aligned(y, 2)) return ARNQ_ERR_ALIGN;
  vec = vec && is_aligned(y, qt == 0 ? 8 : qt == 1 ? 4 : 16);
  NormsParams p;
  p.out.y = static_cast<uint8_t *>(y);
  p.out.scale = scale;
  p.out.rows = rows;
  p.out.n = static_cast<int32_t>(n);
  p.h = static_cast<const uint16_t *>(h);
  p.x = static_cast<const uint16_t *>(x);
  p.gamma_post = static_cast<const uint16_t *>(gamma_post);
  p.gate = static_cast<const uint16_t *>(gate);
  p.gamma = static_cast<const uint16_t *>(gamma);
  p.beta = static_cast<const uint16_t *>(beta);
  p.smooth = static_cast<const uint16_t *>(smooth);
  p.x_out = static_cast<uint16_t *>(x_out);
  p.rows_per_gate = static_cast<int32_t>(gate ? rows / gate_rows : 1);
  p.alpha = residual_scale;
  p.eps_post = eps_post;
  p.eps = eps;
  p.inv_n = 1.0 / static_cast<double>(n);
  int dev = 0, sms = 0, upt = 0, threads = 0;
  st = current_device(&dev, &sms);
  if (st != ARNQ_OK) return st;
  int mode = vec ? WIDE : n % 2 == 0 ? PAIRS : ONES;
  p.out.units = units_of(mode, p.out.n);
  row_threads(p.out.units, mode == WIDE, rows > sms, qt == kQNone ? 288 : 384, &upt, &threads);
  if (upt > 0 && p.out.units != upt * threads) {  // threads hold units behind the row's end
    if (mode == WIDE) mode = TAIL;
    p.out.units = upt * threads;
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dt == ARNQ_BF16 ? by_codes<Bf16>(p, qt, mode, upt, threads, s)
                         : by_codes<Fp16>(p, qt, mode, upt, threads, s);
}
