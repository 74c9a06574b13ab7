// arnq_matmul.cu -- arnq_quant_matmul: argument checks, tensor maps, the
// choice between the kernels, launch.
#include "arnq_matmul.cuh"

#include <cmath>
#include <cstring>

#include "arnq_host.h"
#include "arnq_matmul_shape.h"

namespace {
using namespace arnq;

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// codes [rows, k] in boxes of box_rows x 128, 128-byte swizzled
bool encode(CUtensorMap *map, const void *p, int64_t rows, int64_t k, int box_rows) {
  const EncodeFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k)};
  const cuuint32_t box[2] = {kTileK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t one[2] = {1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// output rows [m, n] in boxes of 32 rows x 128 bytes, 128-byte swizzled
bool encode_out(CUtensorMap *map, void *y, int64_t m, int64_t n, int out) {
  const EncodeFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t esz = out == ARNQ_FP32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(n) * esz};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esz), 32};
  const cuuint32_t one[2] = {1, 1};
  const CUtensorMapDataType type = out == ARNQ_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : out == ARNQ_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return f(map, type, 2, y, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kStatic = 2048;  // the kernels' static shared memory, rounded up
static_assert(kPairSmem >= kTmemColumns * kSmemPerColumn, "a pair's 512 columns leave room for no other CTA");

// ---- the choice of kernel and split, by estimated time in us
//
// Fitted to a B200 (launches back to back, weights from HBM): a CTA of the
// split kernel takes some 0.45 us a chunk of 128 codes of K alone on its SM and
// 0.7 beside another (with plain loads 0.005 us a row of the chunk), streams at
// 5.5 TB/s altogether, and has 2.5 us of fixed cost plus 0.025 us a token of the
// tile for the exchange of partial sums (0.02 without); a CTA pair 0.315 us a
// chunk and 6.5 us.  Of 48 products (the six weights below, m = 1, 16, 64, 128, 192,
// 256, 384, 512) the estimate picks the slower kernel twice: 512 x 4096 x 4096, by
// 6 %, and 256 x 8192 x 1024, by 4 %.  Measured, us, split / pair:
//   n x k          m = 1        64           128          256          512
//   1024 x 4096    5.6 / 15.6   6.6 / 15.7   8.2 / 16.0   9.7 / 15.9   13.7 / 16.1
//   4096 x 4096    6.8 / 15.9   9.6 / 15.9   13.5 / 16.2  13.2 / 16.5  18.2 / 17.1
//   5120 x 7168    11.1 / 23.8  13.6 / 23.4  17.2 / 23.7  23.8 / 24.1  35.1 / 24.6
//   16384 x 4096   15.5 / 23.9  17.7 / 19.3  19.8 / 19.5  28.2 / 20.2  52.0 / 29.0
//   4096 x 16384   16.5 / 44.1  18.9 / 43.9  23.4 / 44.1  26.1 / 44.4  38.6 / 44.5
//   8192 x 1024    4.9 / 10.3   7.4 / 9.1    7.7 / 9.3    9.8 / 9.4    11.6 / 10.4
struct SplitPlan {
  int tokens, split, stages, per_sm;
  double us;
};

double stream_us(const MatmulParams &p) {
  return static_cast<double>(p.n * p.k + p.m * p.k) / 5.5e6;
}

// CTAs resident at once in clusters of `split` (cudaOccupancyMaxActiveClusters:
// 148, 148, 132, 120 at one CTA an SM, 296, 296, 284, 264 at two)
double split_slots(int split, int per_sm, int sms) {
  const double part = split <= 2 ? 1.0 : split == 4 ? (per_sm == 1 ? 0.89 : 0.95) : (per_sm == 1 ? 0.81 : 0.89);
  return part * per_sm * sms;
}

// want: requested tile of tokens and split (0: choose)
SplitPlan plan_split(const MatmulParams &p, bool plain, int sms, int want_tokens, int want_split) {
  SplitPlan best = {};
  const int chunks = static_cast<int>(div_up(p.k, kTileK));
  const int64_t least = div_up(p.m, 256);  // token tiles; more of them spread a small product
  for (int64_t token_tiles = least; token_tiles <= 4 * least; token_tiles *= 2) {
    const int tokens = want_tokens ? want_tokens : static_cast<int>(div_up(div_up(p.m, token_tiles), 16) * 16);
    if (token_tiles > least && (tokens < 32 || want_tokens)) break;
    const int64_t tiles = div_up(p.n, 128) * div_up(p.m, tokens);
    const int stage = 16384 + tokens * 128;
    for (int split = 1; split <= 8 && (split == 1 || split == want_split || chunks >= (plain ? 1 : 2) * split);
         split *= 2) {
      if (want_split && split != want_split) continue;
      const int mine = static_cast<int>(div_up(chunks, split));
      // two CTAs an SM where at least three stages (or all there are) fit half of it
      int stages = (kSmemLimit / 2 - kStatic - 1024) / stage, per_sm = 2;
      if (stages < 3 && stages < mine) {
        stages = (kSmemLimit - kStatic - 1024) / stage;
        per_sm = 1;
      }
      if (tokens * 512 > kSmemLimit / 2 - kStatic - 1024) per_sm = 1;
      if (stages > kSplitMaxStages) stages = kSplitMaxStages;
      if (stages > mine) stages = mine;
      const int64_t ctas = tiles * split;
      const double rounds = std::ceil(static_cast<double>(ctas) / split_slots(split, per_sm, sms));
      const double beside = per_sm == 2 && ctas > sms ? 1.5 : 1.0;
      const double chunk_us = plain ? 0.005 * (128 + tokens) : 0.45;
      double us = rounds * mine * chunk_us * beside;
      if (us < stream_us(p)) us = stream_us(p);
      us += 2.5 + (split > 1 ? 0.025 : 0.02) * tokens * rounds;
      if (best.split == 0 || us < best.us) best = SplitPlan{tokens, split, stages, per_sm, us};
    }
  }
  return best;
}

double pair_us(const MatmulParams &p, int pairs) {
  const int64_t tiles = div_up(p.m, 256) * div_up(p.n, 256);
  const double us = 0.315 * static_cast<double>(div_up(p.k, kTileK)) *
                    static_cast<double>(div_up(tiles, static_cast<int64_t>(pairs)));
  return 6.5 + (us < stream_us(p) ? stream_us(p) : us);
}

arnq_status launch_split(MatmulParams &p, const SplitPlan &plan, bool plain, int dev, cudaStream_t stream) {
  const int64_t token_tiles = div_up(p.m, plan.tokens), tiles = div_up(p.n, 128);
  const int split = plan.split;
  p.tokens = plan.tokens;
  p.split = split;
  p.stages = plan.stages;
  p.channel_tiles = static_cast<int32_t>(tiles);
  if (tiles * token_tiles * split > INT32_MAX) return ARNQ_ERR_SHAPE;
  const int smem = split_smem(p.tokens, p.stages);
  p.tmem_cols = static_cast<uint32_t>(split_columns(p.tokens));
  if (!plain && !(encode(&p.map_w, p.w, p.n, p.k, 128) && encode(&p.map_x, p.x, p.m, p.k, p.tokens)))
    return ARNQ_ERR_CUDA;
  const void *fn = plain ? reinterpret_cast<const void *>(matmul_split_kernel<true>)
                         : reinterpret_cast<const void *>(matmul_split_kernel<false>);
  int per_sm = 0;
  // (raises the shared-memory limit)
  const arnq_status st = resident_ctas(fn, dev, plain ? kPlainThreads : kSplitThreads, smem, &per_sm);
  if (st != ARNQ_OK) return st;
  return launch_dependent(fn, dim3(static_cast<unsigned>(tiles * token_tiles * split)),
                          plain ? kPlainThreads : kSplitThreads, smem, split, stream, &p);
}

arnq_status launch_pair(MatmulParams &p, int pairs, cudaStream_t stream) {
  p.token_tiles = static_cast<int32_t>(div_up(p.m, 256));
  p.channel_tiles = static_cast<int32_t>(div_up(p.n, 256));
  const int esz = p.out == ARNQ_FP32 ? 4 : 2;
  p.tma_out = p.n * esz % 16 == 0 && is_aligned(p.y, 16) ? 1 : 0;
  if (!encode(&p.map_w, p.w, p.n, p.k, 128) || !encode(&p.map_x, p.x, p.m, p.k, 128) ||
      (p.tma_out && !encode_out(&p.map_y, p.y, p.m, p.n, p.out)))
    return ARNQ_ERR_CUDA;
  const int64_t tiles = static_cast<int64_t>(p.token_tiles) * p.channel_tiles;
  if (tiles < pairs) pairs = static_cast<int>(tiles);
  return launch_dependent(reinterpret_cast<const void *>(matmul_pair_kernel), dim3(2 * pairs), kPairThreads,
                          kPairSmem, 2, stream, &p);
}

}  // namespace

extern "C" arnq_status arnq_quant_matmul(const void *x, const float *scale_x, const void *w,
                                         const float *scale_w, const void *bias, int64_t m, int64_t n,
                                         int64_t k, arnq_dtype out_dt, void *y, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  arnq_matmul_plan plan;
  std::memset(&plan, 0, sizeof plan);
  return arnq_quant_matmul_planned(x, scale_x, w, scale_w, bias, m, n, k, out_dt, y, workspace,
                                   workspace_bytes, stream, &plan);
}

extern "C" arnq_status arnq_quant_matmul_planned(const void *x, const float *scale_x, const void *w,
                                                 const float *scale_w, const void *bias, int64_t m,
                                                 int64_t n, int64_t k, arnq_dtype out_dt, void *y,
                                                 void *workspace, size_t workspace_bytes, void *stream,
                                                 const arnq_matmul_plan *plan) {
  if (!plan) return ARNQ_ERR_NULL_PTR;
  if (out_dt != ARNQ_BF16 && out_dt != ARNQ_FP16 && out_dt != ARNQ_FP32) return ARNQ_ERR_DTYPE;
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > ARNQ_MAX_N || k > ARNQ_MAX_K) return ARNQ_ERR_SHAPE;
  if (m == 0 || n == 0 || k == 0) return ARNQ_ERR_EMPTY;
  if (!x || !scale_x || !w || !scale_w || !y) return ARNQ_ERR_NULL_PTR;
  const uintptr_t esz = out_dt == ARNQ_FP32 ? 4 : 2;
  if (!is_aligned(scale_x, 4) || !is_aligned(scale_w, 4) || !is_aligned(y, esz) || !is_aligned(bias, esz))
    return ARNQ_ERR_ALIGN;
  if (!workspace || workspace_bytes < static_cast<size_t>(kStatusBytes)) return ARNQ_ERR_WORKSPACE;
  if (!is_aligned(workspace, 8)) return ARNQ_ERR_ALIGN;
  const bool plain = k % 16 != 0 || !is_aligned(x, 16) || !is_aligned(w, 16);
  const arnq_matmul_plan &q = *plan;
  if (q.kernel < 0 || q.kernel > ARNQ_MATMUL_PAIR || (q.kernel == ARNQ_MATMUL_PAIR && plain) ||
      q.tokens < 0 || q.tokens > 256 || q.tokens % 16 != 0 ||
      (q.split != 0 && q.split != 1 && q.split != 2 && q.split != 4 && q.split != 8) ||
      static_cast<int64_t>(q.split) > div_up(k, kTileK) || q.wait_limit_us < 0 || q.test_hold_bytes < 0 ||
      q.test_hold_bytes > 65536 || (q.test_hold_bytes > 0 && plain))
    return ARNQ_ERR_PLAN;
  int dev = 0, sms = 0;
  arnq_status st = current_device(&dev, &sms);
  if (st != ARNQ_OK) return st;
  MatmulParams p;
  std::memset(&p, 0, sizeof p);
  p.x = static_cast<const int8_t *>(x);
  p.w = static_cast<const int8_t *>(w);
  p.scale_x = scale_x;
  p.scale_w = scale_w;
  p.bias = bias;
  p.y = y;
  p.status = static_cast<int32_t *>(workspace);
  p.m = m;
  p.n = n;
  p.k = k;
  p.out = static_cast<int32_t>(out_dt);
  p.vec_out = n % 4 == 0 && is_aligned(y, 4 * esz) ? 1 : 0;
  p.wait_limit_ns = q.wait_limit_us > 0 ? static_cast<uint64_t>(q.wait_limit_us) * 1000ull
                                        : static_cast<uint64_t>(kWaitLimitNs);
  p.test_hold = static_cast<uint32_t>(q.test_hold_bytes);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const SplitPlan split = plan_split(p, plain, sms, q.tokens, q.split);
  if (!plain && q.kernel != ARNQ_MATMUL_SPLIT) {
    int pairs = 0;
    st = resident_clusters(reinterpret_cast<const void *>(matmul_pair_kernel), dev, kPairThreads, kPairSmem, 2,
                           &pairs);
    if (st != ARNQ_OK) return st;
    if (q.kernel == ARNQ_MATMUL_PAIR || pair_us(p, pairs) < split.us) return launch_pair(p, pairs, cs);
  }
  return launch_split(p, split, plain, dev, cs);
}
