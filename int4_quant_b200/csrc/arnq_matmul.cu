// arnq_matmul.cu -- arnq_quant_matmul: argument checks, tensor maps, the
// choice between the kernels, launch.
#include "arnq_matmul.cuh"

#include <cstring>

#include "arnq_host.h"

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

constexpr int kSmemLimit = 227 * 1024;
constexpr int kStatic = 2048;  // the kernels' static shared memory, rounded up

arnq_status launch_split(MatmulParams &p, bool plain, int sms, int dev, cudaStream_t stream) {
  const int64_t token_tiles = div_up(p.m, 256);
  p.tokens = static_cast<int32_t>(div_up(div_up(p.m, token_tiles), 16) * 16);
  const int64_t tiles = div_up(p.n, 128);
  const int chunks = static_cast<int>(div_up(p.k, kTileK));
  // CTAs for every SM: K shared out while that leaves SMs idle, two chunks each at least
  int split = 1;
  while (split < 8 && tiles * token_tiles * split * 2 <= sms && chunks >= 4 * split) split *= 2;
  p.split = split;
  p.channel_tiles = static_cast<int32_t>(tiles);
  if (tiles * token_tiles * split > INT32_MAX) return ARNQ_ERR_SHAPE;
  const int stage = 16384 + p.tokens * 128;
  int stages = (kSmemLimit - kStatic - 1024) / stage;
  if (stages > kSplitMaxStages) stages = kSplitMaxStages;
  p.stages = stages;
  int smem = stages * stage;
  if (smem < p.tokens * 512) smem = p.tokens * 512;  // the partial sums lie over the stages
  smem += 1024;
  p.tmem_cols = 32;
  while (p.tmem_cols < static_cast<uint32_t>(p.tokens)) p.tmem_cols *= 2;
  if (!plain && !(encode(&p.map_w, p.w, p.n, p.k, 128) && encode(&p.map_x, p.x, p.m, p.k, p.tokens)))
    return ARNQ_ERR_CUDA;
  const void *fn = plain ? reinterpret_cast<const void *>(matmul_split_kernel<true>)
                         : reinterpret_cast<const void *>(matmul_split_kernel<false>);
  int per_sm = 0;
  const arnq_status st = resident_ctas(fn, dev, kSplitThreads, smem, &per_sm);
  if (st != ARNQ_OK) return st;
  return launch_dependent(fn, dim3(static_cast<unsigned>(tiles * token_tiles * split)), kSplitThreads,
                          smem, split, stream, &p);
}

arnq_status launch_pair(MatmulParams &p, int dev, cudaStream_t stream) {
  p.token_tiles = static_cast<int32_t>(div_up(p.m, 256));
  p.channel_tiles = static_cast<int32_t>(div_up(p.n, 256));
  const int esz = p.out == ARNQ_FP32 ? 4 : 2;
  p.tma_out = p.n * esz % 16 == 0 && is_aligned(p.y, 16) ? 1 : 0;
  if (!encode(&p.map_w, p.w, p.n, p.k, 128) || !encode(&p.map_x, p.x, p.m, p.k, 128) ||
      (p.tma_out && !encode_out(&p.map_y, p.y, p.m, p.n, p.out)))
    return ARNQ_ERR_CUDA;
  const void *fn = reinterpret_cast<const void *>(matmul_pair_kernel);
  int pairs = 0;
  const arnq_status st = resident_clusters(fn, dev, kPairThreads, kPairSmem, 2, &pairs);
  if (st != ARNQ_OK) return st;
  const int64_t tiles = static_cast<int64_t>(p.token_tiles) * p.channel_tiles;
  if (tiles < pairs) pairs = static_cast<int>(tiles);
  return launch_dependent(fn, dim3(2 * pairs), kPairThreads, kPairSmem, 2, stream, &p);
}

}  // namespace

extern "C" arnq_status arnq_quant_matmul(const void *x, const float *scale_x, const void *w,
                                         const float *scale_w, const void *bias, int64_t m, int64_t n,
                                         int64_t k, arnq_dtype out_dt, void *y, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  if (out_dt != ARNQ_BF16 && out_dt != ARNQ_FP16 && out_dt != ARNQ_FP32) return ARNQ_ERR_DTYPE;
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > ARNQ_MAX_N || k > ARNQ_MAX_K) return ARNQ_ERR_SHAPE;
  if (m == 0 || n == 0 || k == 0) return ARNQ_ERR_EMPTY;
  if (!x || !scale_x || !w || !scale_w || !y) return ARNQ_ERR_NULL_PTR;
  const uintptr_t esz = out_dt == ARNQ_FP32 ? 4 : 2;
  if (!is_aligned(scale_x, 4) || !is_aligned(scale_w, 4) || !is_aligned(y, esz) || !is_aligned(bias, esz))
    return ARNQ_ERR_ALIGN;
  if (!workspace || workspace_bytes < static_cast<size_t>(kStatusBytes)) return ARNQ_ERR_WORKSPACE;
  if (!is_aligned(workspace, 8)) return ARNQ_ERR_ALIGN;
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
  p.wait_limit_ns = kWaitLimitNs;
  const bool plain = k % 16 != 0 || !is_aligned(x, 16) || !is_aligned(w, 16);
  if (!plain && m > 512) return launch_pair(p, dev, static_cast<cudaStream_t>(stream));
  return launch_split(p, plain, sms, dev, static_cast<cudaStream_t>(stream));
}
