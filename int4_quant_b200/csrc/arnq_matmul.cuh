// arnq_matmul.cuh -- product of INT8 codes with token and channel scales:
//
//   y[t, c] = RN( (sum_k x[t, k] w[c, k]) * scale_x[t] * scale_w[c] + bias[c] )
//
// x [m, k] and w [n, k] int8, the sum exact in 32-bit integers (k <= 131071
// keeps |sum| below 2^31), the rest in binary32 with one rounding to the
// output type.
#pragma once

#include <cooperative_groups.h>

#include "arnq_tc.cuh"

namespace arnq {

struct MatmulParams {
  CUtensorMap map_w, map_x;  // tensor maps of the codes (not used by the plain-load variant)
  const int8_t *x, *w;
  const float *scale_x, *scale_w;
  const void *bias;  // [n] of the output type, or nullptr
  void *y;
  int32_t *status;
  int64_t m, n, k;
  int32_t out;       // 0 bf16, 1 fp16, 2 fp32
  int32_t vec_out;   // y rows take vector stores
  int32_t tokens;    // split kernel: token rows a tile holds (a multiple of 16)
  int32_t channel_tiles;  // split kernel: tiles of 128 channels
  int32_t split;     // split kernel: CTAs (one cluster) sharing a tile's K
  int32_t stages;
  uint32_t tmem_cols;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ void report_timeout(int32_t *status) {
  status[1] = 0;
  reinterpret_cast<int64_t *>(status)[1] = -1;
  __threadfence();
  status[0] = DEV_TIMEOUT;
}

__device__ __forceinline__ float load_bias(const MatmulParams &p, int64_t c) {
  if (!p.bias) return 0.f;
  if (p.out == 2) return static_cast<const float *>(p.bias)[c];
  const uint16_t b = static_cast<const uint16_t *>(p.bias)[c];
  return p.out == 0 ? Cvt<Bf16>::f1(b) : Cvt<Fp16>::f1(b);
}
__device__ __forceinline__ uint32_t pack_out(const MatmulParams &p, float a, float b) {
  return p.out == 0 ? Cvt<Bf16>::pack(a, b) : Cvt<Fp16>::pack(a, b);
}
// four results of consecutive channels; `count` of them exist
__device__ __forceinline__ void store4(const MatmulParams &p, int64_t at, const float v[4], int count) {
  if (p.out == 2) {
    float *y = static_cast<float *>(p.y) + at;
    if (p.vec_out && count == 4) {
      *reinterpret_cast<float4 *>(y) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < count) y[j] = v[j];
    }
    return;
  }
  uint16_t *y = static_cast<uint16_t *>(p.y) + at;
  const uint32_t lo = pack_out(p, v[0], v[1]), hi = pack_out(p, v[2], v[3]);
  if (p.vec_out && count == 4) {
    *reinterpret_cast<uint2 *>(y) = make_uint2(lo, hi);
  } else {
    if (count > 0) y[0] = static_cast<uint16_t>(lo);
    if (count > 1) y[1] = static_cast<uint16_t>(lo >> 16);
    if (count > 2) y[2] = static_cast<uint16_t>(hi);
    if (count > 3) y[3] = static_cast<uint16_t>(hi >> 16);
  }
}

// ------------------------------------------------------------ plain loads

// 16 codes at `at` of the array [0, end), the first `valid` of them (0..16),
// zeros behind; no byte outside the array is read.
__device__ __forceinline__ uint4 load16_any(const int8_t *base, int64_t at, int valid, int64_t end) {
  if (valid <= 0) return make_uint4(0u, 0u, 0u, 0u);
  const uintptr_t a = reinterpret_cast<uintptr_t>(base) + static_cast<uintptr_t>(at);
  const uintptr_t first = a & ~static_cast<uintptr_t>(3);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
  const uintptr_t hi = lo + static_cast<uintptr_t>(end);
  uint32_t w[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const uintptr_t q = first + 4 * i;
    uint32_t v = 0u;
    if (q >= lo && q + 4 <= hi) {
      v = *reinterpret_cast<const uint32_t *>(q);
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (q + b >= lo && q + b < hi)
          v |= static_cast<uint32_t>(*reinterpret_cast<const uint8_t *>(q + b)) << (8 * b);
    }
    w[i] = v;
  }
  const uint32_t sh = static_cast<uint32_t>(a & 3) * 8;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = __funnelshift_r(w[i], w[i + 1], sh);
    const int keep = valid - 4 * i;  // bytes of this word that exist
    if (keep < 4) r[i] = keep <= 0 ? 0u : r[i] & ((1u << (8 * keep)) - 1u);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A tile of `rows` rows of 128 codes into swizzled shared memory, by `nt` threads.
__device__ __forceinline__ void load_tile_any(uint32_t dst, const int8_t *base, int64_t row0, int rows,
                                              int64_t all_rows, int64_t k, int64_t k0, int tid, int nt) {
  for (int i = tid; i < rows * 8; i += nt) {
    const int r = i >> 3, c = i & 7;
    const int64_t at_k = k0 + c * 16, row = row0 + r;
    const int64_t left = row < all_rows ? k - at_k : 0;
    const int valid = left >= 16 ? 16 : static_cast<int>(left);
    const uint4 v = load16_any(base, row * k + at_k, valid, all_rows * k);
    const uint32_t addr = dst + r * 128 + ((c ^ (r & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
  }
}

// ------------------------------------------------------------ few tokens

// One output tile: 128 channels (the instruction's 128 rows: TMEM lanes) by up
// to 256 tokens (TMEM columns), its K shared out over a cluster of `split`
// CTAs.  Each CTA streams its part of the weights once; the partial sums meet
// through distributed shared memory, added as integers (any order, same
// result), each CTA finishing every split-th token.
// Warps: 0 copies, 1 MMA and TMEM, 2-5 the epilogue (and, with PLAIN, the
// loads, for codes that tensor maps cannot describe: k or the pointers not
// multiples of 16).
constexpr int kSplitThreads = 192;
constexpr int kSplitMaxStages = 12;

template <bool PLAIN>
__global__ void __launch_bounds__(kSplitThreads) matmul_split_kernel(const __grid_constant__ MatmulParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ unsigned char dyn[];
  __shared__ __align__(8) uint64_t full[kSplitMaxStages], empty[kSplitMaxStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(dyn) + 1023u) & ~1023u;
  unsigned char *base_ptr = dyn + (base - smem_addr(dyn));
  const int split = p.split, rank = static_cast<int>(blockIdx.x) % split;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int64_t c0 = static_cast<int64_t>(tile % p.channel_tiles) * 128;
  const int64_t t0 = static_cast<int64_t>(tile / p.channel_tiles) * p.tokens;
  const int stages = p.stages;
  const uint32_t stage_bytes = 16384u + static_cast<uint32_t>(p.tokens) * 128u;
  const int chunks = static_cast<int>((p.k + kTileK - 1) / kTileK);
  const int k_begin = static_cast<int>(static_cast<int64_t>(chunks) * rank / split);
  const int k_end = static_cast<int>(static_cast<int64_t>(chunks) * (rank + 1) / split);

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_addr(&full[s]), PLAIN ? 128 : 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    mbar_init(smem_addr(&done), 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (!PLAIN) {
      tma_prefetch_map(&p.map_w);
      tma_prefetch_map(&p.map_x);
    }
  }
  if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_slot), p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // every wait is bounded; whoever gives up tells the others
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (abort_flag) return false;
    if (mbar_wait_bounded(smem_addr(bar), parity, p.wait_limit_ns)) return true;
    abort_flag = 1;
    return false;
  };

  if (!PLAIN && warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (int kc = k_begin; kc < k_end; ++kc, ++i) {
        const int s = i % stages;
        if (i >= stages && !wait(&empty[s], ((i / stages) & 1) ^ 1)) break;
        const uint32_t bar = smem_addr(&full[s]), at = base + s * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        tma_2d(at, &p.map_w, kc * kTileK, static_cast<int>(c0), bar);
        tma_2d(at + 16384u, &p.map_x, kc * kTileK, static_cast<int>(t0), bar);
      }
      if (abort_flag) {  // copies still in flight must land before the CTA ends
        for (int j = i > stages ? i - stages : 0; j < i; ++j)
          mbar_wait_bounded(smem_addr(&full[j % stages]), (j / stages) & 1, p.wait_limit_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = i8_instr_desc(128, p.tokens);
      int i = 0;
      for (int kc = k_begin; kc < k_end; ++kc, ++i) {
        const int s = i % stages;
        if (!wait(&full[s], (i / stages) & 1)) break;
        tc_fence_after();
        const uint64_t a = smem_desc(base + s * stage_bytes);
        const uint64_t b = smem_desc(base + s * stage_bytes + 16384u);
#pragma unroll
        for (int j = 0; j < kTileK / kMmaK; ++j)  // 32 bytes further along the swizzled rows
          mma_i8<1>(tmem, a + 2 * j, b + 2 * j, idesc, i > 0 || j > 0);
        mma_commit(smem_addr(&empty[s]));
      }
      mma_commit(smem_addr(&done));
    }
  } else if (PLAIN && warp >= 2) {
    const int lt = tid - 64;
    int i = 0;
    for (int kc = k_begin; kc < k_end; ++kc, ++i) {
      const int s = i % stages;
      if (i >= stages && !wait(&empty[s], ((i / stages) & 1) ^ 1)) break;
      const uint32_t at = base + s * stage_bytes;
      load_tile_any(at, p.w, c0, 128, p.n, p.k, static_cast<int64_t>(kc) * kTileK, lt, 128);
      load_tile_any(at + 16384u, p.x, t0, p.tokens, p.m, p.k, static_cast<int64_t>(kc) * kTileK, lt, 128);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(smem_addr(&full[s]));
    }
  }
  __syncwarp();

  // ---- partial sums to shared memory: part[t][channel], over the stages
  int32_t *part = reinterpret_cast<int32_t *>(base_ptr);
  const int count = static_cast<int>(p.m - t0 < p.tokens ? p.m - t0 : p.tokens);
  if (warp >= 2) {
    const bool ok = wait(&done, 0);
    tc_fence_after();
    const int quarter = warp & 3;
    if (ok && k_end > k_begin) {
      for (int col = 0; col < p.tokens; col += 16) {
        if (col >= count) break;
        int32_t r[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(col + j) * 128 + quarter * 32 + lane] = r[j];
      }
    } else {
      for (int t = 0; t < count; ++t) part[t * 128 + quarter * 32 + lane] = 0;
    }
    tc_fence_before();
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();  // (a single CTA is a cluster of one)
  tc_fence_after();
  if (warp == 1) tmem_release<1>(tmem, p.tmem_cols);
  const bool failed = abort_flag != 0;
  if (failed && tid == 0) report_timeout(p.status);

  // ---- sums over the cluster, scales, output: a warp a token, four channels a lane
  if (!failed) {
    const int64_t c = c0 + lane * 4;
    const int have = static_cast<int>(p.n - c < 0 ? 0 : p.n - c < 4 ? p.n - c : 4);
    float sw[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sw[j] = j < have ? p.scale_w[c + j] : 0.f;
      b[j] = j < have ? load_bias(p, c + j) : 0.f;
    }
    for (int t = rank + warp * split; t < count; t += split * (kSplitThreads / 32)) {
      int4 sum = make_int4(0, 0, 0, 0);
      for (int r = 0; r < split; ++r) {
        const int4 v = *reinterpret_cast<const int4 *>(
            cluster.map_shared_rank(part + t * 128 + lane * 4, r));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      const float sx = p.scale_x[t0 + t];
      const float v[4] = {__fmaf_rn(__int2float_rn(sum.x) * sx, sw[0], b[0]),
                          __fmaf_rn(__int2float_rn(sum.y) * sx, sw[1], b[1]),
                          __fmaf_rn(__int2float_rn(sum.z) * sx, sw[2], b[2]),
                          __fmaf_rn(__int2float_rn(sum.w) * sx, sw[3], b[3])};
      if (have > 0) store4(p, (t0 + t) * p.n + c, v, have);
    }
  }
  cluster.sync();  // nobody leaves while its partial sums are being read
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace arnq
