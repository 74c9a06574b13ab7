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
  CUtensorMap map_y;         // pair kernel: the output
  CUtensorMap map_w, map_x;  // tensor maps of the codes (not used by the plain-load variant)
  const int8_t *x, *w;
  const float *scale_x, *scale_w;
  const void *bias;  // [n] of the output type, or nullptr
  void *y;
  int32_t *status;
  int64_t m, n, k;
  int32_t out;       // 0 bf16, 1 fp16, 2 fp32
  int32_t vec_out;   // y rows take vector stores
  int32_t tma_out;   // pair kernel: the output goes through map_y
  int32_t token_tiles;    // pair kernel: tiles of 256 tokens
  int32_t tokens;    // split kernel: token rows a tile holds (a multiple of 16)
  int32_t channel_tiles;  // tiles of 128 (split kernel) or 256 (pair kernel) channels
  int32_t split;     // split kernel: CTAs (one cluster) sharing a tile's K
  int32_t stages;
  uint32_t tmem_cols;
  uint64_t wait_limit_ns;
  uint32_t test_hold;  // testing only: bytes the first stage waits for in vain
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
  if (first >= lo && first + 20 <= hi) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(first);
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = q[i];
  } else {
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

// A tile of `rows` rows of 128 codes into swizzled shared memory, by `nt`
// threads, four 16-byte pieces of each in flight.
__device__ __forceinline__ void load_tile_any(uint32_t dst, const int8_t *base, int64_t row0, int rows,
                                              int64_t all_rows, int64_t k, int64_t k0, int tid, int nt) {
  for (int i0 = tid; i0 < rows * 8; i0 += 4 * nt) {
    uint4 v[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int i = i0 + g * nt;
      const int64_t at_k = k0 + (i & 7) * 16, row = row0 + (i >> 3);
      const int64_t left = i < rows * 8 && row < all_rows ? k - at_k : 0;
      v[g] = load16_any(base, row * k + at_k, left >= 16 ? 16 : static_cast<int>(left), all_rows * k);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int i = i0 + g * nt, r = i >> 3;
      if (i >= rows * 8) break;
      const uint32_t addr = dst + r * 128 + (((i & 7) ^ (r & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[g].x), "r"(v[g].y),
                   "r"(v[g].z), "r"(v[g].w)
                   : "memory");
    }
  }
}

// ------------------------------------------------------------ few tokens

// One output tile: 128 channels (the instruction's 128 rows: TMEM lanes) by up
// to 256 tokens (TMEM columns), its K shared out over a cluster of `split`
// CTAs.  Each CTA streams its part of the weights once; the partial sums meet
// through distributed shared memory, added as integers (any order, same
// result), each CTA finishing every split-th token.
// Two waits have no limit of their own: for TMEM, which only CTAs of other
// launches could hold (see arnq_matmul_shape.h; those of other libraries, which
// must give it up without waiting for this kernel), and at the cluster's
// barriers, for CTAs whose own waits are bounded.
// Warps: 0 copies, 1 MMA and TMEM, 2-5 the epilogue.  With PLAIN, for codes
// that tensor maps cannot describe (k or the pointers not multiples of 16),
// warps 2-9 load.  (That variant gets 64 registers and spills 36 bytes.)
constexpr int kSplitThreads = 192, kPlainThreads = 320;
constexpr int kSplitMaxStages = 12;

template <bool PLAIN>
__global__ void __launch_bounds__(PLAIN ? kPlainThreads : kSplitThreads)
    matmul_split_kernel(const __grid_constant__ MatmulParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ unsigned char dyn[];
  __shared__ __align__(8) uint64_t full[kSplitMaxStages], empty[kSplitMaxStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ float sx[256];
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
      mbar_init(smem_addr(&full[s]), PLAIN ? kPlainThreads - 64 : 1);
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

  // what the epilogue needs besides the sums, fetched while they form
  const int count = static_cast<int>(p.m - t0 < p.tokens ? p.m - t0 : p.tokens);
  const int64_t c = c0 + lane * 4;
  const int have = static_cast<int>(p.n - c < 0 ? 0 : p.n - c < 4 ? p.n - c : 4);
  float sw[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sw[j] = j < have ? p.scale_w[c + j] : 0.f;
    b[j] = j < have ? load_bias(p, c + j) : 0.f;
  }
  for (int t = tid; t < count; t += blockDim.x) sx[t] = p.scale_x[t0 + t];

  // The next kernel on the stream may become resident beside this one (it waits
  // for this grid's completion before touching memory).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // every wait for copies and MMAs is bounded; whoever gives up tells the others
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (mbar_try_wait(smem_addr(bar), parity)) return true;
    if (!abort_flag && mbar_wait_bounded(smem_addr(bar), parity, p.wait_limit_ns)) return true;
    abort_flag = 1;
    return false;
  };

  int issued = 0;  // (thread 0) chunks whose copies were started
  if (!PLAIN && warp == 0) {
    if (lane == 0) {
      for (int kc = k_begin; kc < k_end; ++kc, ++issued) {
        const int i = issued, s = i % stages;
        if (i >= stages && !wait(&empty[s], ((i / stages) & 1) ^ 1)) break;
        const uint32_t bar = smem_addr(&full[s]), at = base + s * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes + (i == 0 ? p.test_hold : 0u));
        tma_2d(at, &p.map_w, kc * kTileK, static_cast<int>(c0), bar);
        tma_2d(at + 16384u, &p.map_x, kc * kTileK, static_cast<int>(t0), bar);
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
      // whoever gave up: MMAs still at work must end before TMEM is freed
      mbar_wait_bounded(smem_addr(&done), 0, p.wait_limit_ns);
    }
  } else if (PLAIN && warp >= 2) {
    const int lt = tid - 64;
    int i = 0;
    for (int kc = k_begin; kc < k_end; ++kc, ++i) {
      const int s = i % stages;
      if (i >= stages && !wait(&empty[s], ((i / stages) & 1) ^ 1)) break;
      const uint32_t at = base + s * stage_bytes;
      load_tile_any(at, p.w, c0, 128, p.n, p.k, static_cast<int64_t>(kc) * kTileK, lt,
                    kPlainThreads - 64);
      load_tile_any(at + 16384u, p.x, t0, p.tokens, p.m, p.k, static_cast<int64_t>(kc) * kTileK, lt,
                    kPlainThreads - 64);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(smem_addr(&full[s]));
    }
  }
  __syncwarp();

  // ---- partial sums to shared memory: part[t][channel], over the stages
  int32_t *part = reinterpret_cast<int32_t *>(base_ptr);
  if (warp >= 2 && warp < 6) {
    // one answer for the warp: reading TMEM takes all of its lanes
    const bool ok = __all_sync(0xFFFFFFFFu, wait(&done, 0));
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
  // TMEM is given back before the cluster's barrier: a CTA that holds some never
  // waits for another one, which may itself wait for TMEM on its SM.
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_release<1>(tmem, p.tmem_cols);
  if (abort_flag && tid == 0)  // copies still in flight must land before the CTA ends
    for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
      mbar_wait_bounded(smem_addr(&full[j % stages]), (j / stages) & 1, p.wait_limit_ns);
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();  // (a single CTA is a cluster of one)
  const bool failed = abort_flag != 0;
  if (failed && tid == 0) report_timeout(p.status);

  // ---- sums over the cluster, scales, output: a warp a token, four channels a
  // lane, four tokens at a time
  if (!failed && have > 0) {
    constexpr int kStep = (PLAIN ? kPlainThreads : kSplitThreads) / 32;
    for (int t = rank + warp * split; t < count; t += 4 * split * kStep) {
      int4 sum[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) sum[g] = make_int4(0, 0, 0, 0);
      for (int r = 0; r < split; ++r) {
        const int32_t *from = cluster.map_shared_rank(part, r) + lane * 4;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int tg = t + g * split * kStep;
          if (tg >= count) continue;
          const int4 v = *reinterpret_cast<const int4 *>(from + tg * 128);
          sum[g].x += v.x;
          sum[g].y += v.y;
          sum[g].z += v.z;
          sum[g].w += v.w;
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int tg = t + g * split * kStep;
        if (tg >= count) continue;
        const float f = sx[tg];
        const float v[4] = {__fmaf_rn(__int2float_rn(sum[g].x) * f, sw[0], b[0]),
                            __fmaf_rn(__int2float_rn(sum[g].y) * f, sw[1], b[1]),
                            __fmaf_rn(__int2float_rn(sum[g].z) * f, sw[2], b[2]),
                            __fmaf_rn(__int2float_rn(sum[g].w) * f, sw[3], b[3])};
        store4(p, (t0 + tg) * p.n + c, v, have);
      }
    }
  }
  __syncwarp();
  cluster_part();  // nobody leaves while its partial sums are being read
}

// ------------------------------------------------------------ many tokens

// Output tiles of 256 tokens x 256 channels by pairs of CTAs (cta_group::2):
// each CTA brings 128 tokens and 128 channels of a stage, one thread of the
// pair's first CTA issues the MMAs of both, and each CTA holds its 128 tokens
// (TMEM lanes) by 256 channels (columns), twice: one tile's sums are turned into
// outputs while the next one's are formed.  Persistent: pair i takes tiles i,
// i + pairs, ... in groups of eight token tiles, so that the pairs at work
// share operands in L2.
//
// What bounds it is shared memory: an MMA of 32 codes reads 4 KB of tokens and 8
// KB of channels in an SM, and its share of the stage's copies writes 8 KB,
// against 128 bytes a cycle: some 160 cycles where the tensor core needs 128.
// Measured on 8192 x 7168 x 4096: 162-165 us, 155 cycles an MMA (the tensor pipe
// 83 % active), and a thirteenth tile for eight of the 74 pairs; 186 us in the long
// run, under the power limit.  At an earlier step (172 us, 175 cycles) half of
// the MMAs left out gave 133 us, each done twice 266 us (132 cycles an MMA); a pair
// working on two tiles of tokens with the same channels (6 KB of copies an MMA)
// had no second accumulator left to overlap the epilogue with and came to 175 us.
// Warps: 0 copies, 1 MMA and TMEM, 2-5 the epilogue: a thread has a token's
// row, scales it (token scale in a register, channel scales and bias from the
// warp's shared memory), packs 128 bytes of it into the warp's swizzled buffer
// and sends 32 rows of them as one tensor-map store (or, for rows that tensor
// maps cannot describe, element by element).
constexpr int kPairThreads = 192;
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = 32768;  // 128 tokens and 128 channels
constexpr int kPairGroup = 8;
constexpr int kPairSmem = kPairStages * kPairStageBytes + 4 * 4096 + 4 * 2048 + 1024;

__global__ void __launch_bounds__(kPairThreads) matmul_pair_kernel(const __grid_constant__ MatmulParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ unsigned char dyn[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const uint32_t base = (smem_addr(dyn) + 1023u) & ~1023u;
  const int pairs = static_cast<int>(gridDim.x) >> 1;
  const int64_t tiles = static_cast<int64_t>(p.token_tiles) * p.channel_tiles;
  const int chunks = static_cast<int>((p.k + kTileK - 1) / kTileK);

  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&acc_full[i]), 1);
      mbar_init(smem_addr(&acc_empty[i]), 8);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_addr(&drained), 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&p.map_w);
    tma_prefetch_map(&p.map_x);
    if (p.tma_out) tma_prefetch_map(&p.map_y);
  }
  if (warp == 1) tmem_alloc<2>(smem_addr(&tmem_slot), 512);
  tc_fence_before();
  cluster.sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // every wait for copies, MMAs and accumulators is bounded; whoever gives up
  // tells this CTA's others (the peer's waits run out too)
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (mbar_try_wait(smem_addr(bar), parity)) return true;
    if (!abort_flag && mbar_wait_bounded(smem_addr(bar), parity, p.wait_limit_ns)) return true;
    abort_flag = 1;
    return false;
  };
  // tile i of the pair -> (token tile, channel tile)
  auto tile_at = [&](int64_t t, int64_t *t0, int64_t *c0) {
    const int64_t group = static_cast<int64_t>(kPairGroup) * p.channel_tiles;
    const int64_t first = t / group * kPairGroup, in = t % group;
    const int64_t size = p.token_tiles - first < kPairGroup ? p.token_tiles - first : kPairGroup;
    *t0 = (first + in % size) * 256;
    *c0 = in / size * 256;
  };

  // (thread 0) the next stage, its round's parity, stages filled so far; both CTAs'
  // copies complete on the first one's barrier
  int s = 0, filled = 0;
  uint32_t round = 0;
  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      const uint32_t full0 = peer_addr(smem_addr(&full[0]), 0);
      for (int64_t t = blockIdx.x >> 1; ok && t < tiles; t += pairs) {
        int64_t t0, c0;
        tile_at(t, &t0, &c0);
        const int tx = static_cast<int>(t0 + rank * 128), cw = static_cast<int>(c0 + rank * 128);
        for (int kc = 0; kc < chunks; ++kc) {
          if (filled == kPairStages && !wait(&empty[s], round ^ 1)) {
            ok = false;
            break;
          }
          if (rank == 0)
            mbar_arrive_expect_tx(smem_addr(&full[s]), 2 * kPairStageBytes + (filled == 0 ? p.test_hold : 0u));
          const uint32_t bar = full0 + 8 * s, at = base + s * kPairStageBytes;
          tma_2d_pair(at, &p.map_x, kc * kTileK, tx, bar);
          tma_2d_pair(at + 16384, &p.map_w, kc * kTileK, cw, bar);
          if (filled < kPairStages) ++filled;
          if (++s == kPairStages) {
            s = 0;
            round ^= 1;
          }
        }
      }
      // the last stages' MMAs signal both CTAs too: neither leaves before
      uint32_t r = round;
      for (int j = filled, e = s; ok && j > 0; --j) {
        if (e == 0) r ^= 1;
        e = e == 0 ? kPairStages - 1 : e - 1;
        ok = wait(&empty[e], r);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = i8_instr_desc(256, 256);
      int n_tile = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x >> 1; ok && t < tiles; t += pairs, ++n_tile) {
        const int buf = n_tile & 1;
        if (n_tile >= 2 && !wait(&acc_empty[buf], ((n_tile >> 1) & 1) ^ 1)) break;
        tc_fence_after();
        for (int kc = 0; kc < chunks; ++kc) {
          if (!wait(&full[s], round)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = smem_desc(base + s * kPairStageBytes);
          const uint64_t b = smem_desc(base + s * kPairStageBytes + 16384);
#pragma unroll
          for (int j = 0; j < kTileK / kMmaK; ++j)
            mma_i8<2>(tmem + buf * 256, a + 2 * j, b + 2 * j, idesc, kc > 0 || j > 0);
          mma_commit_pair(smem_addr(&empty[s]));
          if (++s == kPairStages) {
            s = 0;
            round ^= 1;
          }
        }
        if (ok) mma_commit_pair(smem_addr(&acc_full[buf]));
      }
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t buffers = base + kPairStages * kPairStageBytes + (warp - 2) * 4096;
    float *sw = reinterpret_cast<float *>(dyn + (base - smem_addr(dyn)) + kPairStages * kPairStageBytes +
                                          4 * 4096 + (warp - 2) * 2048);
    float *bias = sw + 256;
    const int esz = p.out == 2 ? 4 : 2, cols = 128 / esz;  // columns of 128 bytes
    int n_tile = 0;
    for (int64_t t = blockIdx.x >> 1; t < tiles; t += pairs, ++n_tile) {
      int64_t t0, c0;
      tile_at(t, &t0, &c0);
      const int buf = n_tile & 1;
      const int64_t row = t0 + rank * 128 + quarter * 32 + lane;
      __syncwarp();
      for (int j = lane; j < 256; j += 32) {
        const bool in = c0 + j < p.n;
        sw[j] = in ? p.scale_w[c0 + j] : 0.f;
        bias[j] = in ? load_bias(p, c0 + j) : 0.f;
      }
      const float sx = row < p.m ? p.scale_x[row] : 0.f;
      __syncwarp();
      const bool ok = wait(&acc_full[buf], (n_tile >> 1) & 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      for (int col = 0; col < 256; col += 32) {
        int32_t r[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * 256 + col, r);
        tmem_ld_wait();
        // this warp has read its part of the tile (said only where a later tile
        // waits for it: a signal that nobody waits for may reach a CTA that has left)
        if (col == 224 && t + 2 * pairs < tiles) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(peer_addr(smem_addr(&acc_empty[buf]), 0));
        }
        // 128 more bytes of the rows: the last store must have read the buffer
        const uint32_t at = buffers + lane * 128;
        const int chunk0 = (col % cols) * esz / 16;
        if (chunk0 == 0) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 8 columns: 16 bytes, or 32 of binary32
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            f[j] = __fmaf_rn(__int2float_rn(r[8 * q + j]) * sx, sw[col + 8 * q + j], bias[col + 8 * q + j]);
          if (p.out == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               at + (((chunk0 + 2 * q + h) ^ (lane & 7)) << 4)),
                           "r"(__float_as_uint(f[4 * h])), "r"(__float_as_uint(f[4 * h + 1])),
                           "r"(__float_as_uint(f[4 * h + 2])), "r"(__float_as_uint(f[4 * h + 3]))
                           : "memory");
          } else {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             at + (((chunk0 + q) ^ (lane & 7)) << 4)),
                         "r"(pack_out(p, f[0], f[1])), "r"(pack_out(p, f[2], f[3])),
                         "r"(pack_out(p, f[4], f[5])), "r"(pack_out(p, f[6], f[7]))
                         : "memory");
          }
        }
        if ((col + 32) % cols != 0) continue;
        // 128 bytes of 32 rows are ready
        const int64_t c = c0 + col + 32 - cols, first = row - lane;
        if (p.tma_out) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (c < p.n && first < p.m)
              tma_store_2d(&p.map_y, static_cast<int>(c), static_cast<int>(first),
                           buffers);
            bulk_commit();  // (an empty group too: the waits count groups)
          }
        } else {
          __syncwarp();
          const unsigned char *from = dyn + (buffers - smem_addr(dyn));
          for (int r2 = 0; r2 < 32 && first + r2 < p.m; ++r2)
            for (int j = lane; j < cols && c + j < p.n; j += 32) {
              const unsigned char *e = from + r2 * 128 + (((j * esz / 16) ^ (r2 & 7)) << 4) + (j * esz) % 16;
              const int64_t o = (first + r2) * p.n + c + j;
              if (esz == 4) static_cast<uint32_t *>(p.y)[o] = *reinterpret_cast<const uint32_t *>(e);
              else static_cast<uint16_t *>(p.y)[o] = *reinterpret_cast<const uint16_t *>(e);
            }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_read<0>();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (abort_flag && rank == 0) {  // whoever gave up: what is still at work must end
    if (tid == 32) {              // the MMAs, before TMEM is freed
      mma_commit_pair(smem_addr(&drained), 1);
      mbar_wait_bounded(smem_addr(&drained), 0, p.wait_limit_ns);
    }
    if (tid == 0)  // the copies, before the pair ends
      for (; filled > 0; --filled) {
        if (s == 0) round ^= 1;
        s = s == 0 ? kPairStages - 1 : s - 1;
        mbar_wait_bounded(smem_addr(&full[s]), round, p.wait_limit_ns);
      }
    __syncwarp();
  }
  // neither leaves while the other reads its memory or signals it; signals are all
  // waited for, unless a wait ran out: the barrier then orders them
  if (abort_flag) cluster_sync();
  else cluster_part();
  tc_fence_after();
  if (warp == 1) tmem_release<2>(tmem, 512);
  if (abort_flag && tid == 0) report_timeout(p.status);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace arnq
