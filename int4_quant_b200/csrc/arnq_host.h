// arnq_host.h -- host helpers shared by the operators' launch code: pointer
// alignment, the device's SM count, kernel set-up and resident CTAs per SM.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "arnq.h"

namespace arnq {

inline bool is_aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The current device and its SM count (looked up once per device).
arnq_status current_device(int *dev, int *sms);

// CTAs of `fn` resident on an SM of `dev` with `threads` threads and `smem`
// bytes of dynamic shared memory; raises the kernel's shared-memory limit
// first.  Looked up once per (fn, dev, threads, smem).
arnq_status resident_ctas(const void *fn, int dev, int threads, int smem, int *per_sm);

// Clusters of `cluster` CTAs of `fn` resident on `dev` at once.
arnq_status resident_clusters(const void *fn, int dev, int threads, int smem, int cluster, int *clusters);

// Launches as a programmatic dependent of the preceding work on the stream,
// in clusters of `cluster` CTAs.
arnq_status launch_dependent(const void *fn, dim3 grid, int threads, int smem, int cluster,
                             cudaStream_t stream, void *params);

}  // namespace arnq
