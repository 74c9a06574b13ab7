// arnq_host.cu -- the helpers declared in arnq_host.h.
#include "arnq_host.h"

#include <mutex>

namespace arnq {
namespace {

constexpr int kDevices = 64;
constexpr int kEntries = 256;
struct Entry {
  const void *fn;
  int dev, threads, smem, cluster;  // cluster: 0 for CTAs per SM
  int count;
};
std::mutex g_mutex;
int g_sms[kDevices];       // 0: not looked up yet
Entry g_entries[kEntries];  // a full table is written over from its start
int g_count = 0;

}  // namespace

arnq_status current_device(int *dev, int *sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return ARNQ_ERR_CUDA;
  if (*dev < 0 || *dev >= kDevices) return ARNQ_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_sms[*dev] == 0 &&
      cudaDeviceGetAttribute(&g_sms[*dev], cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
    g_sms[*dev] = 0;
    return ARNQ_ERR_CUDA;
  }
  *sms = g_sms[*dev];
  return ARNQ_OK;
}

static arnq_status resident(const void *fn, int dev, int threads, int smem, int cluster, int *count) {
  std::lock_guard<std::mutex> lock(g_mutex);
  const int have = g_count < kEntries ? g_count : kEntries;
  for (int i = 0; i < have; ++i) {
    const Entry &e = g_entries[i];
    if (e.fn == fn && e.dev == dev && e.threads == threads && e.smem == smem && e.cluster == cluster) {
      *count = e.count;
      return ARNQ_OK;
    }
  }
  if (smem > 0) {
    // the limit only ever needs to be as large as the largest request: a
    // smaller one must not lower it for launches already planned
    int limit = smem;
    for (int i = 0; i < have; ++i)
      if (g_entries[i].fn == fn && g_entries[i].dev == dev && g_entries[i].smem > limit)
        limit = g_entries[i].smem;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess)
      return ARNQ_ERR_CUDA;
  }
  int found = 0;
  if (cluster == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&found, fn, threads, smem) != cudaSuccess)
      return ARNQ_ERR_CUDA;
  } else {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(cluster * 1024, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&found, fn, &cfg) != cudaSuccess) return ARNQ_ERR_CUDA;
  }
  if (found < 1) return ARNQ_ERR_CUDA;
  g_entries[g_count % kEntries] = Entry{fn, dev, threads, smem, cluster, found};
  ++g_count;
  if (g_count >= 2 * kEntries) g_count -= kEntries;
  *count = found;
  return ARNQ_OK;
}

arnq_status resident_ctas(const void *fn, int dev, int threads, int smem, int *per_sm) {
  return resident(fn, dev, threads, smem, 0, per_sm);
}
arnq_status resident_clusters(const void *fn, int dev, int threads, int smem, int cluster, int *clusters) {
  return resident(fn, dev, threads, smem, cluster, clusters);
}

arnq_status launch_dependent(const void *fn, dim3 grid, int threads, int smem, int cluster,
                             cudaStream_t stream, void *params) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  void *args[] = {params};
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) return ARNQ_ERR_CUDA;
  return ARNQ_OK;
}

}  // namespace arnq
