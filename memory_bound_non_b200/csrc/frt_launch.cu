#include "frt_launch.h"

namespace frt {
namespace {
// Never launched: what cluster_room asks the GPU about.
__global__ void room_kernel() {}
}  // namespace

int cluster_room(int per_sm, int ranks) {
  if (ranks == 1) return kSMs * per_sm;
  static std::atomic<int> known[3][4];  // [per_sm 1, 2, 4][ranks 1, 2, 4, 8]; asked once, of the device then current
  std::atomic<int>& slot = known[per_sm >> 1][ranks == 2 ? 1 : ranks == 4 ? 2 : 3];
  int n = slot.load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kSMs * per_sm / ranks * ranks));
  cfg.blockDim = dim3((unsigned)(512 / per_sm));
  cfg.dynamicSmemBytes = (size_t)(216 * 1024 / per_sm);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(room_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, room_kernel, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return kSMs * per_sm / ranks;
  }
  slot.store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace frt
