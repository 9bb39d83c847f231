// Host-side helpers of the kernels that run in clusters or with a large part of an
// SM's shared memory.
#pragma once

#include <thread>

#include "frt_host.h"

namespace frt {

constexpr int kSMs = 148;
// Clusters of `ranks` CTAs (1, 2, 4 or 8) that the GPU holds at once, per_sm (1, 2
// or 4) to an SM.  A cluster lies inside one GPC and the GPCs' SMs are no
// multiple of 4 or 8: 33 of 4 and 15 of 8 where 148 SMs would hold 37 and 18.  A
// grid cut for the latter runs a second wave, twice the time.
int cluster_room(int per_sm, int ranks);

// Raises a kernel's dynamic shared memory limit on the current device to `bytes`
// (needed above the 48 KB default); `opted` keeps the largest size that each
// device has seen.  The limit is set under a lock, so that a thread with a
// smaller size never lowers it behind one with a larger.
struct SmemOptIn {
  static constexpr int kDevices = 64;
  std::atomic<int> bytes[kDevices] = {};
  std::atomic_flag busy = ATOMIC_FLAG_INIT;
};
template <typename Kern>
frt_status opt_in_smem(Kern kern, size_t bytes, SmemOptIn& opted) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= SmemOptIn::kDevices) {
    (void)cudaGetLastError();
    return FRT_ERR_CUDA;
  }
  std::atomic<int>& seen = opted.bytes[device];
  if ((int)bytes <= seen.load(std::memory_order_acquire)) return FRT_OK;
  while (opted.busy.test_and_set(std::memory_order_acquire)) std::this_thread::yield();
  frt_status st = FRT_OK;
  if ((int)bytes > seen.load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess) {
      seen.store((int)bytes, std::memory_order_release);
    } else {
      (void)cudaGetLastError();
      st = FRT_ERR_CUDA;
    }
  }
  opted.busy.clear(std::memory_order_release);
  return st;
}

}  // namespace frt
