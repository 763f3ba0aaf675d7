// lm_host.cuh -- host pieces that the entry points of a token model's operators share (lm_*.cu): errors,
// the device's limits, launches.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "vocoder.h"

#define VOC_API extern "C" __attribute__((visibility("default")))

namespace voc {
namespace lm {

constexpr int kMaxDevices = 64;

struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int sms = 0;
  int *timeout = nullptr;
  int clusters[9] = {};  // clusters of 1..8 CTAs of the split-K product that run at once
};

// Sets the thread's error without a context (vocoder_last_error(NULL)) and hands back the status.
voc_status fail(voc_status st, const char *msg) noexcept;
voc_status cuda_fail(cudaError_t e, const char *what) noexcept;

// The current device, set up on first use (shared-memory limits of the kernels, SM count).
voc_status device(Device **out);

// With VOC_FLAG_SYNC: wait for the stream and report a kernel that gave up a wait.
voc_status finish(const Device &dev, voc_stream_t stream, unsigned flags);

template <typename K>
void allow_smem(cudaError_t &e, K kernel, size_t bytes) {
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
}

// Launch with programmatic stream serialization (see pdl_wait), in clusters of `cluster` CTAs
// along z where that is above 1.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                   voc_stream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = cluster;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool known_flags(unsigned f) { return (f & ~static_cast<unsigned>(VOC_FLAG_SYNC)) == 0; }

}  // namespace lm
}  // namespace voc
