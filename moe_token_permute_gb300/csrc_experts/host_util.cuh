// host_util.cuh -- host helpers of the expert operators' entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>

namespace moe {
namespace experts {

constexpr int kMaxDevices = 64;

// SM count of the current device; 0 if it is not an sm_103 GPU or cannot be
// queried.
inline int supported_sm_count() {
  static std::mutex mu;
  static int sms[kMaxDevices];
  static bool ready[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!ready[dev]) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    sms[dev] = major == 10 && minor == 3 ? n : 0;
    ready[dev] = true;
  }
  return sms[dev];
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Raises a kernel's dynamic shared memory limit where it is below `bytes`; asked of
// the runtime once per device and size (a fixed table: nothing here may throw).
inline cudaError_t allow_smem(const void* kern, size_t bytes) {
  struct Limit {
    const void* kern;
    size_t bytes;
  };
  constexpr int kKernels = 32;
  static std::mutex mu;
  static Limit limits[kMaxDevices][kKernels];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> lock(mu);
  Limit* at = nullptr;
  for (int i = 0; dev < kMaxDevices && i < kKernels && at == nullptr; ++i)
    if (limits[dev][i].kern == kern || limits[dev][i].kern == nullptr) at = &limits[dev][i];
  if (at != nullptr && at->kern == kern && bytes <= at->bytes) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
  if (err == cudaSuccess && at != nullptr) *at = {kern, bytes};
  return err;
}

// Launch with programmatic stream serialization: the grid may be scheduled as
// soon as the previous grid in the stream allows it; every kernel here calls
// griddepcontrol.wait before it touches memory a previous grid may write.
// cluster: blocks of a cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), dim3 grid, dim3 cluster, unsigned block,
                            size_t smem, cudaStream_t stream, Args... args) {
  if (smem > 48 * 1024) {
    const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), smem);
    if (err != cudaSuccess) return err;
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.x;
  attr[1].val.clusterDim.y = cluster.y;
  attr[1].val.clusterDim.z = cluster.z;
  cfg.attrs = attr;
  cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem,
                   cudaStream_t stream, Args... args) {
  return launch_clusters(kern, grid, dim3(1), block, smem, stream, args...);
}

}  // namespace experts
}  // namespace moe
