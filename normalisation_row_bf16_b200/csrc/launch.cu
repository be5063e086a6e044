// launch.cu -- see launch.h.
#include "launch.h"

#include <mutex>
#include <set>
#include <utility>

namespace mxn {

cudaError_t allow_shared_memory(const void* kernel) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (done.count({dev, kernel})) return cudaSuccess;
  int most = 0;
  cudaFuncAttributes fa;
  if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)fa.sharedSizeBytes);
  if (e == cudaSuccess) done.insert({dev, kernel});
  return e;
}

int launch_kernel(const void* kernel, int64_t grid, int threads, size_t smem, void** argv, cudaStream_t stream,
                  const char* what, const char** why, bool pair) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  cudaError_t e = smem > 48 * 1024 ? allow_shared_memory(kernel) : cudaSuccess;
  if (e == cudaSuccess) e = cudaLaunchKernelExC(&cfg, kernel, argv);
  if (e != cudaSuccess) *why = what;
  return (int)e;
}

}  // namespace mxn
