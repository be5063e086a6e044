// launch.h -- kernel launches shared by the layer-norm and feed-forward files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxn {

// Lets `kernel` take all the dynamic shared memory a block may have on the current device.  The limit is a property of
// the kernel in the whole process: it is raised once a device and never lowered, since another thread's launch, or a
// captured one, may need more than this call does.
cudaError_t allow_shared_memory(const void* kernel);

// A launch with programmatic stream serialization (the kernel may start while the previous one in the stream drains; it
// waits, griddepcontrol.wait, before it touches a tensor), of clusters of two CTAs with `pair`.  Returns 0, or a
// cudaError_t with *why naming the failed step.
int launch_kernel(const void* kernel, int64_t grid, int threads, size_t smem, void** argv, cudaStream_t stream,
                  const char* what, const char** why, bool pair = false);

}  // namespace mxn
