// What kernels that follow the SM count or launch one another need.
#pragma once
#include <cuda_runtime.h>

namespace oomb {

// SMs of a device; those of a B200 where they cannot be asked for (no GPU, as when a
// workspace is sized on the host).  That is no error of the call: none is left behind
// for check_launch to find.
inline int sm_count(int device) {
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = 148;
  }
  return n;
}

// Programmatic dependent launch: lets the next kernel of the stream start, and waits in
// that kernel until the one before is complete.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace oomb
