// host_util.cuh -- what the C entry points of the attention and sampling
// operators share on the host: error texts, pointer checks, the device check
// and a launch chained to the previous work with Programmatic Dependent
// Launch.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "kernels.cuh"
#include "moe.h"

namespace wse {

inline int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int status, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error_text(buf);
  return status;
}

inline int fail_cuda(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// MOE_OK if the current device is one that the library is built for.  The
// answer is kept per device: it cannot change.
inline int check_device() {
  static thread_local int good = -1;
  int dev = 0, major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (dev == good) return MOE_OK;
  if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess)
    return fail_cuda(e, "cudaDeviceGetAttribute");
  if (major != 10 || minor != 3)
    return fail(MOE_ERR_UNSUPPORTED, "device is sm_%d%d; this library is built for sm_103a (GB300)", major, minor);
  good = dev;
  return MOE_OK;
}

// SMs of the current device, asked once per device.
inline int sm_count() {
  static thread_local int of = -1, count = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev != of && cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) of = dev;
  return count;
}

// Launches `kernel` so that its prologue may overlap the end of the previous
// kernel on the stream; the kernel waits with pdl_wait() before it touches
// global memory.  cluster > 1: thread-block clusters of that many CTAs.
template <typename... P, typename... A>
int launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, moe_stream_t stream, int cluster,
               A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  c.attrs = attr;
  c.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    c.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
  return e == cudaSuccess ? MOE_OK : fail_cuda(e, "kernel launch");
}

}  // namespace wse
