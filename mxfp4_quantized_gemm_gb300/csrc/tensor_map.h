// What encoding a tensor map needs of the driver, shared by the kernels that
// read or write through one.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace mx {

// A driver function looked up once (thread-safe static initialisation).
template <typename Fn>
Fn driver_function(const char* name, unsigned version) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion(name, &p, version, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<Fn>(p);
  return nullptr;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const auto fn = driver_function<PFN_cuTensorMapEncodeTiled_v12000>("cuTensorMapEncodeTiled", 12000);
  return fn;
}

// Makes the current device's context current in the calling host thread where
// it has none: cuTensorMapEncodeTiled is a driver call and runs in the thread's
// current context, which the runtime binds lazily.  Allowed while a stream is
// captured, as cudaFree(nullptr) is not: that ends the capture with an error.
inline cudaError_t bind_device_context() {
  static const auto current = driver_function<PFN_cuCtxGetCurrent_v4000>("cuCtxGetCurrent", 4000);
  CUcontext ctx = nullptr;
  if (current != nullptr && current(&ctx) == CUDA_SUCCESS && ctx != nullptr) return cudaSuccess;
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  return e == cudaSuccess ? cudaSetDevice(device) : e;
}

}  // namespace mx
