// Host-side argument checks shared by the prompt operators (declared in include/tre.h).
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <string>

#include "tre_internal.h"

#define TRE_EXPORT extern "C" __attribute__((visibility("default")))

namespace tre {

inline tre_status op_error(tre_status st, const char* op, const std::string& what) {
  set_error(std::string(op) + ": " + what);
  return st;
}

// A failed runtime call: its error is reported here and must not be the next call's as well.
inline tre_status op_cuda_error(const char* op, const char* what) {
  cudaGetLastError();
  return op_error(TRE_ERR_CUDA, op, what);
}

// kernel<<<grid, block, smem, stream>>>(args...) with the launch's own status: what the thread's
// earlier calls left for cudaGetLastError is not this launch's error, and stays for whom it
// concerns.
template <class... Params, class... Args>
tre_status op_launch(const char* op, void (*kernel)(Params...), dim3 grid, unsigned block,
                     size_t smem, tre_stream stream, Args... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = (cudaStream_t)stream;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, Params(args)...);
  return e == cudaSuccess ? TRE_OK : op_cuda_error(op, cudaGetErrorString(e));
}

inline bool ptr16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SMs of the current device (cached per device: the attribute query costs microseconds).
int device_sms();

// Device address of the status word that tre_ops_status reports (NULL when the module
// cannot be loaded).
int32_t* ops_status_ptr();

// Allow `kernel` its dynamic shared memory on the current device, once per device
// (`devices`: the kernel's own record of where that is done).
bool allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* devices);

}  // namespace tre

#define OP_ARG(cond, op, what) \
  if (!(cond)) return tre::op_error(TRE_ERR_INVALID_ARG, op, what)
