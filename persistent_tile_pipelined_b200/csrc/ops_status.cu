// The operators' device status word (declared in include/tre.h as tre_ops_status).
#include "ops_host.h"

namespace tre {

// One word per device: the module's copy on the current one.
__device__ int32_t g_ops_status;

int32_t* ops_status_ptr() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_ops_status) == cudaSuccess ? static_cast<int32_t*>(p)
                                                               : nullptr;
}

int device_sms() {
  static int sms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!sms[dev]) cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
  return sms[dev] > 0 ? sms[dev] : 148;
}

}  // namespace tre

using namespace tre;

TRE_EXPORT tre_status tre_ops_status(int32_t* device_status) {
  static const char* op = "tre_ops_status";
  OP_ARG(device_status, op, "NULL argument");
  int32_t v = 0;
  const int32_t zero = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_ops_status, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_ops_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return op_error(TRE_ERR_CUDA, op, cudaGetErrorString(e));
  *device_status = v;
  return TRE_OK;
}
