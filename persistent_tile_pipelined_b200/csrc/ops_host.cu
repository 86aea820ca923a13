// What the operators share on the host: the device status word (declared in include/tre.h as
// tre_ops_status), the device's size and tensor maps.
#include "tc.cuh"
#include "tensor_map.h"

namespace tre {

// One word per device: the module's copy on the current one.
__device__ int32_t g_ops_status;

namespace {

constexpr int kDevices = 64;

// What a wait of the tensor-core operators does when it runs out of time: nothing arrives at
// `bar`, whose second half of the warps are told by the first to give up.  No copy or product is
// in flight.
__global__ void __launch_bounds__(256) timeout_kernel(long long limit, int32_t* status) {
  __shared__ uint64_t bar;
  __shared__ int gave_up;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  __syncthreads();
  tc::wait_warp(&bar, 0, &gave_up, threadIdx.x < blockDim.x / 2 ? limit : tc::kWaitClocks);
  __syncthreads();
  if (threadIdx.x == 0 && gave_up) atomicExch(status, TRE_ERR_DEP_TIMEOUT);
}

// Whether a call failed; its error must not be the next call's as well.
bool failed(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e != cudaSuccess;
}

int current_device() {
  int dev = 0;
  return !failed(cudaGetDevice(&dev)) && dev >= 0 && dev < kDevices ? dev : -1;
}

}  // namespace

int32_t* ops_status_ptr() {
  static std::atomic<int32_t*> known[kDevices];
  const int dev = current_device();
  if (dev < 0) return nullptr;
  int32_t* at = known[dev].load(std::memory_order_relaxed);
  if (!at) {
    void* p = nullptr;
    if (failed(cudaGetSymbolAddress(&p, g_ops_status))) return nullptr;
    known[dev].store(at = static_cast<int32_t*>(p), std::memory_order_relaxed);
  }
  return at;
}

int device_sms() {
  static std::atomic<int> known[kDevices];
  const int dev = current_device();
  if (dev < 0) return 148;
  int sms = known[dev].load(std::memory_order_relaxed);
  if (!sms) {
    if (failed(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev))) return 148;
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

bool allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* devices) {
  const int dev = current_device();
  if (dev < 0) return false;
  if (devices->load(std::memory_order_relaxed) >> dev & 1) return true;
  if (failed(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)))
    return false;
  devices->fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return true;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
    return reinterpret_cast<EncodeTiledFn>(
        e == cudaSuccess && q == cudaDriverEntryPointSuccess ? f : nullptr);
  }();
  return fn;
}

tre_status encode_map(const char* op, CUtensorMapDataType type, int rank, const void* base,
                      const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swizzle, CUtensorMap* out) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return op_cuda_error(op, "cuTensorMapEncodeTiled is not available");
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], one[5];
  for (int i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i], one[i] = 1;
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  const CUresult r = fn(out, type, rank, const_cast<void*>(base), d, st, b, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TRE_OK
                           : op_error(TRE_ERR_CUDA, op,
                                      "cuTensorMapEncodeTiled failed (" +
                                          std::to_string((int)r) + ")");
}

}  // namespace tre

using namespace tre;

TRE_EXPORT tre_status tre_debug_ops_timeout(int64_t clocks, tre_stream stream) {
  static const char* op = "tre_debug_ops_timeout";
  OP_ARG(clocks >= 0 && clocks <= tc::kWaitClocks, op, "clocks must be 0 .. 4e9");
  int32_t* status = ops_status_ptr();
  if (!status) return op_cuda_error(op, "the operators' status word is not available");
  return op_launch(op, timeout_kernel, dim3(1), 256, 0, stream, clocks, status);
}

TRE_EXPORT tre_status tre_ops_status(int32_t* device_status) {
  static const char* op = "tre_ops_status";
  OP_ARG(device_status, op, "NULL argument");
  int32_t v = 0;
  const int32_t zero = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_ops_status, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_ops_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return op_cuda_error(op, cudaGetErrorString(e));
  *device_status = v;
  return TRE_OK;
}
