// Rows of activations times MXFP4 matrices, grouped by expert (declared in include/tre.h as
// tre_mxfp4_matmul).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

#include "ops_host.h"

namespace tre {
namespace {

constexpr int kWarps = 8;
constexpr int kTok = 4;  // rows of x per pass over a matrix row

// One warp per matrix row: lane l takes the groups of 8 weights l, l + 32, ... against
// kTok rows of x at a time.
template <class Out>
__global__ void __launch_bounds__(kWarps * 32)
    mxfp4_matmul_kernel(const __nv_bfloat16* __restrict__ x, int64_t x_stride,
                        const uint8_t* __restrict__ w, const int32_t* __restrict__ offsets,
                        int rows, int64_t n, int64_t k, int64_t pitch, Out* __restrict__ out,
                        int64_t out_stride) {
  const int e = blockIdx.y;
  const int lo = offsets ? min(max(offsets[e], 0), rows) : 0;
  const int hi = offsets ? min(max(offsets[e + 1], 0), rows) : rows;
  const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= n) return;
  const int lane = threadIdx.x & 31;
  const uint8_t* wr = w + ((int64_t)e * n + r) * pitch;
  for (int t0 = lo; t0 < hi; t0 += kTok) {
    float acc[kTok] = {};
    for (int64_t g = lane; g < k / 8; g += 32) {
      const uint32_t codes = *reinterpret_cast<const uint32_t*>(wr + g * 4);
      const uint32_t s = wr[k / 2 + g / 4];
      const float scale =
          __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
            (__nv_fp4x2_storage_t)(codes >> (8 * j) & 0xffu), __NV_E2M1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * j] = f.x * scale;
        v[2 * j + 1] = f.y * scale;
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        if (t0 + i >= hi) continue;
        const uint4 q = *reinterpret_cast<const uint4*>(x + (int64_t)(t0 + i) * x_stride + g * 8);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i] = fmaf(v[2 * j], __uint_as_float(u[j] << 16), acc[i]);
          acc[i] = fmaf(v[2 * j + 1], __uint_as_float(u[j] & 0xffff0000u), acc[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
#pragma unroll
      for (int sft = 16; sft; sft >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], sft);
      if (lane == 0 && t0 + i < hi) {
        if constexpr (sizeof(Out) == 4) out[(int64_t)(t0 + i) * out_stride + r] = acc[i];
        else out[(int64_t)(t0 + i) * out_stride + r] = __float2bfloat16_rn(acc[i]);
      }
    }
  }
}

}  // namespace
}  // namespace tre

using namespace tre;

TRE_EXPORT tre_status tre_mxfp4_matmul(const void* x, int64_t x_row_stride, const void* w,
                                       const int32_t* offsets, int32_t n_experts, int64_t rows,
                                       int64_t n, int64_t k, int32_t out_type, void* out,
                                       int64_t out_row_stride, tre_stream stream) {
  static const char* op = "tre_mxfp4_matmul";
  OP_ARG(out_type == TRE_BF16 || out_type == TRE_F32, op, "unknown output type");
  OP_ARG(n_experts >= 1 && n_experts <= 65535, op, "n_experts must be 1 .. 65535");
  OP_ARG(offsets || n_experts == 1, op, "several experts need offsets");
  OP_ARG(rows >= 0 && rows < ((int64_t)1 << 30), op, "rows out of range");
  OP_ARG(n >= 1 && n < ((int64_t)1 << 30) && n * n_experts < ((int64_t)1 << 31), op,
         "n out of range");
  OP_ARG(k > 0 && k % 32 == 0 && k < ((int64_t)1 << 30), op,
         "k must be a positive multiple of 32");
  if (rows == 0) return TRE_OK;
  OP_ARG(ptr16(x) && ptr16(w) && out && ((uintptr_t)out & (out_type == TRE_BF16 ? 1 : 3)) == 0,
         op, "NULL or misaligned pointer");
  OP_ARG(((uintptr_t)offsets & 3) == 0, op, "misaligned offsets");
  OP_ARG(rows == 1 || (x_row_stride % 8 == 0 && x_row_stride >= k), op,
         "x rows must not overlap and their stride be whole 16-byte units");
  OP_ARG(rows == 1 || out_row_stride >= n, op, "output rows overlap");
  const int64_t pitch = (k / 2 + k / 32 + 15) / 16 * 16;
  const dim3 grid((unsigned)((n + kWarps - 1) / kWarps), (unsigned)n_experts);
  if (out_type == TRE_BF16)
    mxfp4_matmul_kernel<<<grid, kWarps * 32, 0, (cudaStream_t)stream>>>(
        static_cast<const __nv_bfloat16*>(x), x_row_stride, static_cast<const uint8_t*>(w),
        offsets, (int)rows, n, k, pitch, static_cast<__nv_bfloat16*>(out), out_row_stride);
  else
    mxfp4_matmul_kernel<<<grid, kWarps * 32, 0, (cudaStream_t)stream>>>(
        static_cast<const __nv_bfloat16*>(x), x_row_stride, static_cast<const uint8_t*>(w),
        offsets, (int)rows, n, k, pitch, static_cast<float*>(out), out_row_stride);
  return op_launch_status(op);
}
