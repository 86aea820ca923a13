// Residual addition with RMS norm (declared in include/tre.h as tre_add_rmsnorm).
//
// A row's sum of squares is needed before its first result, so a CTA keeps the row in registers
// between the two (8 elements a thread and group, at most 4 groups) and every byte moves once:
// the copy rate bounds it.  Measured, B200: 8192 rows of 7168, fp32 addend: 125 us, 6.6 TB/s, the
// measured copy rate; one row of 4096: 2.3 us on the device, the launch.
#include <cuda_bf16.h>

#include <algorithm>

#include "ops_host.h"

namespace tre {

namespace {

__device__ __forceinline__ float2 bf16x2_f2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t f2_bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 consecutive elements of the row: x + delta.
template <int DELTA>  // 0: none, 1: bf16, 2: fp32
__device__ __forceinline__ void load8(const float* x, const void* delta, int64_t i, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(x + i);
  const float4 b = *reinterpret_cast<const float4*>(x + i + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  if (DELTA == 1) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(delta) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = bf16x2_f2(u[j]);
      v[2 * j] += f.x;
      v[2 * j + 1] += f.y;
    }
  } else if (DELTA == 2) {
    const float* dl = static_cast<const float*>(delta) + i;
    const float4 c = *reinterpret_cast<const float4*>(dl);
    const float4 e = *reinterpret_cast<const float4*>(dl + 4);
    v[0] += c.x, v[1] += c.y, v[2] += c.z, v[3] += c.w;
    v[4] += e.x, v[5] += e.y, v[6] += e.z, v[7] += e.w;
  }
}

__device__ __forceinline__ void norm_store8(const float* v, const __nv_bfloat16* gain, float r,
                                            __nv_bfloat16* out, int64_t i) {
  const uint4 g = *reinterpret_cast<const uint4*>(gain + i);
  const uint32_t u[4] = {g.x, g.y, g.z, g.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = bf16x2_f2(u[j]);
    o[j] = f2_bf16x2(v[2 * j] * r * f.x, v[2 * j + 1] * r * f.y);
  }
  *reinterpret_cast<uint4*>(out + i) = make_uint4(o[0], o[1], o[2], o[3]);
}

// One CTA per row.  NV > 0: a thread keeps its NV groups of 8 elements in registers, so
// every byte is read and written once.  NV = 0 (rows longer than the registers hold): the
// row is read again for the second step.
template <int DELTA, int NV>
__global__ void add_rmsnorm_kernel(const float* __restrict__ x, int64_t x_stride,
                                   const void* __restrict__ delta, int64_t delta_stride,
                                   const __nv_bfloat16* __restrict__ gain, float eps, int64_t d,
                                   float* x_out, int64_t x_out_stride,
                                   __nv_bfloat16* __restrict__ out, int64_t out_stride) {
  const int64_t row = blockIdx.x;
  const float* xr = x + row * x_stride;
  const void* dr = DELTA == 1
                       ? static_cast<const void*>(static_cast<const __nv_bfloat16*>(delta) +
                                                  row * delta_stride)
                       : static_cast<const void*>(static_cast<const float*>(delta) +
                                                  row * delta_stride);
  float* xo = x_out ? x_out + row * x_out_stride : nullptr;
  __nv_bfloat16* o = out + row * out_stride;
  float v[NV > 0 ? NV : 1][8];
  float ss = 0.f;
  const int64_t step = (int64_t)blockDim.x * 8;
  auto first = [&](int64_t i, float* e) {
    load8<DELTA>(xr, dr, i, e);
    if (xo && (DELTA != 0 || xo != xr)) {
      *reinterpret_cast<float4*>(xo + i) = make_float4(e[0], e[1], e[2], e[3]);
      *reinterpret_cast<float4*>(xo + i + 4) = make_float4(e[4], e[5], e[6], e[7]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(e[j], e[j], ss);
  };
  if (NV > 0) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int64_t i = n * step + (int64_t)threadIdx.x * 8;
      if (i < d) first(i, v[n]);
    }
  } else {
    for (int64_t i = (int64_t)threadIdx.x * 8; i < d; i += step) first(i, v[0]);
  }
  __shared__ float part[32];
#pragma unroll
  for (int s = 16; s; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) ss += part[w];
  const float r = 1.f / sqrtf(ss / (float)d + eps);
  if (NV > 0) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int64_t i = n * step + (int64_t)threadIdx.x * 8;
      if (i < d) norm_store8(v[n], gain, r, o, i);
    }
  } else {
    for (int64_t i = (int64_t)threadIdx.x * 8; i < d; i += step) {
      // in place, x already holds the sum
      if (xo) load8<0>(xo, nullptr, i, v[0]);
      else load8<DELTA>(xr, dr, i, v[0]);
      norm_store8(v[0], gain, r, o, i);
    }
  }
}

}  // namespace
}  // namespace tre

using namespace tre;

TRE_EXPORT tre_status tre_add_rmsnorm(const float* x, int64_t x_row_stride, const void* delta,
                                      int32_t delta_type, int64_t delta_row_stride,
                                      const void* gain, float eps, int64_t rows, int64_t d,
                                      float* x_out, int64_t x_out_row_stride, void* out,
                                      int64_t out_row_stride, tre_stream stream) {
  static const char* op = "tre_add_rmsnorm";
  OP_ARG(rows >= 0 && rows <= 0x7fffffff && d > 0 && d <= 0x7fffffff && d % 8 == 0, op,
         "rows must fit 31 bits and d be a positive multiple of 8");
  OP_ARG(eps >= 0.f && eps < 3e38f, op, "eps must be finite and not negative");
  OP_ARG(!delta || delta_type == TRE_BF16 || delta_type == TRE_F32, op, "unknown delta type");
  if (rows == 0) return TRE_OK;
  OP_ARG(ptr16(x) && ptr16(gain) && ptr16(out) && (!delta || ptr16(delta)) &&
             (!x_out || ptr16(x_out)),
         op, "NULL or misaligned pointer");
  OP_ARG(rows == 1 || (x_row_stride % 4 == 0 && out_row_stride % 8 == 0 &&
                       (!x_out || x_out_row_stride % 4 == 0) &&
                       (!delta || delta_row_stride % (delta_type == TRE_BF16 ? 8 : 4) == 0)),
         op, "row strides must be whole 16-byte units");
  OP_ARG(rows == 1 || (x_row_stride >= d || x_row_stride == 0) , op, "x rows overlap");
  OP_ARG(rows == 1 || (out_row_stride >= d && (!x_out || x_out_row_stride >= d)), op,
         "output rows overlap");
  OP_ARG(x_out != x || x_out_row_stride == x_row_stride || rows == 1, op,
         "x_out in place needs x's row stride");
  const int64_t groups = d / 8;
  int threads, nv;
  if (groups <= 4 * 1024) {
    nv = groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4;
    // Two groups a thread where there are many long rows: 1100 rows of 7168 18.5 us against 20.5
    // with one, of 8192 20.9 against 22.6 (8192 rows 123.0 against 121.2 and 140.0 against 137.3);
    // 1024 rows of 512 take 4.2 us with one and 9.6 with two, 64 rows of 7168 5.2 and 5.8.
    if (rows > 1024 && groups >= 512) nv = std::max<int>(nv, 2);
    threads = (int)std::max<int64_t>(32, ((groups + nv - 1) / nv + 31) / 32 * 32);
  } else {
    nv = 0;
    threads = 1024;
  }
  const int kind = !delta ? 0 : delta_type == TRE_BF16 ? 1 : 2;
#define KERNELS(N) {add_rmsnorm_kernel<0, N>, add_rmsnorm_kernel<1, N>, add_rmsnorm_kernel<2, N>}
  static constexpr decltype(&add_rmsnorm_kernel<0, 0>) kernels[][3] = {KERNELS(0), KERNELS(1),
                                                                       KERNELS(2), KERNELS(4)};
#undef KERNELS
  return op_launch(op, kernels[nv == 4 ? 3 : nv][kind], dim3((unsigned)rows), threads, 0, stream, x,
                   x_row_stride, delta, delta_row_stride, static_cast<const __nv_bfloat16*>(gain),
                   eps, d, x_out, x_out_row_stride, static_cast<__nv_bfloat16*>(out),
                   out_row_stride);
}
