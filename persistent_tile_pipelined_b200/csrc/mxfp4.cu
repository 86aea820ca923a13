// MXFP4 rows: quantiser and its inverse (declared in include/tre.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

#include "ops_host.h"

namespace tre {

namespace {

constexpr int kRowThreads = 256;
constexpr int kGroupsPerCta = kRowThreads / 4;  // 4 lanes share a group of 32 weights

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}

// Four lanes take one group of 32 weights, 8 each: the largest magnitude by two
// exchanges, its binary exponent from the bits, then 8 codes as one word.
template <class T>
__global__ void __launch_bounds__(kRowThreads)
    mxfp4_quantize_kernel(const T* __restrict__ w, int64_t w_stride, uint32_t groups,
                          uint32_t groups_per_row, int64_t k, int64_t pitch,
                          uint8_t* __restrict__ out) {
  const uint32_t g = blockIdx.x * kGroupsPerCta + (threadIdx.x >> 2);
  const uint32_t lane4 = threadIdx.x & 3u;
  const bool live = g < groups;
  const uint32_t row = live ? g / groups_per_row : 0u, b = live ? g - row * groups_per_row : 0u;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (live) load8(w + (int64_t)row * w_stride + (int64_t)b * 32 + lane4 * 8, v);
  // magnitudes compare like their bits, and a NaN's or infinity's bits exceed every number's
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (!live) return;
  // floor(log2(max)) + 127 is the exponent field (0 for subnormals, which clamp anyway);
  // the scale's exponent is 2 less, so that the largest code's exponent (4 = 2^2) meets it
  const int field = (int)(top >> 23);
  const bool bad = field == 255;
  const int byte = bad ? 255 : max(field - 2, 0);
  uint32_t codes = 0;
  if (!bad) {
    // w / scale = w * 2^(127 - byte), exact: byte <= 252, so the factor is a normal number
    const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = make_float2(v[2 * j] * inv, v[2 * j + 1] * inv);
      codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(p, __NV_E2M1, cudaRoundNearest) << (8 * j);
    }
  }
  uint8_t* orow = out + (int64_t)row * pitch;
  *reinterpret_cast<uint32_t*>(orow + (int64_t)b * 16 + lane4 * 4) = codes;
  if (lane4 == 0) orow[k / 2 + b] = (uint8_t)byte;
  if (b + 1 == groups_per_row)
    for (int64_t i = k / 2 + groups_per_row + lane4; i < pitch; i += 4) orow[i] = 0;
}

template <class T>
__global__ void __launch_bounds__(kRowThreads)
    mxfp4_dequantize_kernel(const uint8_t* __restrict__ w, uint32_t groups,
                            uint32_t groups_per_row, int64_t k, int64_t pitch,
                            T* __restrict__ out) {
  const uint32_t g = blockIdx.x * kGroupsPerCta + (threadIdx.x >> 2);
  const uint32_t lane4 = threadIdx.x & 3u;
  if (g >= groups) return;
  const uint32_t row = g / groups_per_row, b = g - row * groups_per_row;
  const uint8_t* wr = w + (int64_t)row * pitch;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(wr + (int64_t)b * 16 + lane4 * 4);
  const uint32_t s = wr[k / 2 + b];
  const float scale =
      __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h =
        __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(codes >> (8 * j) & 0xffu), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * j] = f.x * scale;
    v[2 * j + 1] = f.y * scale;
  }
  T* o = out + (int64_t)row * k + (int64_t)b * 32 + lane4 * 8;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

int64_t pitch_of(int64_t k) { return (k / 2 + k / 32 + 15) / 16 * 16; }

// Rows per launch: a launch's groups stay below 2^31, so their index divides in 32 bits.
template <class Launch>
void in_slabs(int64_t rows, int64_t groups_per_row, Launch launch) {
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 30) / groups_per_row);
  for (int64_t r = 0; r < rows; r += most) launch(r, std::min(most, rows - r));
}

tre_status check_rows(const char* op, int32_t type, int64_t rows, int64_t k) {
  OP_ARG(type == TRE_BF16 || type == TRE_F32, op, "unknown element type");
  OP_ARG(rows >= 0 && rows <= ((int64_t)1 << 40), op, "rows out of range");
  OP_ARG(k > 0 && k % 32 == 0 && k <= ((int64_t)1 << 30), op,
         "k must be a positive multiple of 32");
  return TRE_OK;
}

}  // namespace
}  // namespace tre

using namespace tre;

TRE_EXPORT tre_status tre_mxfp4_quantize(const void* w, int32_t type, int64_t rows, int64_t k,
                                         int64_t w_row_stride, void* out, tre_stream stream) {
  static const char* op = "tre_mxfp4_quantize";
  const tre_status st = check_rows(op, type, rows, k);
  if (st != TRE_OK || rows == 0) return st;
  OP_ARG(ptr16(w) && ptr16(out), op, "NULL or misaligned pointer");
  OP_ARG(rows == 1 || (w_row_stride >= 0 && w_row_stride % (type == TRE_BF16 ? 8 : 4) == 0), op,
         "the row stride must be whole 16-byte units");
  const int64_t gpr = k / 32, pitch = pitch_of(k);
  in_slabs(rows, gpr, [&](int64_t r, int64_t n) {
    const uint32_t groups = (uint32_t)(n * gpr);
    const unsigned grid = (groups + kGroupsPerCta - 1) / kGroupsPerCta;
    uint8_t* o = static_cast<uint8_t*>(out) + r * pitch;
    if (type == TRE_BF16)
      mxfp4_quantize_kernel<<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(
          static_cast<const __nv_bfloat16*>(w) + r * w_row_stride, w_row_stride, groups,
          (uint32_t)gpr, k, pitch, o);
    else
      mxfp4_quantize_kernel<<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(
          static_cast<const float*>(w) + r * w_row_stride, w_row_stride, groups, (uint32_t)gpr, k,
          pitch, o);
  });
  return op_launch_status(op);
}

TRE_EXPORT tre_status tre_mxfp4_dequantize(const void* w, int64_t rows, int64_t k, int32_t type,
                                           void* out, tre_stream stream) {
  static const char* op = "tre_mxfp4_dequantize";
  const tre_status st = check_rows(op, type, rows, k);
  if (st != TRE_OK || rows == 0) return st;
  OP_ARG(ptr16(w) && ptr16(out), op, "NULL or misaligned pointer");
  const int64_t gpr = k / 32, pitch = pitch_of(k);
  in_slabs(rows, gpr, [&](int64_t r, int64_t n) {
    const uint32_t groups = (uint32_t)(n * gpr);
    const unsigned grid = (groups + kGroupsPerCta - 1) / kGroupsPerCta;
    const uint8_t* in = static_cast<const uint8_t*>(w) + r * pitch;
    if (type == TRE_BF16)
      mxfp4_dequantize_kernel<<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(
          in, groups, (uint32_t)gpr, k, pitch, static_cast<__nv_bfloat16*>(out) + r * k);
    else
      mxfp4_dequantize_kernel<<<grid, kRowThreads, 0, (cudaStream_t)stream>>>(
          in, groups, (uint32_t)gpr, k, pitch, static_cast<float*>(out) + r * k);
  });
  return op_launch_status(op);
}
