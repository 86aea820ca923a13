// MXFP4 rows: quantiser and its inverse (declared in include/tre.h).
//
// One pass: a group of 32 weights is four lanes' loads, its scale two exchanges between them, so
// the copy rate bounds both directions.  Measured, B200: 24 x 1999 x 7168 fp32 to rows and back to
// bf16: 400-404 us, 6.0 TB/s (0.92 of the measured copy rate).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

#include "ops_host.h"

namespace tre {

namespace {

constexpr int kRowThreads = 256;
constexpr int kGroupsPerPass = kRowThreads / 4;  // 4 lanes share a group of 32 weights
// kPasses: groups of a lane, loaded together.  4 where the grid is long (24 x 1999 x 7168 fp32 and
// back: 384 us against 437 with 1), 1 where it is short and its last wave counts
// (2048 x 7168 bf16 and back: 23 us against 29 with 4).
constexpr uint32_t kLongGrid = 4096;  // CTAs of 4 passes

// Row and group within the row of a group's number (below 2^30): `inv` is ceil(2^32 / per_row),
// whose quotient is at most one too large.
__device__ __forceinline__ void place_of(uint32_t g, uint32_t per_row, uint32_t inv, uint32_t& row,
                                         uint32_t& b) {
  row = inv ? __umulhi(g, inv) : g;  // (per_row 1: 2^32 does not fit)
  if (row * per_row > g) --row;
  b = g - row * per_row;
}

// 8 numbers: fp32 as one 32-byte load where the rows are aligned to that (kWide), bf16 as one of
// 16 bytes.
template <bool kWide>
__device__ __forceinline__ void load8(const float* p, float* v) {
  if (kWide) {
    asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

template <bool kWide>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}

// Four lanes take a group of 32 weights, 8 each: the largest magnitude by two exchanges, its
// binary exponent from the bits, then 8 codes as one word.
template <int kPasses, bool kWide, class T>
__global__ void __launch_bounds__(kRowThreads)
    mxfp4_quantize_kernel(const T* __restrict__ w, int64_t w_stride, uint32_t groups,
                          uint32_t per_row, uint32_t inv_per_row, int64_t k, int64_t pitch,
                          uint8_t* __restrict__ out) {
  const uint32_t g0 = blockIdx.x * (kPasses * kGroupsPerPass) + (threadIdx.x >> 2);
  const uint32_t lane4 = threadIdx.x & 3u;
  float v[kPasses][8];
  uint32_t row[kPasses], b[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t g = g0 + i * kGroupsPerPass;
    if (g < groups) {
      place_of(g, per_row, inv_per_row, row[i], b[i]);
      load8<kWide>(w + (int64_t)row[i] * w_stride + (int64_t)b[i] * 32 + lane4 * 8, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const bool live = g0 + i * kGroupsPerPass < groups;
    // magnitudes compare like their bits, and a NaN's or infinity's bits exceed every number's
    uint32_t top = 0;
    if (live)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (!live) continue;
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
        const float2 p = make_float2(v[i][2 * j] * inv, v[i][2 * j + 1] * inv);
        codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(p, __NV_E2M1, cudaRoundNearest) << (8 * j);
      }
    }
    uint8_t* orow = out + (int64_t)row[i] * pitch;
    *reinterpret_cast<uint32_t*>(orow + (int64_t)b[i] * 16 + lane4 * 4) = codes;
    if (lane4 == 0) orow[k / 2 + b[i]] = (uint8_t)byte;
    if (b[i] + 1 == per_row)
      for (int64_t x = k / 2 + per_row + lane4; x < pitch; x += 4) orow[x] = 0;
  }
}

template <int kPasses, class T>
__global__ void __launch_bounds__(kRowThreads)
    mxfp4_dequantize_kernel(const uint8_t* __restrict__ w, uint32_t groups, uint32_t per_row,
                            uint32_t inv_per_row, int64_t k, int64_t pitch, T* __restrict__ out) {
  const uint32_t g0 = blockIdx.x * (kPasses * kGroupsPerPass) + (threadIdx.x >> 2);
  const uint32_t lane4 = threadIdx.x & 3u;
  uint32_t codes[kPasses], s[kPasses], row[kPasses], b[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t g = g0 + i * kGroupsPerPass;
    if (g < groups) {
      place_of(g, per_row, inv_per_row, row[i], b[i]);
      const uint8_t* wr = w + (int64_t)row[i] * pitch;
      codes[i] = __ldg(reinterpret_cast<const uint32_t*>(wr + (int64_t)b[i] * 16 + lane4 * 4));
      s[i] = __ldg(wr + k / 2 + b[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (g0 + i * kGroupsPerPass >= groups) continue;
    const float scale = __uint_as_float(s[i] == 0u     ? 0x00400000u
                                        : s[i] == 255u ? 0x7fc00000u
                                                       : s[i] << 23);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
          (__nv_fp4x2_storage_t)(codes[i] >> (8 * j) & 0xffu), __NV_E2M1);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * j] = f.x * scale;
      v[2 * j + 1] = f.y * scale;
    }
    T* o = out + (int64_t)row[i] * k + (int64_t)b[i] * 32 + lane4 * 8;
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
}

int64_t pitch_of(int64_t k) { return (k / 2 + k / 32 + 15) / 16 * 16; }

uint32_t inverse(int64_t d) { return d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); }

// Rows per launch: a launch's groups stay within 2^30, so their numbers divide in 32 bits.
template <class Launch>
tre_status in_slabs(int64_t rows, int64_t groups_per_row, Launch launch) {
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 30) / groups_per_row);
  tre_status st = TRE_OK;
  for (int64_t r = 0; r < rows && st == TRE_OK; r += most) st = launch(r, std::min(most, rows - r));
  return st;
}

template <class T>
tre_status quantize(const char* op, const T* w, int64_t stride, int64_t rows, int64_t k,
                    int64_t pitch, uint8_t* out, tre_stream stream) {
  const uint32_t per_row = (uint32_t)(k / 32), groups = (uint32_t)(rows * per_row);
  const uint32_t ctas = (groups + kGroupsPerPass - 1) / kGroupsPerPass;
  const bool wide = sizeof(T) == 4 && (reinterpret_cast<uintptr_t>(w) & 31u) == 0 &&
                    (rows == 1 || stride % 8 == 0);
  const bool longer = ctas >= 4 * kLongGrid;
  auto kernel = longer ? mxfp4_quantize_kernel<4, false, T> : mxfp4_quantize_kernel<1, false, T>;
  if (wide) kernel = longer ? mxfp4_quantize_kernel<4, true, T> : mxfp4_quantize_kernel<1, true, T>;
  return op_launch(op, kernel, dim3(longer ? (ctas + 3) / 4 : ctas), kRowThreads, 0, stream, w,
                   stride, groups, per_row, inverse(per_row), k, pitch, out);
}

template <class T>
tre_status dequantize(const char* op, const uint8_t* w, int64_t rows, int64_t k, int64_t pitch,
                      T* out, tre_stream stream) {
  const uint32_t per_row = (uint32_t)(k / 32), groups = (uint32_t)(rows * per_row);
  const uint32_t ctas = (groups + kGroupsPerPass - 1) / kGroupsPerPass;
  const bool longer = ctas >= 4 * kLongGrid;
  auto kernel = longer ? mxfp4_dequantize_kernel<4, T> : mxfp4_dequantize_kernel<1, T>;
  return op_launch(op, kernel, dim3(longer ? (ctas + 3) / 4 : ctas), kRowThreads, 0, stream, w,
                   groups, per_row, inverse(per_row), k, pitch, out);
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
  const int64_t pitch = pitch_of(k);
  return in_slabs(rows, k / 32, [&](int64_t r, int64_t n) {
    uint8_t* o = static_cast<uint8_t*>(out) + r * pitch;
    return type == TRE_BF16 ? quantize(op, static_cast<const __nv_bfloat16*>(w) + r * w_row_stride,
                                       w_row_stride, n, k, pitch, o, stream)
                            : quantize(op, static_cast<const float*>(w) + r * w_row_stride,
                                       w_row_stride, n, k, pitch, o, stream);
  });
}

TRE_EXPORT tre_status tre_mxfp4_dequantize(const void* w, int64_t rows, int64_t k, int32_t type,
                                           void* out, tre_stream stream) {
  static const char* op = "tre_mxfp4_dequantize";
  const tre_status st = check_rows(op, type, rows, k);
  if (st != TRE_OK || rows == 0) return st;
  OP_ARG(ptr16(w) && ptr16(out), op, "NULL or misaligned pointer");
  const int64_t pitch = pitch_of(k);
  return in_slabs(rows, k / 32, [&](int64_t r, int64_t n) {
    const uint8_t* in = static_cast<const uint8_t*>(w) + r * pitch;
    return type == TRE_BF16
               ? dequantize(op, in, n, k, pitch, static_cast<__nv_bfloat16*>(out) + r * k, stream)
               : dequantize(op, in, n, k, pitch, static_cast<float*>(out) + r * k, stream);
  });
}
