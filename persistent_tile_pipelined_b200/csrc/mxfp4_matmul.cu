// Rows of activations times MXFP4 matrices, grouped by expert (declared in include/tre.h as
// tre_mxfp4_matmul).
//
// out^T = W x^T on the tensor cores: 128 matrix rows are the M side, kN rows of x the N side.
// An E2M1 number times a power of two has two significant bits, so the decoded weight is
// exact in bf16 and the product is kind::f16 with fp32 sums; the activations keep their
// bits.  Per stage of kKS weights the copy warp brings the codes of 128 rows and the kN rows
// of x into shared memory; two warpgroups take stages in turn, one thread per matrix row,
// and write the decoded weights straight into tensor memory, where the product reads its A
// side (no second trip through shared memory, no swizzle, no proxy fence); one thread issues
// the products.
#include <cuda_bf16.h>

#include <algorithm>

#include "tc.cuh"
#include "tensor_map.h"

namespace tre {
namespace {

constexpr int kRows = 128;          // matrix rows per CTA
constexpr int kCopyWarp = 8, kMmaWarp = 9, kThreadsMm = 320;  // warps 0-7: two decode warpgroups

template <int N>
struct Tile {
  static constexpr int KW = 256;                     // weights of a row per copy: 128 bytes
  static constexpr int KS = N >= 128 ? 64 : 128;     // weights per step: decode, product
  static constexpr int kSteps = KW / KS;             // steps per copy of weights
  static constexpr int WST = N == 256 ? 3 : N == 128 ? 2 : N == 64 ? 3 : N == 32 ? 4 : 5;
  static constexpr int XST = N == 256 ? 5 : N == 64 ? 3 : 4;
  static constexpr int kABufs = N == 256 ? 8 : N == 128 ? 4 : 2;  // an equal number per warpgroup
  static constexpr int kACols = KS / 2;              // tensor-memory columns of one A step
  static constexpr int kCols = N == 256 ? 512 : 256;
  static constexpr int kDCol = kABufs * kACols;
  static constexpr int kXBytes = N * KS * 2, kWBytes = kRows * KW / 2;
  static constexpr int kSmem = WST * kWBytes + XST * kXBytes + 1024 + 512;
  static constexpr int kCtas = N == 256 ? 1 : 2;     // per SM
  static_assert(kDCol + N <= kCols, "tensor memory");
  static_assert(kCtas * (kSmem + 1024 + 64) <= 228 * 1024, "shared memory");
};

struct MatmulParams {
  const uint8_t* w;
  const int32_t* offsets;
  void* out;
  int64_t out_stride, pitch;
  int32_t rows, n, k, n_experts, splits;
  uint32_t four;  // 4 (see e2m1x8)
  int32_t* status;
};

// The bf16 pairs of 8 codes (a little-endian word: element 2i in the low nibble of byte i),
// unscaled: the code's exponent and mantissa bits sit in bf16's lowest exponent and highest
// mantissa bits, which is the number times 2^-126 (its subnormal 0.5 included).  A byte
// permute doubles the nibble's byte into both bytes of its half, once shifted so that both
// nibbles stand high: the sign is then in place and the magnitude two bits below its own.
// `four` is 4, but not a constant: the shift by two is then an integer multiply-add, off the
// logic unit, which is what bounds the decoding.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t four, uint32_t* o) {
  const uint32_t w4 = w << 4;
  constexpr uint32_t sel[4] = {0x4400, 0x5511, 0x6622, 0x7733};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = __byte_perm(w4, w, sel[i]);
    o[i] = (p & 0x00700070u) * four + (p & 0x80008000u);
  }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 32 codes times their scale 2^(s - 127) as 16 bf16 pairs, s the byte `at` of `word`.  The
// pattern's 2^-126 and the scale make one exact factor 2^(s - 1), representable up to s = 128;
// larger scales (and NaN, 255) multiply once more (kBig: there may be such).
template <bool kBig>
__device__ __forceinline__ void decode32(const uint4 c, uint32_t word, int at, uint32_t four,
                                         uint32_t* o) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const uint32_t s2 = __byte_perm(word, 0, 0x4040 + 0x0101 * at);  // s in both halves
  const uint32_t s = s2 & 0xffffu;
  uint32_t f2 = s2 * 128u + (126u << 7 | 126u << 23);
  if (kBig && s > 128u) f2 = 0x7f007f00u;
#pragma unroll
  for (int j = 0; j < 4; ++j) e2m1x8(w[j], four, o + 4 * j);
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = mul_bf16x2(o[j], f2);
  if (kBig && s > 128u) {
    const uint32_t h = s == 255u ? 0x7fc0u : (s - 1u) << 7;
    const uint32_t h2 = h | h << 16;
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = mul_bf16x2(o[j], h2);
  }
}

// A step's codes (16-byte chunks q) into tensor memory, 32 columns (64 weights) at a time: the
// first half is decoded before the place is waited for, the second while the first is stored.
// By whole warps; false when the wait gave up.
template <int kChunks, bool kBig>
__device__ __forceinline__ bool decode_step(const uint4* q, uint32_t word, uint32_t four,
                                            uint32_t addr, uint64_t* empty, uint32_t parity,
                                            volatile int* gave_up) {
#pragma unroll
  for (int c = 0; c < kChunks; c += 2) {
    uint32_t v[32];
    decode32<kBig>(q[c], word, c, four, v);
    decode32<kBig>(q[c + 1], word, c + 1, four, v + 16);
    if (c == 0) {
      if (!tc::wait_warp(empty, parity, gave_up)) return false;
      tc::fence_after();
    }
    tc::tmem_st32(addr + c * 16, v);
  }
  return true;
}

// Whether any of 4 bytes exceeds 128.
__device__ __forceinline__ uint32_t over128(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) & w & 0x80808080u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t smem_addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <class Out>
__device__ __forceinline__ void put(Out* p, float v) {
  if constexpr (sizeof(Out) == 4) *p = v;
  else *p = __float2bfloat16_rn(v);
}

// Rows of x per copy: a tile brings only the boxes that hold rows of its expert (what the
// product makes of the rest of its N side is not stored).
template <int N>
constexpr int kBoxOf = N > 64 ? 64 : 16;

template <int N, class Out>
__global__ void __launch_bounds__(kThreadsMm, Tile<N>::kCtas)
    mxfp4_matmul_kernel(const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ CUtensorMap wmap, const MatmulParams p) {
  using T = Tile<N>;
  constexpr int kBox = kBoxOf<N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* xring = ring + T::WST * T::kWBytes;
  uint64_t* w_full = reinterpret_cast<uint64_t*>(xring + T::XST * T::kXBytes);
  uint64_t* w_empty = w_full + T::WST;
  uint64_t* x_full = w_empty + T::WST;
  uint64_t* x_empty = x_full + T::XST;
  uint64_t* a_full = x_empty + T::XST;
  uint64_t* a_empty = a_full + T::kABufs;
  uint64_t* done = a_empty + T::kABufs;
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up, tile[3];  // expert, first row of x, rows of x
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the tile's expert: tiles of kN rows, expert by expert
  if (warp == 0) {
    int y = blockIdx.y, found = -1, row = 0, count = 0;
    if (!p.offsets) {
      found = 0;
      row = y * N;
      count = p.rows - row;
    } else {
      // a lane takes `per` experts in a row; their counts load together
      const int per = (p.n_experts + 31) / 32, first = lane * per;
      auto bounds = [&](int e, int& lo, int& hi) {
        lo = hi = 0;
        if (e < p.n_experts && e < first + per) {
          lo = min(max(p.offsets[e], 0), p.rows);
          hi = max(min(max(p.offsets[e + 1], 0), p.rows), lo);
        }
      };
      int tiles = 0;
      for (int e = first; e < first + per; e += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          int lo, hi;
          bounds(e + i, lo, hi);
          tiles += (hi - lo + N - 1) / N;
        }
      }
      int sum = tiles;  // inclusive over the lanes
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      const uint32_t mine = __ballot_sync(0xffffffffu, sum > y);
      if (mine) {
        const int l = __ffs(mine) - 1;
        if (lane == l) {
          y -= sum - tiles;
          for (int e = first; found < 0; ++e) {
            int lo, hi;
            bounds(e, lo, hi);
            const int t = (hi - lo + N - 1) / N;
            if (y < t) {
              found = e;
              row = lo + y * N;
              count = hi - row;
            }
            y -= t;
          }
        }
        found = __shfl_sync(0xffffffffu, found, l);
        row = __shfl_sync(0xffffffffu, row, l);
        count = __shfl_sync(0xffffffffu, count, l);
      }
    }
    if (lane == 0) {
      tile[0] = found;
      tile[1] = row;
      tile[2] = min(count, N);
      gave_up = 0;
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < T::WST; ++i) {
      mbar_init(w_full + i, 1);
      mbar_init(w_empty + i, 8);  // a lane of each decode warp
    }
    for (int i = 0; i < T::XST; ++i) {
      mbar_init(x_full + i, 1);
      mbar_init(x_empty + i, 1);
    }
    for (int i = 0; i < T::kABufs; ++i) {
      mbar_init(a_full + i, 4);
      mbar_init(a_empty + i, 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  } else if (warp == kCopyWarp && lane == 0) {
    tc::prefetch_map(&wmap);
    tc::prefetch_map(&xmap);
  }
  __syncthreads();
  const int expert = tile[0], t0 = tile[1], nt = tile[2];
  if (expert < 0) return;  // the same for every CTA of the cluster
  if (warp == kMmaWarp) tc::tmem_alloc(&tmem_base, T::kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;

  const int split = p.splits > 1 ? (int)cluster_rank() : 0;
  const int r0 = (int)(blockIdx.x / p.splits) * kRows;
  // whole groups of 512 weights (16 scale bytes) per part of a split
  const int groups = (p.k + 511) / 512;
  const int k_begin = (int)((int64_t)groups * split / p.splits) * 512;
  const int k_end = min((int)((int64_t)groups * (split + 1) / p.splits) * 512, p.k);
  const int stages = (max(k_end - k_begin, 0) + T::KS - 1) / T::KS;

  if (warp == kCopyWarp) {
    if (tc::elect_one()) {
      int it = 0, w = 0;
      const int boxes = (nt + kBox - 1) / kBox;  // rows of x that the expert has, by the box
      const int copies = (stages + T::kSteps - 1) / T::kSteps;
      long long since = clock64();  // the last copy
      while (it < stages) {  // whichever ring has a free place
        bool idle = true;
        if (w < copies && mbar_test_wait(w_empty + w % T::WST, (w / T::WST & 1) ^ 1)) {
          const int slot = w % T::WST;
          mbar_arrive_expect_tx(w_full + slot, T::kWBytes);
          tc::load_2d(ring + slot * T::kWBytes, &wmap, k_begin / 2 + w * (T::KW / 2),
                      expert * p.n + r0, w_full + slot);
          ++w;
          idle = false;
        }
        if (it / T::kSteps < w && mbar_test_wait(x_empty + it % T::XST, (it / T::XST & 1) ^ 1)) {
          const int slot = it % T::XST;
          uint8_t* x = xring + slot * T::kXBytes;
          const int k0 = k_begin + it * T::KS;
          mbar_arrive_expect_tx(x_full + slot, boxes * kBox * T::KS * 2);
#pragma unroll
          for (int h = 0; h < T::KS / 64; ++h)
            for (int b = 0; b < boxes; ++b)
              tc::load_2d(x + h * N * 128 + b * kBox * 128, &xmap, k0 + h * 64, t0 + b * kBox,
                          x_full + slot);
          ++it;
          idle = false;
        }
        if (!idle) {
          since = clock64();
        } else {
          __nanosleep(32);
          if (*(volatile int*)&gave_up || clock64() - since > tc::kWaitClocks) {
            gave_up = 1;
            break;
          }
        }
      }
      if (gave_up) {  // copies in flight land before the CTA ends
        for (int i = max(0, it - T::XST); i < it; ++i)
          for (int n = 0; n < 100000 && !mbar_try_wait(x_full + i % T::XST, i / T::XST & 1); ++n) {
          }
        for (int i = max(0, w - T::WST); i < w; ++i)
          for (int n = 0; n < 100000 && !mbar_try_wait(w_full + i % T::WST, i / T::WST & 1); ++n) {
          }
      }
    }
  } else if (warp == kMmaWarp) {
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_bf16(kRows, min(N, (nt + 15) & ~15), 0);
      bool ok = true;
      for (int it = 0; it < stages && ok; ++it) {
        const int slot = it % T::XST, buf = it % T::kABufs;
        ok = tc::wait(x_full + slot, it / T::XST & 1, &gave_up) &&
             tc::wait(a_full + buf, it / T::kABufs & 1, &gave_up);
        if (!ok) break;
        tc::fence_after();
        const uint32_t x = smem_u32(xring + slot * T::kXBytes);
#pragma unroll
        for (int j = 0; j < T::KS / 16; ++j) {
          const uint64_t b = tc::smem_desc(x + (j / 4) * N * 128 + (j % 4) * 32, 16, 1024);
          tc::mma_ts(tmem + T::kDCol, tmem + buf * T::kACols + j * 8, b, idesc, it + j > 0);
        }
        tc::commit(x_empty + slot);
        tc::commit(a_empty + buf);
      }
      tc::commit(done);
      if (!ok)
        for (int n = 0; n < 100000 && !mbar_try_wait(done, 0); ++n) {
        }
    }
  } else {
    // decode: thread = matrix row r0 + 32 (warp mod 4) + lane, warpgroup = step parity
    const int wg = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const int64_t row = (int64_t)expert * p.n + min(r0 + r, p.n - 1);
    const uint8_t* scales = p.w + row * p.pitch + p.k / 2;
    const int blocks = p.k / 32;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    // 16 scales; zero behind the row's last, where the copies bring zero codes
    auto fetch = [&](int g) {
      if (g * 16 >= blocks) return make_uint4(0, 0, 0, 0);
      uint4 v = *reinterpret_cast<const uint4*>(scales + g * 16);
      const int left = blocks - g * 16;
      if (left < 16) {
        auto keep = [&](int n) { return n >= 4 ? ~0u : n <= 0 ? 0u : ~0u >> (32 - 8 * n); };
        v.x &= keep(left);
        v.y &= keep(left - 4);
        v.z &= keep(left - 8);
        v.w &= keep(left - 12);
      }
      return v;
    };
    const uint8_t* my_codes = ring + r * (T::KW / 2);
    constexpr int kChunks = T::KS / 32;  // 16-byte chunks of a step
    uint4 sc = fetch(k_begin / 512), next = make_uint4(0, 0, 0, 0);
    bool ok = true;
    int slot = 0, phase = 0, mine = 0;  // `mine`: steps that this warpgroup has taken
#pragma unroll 1
    for (int first = 0; first < stages && ok; first += T::kSteps) {  // a copy of 256 weights
      const bool odd = (first / T::kSteps) & 1;
      if (!odd) next = fetch(k_begin / 512 + first / (2 * T::kSteps) + 1);
      const uint32_t lo = odd ? sc.z : sc.x, hi = odd ? sc.w : sc.y;  // the copy's 8 scales
      // the same way for the whole warp: its stores to tensor memory go together
      const bool big = __any_sync(0xffffffffu, (over128(lo) | over128(hi)) != 0);
      ok = tc::wait_warp(w_full + slot, phase, &gave_up);
#pragma unroll
      for (int u = 0; u < T::kSteps / 2; ++u) {
        const int h = 2 * u + wg;
        if (!ok || first + h >= stages) continue;
        uint4 q[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)  // the 128-byte swizzle: chunk c of row r at c ^ (r mod 8)
          q[c] = *reinterpret_cast<const uint4*>(my_codes + slot * T::kWBytes +
                                                 ((h * kChunks + c) ^ (r & 7)) * 16);
        const uint32_t word = kChunks == 4 ? (wg ? hi : lo) : (u ? hi : lo) >> (16 * wg);
        const int buf = (2 * mine + wg) % T::kABufs;
        const uint32_t free = (2 * mine / T::kABufs & 1) ^ 1, at = lane_addr + buf * T::kACols;
        ok = big ? decode_step<kChunks, true>(q, word, p.four, at, a_empty + buf, free, &gave_up)
                 : decode_step<kChunks, false>(q, word, p.four, at, a_empty + buf, free, &gave_up);
        if (!ok) continue;
        ++mine;
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(a_full + buf);
      }
      if (lane == 0) mbar_arrive(w_empty + slot);
      if (++slot == T::WST) slot = 0, phase ^= 1;
      if (odd) sc = next;
    }
    __syncwarp();
    // the sums: warpgroup = half of the rows of x
    ok = ok && (stages == 0 || tc::wait_warp(done, 0, &gave_up));
    tc::fence_after();
    Out* out = static_cast<Out*>(p.out);
    float* part = reinterpret_cast<float*>(ring);  // split along k: [N][128], ring is idle
    constexpr int kStep = N >= 64 ? 32 : 8;
    for (int c0 = wg * (N / 2); c0 < min((wg + 1) * (N / 2), nt); c0 += kStep) {
      uint32_t v[kStep];
      __syncwarp();
      if (kStep == 32) tc::tmem_ld32(lane_addr + T::kDCol + c0, v);
      else tc::tmem_ld8(lane_addr + T::kDCol + c0, v);
      tc::wait_ld();
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const float f = stages == 0 ? 0.f : __uint_as_float(v[j]);
        if (p.splits > 1) {
          part[(c0 + j) * kRows + r] = f;
        } else if (ok && c0 + j < nt && r0 + r < p.n) {
          put(out + (int64_t)(t0 + c0 + j) * p.out_stride + r0 + r, f);
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::fence_after();
    tc::tmem_free(tmem, T::kCols);
  }
  if (p.splits > 1) {
    // every CTA joins its share of the rows of x, always adding the parts in the same order
    cluster_sync();
    const int r = threadIdx.x & (kRows - 1);
    if (threadIdx.x < 2 * kRows && r0 + r < p.n) {
      for (int j = split * 2 + (threadIdx.x >> 7); j < nt; j += 2 * p.splits) {
        float sum = 0.f;
        for (int s = 0; s < p.splits; ++s)
          sum += ld_cluster(smem_u32(ring) + (uint32_t)(j * kRows + r) * 4, s);
        put(static_cast<Out*>(p.out) + (int64_t)(t0 + j) * p.out_stride + r0 + r, sum);
      }
    }
    cluster_sync();
  }
  if (threadIdx.x == 0 && gave_up) atomicExch(p.status, TRE_ERR_DEP_TIMEOUT);
}

template <int N, class Out>
tre_status launch(const char* op, const MatmulParams& p, const CUtensorMap& xmap,
                  const CUtensorMap& wmap, cudaStream_t stream) {
  using T = Tile<N>;
  auto kernel = mxfp4_matmul_kernel<N, Out>;
  static std::atomic<uint64_t> devices;
  if (!allow_smem(reinterpret_cast<const void*>(kernel), T::kSmem, &devices))
    return op_error(TRE_ERR_CUDA, op, "the device refuses the kernel's shared memory");
  cudaLaunchConfig_t c = {};
  const int64_t tiles = p.offsets ? (int64_t)p.rows / N + std::min<int64_t>(p.n_experts, p.rows)
                                  : ((int64_t)p.rows + N - 1) / N;
  OP_ARG(tiles <= 65535, op, "too many rows for one call");
  c.gridDim = dim3((unsigned)((p.n + kRows - 1) / kRows * p.splits), (unsigned)tiles);
  c.blockDim = dim3(kThreadsMm);
  c.dynamicSmemBytes = T::kSmem;
  c.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = p.splits > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, xmap, wmap, p);
  return e == cudaSuccess ? TRE_OK : op_error(TRE_ERR_CUDA, op, cudaGetErrorString(e));
}

// Rows of x per tile: the least of 16 .. 256 that covers three times an expert's average (few
// experts' weights are decoded twice), but no more than leaves the device without tiles to fill it.
int tile_rows(const MatmulParams& p, int sms) {
  const int64_t avg = ((int64_t)p.rows * (p.n_experts > 1 ? 3 : 1) + p.n_experts - 1) / p.n_experts;
  int best = 16;
  while (best < 256 && best < avg) best *= 2;
  const int64_t row_tiles = (p.n + kRows - 1) / kRows;
  while (best > 64 && row_tiles * ((p.rows + best - 1) / best) < sms) best /= 2;
  return best;
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
  tre_status st;
  OP_ARG(ptr16(x) && ptr16(w) && out && ((uintptr_t)out & (out_type == TRE_BF16 ? 1 : 3)) == 0,
         op, "NULL or misaligned pointer");
  OP_ARG(((uintptr_t)offsets & 3) == 0, op, "misaligned offsets");
  OP_ARG(rows == 1 || (x_row_stride % 8 == 0 && x_row_stride >= k), op,
         "x rows must not overlap and their stride be whole 16-byte units");
  OP_ARG(rows == 1 || out_row_stride >= n, op, "output rows overlap");
  const int64_t pitch = (k / 2 + k / 32 + 15) / 16 * 16;
  const int sms = device_sms();
  MatmulParams p{static_cast<const uint8_t*>(w), offsets, out, out_row_stride, pitch,
                 (int32_t)rows, (int32_t)n, (int32_t)k, n_experts, 1, 4u, ops_status_ptr()};
  OP_ARG(p.status, op, "the operators' status word is not available");
  const int tile = tile_rows(p, sms);
  if (tile <= 32) {  // few tiles: split k over a cluster until the device is busy
    const int64_t tiles = (n + kRows - 1) / kRows * ((rows + tile - 1) / tile);
    const int groups = (int)((k + 511) / 512);
    const int most = (int)std::min<int64_t>({8, groups, std::max<int64_t>(1, 2 * sms / tiles)});
    const int each = (groups + most - 1) / most;
    p.splits = (groups + each - 1) / each;
  }
  CUtensorMap xmap, wmap;
  const uint64_t xd[2] = {(uint64_t)k, (uint64_t)rows};
  const uint64_t xs[1] = {(uint64_t)(rows == 1 ? k : x_row_stride) * 2};
  const uint32_t xb[2] = {64, tile > 64 ? 64u : 16u};  // kBoxOf
  st = encode_map(op, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, xd, xs, xb,
                  CU_TENSOR_MAP_SWIZZLE_128B, &xmap);
  if (st != TRE_OK) return st;
  const uint64_t wd[2] = {(uint64_t)k / 2, (uint64_t)n * n_experts};
  const uint64_t ws[1] = {(uint64_t)pitch};
  const uint32_t wb[2] = {Tile<16>::KW / 2, kRows};
  st = encode_map(op, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w, wd, ws, wb,
                  CU_TENSOR_MAP_SWIZZLE_128B, &wmap);
  if (st != TRE_OK) return st;
#define MM(N)                                                                            \
  case N:                                                                                \
    return out_type == TRE_BF16                                                          \
               ? launch<N, __nv_bfloat16>(op, p, xmap, wmap, (cudaStream_t)stream)       \
               : launch<N, float>(op, p, xmap, wmap, (cudaStream_t)stream)
  switch (tile) {
    MM(16);
    MM(32);
    MM(64);
    MM(128);
    default:
      MM(256);
  }
#undef MM
}
