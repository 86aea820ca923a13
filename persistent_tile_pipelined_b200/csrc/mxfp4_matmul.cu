// Rows of activations times MXFP4 matrices, grouped by expert (declared in include/tre.h as
// tre_mxfp4_matmul).
//
// out^T = W x^T on the tensor cores: 128 matrix rows are the M side, 16 to 256 rows of x the N
// side.  An E2M1 number times a power of two has two significant bits, so the decoded weight is
// exact in bf16 and the product is kind::f16 with fp32 sums; the activations keep their bits.
// One warp copies the codes of 128 rows (256 weights at a time) and the rows of x to shared
// memory; two warpgroups take steps of 64 or 128 weights in turn, one thread per matrix row, and
// write the decoded weights straight into tensor memory, where the product reads its A side (no
// second trip through shared memory, no swizzle, no proxy fence); one warp issues the products.
//
// A job is a tile of x times 128 matrix rows.  The experts' counts are known on the device only:
// each CTA sums their tiles and finds its job.  Tiles up to 128 rows run two CTAs an SM, one job
// each, so that one starts or ends while the other multiplies (resident CTAs: 732 us against 620
// on the case below); the 256-row tile has the SM alone, stays, and lets two further
// warpgroups carry the sums out (278 -> 247 us).  For few rows k is split over a cluster of up
// to 8 CTAs, which adds the parts through distributed shared memory, in order.
//
// What bounds it, B200.  Few rows per expert (4096 rows over 256 experts of 2048 x 7168, 219
// with rows: 1.7 GB of codes, 272 us at the measured copy rate): decoding, 590 us, 3.0 TB/s.
// A pair of weights takes three operations of the logic unit (half a warp a clock) and two
// multiply-adds: 250 ns per 128 x 128 weights and SM when nothing else runs, 340 us of the case.
// A CTA's start and end take 90 us of it, the barriers between copies, decoding and products
// some 50 each.  Steps of 64 weights are slower than of 128 (640 us), more places for decoded
// weights or for x change nothing, the codes read a step ahead 626, a third decoding warpgroup
// 638, the conversion instruction (e2m1 pair to f16, then to bf16) 719 against 677.  Many rows
// (8192 x 2048 over 4 experts of 7168 rows): 241-245 us, 990 TFLOP/s, 0.61 of the measured 1615;
// every 128 matrix rows read their x again, 8.4 TB/s from L2.
#include <cuda_bf16.h>

#include <algorithm>

#include "tc.cuh"
#include "tensor_map.h"

namespace tre {
namespace {

constexpr int kRows = 128;          // matrix rows per CTA
constexpr int kDecodeWarps = 8;     // warps 0-7: two warpgroups

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
  // The largest tile has the SM to itself: a CTA stays and takes job after job, and two
  // warpgroups of their own carry the sums out while the next job's products run (its sums
  // take half of the tensor memory, so they have to be out of it first).
  static constexpr bool kStay = N == 256;
  static constexpr int kOutWarps = kStay ? 8 : 0;
  static constexpr int kCopyWarp = kDecodeWarps + kOutWarps, kMmaWarp = kCopyWarp + 1;
  static constexpr int kThreads = kStay ? 640 : 320; // (whole warpgroups where registers move)
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
  int32_t most_jobs;  // tiles of x times tiles of matrix rows: an upper bound
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

// A step's codes (16-byte chunks q; their scales are `word` from `byte` on) into tensor memory,
// 32 columns (64 weights) at a time: the first half is decoded before the place is waited for,
// the second while the first is stored.  By whole warps; false when the wait gave up.
template <int kChunks, bool kBig>
__device__ __forceinline__ bool decode_step(const uint4* q, uint32_t word, int byte,
                                            uint32_t four, uint32_t addr, uint64_t* empty,
                                            uint32_t parity, volatile int* gave_up) {
#pragma unroll
  for (int c = 0; c < kChunks; c += 2) {
    uint32_t v[32];
    decode32<kBig>(q[c], word, byte + c, four, v);
    decode32<kBig>(q[c + 1], word, byte + c + 1, four, v + 16);
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

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
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

struct Job {
  int expert, r0, t0, nt;  // rows r0 .. r0 + 127 of its matrix, rows t0 .. t0 + nt - 1 of x
};

template <int N, class Out>
__global__ void __launch_bounds__(Tile<N>::kThreads, Tile<N>::kCtas)
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
  uint64_t* d_free = done + 1;
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up, lane_tiles[32], lane_last[32];
  __shared__ Job first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Tiles of N rows of x, expert by expert.  A lane counts those of `per` experts in a row
  // (their bounds load together): lane_tiles, and lane_last = the sum up to and with it.
  const int per = (p.n_experts + 31) / 32;
  auto bounds = [&](int e, int first, int& lo, int& hi) {
    lo = hi = 0;
    if (e < p.n_experts && e < first + per) {
      lo = p.offsets ? min(max(p.offsets[e], 0), p.rows) : 0;
      hi = p.offsets ? max(min(max(p.offsets[e + 1], 0), p.rows), lo) : p.rows;
    }
  };
  // A job is a tile of x times 128 rows of its expert; the CTA (a cluster when k is split)
  // takes every gridDim-th, neighbours the same x.
  const int row_tiles = (p.n + kRows - 1) / kRows;
  const int job_step = gridDim.x / p.splits, first_job = blockIdx.x / p.splits;
  auto find_job = [&](int job) {  // whole warp
    int y = job / row_tiles;
    Job j{0, (job - y * row_tiles) * kRows, 0, 0};
    const int l = __ffs(__ballot_sync(0xffffffffu, lane_last[lane] > y)) - 1;
    y -= lane_last[l] - lane_tiles[l];
    for (int e0 = l * per;; e0 += 32) {  // the lane's experts, 32 at a time
      int lo, hi;
      bounds(e0 + lane, l * per, lo, hi);
      const int t = (hi - lo + N - 1) / N;
      int sum = t;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      const uint32_t mine = __ballot_sync(0xffffffffu, sum > y);
      const int last = __shfl_sync(0xffffffffu, sum, 31);
      if (mine || e0 + 32 >= l * per + per) {
        const int m = mine ? __ffs(mine) - 1 : 0;
        j.expert = e0 + m;
        j.t0 = __shfl_sync(0xffffffffu, lo + (y - (sum - t)) * N, m);
        j.nt = min(__shfl_sync(0xffffffffu, hi, m) - j.t0, N);
        if (!mine) j.nt = 0;  // the offsets changed under the call: no rows
        return j;
      }
      y -= last;
    }
  };

  if (warp == 0) {
    int tiles = 0;
    for (int e = lane * per; e < lane * per + per; e += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int lo, hi;
        bounds(e + i, lane * per, lo, hi);
        tiles += (hi - lo + N - 1) / N;
      }
      tiles = min(tiles, 1 << 25);  // (offsets that decrease cannot make the sums overflow)
    }
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    lane_tiles[lane] = tiles;
    lane_last[lane] = sum;
    __syncwarp();
    Job j{0, 0, 0, 0};
    if (first_job < (int64_t)lane_last[31] * row_tiles) j = find_job(first_job);
    if (lane == 0) {
      gave_up = 0;
      first = j;
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
    mbar_init(d_free, 8);  // a lane of each warp that carries sums out
    fence_mbar_init();
  } else if (warp == T::kCopyWarp && lane == 0) {
    tc::prefetch_map(&wmap);
    tc::prefetch_map(&xmap);
  } else if (warp == T::kMmaWarp) {
    tc::tmem_alloc(&tmem_base, T::kCols);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;

  const int split = p.splits > 1 ? (int)cluster_rank() : 0;
  // whole groups of 512 weights (16 scale bytes) per part of a split
  const int groups = (p.k + 511) / 512;
  const int k_begin = (int)((int64_t)groups * split / p.splits) * 512;
  const int k_end = min((int)((int64_t)groups * (split + 1) / p.splits) * 512, p.k);
  const int steps = (k_end - k_begin + T::KS - 1) / T::KS;
  const int copies = (steps + T::kSteps - 1) / T::kSteps;

  const int jobs = (int)min((int64_t)lane_last[31] * row_tiles, (int64_t)p.most_jobs);
  Job job{0, 0, 0, 0};  // of the reduction at the end
  // registers where the sums have warps of their own: 640 x 96 at launch, 256 x 80 + 256 x 136 +
  // 128 x 48 now
  if (T::kStay && warp >= T::kCopyWarp) tc::regs_less<48>();
  if (warp == T::kCopyWarp) {
    // (the whole warp, one lane issues: see the products)
    const bool leader = tc::elect_one();
    int wslot = 0, wphase = 1, xslot = 0, xphase = 1;  // places and the parity that frees them
    int w_used = 0, x_used = 0;
    bool ok = true;
    for (int n = first_job; n < jobs && ok; n = T::kStay ? n + job_step : jobs) {
      const Job j = n == first_job ? first : find_job(n);
      const int boxes = (j.nt + kBox - 1) / kBox;  // rows of x that the expert has, by the box
      const int wrow = j.expert * p.n + j.r0;
      long long since = clock64();  // the last copy
      for (int x = 0, w = 0; x < steps;) {  // whichever ring has a free place
        bool idle = true;
        if (w < copies && __all_sync(0xffffffffu, mbar_test_wait(w_empty + wslot, wphase))) {
          if (leader) {
            mbar_arrive_expect_tx(w_full + wslot, T::kWBytes);
            tc::load_2d(ring + wslot * T::kWBytes, &wmap, k_begin / 2 + w * (T::KW / 2), wrow,
                        w_full + wslot);
          }
          if (++wslot == T::WST) wslot = 0, wphase ^= 1;
          ++w, ++w_used;
          idle = false;
        }
        if (x / T::kSteps < w &&
            __all_sync(0xffffffffu, mbar_test_wait(x_empty + xslot, xphase))) {
          if (leader) {
            uint8_t* dst = xring + xslot * T::kXBytes;
            const int k0 = k_begin + x * T::KS;
            mbar_arrive_expect_tx(x_full + xslot, boxes * kBox * T::KS * 2);
#pragma unroll
            for (int h = 0; h < T::KS / 64; ++h)
              for (int b = 0; b < boxes; ++b)
                tc::load_2d(dst + h * N * 128 + b * kBox * 128, &xmap, k0 + h * 64,
                            j.t0 + b * kBox, x_full + xslot);
          }
          if (++xslot == T::XST) xslot = 0, xphase ^= 1;
          ++x, ++x_used;
          idle = false;
        }
        if (!idle) {
          since = clock64();
        } else {
          __nanosleep(32);
          if (__any_sync(0xffffffffu, *(volatile int*)&gave_up ||
                                          clock64() - since > tc::kWaitClocks)) {
            gave_up = 1;
            ok = false;
            break;
          }
        }
      }
    }
    const long long since = clock64();
    tc::settle_copies(x_full, x_used, T::XST, since);
    tc::settle_copies(w_full, w_used, T::WST, since);
  } else if (warp == T::kMmaWarp) {
    // The whole warp runs the loop, so that what the products take is uniform; one lane issues.
    const bool leader = tc::elect_one();
    constexpr uint32_t kHi = tc::desc_hi(1024);
    const uint32_t lo0 = tc::desc_lo(smem_u32(xring), 16);
    int xslot = 0, xphase = 0, abuf = 0, aphase = 0, dphase = 1;
    bool ok = true;
    for (int n = first_job; n < jobs && ok; n = T::kStay ? n + job_step : jobs) {
      const Job j = n == first_job ? first : find_job(n);
      const uint32_t idesc = tc::idesc_bf16(kRows, max(min(N, (j.nt + 15) & ~15), 16), 0);
      ok = tc::wait_warp(d_free, dphase, &gave_up);
      for (int x = 0; x < steps && ok; ++x) {
        ok = tc::wait_warp(x_full + xslot, xphase, &gave_up) &&
             tc::wait_warp(a_full + abuf, aphase, &gave_up);
        if (!ok) break;
        tc::fence_after();
        const uint32_t lo = lo0 + xslot * (T::kXBytes / 16);
        const uint32_t at = tmem + abuf * T::kACols;
        if (leader) {
#pragma unroll
          for (int i = 0; i < T::KS / 16; ++i)
            tc::mma_ts(tmem + T::kDCol, at + i * 8,
                       tc::desc_of(lo + (i / 4) * (N * 128 / 16) + (i % 4) * 2, kHi), idesc,
                       i > 0 || x > 0);
          tc::commit(x_empty + xslot);
          tc::commit(a_empty + abuf);
        }
        if (++xslot == T::XST) xslot = 0, xphase ^= 1;
        if (++abuf == T::kABufs) abuf = 0, aphase ^= 1;
      }
      if (leader) tc::commit(done);
      __syncwarp();
      dphase ^= 1;
    }
    if (first_job < jobs) tc::settle(done, dphase, clock64());
  } else if (T::kStay && warp >= kDecodeWarps) {
    // The sums of a job: thread = matrix row, warpgroup = 128 of the rows of x.  Three
    // quarters wait in registers so that the tensor memory is free after one is stored.
    if (warp >= T::kMmaWarp) {
      // (fills the last warpgroup)
    } else {
      if (T::kStay) tc::regs_more<136>();
      const int wg = (warp - kDecodeWarps) >> 2, quad = warp & 3, r = quad * 32 + lane;
      const uint32_t d_addr = tmem + ((uint32_t)(quad * 32) << 16) + T::kDCol + wg * 128;
      bool ok = true;
      int phase = 0;
      for (int n = first_job; n < jobs && ok; n += job_step) {
        const Job j = n == first_job ? first : find_job(n);
        ok = tc::wait_warp(done, phase, &gave_up);
        phase ^= 1;
        if (!ok) break;
        tc::fence_after();
        const int64_t stride = p.out_stride;
        Out* out = static_cast<Out*>(p.out) + (int64_t)(j.t0 + wg * 128) * stride + j.r0 + r;
        const int count = j.r0 + r < p.n ? j.nt - wg * 128 : 0;
        uint32_t v[3][32];
        auto store = [&](const uint32_t* s, int c0) {
          Out* o = out + (int64_t)c0 * stride;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < count) put(o + c * stride, __uint_as_float(s[c]));
        };
        tc::tmem_ld32(d_addr, v[0]);
        tc::tmem_ld32(d_addr + 32, v[1]);
        tc::tmem_ld32(d_addr + 64, v[2]);
        tc::wait_ld();
        store(v[0], 0);
        __syncwarp();
        tc::tmem_ld32(d_addr + 96, v[0]);
        tc::wait_ld();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_free);
        store(v[1], 32);
        store(v[2], 64);
        store(v[0], 96);
        __syncwarp();
      }
    }
  } else {
    if (T::kStay) tc::regs_less<80>();
    // decode: thread = matrix row r0 + 32 (warp mod 4) + lane, warpgroup = step parity
    const int wg = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const int blocks = p.k / 32;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int kChunks = T::KS / 32;  // 16-byte chunks of a step
    // 128-byte swizzle: chunk c of row r lies at c ^ (r mod 8); the warpgroup takes chunks
    // wg * kChunks + 0 .. of every 2 kChunks
    const uint32_t my_codes =
        (smem_u32(ring) + r * (T::KW / 2) + (r & 7) * 16) ^ (wg * kChunks * 16);
    bool ok = true;
    int slot = 0, phase = 0;
    int taken = 0;  // steps of the jobs so far: the A buffers go round with them
    for (int n = first_job; n < jobs && ok; n = T::kStay ? n + job_step : jobs) {
      job = n == first_job ? first : find_job(n);
      const int64_t row = (int64_t)job.expert * p.n + min(job.r0 + r, p.n - 1);
      const uint8_t* scales = p.w + row * p.pitch + p.k / 2;
      // 16 scales: two copies' worth
      auto fetch = [&](int g) {
        return g * 16 < blocks ? *reinterpret_cast<const uint4*>(scales + g * 16)
                               : make_uint4(0, 0, 0, 0);
      };
      // Of those the warpgroup's own, a word for each copy (when they are used: the load has
      // had two copies' time); zero behind the row's last, where the copies bring zero codes.
      auto own = [&](uint4 v, int g) {
        const int left = blocks - g * 16;
        if (left < 16) {
          auto keep = [&](int b) { return b >= 4 ? ~0u : b <= 0 ? 0u : ~0u >> (32 - 8 * b); };
          v.x &= keep(left);
          v.y &= keep(left - 4);
          v.z &= keep(left - 8);
          v.w &= keep(left - 12);
        }
        if (kChunks == 4) return wg ? make_uint2(v.y, v.w) : make_uint2(v.x, v.z);
        const uint32_t sel = wg ? 0x7632 : 0x5410;
        return make_uint2(__byte_perm(v.x, v.y, sel), __byte_perm(v.z, v.w, sel));
      };
      int g = k_begin / 512;
      uint4 next = fetch(g);
      uint2 sc = make_uint2(0, 0);
#pragma unroll 1
      for (int first = 0; first < steps && ok; first += T::kSteps) {  // a copy of 256 weights
        const bool odd = (first / T::kSteps) & 1;
        if (!odd) {
          sc = own(next, g);
          next = fetch(++g);
        }
        const uint32_t word = odd ? sc.y : sc.x;
        // the same way for the whole warp: its stores to tensor memory go together
        const bool big = __any_sync(0xffffffffu, over128(word) != 0);
        ok = tc::wait_warp(w_full + slot, phase, &gave_up);
        const uint32_t codes = my_codes + slot * T::kWBytes;
#pragma unroll
        for (int u = 0; u < T::kSteps / 2; ++u) {
          const int h = 2 * u + wg;
          if (!ok || first + h >= steps) continue;
          const int step = taken + first + h;
          uint4 q[kChunks];
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            q[c] = ld_shared16(codes ^ ((2 * u * kChunks + c) * 16));
          const int buf = step % T::kABufs;
          const uint32_t free = (step / T::kABufs & 1) ^ 1, at = lane_addr + buf * T::kACols;
          uint64_t* place = a_empty + buf;
          ok = big ? decode_step<kChunks, true>(q, word, u * kChunks, p.four, at, place, free,
                                                &gave_up)
                   : decode_step<kChunks, false>(q, word, u * kChunks, p.four, at, place, free,
                                                 &gave_up);
          if (!ok) continue;
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(a_full + buf);
        }
        if (lane == 0) mbar_arrive(w_empty + slot);
        if (++slot == T::WST) slot = 0, phase ^= 1;
      }
      taken += steps;
      __syncwarp();
      if (T::kStay) continue;
      // the sums: warpgroup = half of the rows of x
      ok = ok && tc::wait_warp(done, 0, &gave_up);
      if (!ok) break;
      tc::fence_after();
      Out* out = static_cast<Out*>(p.out);
      float* part = reinterpret_cast<float*>(ring);  // split along k: [N][128], ring is idle
      constexpr int kStep = N >= 64 ? 32 : 8;
      const uint32_t d_addr = lane_addr + T::kDCol;
      for (int c0 = wg * (N / 2); c0 < min((wg + 1) * (N / 2), job.nt); c0 += kStep) {
        uint32_t v[kStep];
        __syncwarp();
        if (kStep == 32) tc::tmem_ld32(d_addr + c0, v);
        else tc::tmem_ld8(d_addr + c0, v);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          const float f = __uint_as_float(v[j]);
          if (p.splits > 1) {
            part[(c0 + j) * kRows + r] = f;
          } else if (c0 + j < job.nt && job.r0 + r < p.n) {
            put(out + (int64_t)(job.t0 + c0 + j) * p.out_stride + job.r0 + r, f);
          }
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == T::kMmaWarp) {
    __syncwarp();
    tc::fence_after();
    tc::tmem_free(tmem, T::kCols);
  }
  if (p.splits > 1) {
    // every CTA joins its share of the rows of x, always adding the parts in the same order
    cluster_sync();
    const int r = threadIdx.x & (kRows - 1);
    if (threadIdx.x < 2 * kRows && job.r0 + r < p.n) {
      for (int j = split * 2 + (threadIdx.x >> 7); j < job.nt; j += 2 * p.splits) {
        float sum = 0.f;
        for (int s = 0; s < p.splits; ++s)
          sum += ld_cluster(smem_u32(ring) + (uint32_t)(j * kRows + r) * 4, s);
        put(static_cast<Out*>(p.out) + (int64_t)(job.t0 + j) * p.out_stride + job.r0 + r, sum);
      }
    }
    cluster_sync();
  }
  if (threadIdx.x == 0 && gave_up) atomicExch(p.status, TRE_ERR_DEP_TIMEOUT);
}

template <int N, class Out>
tre_status launch(const char* op, MatmulParams p, const CUtensorMap& xmap,
                  const CUtensorMap& wmap, int sms, cudaStream_t stream) {
  using T = Tile<N>;
  auto kernel = mxfp4_matmul_kernel<N, Out>;
  static std::atomic<uint64_t> devices;
  if (!allow_smem(reinterpret_cast<const void*>(kernel), T::kSmem, &devices))
    return op_cuda_error(op, "the device refuses the kernel's shared memory");
  cudaLaunchConfig_t c = {};
  const int64_t tiles = p.offsets ? (int64_t)p.rows / N + std::min<int64_t>(p.n_experts, p.rows)
                                  : ((int64_t)p.rows + N - 1) / N;
  const int64_t jobs = tiles * ((p.n + kRows - 1) / kRows);
  OP_ARG(jobs < ((int64_t)1 << 28), op, "too many rows for one call");
  p.most_jobs = (int32_t)jobs;
  c.gridDim = dim3((unsigned)(T::kStay ? std::min<int64_t>(jobs, sms) : jobs * p.splits));
  c.blockDim = dim3(T::kThreads);
  c.dynamicSmemBytes = T::kSmem;
  c.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = p.splits > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, xmap, wmap, p);
  return e == cudaSuccess ? TRE_OK : op_cuda_error(op, cudaGetErrorString(e));
}

// Rows of x per tile: the least of 16 .. 256 that covers three times an expert's average, so that
// few experts' weights are decoded twice.  Measured, 64 experts of 2048 x 7168 with a skewed
// spread, against twice and once the average: 1024 rows 141, 160 and 240 us, 2048 rows 167, 181
// and 241; but 4096 rows 303, 221 and 251, where it is the 256-row tile that loses.  No more than
// leaves the device without tiles to fill it, though never below 64: 512 rows of one such matrix
// 34.9 us against 50.2 with tiles of 32, which split k; but 33 to 256 rows 33 us against 16 to 31.
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
                 (int32_t)rows, (int32_t)n, (int32_t)k, n_experts, 1, 0, 4u, ops_status_ptr()};
  if (!p.status) return op_cuda_error(op, "the operators' status word is not available");
  const int tile = tile_rows(p, sms);
  // Few tiles: split k over a cluster until the device is busy.  Rows count as if they lay
  // together; spread over experts they make up to n_experts tiles more, and each part has a start
  // and an end: 8 rows over 64 experts of 2048 x 7168 45 us, 64 rows 137; with the tiles that there
  // can be 29 and 94, from 256 rows on the same.
  if (tile <= 32) {
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
               ? launch<N, __nv_bfloat16>(op, p, xmap, wmap, sms, (cudaStream_t)stream)       \
               : launch<N, float>(op, p, xmap, wmap, sms, (cudaStream_t)stream)
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
