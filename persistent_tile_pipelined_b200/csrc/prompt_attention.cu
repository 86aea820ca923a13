// Causal attention of packed prompts (declared in include/tre.h as tre_prompt_attention).
//
// One CTA takes 256 rows of one key/value head's query group: row r of a sequence is query
// token r / g, head r mod g of the group, so grouped heads share every key and value tile and
// a single token of a large group still fills matrix rows.  The rows are two tiles of 128,
// each with its scores S (fp32, tensor memory), its probabilities P (bf16, over the first half
// of S) and its output sums O (fp32, tensor memory).  Per 128 keys and tile:
//   S = Q K^T (operands in shared memory);  a warpgroup, one thread per row, takes the row's
//   maximum, P = 2^(S c - m) and the row's sum;  O += P V (P read from tensor memory).
// While one tile is in its softmax the matrix unit works on the other.  The running maximum is
// only raised, and O rescaled, when it grows by more than 2^8: P then stays below 2^8, which
// costs bf16 P and fp32 sums no precision, and the rescaling all but disappears.
//
// Rows are q token by q token, so that a tile of 256 rows is 256 / g tokens and the part of the
// last key tiles that causal rows do not see stays small; the grid starts with the last rows,
// which take longest.  A lone row tile (128 rows or fewer: one token, a short chunk) would
// wait for its own softmax at every step, so two warpgroups take it with the even and the odd
// key tiles; few rows over many keys are further split over CTAs and joined by a second kernel.
//
// What bounds it.  Per row tile and 128 keys of width 128 the two products take 1024 clocks of
// the matrix unit, the 16384 exponentials 1024 of the special-function unit; the chain softmax ->
// P V -> next S of a tile measures 3150 clocks for the two tiles (1040 of them waiting for S, 450
// for the maximum, 1180 for the exponentials), an item's start and end about 13000 more.
// Measured, B200: 8192 tokens, 32 / 8 heads of 128: 508-516 us, 1065-1080 TFLOP/s of the causal
// half (0.67 of the measured 1615, 0.78 of the 1378 that the power cap sustains); eight packed
// prompts of 1 to 1500 tokens, 64 / 8 heads: 160-162 us; one token over 131072 keys: 96 us (90 in a
// graph, 6.0 TB/s, 0.91 of the measured copy rate).
// Tried and slower: three eighths or half of the exponentials on the multiply-add units (597 and
// 579 us against 549 with a quarter); the first half of P by the old maximum (566 against 545);
// resident CTAs that take the next item while one ends (872 against 526).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "tc.cuh"
#include "tensor_map.h"

namespace tre {
namespace {

constexpr int kTile = 128;                     // rows of a tile, keys of a step
constexpr int kItemRows = 2 * kTile;           // rows per CTA
constexpr int kCopyWarp = 8, kMmaWarp = 9, kFixWarp = 10, kFixWarps = 2;
constexpr int kThreadsAttn = 384;
constexpr float kRaise = 8.f;                  // log2 of how far P may exceed 1
constexpr float kFar = 67108864.f;             // 2^26, see rest_of
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Shape {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int ST = D == 128 ? 5 : 10;  // key and value tiles in flight (one more
                                                // where the second row tile's q is not needed)
  static constexpr int kSmem = (2 + ST) * kTileBytes + 1024 + 512;
  static constexpr int kO = 2 * kTile;          // tensor-memory column of the first O
};

// Division by a number that the host knows, of numbers below 2^31: inv is ceil(2^32 / d) (0 for
// 1), whose quotient is at most one too large.
struct Divisor {
  uint32_t d, inv;
};

__device__ __forceinline__ int quotient(int n, Divisor d) {
  uint32_t q = d.inv ? __umulhi((uint32_t)n, d.inv) : (uint32_t)n;
  if (q * d.d > (uint32_t)n) --q;
  return (int)q;
}

struct AttnParams {
  tre_attention a;
  Divisor group, kv_heads;  // query heads of a kv head; kv heads
  const __nv_bfloat16* q;
  const __nv_bfloat16 *k, *v;  // the slow path's view of what the tensor maps describe
  __nv_bfloat16* out;
  const int32_t *q_offsets, *kv_offsets;
  float* part_o;       // [splits][n_q_rows * Hq][D]
  float2* part_ml;     // [splits][n_q_rows * Hq]: maximum of q . k, sum (sum -1: no key seen)
  int32_t tiles;       // upper bound of the row tiles of a kv head
  int32_t splits;
  float c;             // scale * log2(e)
  int32_t* status;
};

// Work of one CTA: rows [row0, row0 + rows) of sequence rows q0 .. (nq tokens), keys k0 ..
struct Item {
  int q0, nq, k0, nk, row0, rows;
};

// The y-th row tile over all sequences (whole warp); rows = 0 when there is none.
__device__ Item find_item(const AttnParams& p, int g, int y) {
  const int lane = threadIdx.x & 31;
  Item it{0, p.a.n_q_rows, 0, p.a.n_kv_rows, 0, 0};
  if (p.a.n_seqs == 0) {
    it.row0 = y * kItemRows;
  } else {
    bool found = false;
    for (int i0 = 0; i0 < p.a.n_seqs && !found; i0 += 32) {
      const int i = i0 + lane;
      int qa = 0, qb = 0;
      if (i < p.a.n_seqs) {
        qa = min(max(p.q_offsets[i], 0), p.a.n_q_rows);
        qb = min(max(p.q_offsets[i + 1], 0), p.a.n_q_rows);
      }
      const int tiles = qb > qa ? (int)(((int64_t)(qb - qa) * g + kItemRows - 1) / kItemRows) : 0;
      int sum = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      const uint32_t mine = __ballot_sync(0xffffffffu, sum > y);
      if (mine) {
        const int l = __ffs(mine) - 1;
        found = true;
        it.row0 = (y - __shfl_sync(0xffffffffu, sum - tiles, l)) * kItemRows;
        it.q0 = __shfl_sync(0xffffffffu, qa, l);
        it.nq = __shfl_sync(0xffffffffu, qb, l) - it.q0;
        it.k0 = min(max(p.kv_offsets[i0 + l], 0), p.a.n_kv_rows);
        it.nk = max(min(max(p.kv_offsets[i0 + l + 1], 0), p.a.n_kv_rows) - it.k0, 0);
      } else {
        y -= __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    if (!found) return it;
  }
  const int64_t left = (int64_t)it.nq * g - it.row0;
  it.rows = left > kItemRows ? kItemRows : left > 0 ? (int)left : 0;
  return it;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of three; NaN if any is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^x of two numbers below 128 on the fused multiply-add units: x = i + f with |f| <= 1/2,
// 2^f by a cubic whose relative error is at most 1.02e-4 (below 2^-13; its constant
// is 1, so that x <= -127 gives exact zero), i added to the exponent bits.  Not for NaN.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  const float2 magic = make_float2(12582912.f, 12582912.f);  // 1.5 x 2^23: x rounds to i
  const float2 minus = make_float2(-12582912.f, -12582912.f);
  const float2 none = make_float2(-1.f, -1.f);
  x.x = fmaxf(x.x, -127.f);
  x.y = fmaxf(x.y, -127.f);
  const float2 t = tc::add2(x, magic);
  const float2 f = tc::fma2(tc::add2(t, minus), none, x);
  float2 q = tc::fma2(f, make_float2(0.05500893f, 0.05500893f),
                      make_float2(0.24221096f, 0.24221096f));
  q = tc::fma2(q, f, make_float2(0.69328293f, 0.69328293f));
  q = tc::fma2(q, f, make_float2(1.f, 1.f));
  return make_float2(
      __uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23)),
      __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23)));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row's exponentials are relative to its maximum m (a product q . k) times c = scale log2(e).
// fl(m c) alone is off by up to half a unit in its last place, the same for every key of the row:
// up to kFar a factor of at most 4 that P and its sum share; from 2^31 on an overflow, or nothing
// but zeros.  Beyond kFar the rest of the product, exact in fp32, is taken off as well.
__device__ __forceinline__ bool is_far(float mc) { return fabsf(mc) > kFar && mc > -INFINITY; }

__device__ __forceinline__ float rest_of(float m, float c) {
  const float mc = __fmul_rn(m, c);
  return is_far(mc) ? fmaf(m, c, -mc) : 0.f;
}

// 2^((from - to) c) as the rows' exponentials have it, from <= to; 0 when from is -infinity (no
// score yet).  (Far maxima branch away: code that runs once waits for every line of it.)
__device__ __forceinline__ float share_of(float from, float to, float c) {
  const float a = __fmul_rn(from, c), b = __fmul_rn(to, c);
  float d = a - b;
  if (__builtin_expect(fmaxf(fabsf(a), fabsf(b)) > kFar, 0))
    d = from == -INFINITY ? -INFINITY : d + (rest_of(from, c) - rest_of(to, c));
  return exp2_approx(d);
}

// Where a row's result goes: the output, or its part [split] when the keys are split.
struct RowOut {
  __nv_bfloat16* out;
  float* o;
  float2* ml;
};

__device__ __forceinline__ RowOut row_out(const AttnParams& p, int D, int split, int tok, int h) {
  const int64_t at = ((int64_t)split * p.a.n_q_rows + tok) * p.a.n_q_heads + h;
  return {p.out + (int64_t)tok * p.a.out_row_stride + (int64_t)h * p.a.out_head_stride,
          p.part_o + at * D, p.part_ml + at};
}

// One row the long way, by one warp: keys [from, to) of the sequence in order, the lanes
// sharing the width.  Taken by every row of a CTA whose partly visible key tiles hold a NaN or
// an infinity in v: the matrix product would carry 0 x NaN into rows that do not see the key.
// Right, but slow: 8192 tokens, 32 / 8 heads of 128 take 0.44 ms without such a value, 63 ms with
// one at key 4000 of one head and 442 ms with one at every 64th key of all.
template <int D>
__device__ __forceinline__ void slow_row(const AttnParams& p, int split, int tok, int h, int k0,
                                         int from, int to, int see) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, kh = quotient(h, p.group);
  const __nv_bfloat16* qr =
      p.q + (int64_t)tok * p.a.q_row_stride + (int64_t)h * p.a.q_head_stride + lane;
  const __nv_bfloat16* k = p.k + (int64_t)kh * p.a.k_head_stride + lane;
  const __nv_bfloat16* v = p.v + (int64_t)kh * p.a.v_head_stride + lane;
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(qr[32 * e]), acc[e] = 0.f;
#pragma unroll 1
  for (int s = from; s < to; ++s) {
    const int64_t at = k0 + s;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      x = fmaf(q[e], __bfloat162float(k[at * p.a.k_row_stride + 32 * e]), x);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float mn = fmaxf(m, x), old = share_of(m, mn, p.c);
    const float to = mn == -INFINITY ? 0.f : mn;
    const float w = exp2_approx(fmaf(x, p.c, -__fmul_rn(to, p.c)) - rest_of(to, p.c));
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = fmaf(w, __bfloat162float(v[at * p.a.v_row_stride + 32 * e]), acc[e] * old);
    l = fmaf(l, old, w);
    m = mn;
  }
  const RowOut r = row_out(p, D, split, tok, h);
  if (p.splits > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) r.o[lane + 32 * e] = acc[e];
    if (lane == 0) *r.ml = make_float2(m, to > from ? l : -1.f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      r.out[lane + 32 * e] = __float2bfloat16_rn(see > 0 ? acc[e] / l : 0.f);
  }
}

// The barriers behind the tiles in shared memory: `full` and, ST + 1 further, `empty` of the
// ring's places, then these.
enum {
  kBarQ = 0,
  kBarS = 2,
  kBarHalf = 4,  // the first half of P is there
  kBarP = 6,
  kBarO = 8,
  kBarFixed = 10,
  kBarCheck = 11,
  kBarDrained = 12
};

// The matrix products of key tiles [kb, ke) by one thread; n0, n1: the row tiles' key tiles.
// kAlternate: key tile i belongs to row tile (i - kb) mod 2, whose S runs two key tiles ahead of
// its O; else both row tiles take every key tile, S one ahead.
template <int D, bool kAlternate>
__device__ __forceinline__ void issue_products(uint8_t* qs, uint64_t* full, uint64_t* bars,
                                               uint32_t tmem, int kb, int ke, int n0, int n1,
                                               int least, volatile int* gave_up) {
  using T = Shape<D>;
  constexpr uint32_t id_s = tc::idesc_bf16(kTile, kTile, 0);
  constexpr uint32_t id_o = tc::idesc_bf16(kTile, D, 1);
  constexpr int kPlaces = kAlternate ? T::ST + 1 : T::ST, kAhead = kAlternate ? 2 : 1;
  uint64_t* empty = full + T::ST + 1;
  const uint32_t ring = smem_u32(qs + (kAlternate ? 1 : 2) * T::kTileBytes);
  const int total = ke - kb;
  const int count[2] = {n0 - kb, n1 - kb};
  auto takes = [&](int sub, int i) {
    return i < count[sub] && (!kAlternate || (i & 1) == sub);
  };
  auto arrived = [&](int n) {
    return tc::wait(full + n % kPlaces, n / kPlaces & 1, gave_up);
  };
  auto scores = [&](int sub, int n) {
    const uint32_t q = smem_u32(qs) + (kAlternate ? 0 : sub * T::kTileBytes);
    const uint32_t k = ring + n % kPlaces * T::kTileBytes;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const uint32_t at = (j / 4) * kTile * 128 + (j % 4) * 32;
      tc::mma_ss(tmem + sub * kTile, tc::smem_desc(q + at, 16, 1024),
                 tc::smem_desc(k + at, 16, 1024), id_s, j > 0);
    }
    tc::commit(bars + kBarS + sub);
  };
  auto outputs = [&](int sub, int n, bool add, int half) {
    const uint32_t v = ring + n % kPlaces * T::kTileBytes;
#pragma unroll
    for (int j = half * kTile / 32; j < (half + 1) * kTile / 32; ++j)
      tc::mma_ts(tmem + T::kO + sub * D, tmem + sub * kTile + j * 8,
                 tc::smem_desc(v + j * 2048, kTile * 128, 1024), id_o, add || j > 0);
    if (half) tc::commit(bars + kBarO + sub);
  };
  for (int i = 0; i < min(kAhead, total); ++i) {
    if (!arrived(2 * i)) return;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if (!takes(sub, i)) continue;
      if (!tc::wait(bars + kBarQ + (kAlternate ? 0 : sub), 0, gave_up)) return;
      tc::fence_after();
      scores(sub, 2 * i);
    }
    tc::commit(empty + 2 * i % kPlaces);
  }
  int fixed = 0;
  for (int i = 0; i < total; ++i) {
    const int nv = 2 * i + 1, next = i + kAhead, nk = 2 * next;
    if (!arrived(nv)) return;
    const bool partly = (kb + i + 1) * kTile > least;
    if (partly) mbar_arrive(bars + kBarCheck);
    const int round = kAlternate ? i >> 1 : i;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if (!takes(sub, i)) continue;
      if (!tc::wait(bars + kBarHalf + sub, round & 1, gave_up)) return;
      if (partly && !tc::wait(bars + kBarFixed, fixed & 1, gave_up)) return;
      tc::fence_after();
      outputs(sub, nv, round > 0, 0);
      if (!tc::wait(bars + kBarP + sub, round & 1, gave_up)) return;
      tc::fence_after();
      outputs(sub, nv, true, 1);
      if (takes(sub, next)) {
        if (!arrived(nk)) return;
        scores(sub, nk);
      }
    }
    fixed += partly;
    tc::commit(empty + nv % kPlaces);
    if (next < total) tc::commit(empty + nk % kPlaces);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsAttn, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const AttnParams p) {
  using T = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(qs + (2 + T::ST) * T::kTileBytes);
  uint64_t* empty = full + T::ST + 1;
  uint64_t* q_full = empty + T::ST + 1;
  uint64_t* s_full = q_full + kBarS;
  uint64_t* p_half = q_full + kBarHalf;
  uint64_t* p_full = q_full + kBarP;
  uint64_t* o_done = q_full + kBarO;
  uint64_t* v_fixed = q_full + kBarFixed;
  uint64_t* v_check = q_full + kBarCheck;
  uint64_t* drained = q_full + kBarDrained;
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up, poison;
  __shared__ Item item;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = (int)p.group.d;
  const int place = quotient(blockIdx.x, p.kv_heads);  // of the row tile, from the last
  const int kh = (int)blockIdx.x - place * p.a.n_kv_heads;

  if (warp == 0) {
    // the last row tiles first: with causal rows they take longest
    const Item it = find_item(p, g, p.tiles - 1 - place);
    if (lane == 0) {
      item = it;
      gave_up = 0;
      poison = 0;
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < T::ST + 1; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 4);
      mbar_init(s_full + i, 1);
      mbar_init(p_half + i, 4);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
    }
    mbar_init(v_fixed, kFixWarps);
    mbar_init(v_check, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
  } else if (warp == kCopyWarp && lane == 0 && p.a.n_kv_rows > 0) {
    tc::prefetch_map(&kmap);
    tc::prefetch_map(&vmap);
  } else if (warp == kMmaWarp) {
    tc::tmem_alloc(&tmem_base, 512);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  const Item it = item;
  if (it.rows == 0) {
    if (warp == kMmaWarp) tc::tmem_free(tmem, 512);
    return;
  }

  // keys that a row sees: it.nk - it.nq + (row / g) + 1, not below 0
  auto sees = [&](int row) { return max(it.nk - it.nq + quotient(row, p.group) + 1, 0); };
  const int subs = it.rows > kTile ? 2 : 1;
  const int least = sees(it.row0);  // of the CTA's rows
  int n_sub[2];                     // key tiles of each row tile
  n_sub[0] = (sees(it.row0 + min(it.rows, kTile) - 1) + kTile - 1) / kTile;
  n_sub[1] = subs == 2 ? (sees(it.row0 + it.rows - 1) + kTile - 1) / kTile : 0;
  const int n_all = max(n_sub[0], n_sub[1]);
  const int split = blockIdx.y;
  // (below 2^24 tiles and 2^8 parts: the products fit 32 bits)
  const int kb = p.splits == 1 ? 0 : (int)((uint32_t)n_all * (uint32_t)split / (uint32_t)p.splits);
  const int ke = p.splits == 1 ? n_all
                               : (int)((uint32_t)n_all * (split + 1u) / (uint32_t)p.splits);
  // One row tile alone would wait for its own softmax at every step: both take it, with the
  // even and the odd key tiles, and join their sums at the end.
  const bool alternate = subs == 1;
  n_sub[0] = min(n_sub[0], ke);
  n_sub[1] = alternate ? n_sub[0] : min(n_sub[1], ke);

  uint8_t* ring = qs + (alternate ? 1 : 2) * T::kTileBytes;
  // places of the ring: K and V tiles take them in turn
  const int places = alternate ? T::ST + 1 : T::ST;

  // Registers: 384 threads x 168 at launch; the softmax warps hold a row of scores (256 x 208)
  // and the others give theirs up (128 x 80).
  if (warp >= kCopyWarp) tc::regs_less<80>();
  if (warp == kCopyWarp) {
    if (tc::elect_one()) {
      int n = 0, slot = 0, phase = 0;
      const int total = 2 * (ke - kb);
      for (; n < total; ++n) {
        if (!tc::wait(empty + slot, phase ^ 1, &gave_up)) break;
        uint8_t* dst = ring + slot * T::kTileBytes;
        mbar_arrive_expect_tx(full + slot, T::kTileBytes);
        const int row = it.k0 + (kb + n / 2) * kTile;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tc::load_3d(dst + h * kTile * 128, n & 1 ? &vmap : &kmap, h * 64, row, kh, full + slot);
        if (++slot == places) slot = 0, phase ^= 1;
      }
      tc::settle_copies(full, n, places, clock64());
    }
  } else if (warp == kMmaWarp) {
    if (tc::elect_one()) {
      if (alternate)
        issue_products<D, true>(qs, full, q_full, tmem, kb, ke, n_sub[0], n_sub[1], least,
                                &gave_up);
      else
        issue_products<D, false>(qs, full, q_full, tmem, kb, ke, n_sub[0], n_sub[1], least,
                                 &gave_up);
      tc::commit(drained);
      tc::settle(drained, 0, clock64());
    }
  } else if (warp >= kFixWarp) {
    // Key tiles that some row sees only in part: values of keys behind the sequence become
    // zero (P is zero there, and 0 x NaN is not), others are looked through for NaN and
    // infinities.
    uint32_t bad = 0;
    int checked = 0;
    for (int i = max(kb, least / kTile); i < ke; ++i) {
      // the product's thread says when the tile is there (a wait on the tile's own barrier
      // could mistake an earlier round of the ring for this one)
      if (!tc::wait_warp(v_check, checked++ & 1, &gave_up)) break;
      uint8_t* v = ring + (2 * (i - kb) + 1) % places * T::kTileBytes;
      constexpr int kLanes = D / 8, kRowsAtOnce = kFixWarps * 32 / kLanes;
      const int t64 = threadIdx.x - kFixWarp * 32, ch = t64 % kLanes;
      const int from = max(least - i * kTile, 0) / kRowsAtOnce * kRowsAtOnce;
      v += (ch >> 3) * kTile * 128 + (ch & 7) * 16;
#pragma unroll 8
      for (int j = from + t64 / kLanes; j < kTile; j += kRowsAtOnce) {
        uint4* at = reinterpret_cast<uint4*>(v + j * 128);
        if (i * kTile + j >= it.nk) {
          *at = make_uint4(0, 0, 0, 0);
        } else {
          const uint4 x = *at;
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)  // an exponent of ones carries into the sign's place
            bad |= (w[e] & 0x7f807f80u) + 0x00800080u;
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_fixed);
    }
    if (bad & 0x80008000u) poison = 1;
  } else {
    tc::regs_more<208>();
    const int sub = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
    const int base = alternate ? 0 : sub * kTile;  // of the item's rows
    const int row = it.row0 + base + r;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_addr = lane_addr + sub * kTile, o_addr = lane_addr + T::kO + sub * D;
    const int n_mine = sub == 0 ? n_sub[0] : n_sub[1];
    if (sub < subs && kb < n_mine) {
      // this tile's rows of q, 16 bytes a lane, swizzled; rows that do not exist are zero
      constexpr int kChunks = D / 8, kPass = kTile / kChunks;
      const int ch = r % kChunks, r8 = r / kChunks;
      const int at = it.row0 + sub * kTile + r8, dt = quotient(kPass, p.group), dh = kPass - dt * g;
      int tk = quotient(at, p.group), hd = at - tk * g;
      const __nv_bfloat16* src = p.q + (int64_t)kh * g * p.a.q_head_stride + ch * 8;
      const uint32_t dst = smem_u32(qs) + sub * T::kTileBytes + (ch >> 3) * kTile * 128;
#pragma unroll
      for (int x = 0; x < kChunks; ++x) {
        // past L1, which beside this much shared memory holds less than the rows in flight
        const int rr = r8 + x * kPass;
        const bool there = sub * kTile + rr < it.rows;
        tc::copy16(dst + rr * 128 + (((ch & 7) ^ (rr & 7)) * 16),
                   src + (there ? (int64_t)(it.q0 + tk) * p.a.q_row_stride +
                                      (int64_t)hd * p.a.q_head_stride
                                : 0),
                   there);
        tk += dt;
        hd += dh;
        if (hd >= g) hd -= g, ++tk;
      }
      tc::copy16_wait();
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + sub);
    }
    const bool mine = base + r < it.rows;
    const bool any_row = base + quad * 32 < it.rows;  // of the warp's
    const int see = mine ? sees(row) : 0;
    const int sub_least = sees(it.row0 + base);
    const int step = alternate ? 2 : 1;
    const float c = p.c;
    float m = -INFINITY, l = 0.f;  // the row's maximum (of q . k) and sum
    float limit = -INFINITY;  // of a tile's maximum times c: above it m is looked at; NaN: always
    float factor = c, shift = 0.f;  // exponent = what s holds * factor - shift
    bool ok = true;
    int round = 0;
    for (int i = kb + (alternate ? sub : 0); i < n_mine; i += step, ++round) {
      ok = tc::wait_warp(s_full + sub, round & 1, &gave_up);
      if (!ok) break;
      if (!any_row) {  // rows that do not exist: whatever lies in P stays in their sums
        if (lane == 0) {
          mbar_arrive(p_half + sub);
          mbar_arrive(p_full + sub);
        }
        continue;
      }
      tc::fence_after();
      uint32_t s[kTile];
#pragma unroll
      for (int x = 0; x < kTile; x += 32) tc::tmem_ld32(s_addr + x, s + x);
      tc::wait_ld();
      if ((i + 1) * kTile > sub_least) {
        const int lim = see - i * kTile;
#pragma unroll
        for (int x = 0; x < kTile; ++x)
          if (x >= lim) s[x] = 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < kTile; x += 8)
#pragma unroll
        for (int y = 0; y < 4; ++y)
          mx[y] = max3_nan(mx[y], __uint_as_float(s[x + 2 * y]), __uint_as_float(s[x + 2 * y + 1]));
      float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], -INFINITY);
      // a NaN or an infinite score makes the row NaN (infinity less itself): by its sum, since
      // the exponentials below need not carry it
      float top_c = __fmul_rn(top, c);
      if (!(top_c < INFINITY)) l = NAN, top = top_c = -INFINITY;
      if (__any_sync(0xffffffffu, !(top_c <= limit) || round == 0)) {
        top = fmaxf(m, top);
        top_c = __fmul_rn(top, c);
        const bool far = is_far(top_c);
        const bool up = __any_sync(0xffffffffu, top_c > __fmul_rn(m, c) + kRaise ||
                                                    (far && top > m) || round == 0);
        const float f = up ? share_of(m, top, c) : 1.f;
        if (up) m = top;
        l *= f;
        if (up && round > 0) {
          ok = tc::wait_warp(o_done + sub, (round - 1) & 1, &gave_up);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int x = 0; x < D; x += 32) {
            uint32_t o[32];
            tc::tmem_ld32(o_addr + x, o);
            tc::wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tc::tmem_st32(o_addr + x, o);
          }
        }
        const float mc = __fmul_rn(m, c);
        shift = m == -INFINITY ? 0.f : mc;
        factor = c;
        limit = fminf(mc + kRaise, kFar);
        if (__any_sync(0xffffffffu, far)) {  // the exponents themselves
          const float rest = rest_of(m, c);
#pragma unroll
          for (int x = 0; x < kTile; ++x)
            s[x] = __float_as_uint(fmaf(__uint_as_float(s[x]), c, -shift) - rest);
          factor = 1.f;
          shift = 0.f;
          limit = NAN;
        }
      }
      const float2 cc = make_float2(factor, factor), ms = make_float2(-shift, -shift);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int x = 0; x < kTile; x += 64) {
        uint32_t pk[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          float2 e = tc::fma2(make_float2(__uint_as_float(s[x + 2 * y]),
                                          __uint_as_float(s[x + 2 * y + 1])), cc, ms);
          // a quarter of them on the multiply-add units: the special-function unit alone (16 a
          // clock) takes as long as both matrix products of the tile
          e = (y & 3) == 3 ? exp2_poly(e) : make_float2(exp2_approx(e.x), exp2_approx(e.y));
          sum[y & 1] = tc::add2(sum[y & 1], e);
          pk[y] = pack_bf16(e.x, e.y);
        }
        tc::tmem_st32(s_addr + x / 2, pk);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive((x == 0 ? p_half : p_full) + sub);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    // `round` key tiles are in the row's m, l and O
    if (ok && round > 0) ok = tc::wait_warp(o_done + sub, (round - 1) & 1, &gave_up);
    tc::fence_after();
    asm volatile("bar.sync 2, %0;" ::"n"(256 + 32 * kFixWarps) : "memory");  // poison is known
    float* other_o = reinterpret_cast<float*>(qs);  // [D][128], the products are done with q
    float2* other_ml = reinterpret_cast<float2*>(qs + 2 * T::kTileBytes);
    if (alternate) {
      if (sub == 1) {
        if (round > 0 && any_row && ok) {
#pragma unroll 1
          for (int x = 0; x < D; x += 32) {
            uint32_t o[32];
            __syncwarp();
            tc::tmem_ld32(o_addr + x, o);
            tc::wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) other_o[(x + y) * kTile + r] = __uint_as_float(o[y]);
          }
        }
        other_ml[r] = make_float2(m, round > 0 ? l : -1.f);
      }
      asm volatile("bar.sync 3, 256;" ::: "memory");
    }
    const bool slow = poison != 0;
    const int tok0 = quotient(row, p.group), tok = it.q0 + tok0, h = kh * g + row - tok0 * g;
    if (sub < subs && ok && any_row) {
      if (slow) {
#pragma unroll 1
        for (int x = 0; x < 32; ++x) {
          const int rx = row - lane + x, sx = sees(rx);
          if (rx - it.row0 >= it.rows) break;
          const int tx = quotient(rx, p.group);
          slow_row<D>(p, split, it.q0 + tx, kh * g + rx - tx * g, it.k0, min(kb * kTile, sx),
                      min(ke * kTile, sx), sx);
        }
      } else {
        const RowOut dst = row_out(p, D, split, tok, h);
        // (a lone row tile's q place holds the other half's sums)
        uint8_t* stage = alternate ? qs + 3 * T::kTileBytes : qs + sub * T::kTileBytes;
        float f0 = 1.f, f1 = 0.f;  // this tile's share and the other's
        if (alternate) {
          const float2 ml = other_ml[r];
          if (ml.y != -1.f) {
            const float both = fmaxf(m, ml.x);
            f0 = share_of(m, both, p.c);
            f1 = share_of(ml.x, both, p.c);
            m = both;
            l = fmaf(ml.y, f1, l * f0);
          }
        }
        const bool joined = alternate && n_mine - kb > 1;
        const float inv = see > 0 ? 1.f / l : 0.f;
#pragma unroll
        for (int x = 0; x < D; x += 32) {
          uint32_t o[32];
          if (round > 0) {
            __syncwarp();
            tc::tmem_ld32(o_addr + x, o);
            tc::wait_ld();
          }
          if (joined)
#pragma unroll
            for (int y = 0; y < 32; ++y)
              o[y] = __float_as_uint(fmaf(other_o[(x + y) * kTile + r], f1,
                                          __uint_as_float(o[y]) * f0));
          if (round == 0 || see == 0)
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = 0;
          if (p.splits == 1) {
            // through shared memory (this row tile's q is done with, or the other's), 16 bytes
            // a chunk, so that rows leave whole
            uint4* row_out = reinterpret_cast<uint4*>(stage + r * D * 2);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                w[z] = pack_bf16(__uint_as_float(o[8 * y + 2 * z]) * inv,
                                 __uint_as_float(o[8 * y + 2 * z + 1]) * inv);
              row_out[(x / 8 + y) ^ (r & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (mine) {
            uint4* out = reinterpret_cast<uint4*>(dst.o + x);
#pragma unroll
            for (int y = 0; y < 8; ++y)
              out[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            if (x == 0) *dst.ml = make_float2(m, see > kb * kTile && kb < ke ? l : -1.f);
          }
        }
        if (p.splits == 1) {
          __syncwarp();
          constexpr int kChunks = D / 8, kRows2 = 32 / kChunks;  // rows of a store
          const int ch = lane % kChunks;
#pragma unroll 4
          for (int x = 0; x < 32; x += kRows2) {
            const int rr = x + lane / kChunks;  // of the warp's
            const uint64_t to = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst.out), rr);
            const uint4 val = reinterpret_cast<const uint4*>(
                stage + (quad * 32 + rr) * D * 2)[ch ^ (rr & 7)];
            if (base + quad * 32 + rr < it.rows) reinterpret_cast<uint4*>(to)[ch] = val;
          }
        }
      }
    }
  }
  if (warp >= kFixWarp) asm volatile("bar.sync 2, %0;" ::"n"(256 + 32 * kFixWarps) : "memory");
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc::fence_after();
    tc::tmem_free(tmem, 512);
  }
  if (threadIdx.x == 0 && gave_up) atomicExch(p.status, TRE_ERR_DEP_TIMEOUT);
}

// Joins the parts of the rows of one item, a warp per row.  Lane s reads the maximum and sum of
// part s (and s + 32, ...), so that the parts' shares are known after one wait; then the parts
// are added in order, several loads in flight.  Its launch and the search for its item overlap
// the end of the first kernel, which it then waits for: a programmatic launch, which the first
// kernel lets go only when its last CTA ends.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p) {
  const int g = (int)p.group.d, place = quotient(blockIdx.x, p.kv_heads);
  const int kh = (int)blockIdx.x - place * p.a.n_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Item it = find_item(p, g, place);
  const int rr = blockIdx.y * 8 + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (rr >= it.rows) return;
  const int row = it.row0 + rr, tok0 = quotient(row, p.group);
  const int tok = it.q0 + tok0, h = kh * g + row - tok0 * g;
  const int64_t step = (int64_t)p.a.n_q_rows * p.a.n_q_heads;
  const int64_t at = (int64_t)tok * p.a.n_q_heads + h;
  float m = -INFINITY;
  bool seen = false;
  for (int s = lane; s < p.splits; s += 32) {
    const float2 ml = p.part_ml[s * step + at];
    seen |= ml.y != -1.f;
    m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  seen = __any_sync(0xffffffffu, seen);
  constexpr int E = D / 32;
  float l = 0.f, acc[E] = {};
  for (int s0 = 0; s0 < p.splits; s0 += 32) {
    float share = 0.f, sum = 0.f;  // of part s0 + lane; none without a finite maximum
    if (s0 + lane < p.splits) {
      const float2 ml = p.part_ml[(s0 + lane) * step + at];
      if (ml.x != -INFINITY) {
        share = share_of(ml.x, m, p.c);
        sum = ml.y * share;
      }
      if (ml.y != ml.y) sum = ml.y;
    }
    const int count = min(32, p.splits - s0);
#pragma unroll 8
    for (int s = 0; s < count; ++s) {
      const float f = __shfl_sync(0xffffffffu, share, s);
      l += __shfl_sync(0xffffffffu, sum, s);
      const float* o = p.part_o + ((s0 + s) * step + at) * D;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(o[lane + 32 * e], f, acc[e]);
    }
  }
  __nv_bfloat16* out =
      p.out + (int64_t)tok * p.a.out_row_stride + (int64_t)h * p.a.out_head_stride;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = __float2bfloat16_rn(seen ? acc[e] / l : 0.f);
}

tre_status check(const char* op, const tre_attention* a) {
  OP_ARG(a, op, "NULL argument");
  OP_ARG(a->head_dim == 64 || a->head_dim == 128, op, "head_dim must be 64 or 128");
  OP_ARG(a->n_kv_heads >= 1 && a->n_kv_heads <= 65535 && a->n_q_heads >= 1 &&
             a->n_q_heads <= 65535 && a->n_q_heads % a->n_kv_heads == 0,
         op, "n_q_heads must be a positive multiple of n_kv_heads");
  OP_ARG(a->n_seqs >= 0 && a->n_seqs < (1 << 20), op, "n_seqs out of range");
  OP_ARG(a->n_q_rows >= 0 && a->n_kv_rows >= 0, op, "negative row count");
  OP_ARG((int64_t)a->n_q_rows * a->n_q_heads <= ((int64_t)1 << 30) &&
             a->n_kv_rows <= (1 << 30),
         op, "more than 2^30 rows");
  OP_ARG(a->scale > 0.f && a->scale * kLog2e < INFINITY, op,
         "scale must be positive and scale log2(e) finite");
  const struct {
    int64_t stride;
    int count;  // a dimension of one entry is never stepped over
  } dims[] = {{a->q_row_stride, a->n_q_rows},     {a->q_head_stride, a->n_q_heads},
              {a->k_row_stride, a->n_kv_rows},    {a->k_head_stride, a->n_kv_heads},
              {a->v_row_stride, a->n_kv_rows},    {a->v_head_stride, a->n_kv_heads},
              {a->out_row_stride, a->n_q_rows},   {a->out_head_stride, a->n_q_heads}};
  for (const auto& d : dims)
    OP_ARG(d.count <= 1 || (d.stride >= a->head_dim && d.stride % 8 == 0 &&
                            d.stride < ((int64_t)1 << 38)),
           op, "rows and heads must lie apart by whole 16-byte units");
  OP_ARG(a->n_q_rows <= 1 || a->n_q_heads <= 1 ||
             a->out_row_stride >= (a->n_q_heads - 1) * a->out_head_stride + a->head_dim ||
             a->out_head_stride >= (a->n_q_rows - 1) * a->out_row_stride + a->head_dim,
         op, "output rows and heads overlap");
  return TRE_OK;
}


Divisor divisor(int d) {
  return {(uint32_t)d,
          d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + (uint64_t)d - 1) / (uint64_t)d)};
}

// Row tiles of a kv head: an upper bound, the lengths are known on the device only.
int row_tiles(const tre_attention& a) {
  const int64_t rows = (int64_t)a.n_q_rows * (a.n_q_heads / a.n_kv_heads);
  if (a.n_seqs == 0) return (int)((rows + kItemRows - 1) / kItemRows);
  return (int)(rows / kItemRows + std::min(a.n_seqs, a.n_q_rows));
}

// Parts along the keys: as many as fill the device when the rows alone do not, each of two
// key tiles or more.  Measured, 32 / 8 heads of 128 over 32768 keys: 512 tokens (64 items, two
// parts) 238 us.  From half a device of items on there is one part: 1024 tokens (128 items) 433 us
// against 477 with three, but 640 tokens (80 items) 424 against 322, and 1280 (160 items) 819
// against 670 with two.
int key_splits(const tre_attention& a, int sms) {
  const int64_t items = (int64_t)row_tiles(a) * a.n_kv_heads;
  const int64_t tiles = ((int64_t)a.n_kv_rows + kTile - 1) / kTile;
  if (items == 0 || items * 2 > sms) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(sms / items, tiles / 2));
}

size_t workspace_bytes_of(const tre_attention& a, int sms) {
  const int splits = key_splits(a, sms);
  if (splits == 1) return 0;
  return (size_t)splits * a.n_q_rows * a.n_q_heads * (a.head_dim * 4 + 8);
}

template <int D>
tre_status launch(const char* op, const AttnParams& p, const CUtensorMap& kmap,
                  const CUtensorMap& vmap, cudaStream_t stream) {
  auto kernel = prompt_attention_kernel<D>;
  static std::atomic<uint64_t> devices;
  if (!allow_smem(reinterpret_cast<const void*>(kernel), Shape<D>::kSmem, &devices))
    return op_cuda_error(op, "the device refuses the kernel's shared memory");
  const unsigned items = (unsigned)(p.tiles * p.a.n_kv_heads);
  const tre_status st = op_launch(op, kernel, dim3(items, p.splits), kThreadsAttn, Shape<D>::kSmem,
                                  stream, kmap, vmap, p);
  if (st == TRE_OK && p.splits > 1) {
    const int most = (int)std::min<int64_t>(
        kItemRows, (int64_t)p.a.n_q_rows * (p.a.n_q_heads / p.a.n_kv_heads));
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(items, (most + 7) / 8);
    c.blockDim = dim3(256);
    c.stream = stream;
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &early;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, join_kernel<D>, p);
    if (e != cudaSuccess) return op_cuda_error(op, cudaGetErrorString(e));
  }
  return st;
}

tre_status map_of(const char* op, const void* base, int D, int64_t rows, int heads,
                  int64_t row_stride, int64_t head_stride, CUtensorMap* out) {
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)rows, (uint64_t)heads};
  // the stride of a dimension of one entry is never used, but has to be valid
  const uint64_t st[2] = {(uint64_t)(rows > 1 ? row_stride : D) * 2,
                          (uint64_t)(heads > 1 ? head_stride : D) * 2};
  const uint32_t box[3] = {64, kTile, 1};
  return encode_map(op, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, st, box,
                    CU_TENSOR_MAP_SWIZZLE_128B, out);
}

}  // namespace
}  // namespace tre

using namespace tre;

TRE_EXPORT tre_status tre_prompt_attention_workspace(const tre_attention* a, int32_t num_sms,
                                                     size_t* bytes) {
  static const char* op = "tre_prompt_attention_workspace";
  const tre_status st = check(op, a);
  if (st != TRE_OK) return st;
  OP_ARG(bytes && num_sms > 0, op, "bad argument");
  *bytes = workspace_bytes_of(*a, num_sms);
  return TRE_OK;
}

TRE_EXPORT tre_status tre_prompt_attention(const tre_attention* a, const void* q, const void* k,
                                           const void* v, const int32_t* q_offsets,
                                           const int32_t* kv_offsets, void* out, void* workspace,
                                           size_t workspace_bytes, tre_stream stream) {
  static const char* op = "tre_prompt_attention";
  tre_status st = check(op, a);
  if (st != TRE_OK) return st;
  if (a->n_q_rows == 0) return TRE_OK;
  OP_ARG(ptr16(q) && ptr16(out) && (a->n_kv_rows == 0 || (ptr16(k) && ptr16(v))), op,
         "NULL or misaligned pointer");
  OP_ARG(a->n_seqs == 0 || (q_offsets && kv_offsets && ((uintptr_t)q_offsets & 3) == 0 &&
                            ((uintptr_t)kv_offsets & 3) == 0),
         op, "sequences need offsets");
  const int sms = device_sms();
  const size_t need = workspace_bytes_of(*a, sms);
  OP_ARG(need == 0 || (ptr16(workspace) && workspace_bytes >= need), op,
         "the workspace is too small or misaligned");
  AttnParams p{};
  p.a = *a;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q_offsets = q_offsets;
  p.kv_offsets = kv_offsets;
  p.tiles = row_tiles(*a);
  p.splits = key_splits(*a, sms);
  p.part_o = static_cast<float*>(workspace);
  const size_t parts = (size_t)p.splits * a->n_q_rows * a->n_q_heads;
  p.part_ml = reinterpret_cast<float2*>(p.part_o + parts * a->head_dim);
  p.group = divisor(a->n_q_heads / a->n_kv_heads);
  p.kv_heads = divisor(a->n_kv_heads);
  p.c = a->scale * kLog2e;
  p.status = ops_status_ptr();
  if (!p.status) return op_cuda_error(op, "the operators' status word is not available");
  OP_ARG((int64_t)p.tiles * a->n_kv_heads < ((int64_t)1 << 31), op, "too many query rows");
  CUtensorMap kmap{}, vmap{};
  if (a->n_kv_rows > 0) {
    st = map_of(op, k, a->head_dim, a->n_kv_rows, a->n_kv_heads, a->k_row_stride,
                a->k_head_stride, &kmap);
    if (st == TRE_OK)
      st = map_of(op, v, a->head_dim, a->n_kv_rows, a->n_kv_heads, a->v_row_stride,
                  a->v_head_stride, &vmap);
    if (st != TRE_OK) return st;
  }
  return a->head_dim == 64 ? launch<64>(op, p, kmap, vmap, (cudaStream_t)stream)
                           : launch<128>(op, p, kmap, vmap, (cudaStream_t)stream);
}
