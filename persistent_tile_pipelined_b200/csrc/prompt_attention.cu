// Causal attention of packed prompts (declared in include/tre.h as tre_prompt_attention).
#include <cuda_bf16.h>

#include <algorithm>

#include "ops_host.h"

namespace tre {
namespace {

constexpr int kWarps = 4;

struct AttnParams {
  tre_attention a;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  const int32_t *q_offsets, *kv_offsets;
};

// One warp per (query row, head): the keys in order, 32 at a time, one per lane, with the
// running maximum and sum of the softmax; then the lanes share the width of v.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) prompt_attention_kernel(const AttnParams p) {
  __shared__ float qs[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y * kWarps + warp;
  if (h >= p.a.n_q_heads) return;
  int q0 = 0, q1 = p.a.n_q_rows, k0 = 0, k1 = p.a.n_kv_rows;
  if (p.a.n_seqs) {
    int i = 0;
    for (; i < p.a.n_seqs; ++i) {
      q0 = min(max(p.q_offsets[i], 0), p.a.n_q_rows);
      q1 = min(max(p.q_offsets[i + 1], 0), p.a.n_q_rows);
      if (t >= q0 && t < q1) break;
    }
    if (i == p.a.n_seqs) return;
    k0 = min(max(p.kv_offsets[i], 0), p.a.n_kv_rows);
    k1 = min(max(p.kv_offsets[i + 1], 0), p.a.n_kv_rows);
  }
  const int see = k1 - k0 - (q1 - q0) + (t - q0) + 1;  // keys k0 .. k0 + see - 1
  const int kh = h / (p.a.n_q_heads / p.a.n_kv_heads);
  const __nv_bfloat16* q = p.q + t * p.a.q_row_stride + h * p.a.q_head_stride;
  const __nv_bfloat16* k = p.k + kh * p.a.k_head_stride;
  const __nv_bfloat16* v = p.v + kh * p.a.v_head_stride;
  for (int i = lane; i < D; i += 32) qs[warp][i] = __bfloat162float(q[i]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, acc[D / 32] = {};
  for (int s0 = 0; s0 < see; s0 += 32) {
    float s = -INFINITY;
    if (s0 + lane < see) {
      const __nv_bfloat16* kr = k + (int64_t)(k0 + s0 + lane) * p.a.k_row_stride;
      float dot = 0.f;
      for (int i = 0; i < D; ++i) dot = fmaf(qs[warp][i], __bfloat162float(kr[i]), dot);
      s = dot * p.a.scale;
    }
    float mn = s;
#pragma unroll
    for (int x = 16; x; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    mn = fmaxf(mn, m);
    const float shift = mn == -INFINITY ? 0.f : mn;
    const float c = expf(m - shift);
    const float e = s0 + lane < see ? expf(s - shift) : 0.f;
    m = mn;
    l *= c;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] *= c;
    for (int x = 0; x < 32 && s0 + x < see; ++x) {
      const float ex = __shfl_sync(0xffffffffu, e, x);
      l += ex;
      const __nv_bfloat16* vr = v + (int64_t)(k0 + s0 + x) * p.a.v_row_stride;
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        acc[j] = fmaf(ex, __bfloat162float(vr[lane + 32 * j]), acc[j]);
    }
  }
  __nv_bfloat16* o = p.out + t * p.a.out_row_stride + h * p.a.out_head_stride;
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
    o[lane + 32 * j] = __float2bfloat16_rn(see > 0 ? acc[j] / l : 0.f);
}

tre_status check(const char* op, const tre_attention* a) {
  OP_ARG(a, op, "NULL argument");
  OP_ARG(a->head_dim == 64 || a->head_dim == 128, op, "head_dim must be 64 or 128");
  OP_ARG(a->n_kv_heads >= 1 && a->n_kv_heads <= 65535 && a->n_q_heads >= 1 &&
             a->n_q_heads <= 65535 && a->n_q_heads % a->n_kv_heads == 0,
         op, "n_q_heads must be a positive multiple of n_kv_heads");
  OP_ARG(a->n_seqs >= 0 && a->n_seqs < (1 << 20), op, "n_seqs out of range");
  OP_ARG(a->n_q_rows >= 0 && a->n_kv_rows >= 0, op, "negative row count");
  OP_ARG((int64_t)a->n_q_rows * a->n_q_heads < ((int64_t)1 << 31), op, "too many query rows");
  OP_ARG(a->scale > 0.f && a->scale < 3e38f, op, "scale must be positive and finite");
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
  return TRE_OK;
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
  *bytes = 0;
  return TRE_OK;
}

TRE_EXPORT tre_status tre_prompt_attention(const tre_attention* a, const void* q, const void* k,
                                           const void* v, const int32_t* q_offsets,
                                           const int32_t* kv_offsets, void* out, void* workspace,
                                           size_t workspace_bytes, tre_stream stream) {
  static const char* op = "tre_prompt_attention";
  const tre_status st = check(op, a);
  if (st != TRE_OK) return st;
  if (a->n_q_rows == 0) return TRE_OK;
  OP_ARG(ptr16(q) && ptr16(out) && (a->n_kv_rows == 0 || (ptr16(k) && ptr16(v))), op,
         "NULL or misaligned pointer");
  OP_ARG(a->n_seqs == 0 || (q_offsets && kv_offsets && ((uintptr_t)q_offsets & 3) == 0 &&
                            ((uintptr_t)kv_offsets & 3) == 0),
         op, "sequences need offsets");
  AttnParams p{*a, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
               static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(out), q_offsets,
               kv_offsets};
  const dim3 grid((unsigned)a->n_q_rows, (unsigned)((a->n_q_heads + kWarps - 1) / kWarps));
  if (a->head_dim == 64)
    prompt_attention_kernel<64><<<grid, kWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else
    prompt_attention_kernel<128><<<grid, kWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return op_launch_status(op);
}
