// Attention over the 8-bit cache (msa_kv8_attn): E4M3 keys and values with one FP32 scale for
// each 128-token page and KV head.
//
// For a query row at position p, keys t <= p of the listed blocks (or of all):
//   s_t = sm_scale k_scale (q . k_t),  out = sum_t 2^(s_t log2e - m) v_scale v_t / sum_t 2^(s_t log2e - m)
// with the running maximum m and sum of an online softmax in FP32.
//
// This form is the plain one: a CTA of 128 threads per (query row, query head), a thread per key
// of a page for the scores and a thread per dim for the products with V.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

__device__ __forceinline__ float e4m3_f32(uint32_t c) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(c & 0xFFu));
  return __half2float(__low2half(*reinterpret_cast<const __half2*>(&h)));
}

__device__ __forceinline__ float cta_max(float v, float* s) {
  for (int d = 16; d; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
  __syncthreads();
  return v;
}
__device__ __forceinline__ float cta_sum(float v, float* s) {
  for (int d = 16; d; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  return v;
}

template <bool kBf16>
__global__ void __launch_bounds__(128) kv8_attn_kernel(const Kv8AttnParams p) {
  __shared__ float q[kDim], w[kBlock], red[4];
  const int row = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, h = head / p.q_per_kv;
  const int heads = p.num_kv_heads * p.q_per_kv;
  int lo = 0, hi = p.num_reqs;  // the last request with q_indptr[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.q_indptr[mid] <= row) lo = mid;
    else hi = mid;
  }
  const int b = lo, N = p.context_lens[b], r0 = p.q_indptr[b], R = p.q_indptr[b + 1] - r0;
  const bool ok = N >= 0 && N <= p.max_pages * static_cast<long long>(kBlock) && R >= 0 && R <= p.max_rows && R <= N &&
                  r0 >= 0 && r0 <= p.total_rows - R;
  if (!ok || row >= r0 + R || row < r0) {
    if (!ok && tid == 0) set_flag(p.flags, kFlagBadLength);
    return;
  }
  if (kBf16)
    q[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * p.q_stride + head * kDim + tid]);
  else
    q[tid] = e4m3_f32(static_cast<const uint8_t*>(p.q)[row * p.q_stride + head * kDim + tid]);
  __syncthreads();
  const int nb = (N + kBlock - 1) / kBlock, pos = N - R + (row - r0);
  const int32_t* ids = p.n_ids ? p.block_ids + (static_cast<long long>(b) * p.num_kv_heads + h) * p.n_ids : nullptr;
  const int tiles = ids ? p.n_ids : pos / kBlock + 1;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int j = 0; j < tiles; ++j) {
    const int c = ids ? ids[j] : j;
    if (c < 0 || c >= nb) {
      if (c != -1 && tid == 0) set_flag(p.flags, kFlagBadIds);
      continue;
    }
    bool twice = false;
    for (int i = 0; ids && i < j; ++i) twice |= ids[i] == c;
    if (twice) {
      if (tid == 0) set_flag(p.flags, kFlagBadIds);
      continue;
    }
    const int phys = p.block_table[static_cast<long long>(b) * p.max_pages + c];
    if (phys < 0 || phys >= p.num_pages) {
      if (tid == 0) set_flag(p.flags, kFlagBadPage);
      continue;
    }
    const long long ph = static_cast<long long>(phys) * p.num_kv_heads + h;
    const int seen = pos - c * kBlock + 1 < kBlock ? pos - c * kBlock + 1 : kBlock;
    float s = -INFINITY;
    if (tid < seen) {
      const uint8_t* k = p.k_data + (ph * kBlock + tid) * kDim;
      s = 0.f;
      for (int d = 0; d < kDim; ++d) s += q[d] * e4m3_f32(k[d]);
      s *= p.k_scale[ph] * p.sm_scale_log2;
    }
    const float mx = cta_max(s, red);
    const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;
    const float e = tid < seen ? exp2f(s - ref) : 0.f, alpha = exp2f(m - ref);
    w[tid] = e;
    l = l * alpha + cta_sum(e, red);
    o *= alpha;
    const float vs = p.v_scale[ph];
    for (int t = 0; t < seen; ++t) o += w[t] * vs * e4m3_f32(p.v_data[(ph * kBlock + t) * kDim + tid]);
    m = m_new;
    __syncthreads();
  }
  const long long at = static_cast<long long>(row) * heads + head;
  p.out[at * kDim + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.f ? 0.f : o / l));
  if (tid == 0 && p.lse != nullptr) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

msa_status check_args(const msa_kv8_attn_args* a) {
  if (a == nullptr || a->num_reqs < 0 || a->num_reqs > kMaxReqs || a->total_rows < 0 || a->max_rows_per_req < 1 ||
      a->num_pages < 1 || a->max_pages_per_req < 1)
    return MSA_ERR_INVALID_ARG;
  if (static_cast<long long>(a->total_rows) > static_cast<long long>(a->num_reqs) * a->max_rows_per_req)
    return MSA_ERR_INVALID_ARG;
  if (a->num_kv_heads < 1 || a->num_kv_heads > kKv8MaxHeads || a->q_per_kv < 1 || a->q_per_kv > kKv8MaxQPerKv)
    return MSA_ERR_UNSUPPORTED;
  if (a->q_type != MSA_TYPE_E4M3 && a->q_type != MSA_TYPE_BF16) return MSA_ERR_UNSUPPORTED;
  if (a->n_block_ids < 0 || a->n_block_ids > kKv8MaxIds) return MSA_ERR_INVALID_ARG;
  if (static_cast<long long>(a->num_pages) * a->num_kv_heads * kBlock >= (1LL << 31) ||
      static_cast<long long>(a->max_pages_per_req) * kBlock >= (1LL << 31))
    return MSA_ERR_UNSUPPORTED;
  if (!(a->sm_scale > 0.f) || !std::isfinite(a->sm_scale)) return MSA_ERR_INVALID_ARG;
  return MSA_OK;
}

}  // namespace

cudaError_t launch_kv8_attn(const Kv8AttnParams& prm, bool q_bf16, int, cudaStream_t st) {
  const dim3 grid(prm.total_rows, prm.num_kv_heads * prm.q_per_kv);
  if (q_bf16) kv8_attn_kernel<true><<<grid, 128, 0, st>>>(prm);
  else kv8_attn_kernel<false><<<grid, 128, 0, st>>>(prm);
  return cudaGetLastError();
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_kv8_attn_workspace_size(const msa_kv8_attn_args* a, size_t* bytes) {
  if (bytes == nullptr) return MSA_ERR_INVALID_ARG;
  const msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  *bytes = 256;
  return MSA_OK;
}

msa_status msa_kv8_attn(const msa_kv8_attn_args* a, void* ws, size_t ws_bytes, void* stream) {
  msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  const bool rows = a->total_rows > 0;
  auto unaligned = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) != 0; };
  if (a->num_reqs > 0 && (a->context_lens == nullptr || a->q_indptr == nullptr || a->block_table == nullptr))
    return MSA_ERR_INVALID_ARG;
  if ((a->block_ids != nullptr) != (a->n_block_ids > 0)) return MSA_ERR_INVALID_ARG;
  if (rows && (a->q == nullptr || a->out == nullptr)) return MSA_ERR_INVALID_ARG;
  if (a->k_data == nullptr || a->k_scale == nullptr || a->v_data == nullptr || a->v_scale == nullptr)
    return MSA_ERR_INVALID_ARG;
  const int q_size = a->q_type == MSA_TYPE_BF16 ? 2 : 1;
  if (unaligned(a->q, 16) || unaligned(a->out, 16) || unaligned(a->k_data, 16) || unaligned(a->v_data, 16) ||
      unaligned(a->k_scale, 4) || unaligned(a->v_scale, 4) || unaligned(a->lse, 4) ||
      a->q_row_stride < static_cast<int64_t>(kDim) * a->num_kv_heads * a->q_per_kv || a->q_row_stride * q_size % 16 != 0)
    return MSA_ERR_INVALID_ARG;
  if (ws == nullptr || unaligned(ws, 256)) return MSA_ERR_WORKSPACE;
  int sms = 0;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  size_t need = 0;
  if ((s = msa_kv8_attn_workspace_size(a, &need)) != MSA_OK) return s;
  if (ws_bytes < need) return MSA_ERR_WORKSPACE;
  if (a->num_reqs == 0 || !rows) return MSA_OK;
  Kv8AttnParams p = {};
  p.num_reqs = a->num_reqs;
  p.total_rows = a->total_rows;
  p.max_rows = a->max_rows_per_req;
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages_per_req;
  p.num_kv_heads = a->num_kv_heads;
  p.q_per_kv = a->q_per_kv;
  p.n_ids = a->n_block_ids;
  p.context_lens = a->context_lens;
  p.q_indptr = a->q_indptr;
  p.block_table = a->block_table;
  p.block_ids = a->block_ids;
  p.q = a->q;
  p.q_stride = a->q_row_stride;
  p.k_data = a->k_data;
  p.k_scale = a->k_scale;
  p.v_data = a->v_data;
  p.v_scale = a->v_scale;
  p.sm_scale_log2 = a->sm_scale * 1.4426950408889634f;
  p.flags = static_cast<uint32_t*>(ws);
  p.out = a->out;
  p.lse = a->lse;
  return launch_kv8_attn(p, a->q_type == MSA_TYPE_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MSA_OK
             : MSA_ERR_CUDA;
}

}  // extern "C"
