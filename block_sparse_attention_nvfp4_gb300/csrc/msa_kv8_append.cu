// Append to the 8-bit cache (msa_kv8_append): new tokens' K and V rows quantised to E4M3
// with one scale for each 128-token page and KV head.
//
// The scale of a (page, head) has to hold for all its tokens, and new tokens arrive a few
// at a time: with a the largest finite magnitude of the new rows,
//   need = smallest 2^e, e >= -60, with a <= 448 2^e;   scale = max(need, 2^ceil(log2 old)),
// old codes are rewritten as RNE(code old / scale) only when the scale moved, new ones are
// RNE(x / scale). With a power of two x / scale is exact in FP32, so each code is rounded
// once. Old scales count only when the first new slot is not slot 0: a page that starts anew
// takes nothing from what it held.
//
// Bound: memory (a token reads 2 H 128 source values and writes 2 H 128 bytes); a step of single
// tokens is bound by latency. Units of work are (request, touched page) x (KV head, K or V);
// a request's new tokens are consecutive positions, so a unit's rows are consecutive rows of the
// source and consecutive slots of the page, one CTA or warp sees all of them, and one pass with
// the rows held in registers is enough (amax -> scale -> codes), with no atomics.
//   * append_rows_kernel (at most 8 rows per request, so at most two pages): CTA = (request, first or
//     second page), each warp whole (head, K or V) pairs; the pairs whose scale moved are rescaled by the
//     whole CTA after. The source rows are asked for before the page is known. One token for each of 256
//     requests, 4 heads, BF16: 6.2 us, 20.6 with the other kernel.
//   * append_tile_kernel: CTA = one (request, page, head, K or V), up to 128 x 128 values in
//     registers; the next unit is located while this one's rows are on their way. 8 ragged prompts of
//     44,000 tokens together, 4 heads, BF16 (134 MB read and written): 29 us, 0.69 of the copy rate. What is
//     missing: a CTA loads, takes the maximum, waits, converts and stores one unit after the other, and four
//     CTAs on an SM cover that in part (ALU pipe 64 %, issue 61 %, memory 40 % busy by the counters: neither is
//     full); 4.6 rounds of units leave a tail of about a tenth.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsMost = 8;   // rows per request that append_rows_kernel takes
constexpr int kMinExp = -60;

// The values of 16 loaded bytes of T as FP32.
template <typename T>
__device__ __forceinline__ void widen(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// Bits of |x| for the maximum: non-negative floats order as their bits; infinities and NaN count as 0.
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// Exponent of the smallest 2^e >= 2^kMinExp with amax <= 448 2^e (448 = 1.75 2^8), amax by its bits.
__device__ __forceinline__ int need_exp(uint32_t amax) {
  int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}

struct Scale {
  float scale, inv;  // 2^e, 2^-e
  float ratio;       // old / scale: what the old codes are multiplied by (1: left alone)
};

// f: first new slot of the page.
__device__ __forceinline__ Scale new_scale(uint32_t amax, float old, int f) {
  int e = need_exp(amax);
  float ratio = 1.f;
  if (f > 0) {
    const uint32_t u = __float_as_uint(old);
    if (u - 1u < 0x7F7FFFFFu) {  // positive and finite
      const int eo = static_cast<int>(u >> 23) - 127 + ((u & 0x7FFFFFu) ? 1 : 0);
      e = eo > e ? eo : e;
      e = e > 126 ? 126 : e;
      ratio = old * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    } else {
      ratio = 0.f;
    }
  }
  Scale s;
  s.scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  s.inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  s.ratio = ratio;
  return s;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1; cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3; "
      "mov.b32 %0, {lo, hi}; }"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four codes times a ratio in [0, 1], rounded back to E4M3. The codes are exact in FP16 and
// FP32; a power-of-two ratio keeps the product exact, so it is rounded once.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  uint32_t h0, h1;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi; }"
      : "=r"(h0), "=r"(h1)
      : "r"(c));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  return e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}
__device__ __forceinline__ void rescale_chunk(uint4* p, float ratio) {
  uint4 v = *p;
  v.x = rescale4(v.x, ratio);
  v.y = rescale4(v.y, ratio);
  v.z = rescale4(v.z, ratio);
  v.w = rescale4(v.w, ratio);
  *p = v;
}

// ---- the units of append_tile_kernel: every CTA scans the requests once
struct Units {
  int prefix[kMaxReqs + 1];  // units before request b (a unit = a page that the request writes)
};

__device__ __forceinline__ bool good_request(const Kv8AppendParams& p, int N, int r0, int R) {
  return N >= 0 && N <= p.max_pages * static_cast<long long>(kBlock) && R >= 0 && R <= p.max_rows && R <= N && r0 >= 0 &&
         r0 <= p.total_rows - R;
}

// Pages that request b writes (0 when its geometry is bad, which is flagged).
__device__ __forceinline__ int touched(const Kv8AppendParams& p, int b) {
  const int N = p.context_lens[b], r0 = p.q_indptr[b], R = p.q_indptr[b + 1] - r0;
  if (!good_request(p, N, r0, R)) {
    if (blockIdx.x == 0) set_flag(p.flags, kFlagBadLength);
    return 0;
  }
  return R == 0 ? 0 : (N - 1) / kBlock - (N - R) / kBlock + 1;
}

template <int kThreads>
__device__ __forceinline__ int scan_units(const Kv8AppendParams& p, Units& un) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int part[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (p.num_reqs + kThreads - 1) / kThreads;
  const int b0 = tid * per < p.num_reqs ? tid * per : p.num_reqs;
  const int b1 = b0 + per < p.num_reqs ? b0 + per : p.num_reqs;
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = touched(p, b);
    un.prefix[b] = n;
    mine += n;
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) part[w] = incl;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) base += part[i];
    total += part[i];
  }
  int acc = base + incl - mine;
  for (int b = b0; b < b1; ++b) {
    const int n = un.prefix[b];
    un.prefix[b] = acc;
    acc += n;
  }
  if (tid == 0) un.prefix[p.num_reqs] = total;
  __syncthreads();
  return total;
}

struct Unit {
  int phys;       // physical page, -1 when it is not to be written
  int f, m;       // first slot written, slots written
  long long row;  // first source row
};

__device__ __forceinline__ Unit locate(const Kv8AppendParams& p, const Units& un, int u, bool report) {
  int lo = 0, hi = p.num_reqs;  // prefix[lo] <= u < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (un.prefix[mid] <= u) lo = mid;
    else hi = mid;
  }
  const int b = lo, N = p.context_lens[b], r0 = p.q_indptr[b], R = p.q_indptr[b + 1] - r0;
  const int first = N - R, c = first / kBlock + (u - un.prefix[b]);
  const int a = c * kBlock > first ? c * kBlock : first;
  const int e = (c + 1) * kBlock < N ? (c + 1) * kBlock : N;
  Unit x;
  x.f = a - c * kBlock;
  x.m = e - a;
  x.row = r0 + (a - first);
  x.phys = p.block_table[static_cast<long long>(b) * p.max_pages + c];
  if (x.phys < 0 || x.phys >= p.num_pages) {
    if (report) set_flag(p.flags, kFlagBadPage);
    x.phys = -1;
  }
  return x;
}

// Page `which` of the ones that request b writes, with up to kRowsMost rows; m = 0 when there is none.
__device__ __forceinline__ Unit page_of_request(const Kv8AppendParams& p, int b, int which, bool report) {
  const int N = p.context_lens[b], r0 = p.q_indptr[b], R = p.q_indptr[b + 1] - r0;
  Unit x = {-1, 0, 0, 0};
  if (!good_request(p, N, r0, R)) {
    if (report && which == 0) set_flag(p.flags, kFlagBadLength);
    return x;
  }
  const int first = N - R, c = first / kBlock + which;
  if (R == 0 || c * kBlock >= N) return x;
  const int a = which == 0 ? first : c * kBlock, e = (c + 1) * kBlock < N ? (c + 1) * kBlock : N;
  x.f = a - c * kBlock;
  x.m = e - a;
  x.row = r0 + (a - first);
  x.phys = p.block_table[static_cast<long long>(b) * p.max_pages + c];
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const Kv8AppendParams p, int pages) {
  constexpr int kV = 16 / sizeof(T);       // values a lane loads at once
  constexpr int kLanes = kDim / kV;        // lanes of a row: 16 (2-byte types) or 32
  constexpr int kPer = 32 / kLanes;        // rows a warp loads at once
  constexpr int kIter = kRowsMost / kPer;
  __shared__ int grown[2 * 64];
  __shared__ float grown_ratio[2 * 64];
  __shared__ int n_grown;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int u = blockIdx.x; u < pages * p.num_reqs; u += gridDim.x) {
    const Unit x = page_of_request(p, pages == 1 ? u : u >> 1, pages == 1 ? 0 : u & 1, tid == 0);
    if (x.m == 0) continue;
    if (tid == 0) n_grown = 0;
    __syncthreads();
    for (int s = w; s < 2 * p.num_kv_heads; s += kWarps) {
      const int h = s >> 1, kv = s & 1;
      const T* src = static_cast<const T*>(kv ? p.v : p.k);
      if (src == nullptr) continue;
      const long long stride = kv ? p.v_stride : p.k_stride;
      uint4 raw[kIter];
      uint32_t amax = 0u;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int r = i * kPer + lane / kLanes;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < x.m)
          raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + (x.row + r) * stride + h * kDim) + lane % kLanes);
      }
      if (x.phys < 0 || x.phys >= p.num_pages) break;
      const long long ph = static_cast<long long>(x.phys) * p.num_kv_heads + h;
      float* scale = (kv ? p.v_scale : p.k_scale) + ph;
      const float old = *scale;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        float f[kV];
        widen<T>(raw[i], f);
#pragma unroll
        for (int j = 0; j < kV; ++j) amax = max(amax, finite_abs_bits(f[j]));
      }
      amax = __reduce_max_sync(0xFFFFFFFFu, amax);
      const Scale sc = new_scale(amax, old, x.f);
      uint8_t* data = (kv ? p.v_data : p.k_data) + ph * (kBlock * kDim);
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int r = i * kPer + lane / kLanes;
        float f[kV];
        widen<T>(raw[i], f);
        uint32_t c[kV / 4];
#pragma unroll
        for (int j = 0; j < kV / 4; ++j)
          c[j] = e4m3x4(f[4 * j] * sc.inv, f[4 * j + 1] * sc.inv, f[4 * j + 2] * sc.inv, f[4 * j + 3] * sc.inv);
        if (r < x.m) {
          uint8_t* dst = data + (x.f + r) * kDim + (lane % kLanes) * kV;
          if constexpr (kV == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
          else *reinterpret_cast<uint32_t*>(dst) = c[0];
        }
      }
      if (lane == 0) {
        *scale = sc.scale;
        if (sc.ratio != 1.f) {
          const int g = atomicAdd(&n_grown, 1);
          grown[g] = s;
          grown_ratio[g] = sc.ratio;
        }
      }
    }
    if (tid == 0 && (x.phys < 0 || x.phys >= p.num_pages)) set_flag(p.flags, kFlagBadPage);
    __syncthreads();
    const int ng = n_grown;
    for (int g = 0; g < ng; ++g) {
      const int h = grown[g] >> 1, kv = grown[g] & 1;
      const float ratio = grown_ratio[g];
      uint4* data = reinterpret_cast<uint4*>((kv ? p.v_data : p.k_data) +
                                             (static_cast<long long>(x.phys) * p.num_kv_heads + h) * (kBlock * kDim));
      for (int c = tid; c < x.f * (kDim / 16); c += kThreads) rescale_chunk(data + c, ratio);
    }
    __syncthreads();
  }
}

// The largest finite magnitude among 16 loaded bytes of T, by its FP32 bits.
template <typename T>
__device__ __forceinline__ uint32_t amax_bits(const uint4& v) {
  float f[16 / sizeof(T)];
  widen<T>(v, f);
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < static_cast<int>(16 / sizeof(T)); ++j) m = max(m, finite_abs_bits(f[j]));
  return m;
}

// kThreads x 8 loads of 16 bytes cover a tile of 2-byte (256) or 4-byte (512) values: 64 registers a
// thread keep four (two) CTAs on an SM, 128 KB of loads in flight.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) append_tile_kernel(const Kv8AppendParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kV = 16 / sizeof(T);
  constexpr int kLanes = kDim / kV;
  constexpr int kPer = kThreads / kLanes;  // rows the CTA loads at once
  constexpr int kIter = kBlock / kPer;
  static_assert(kIter == 8, "registers");
  __shared__ Units un;
  __shared__ uint32_t wmax[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int total = scan_units<kThreads>(p, un);
  const int pairs = 2 * p.num_kv_heads;
  const long long work = static_cast<long long>(total) * pairs;
  const int r_lane = tid / kLanes, c_lane = tid % kLanes;
  int buf = 0;
  long long t = blockIdx.x;
  Unit x = {};
  if (t < work) x = locate(p, un, static_cast<int>(t / pairs), tid == 0);
  while (t < work) {
    const int s = static_cast<int>(t % pairs), h = s >> 1, kv = s & 1;
    const T* src = static_cast<const T*>(kv ? p.v : p.k);
    const bool on = src != nullptr && x.phys >= 0;
    const long long stride = kv ? p.v_stride : p.k_stride;
    uint4 raw[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = i * kPer + r_lane;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (on && r < x.m) raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + (x.row + r) * stride + h * kDim) + c_lane);
    }
    const long long ph = static_cast<long long>(on ? x.phys : 0) * p.num_kv_heads + h;
    float* scale = (kv ? p.v_scale : p.k_scale) + ph;
    const float old = on ? *scale : 1.f;
    const Unit cur = x;
    t += gridDim.x;
    if (t < work) x = locate(p, un, static_cast<int>(t / pairs), tid == 0);  // while the loads are on their way
    if (!on) continue;
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < kIter; ++i) amax = max(amax, amax_bits<T>(raw[i]));
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if (lane == 0) wmax[buf][w] = amax;
    __syncthreads();  // also: every thread has read the old scale
    amax = 0u;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) amax = max(amax, wmax[buf][i]);
    buf ^= 1;  // the other half is free: its readers passed the barrier above
    const Scale sc = new_scale(amax, old, cur.f);
    uint8_t* data = (kv ? p.v_data : p.k_data) + ph * (kBlock * kDim);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = i * kPer + r_lane;
      float f[kV];
      widen<T>(raw[i], f);
      uint32_t c[kV / 4];
#pragma unroll
      for (int j = 0; j < kV / 4; ++j)
        c[j] = e4m3x4(f[4 * j] * sc.inv, f[4 * j + 1] * sc.inv, f[4 * j + 2] * sc.inv, f[4 * j + 3] * sc.inv);
      if (r < cur.m) {
        uint8_t* dst = data + (cur.f + r) * kDim + c_lane * kV;
        if constexpr (kV == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
        else *reinterpret_cast<uint32_t*>(dst) = c[0];
      }
    }
    if (tid == 0) *scale = sc.scale;
    if (sc.ratio != 1.f)
      for (int c = tid; c < cur.f * (kDim / 16); c += kThreads)
        rescale_chunk(reinterpret_cast<uint4*>(data) + c, sc.ratio);
  }
}

template <typename T>
cudaError_t launch(const Kv8AppendParams& prm, int sm_count, cudaStream_t st) {
  // units that the host can bound: pages of a request's rows, at most total_rows / 128 + 2 each
  const long long units = prm.total_rows / kBlock + 2LL * prm.num_reqs;
  if (prm.max_rows <= kRowsMost) {
    const long long cap = static_cast<long long>(sm_count) * 4;
    const int pages = prm.max_rows > 1 ? 2 : 1;  // that a request can write
    const long long work = static_cast<long long>(pages) * prm.num_reqs;
    append_rows_kernel<T><<<static_cast<int>(work < cap ? work : cap), kThreads, 0, st>>>(prm, pages);
  } else {
    const long long cap = static_cast<long long>(sm_count) * 4, work = units * 2 * prm.num_kv_heads;
    constexpr int kTh = sizeof(T) == 2 ? 256 : 512;
    append_tile_kernel<T, kTh><<<static_cast<int>(work < cap ? work : cap), kTh, 0, st>>>(prm);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_kv8_append(const msa_kv8_append_args* a, void* ws, size_t ws_bytes, void* stream) {
  if (a == nullptr || a->num_reqs < 0 || a->num_reqs > kMaxReqs || a->total_rows < 0 || a->max_rows_per_req < 1 ||
      a->num_pages < 1 || a->max_pages_per_req < 1)
    return MSA_ERR_INVALID_ARG;
  if (static_cast<long long>(a->total_rows) > static_cast<long long>(a->num_reqs) * a->max_rows_per_req)
    return MSA_ERR_INVALID_ARG;
  if (a->num_kv_heads < 1 || a->num_kv_heads > kKv8MaxHeads) return MSA_ERR_UNSUPPORTED;
  if (a->src_type != MSA_TYPE_BF16 && a->src_type != MSA_TYPE_F16 && a->src_type != MSA_TYPE_F32)
    return MSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->num_pages) * a->num_kv_heads * kBlock >= (1LL << 31) ||
      static_cast<long long>(a->max_pages_per_req) * kBlock >= (1LL << 31))
    return MSA_ERR_UNSUPPORTED;
  if (a->num_reqs > 0 && (a->context_lens == nullptr || a->q_indptr == nullptr || a->block_table == nullptr))
    return MSA_ERR_INVALID_ARG;
  const int size = a->src_type == MSA_TYPE_F32 ? 4 : 2;
  auto bad_source = [&](const void* x, int64_t stride, const void* data, const void* scale) {
    return x != nullptr && (data == nullptr || scale == nullptr || (reinterpret_cast<uintptr_t>(x) & 15u) != 0 ||
                            (reinterpret_cast<uintptr_t>(data) & 15u) != 0 ||
                            (reinterpret_cast<uintptr_t>(scale) & 3u) != 0 || stride < kDim * a->num_kv_heads ||
                            stride * size % 16 != 0);
  };
  if (bad_source(a->k, a->k_token_stride, a->k_data, a->k_scale) ||
      bad_source(a->v, a->v_token_stride, a->v_data, a->v_scale))
    return MSA_ERR_INVALID_ARG;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < 256) return MSA_ERR_WORKSPACE;
  int sms = 0;
  const msa_status s = check_device(&sms);
  if (s != MSA_OK) return s;
  if (a->num_reqs == 0 || a->total_rows == 0 || (a->k == nullptr && a->v == nullptr)) return MSA_OK;
  Kv8AppendParams p = {};
  p.num_reqs = a->num_reqs;
  p.total_rows = a->total_rows;
  p.max_rows = a->max_rows_per_req;
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages_per_req;
  p.num_kv_heads = a->num_kv_heads;
  p.context_lens = a->context_lens;
  p.q_indptr = a->q_indptr;
  p.block_table = a->block_table;
  p.k = a->k;
  p.v = a->v;
  p.k_stride = a->k_token_stride;
  p.v_stride = a->v_token_stride;
  p.k_data = a->k_data;
  p.k_scale = a->k_scale;
  p.v_data = a->v_data;
  p.v_scale = a->v_scale;
  p.flags = static_cast<uint32_t*>(ws);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->src_type == MSA_TYPE_BF16  ? launch<__nv_bfloat16>(p, sms, st)
                        : a->src_type == MSA_TYPE_F16 ? launch<__half>(p, sms, st)
                                                      : launch<float>(p, sms, st);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
