// What the warp-specialised kernels over the 8-bit cache share: bounded waits, products issued by a converged warp,
// tensor-memory and conversion helpers, chained launches, and the checks of their arguments.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

// Counts round N places; `phase` flips every time round (a barrier's parity), without divisions.
template <int N>
struct Ring {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++at == N) at = 0, phase ^= 1u;
  }
};

// A bounded wait: 2^31 cycles, about a second. A try suspends the warp for a while by itself.
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr uint32_t kWaitCycles = 0x7FFFFFFFu;
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint32_t* flags) {
  const uint32_t t0 = clock();
  while (!try_bar(bar, parity))
    if (static_cast<uint32_t>(clock()) - t0 > kWaitCycles) {
      set_flag(flags, kFlagTimeout);
      return false;
    }
  return true;
}
// The whole warp waits, converged: its lanes vote on every try (one lane asking for all leaves the
// others to a divergent barrier, which wakes ~1,500 cycles late). The loop stands in line: as a
// function of its own, the call's registers cost the roles more than the code (64 ragged requests
// 193 us instead of 164, a BF16 prompt 409 instead of 370), and a loop that counts its tries and does not
// read the clock between them takes the issue slots of the working warps (64 ragged requests 173 us).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t* flags) {
  if (__all_sync(0xFFFFFFFFu, try_bar(bar, parity))) return true;
  const uint32_t t0 = clock();
  do {
    if (__any_sync(0xFFFFFFFFu, static_cast<uint32_t>(clock()) - t0 > kWaitCycles)) {
      set_flag(flags, kFlagTimeout);
      return false;
    }
  } while (!__all_sync(0xFFFFFFFFu, try_bar(bar, parity)));
  return true;
}
// The MMAs and commits with the election inside: the issuing warp stays converged, so that its
// descriptors live in uniform registers (8 products issue in 260 cycles against 450 from a
// one-lane branch).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_f8_ss_elect(uint32_t elected, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; "
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_f16_tmemA_elect(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                    uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; "
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint32_t elected, uint32_t bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0; "
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr) : "memory");
}
// 16 bytes to shared memory, asynchronously; the first `bytes` (0 or 16) are copied, the others zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// A sum brought from reference m to m_to >= m: in two steps, because a sum is relative to a reference with a
// value scale in it, may be as large as 2^67 for that, and counts although 2^(m - m_to) is below FP32's range.
__device__ __forceinline__ float carry(float sum, float m, float m_to) {
  const float h = ex2(0.5f * (m - m_to));
  return sum * h * h;
}
// 32 columns of the warp's lanes times a factor per lane.
__device__ __forceinline__ void tmem_scale32(uint32_t taddr, float a) {
  uint32_t o[32];
  tmem_ld32(taddr, o);
  tc_wait_ld();
#pragma unroll
  for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * a);
  tmem_st32(taddr, o);
}
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t c) {  // the low two codes
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(c));
  return h;
}
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ uint32_t f32x2_e4m3x2(float a, float b) {  // a in the low byte
  uint32_t r;
  asm("{ .reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %2, %1; cvt.u32.u16 %0, t; }" : "=r"(r) : "f"(a), "f"(b));
  return r;
}

// A launch chained to the kernel before it, which the kernel itself waits for.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What every call over the 8-bit cache with these arguments checks first.
inline msa_status check_args(const msa_kv8_attn_args* a) {
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
}  // namespace msa
