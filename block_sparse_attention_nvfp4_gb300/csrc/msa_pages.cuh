// What the operators of a page pool share: the pool as the kernels see it, sums and free pages within a plan CTA,
// checks of the arguments, chained launches.
#pragma once
#include <climits>
#include <cstdint>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kChunk = 16384;   // bytes of a unit of copying: 4 x 16 bytes per thread
constexpr int kMaxPages = 1 << 20;  // sums over a plan CTA's entries stay within 32 bits

struct Plane {
  uint8_t* data;
  long long page_bytes;
  int strips, strip_bytes, slot_bytes;  // slot_bytes 0: page_bytes kept once for a page
  int chunks;                           // per strip
  int first;                            // first chunk of the plane among a page's chunks
};

struct Pool {
  int num_seqs, num_pages, max_pages, num_planes;
  int chunks;  // of a page, over all planes
  int32_t* seq_lens;
  int32_t* table;
  int32_t* refs;
  uint32_t* flags;
  Plane planes[MSA_MAX_PLANES];
};

// Workspace after the flags: five lists of num_seqs and two of num_pages.
struct Lists {
  int32_t* claim;   // [num_seqs] by sequence
  int32_t* src;     // [n] by list entry: pages to copy (-1: none), from
  int32_t* dst;     //     and to
  int32_t* tokens;  //     slots to copy
  int32_t* len;     //     fork: the parent's length before the call (-1: the entry does nothing)
  int32_t* free_ids;  // [num_pages] free pages in id order; compact: targets
  int32_t* map;       // [num_pages] compact: new id of a page, -1 when its count is 0
  int32_t* count;     // compact: number of moves, then where the sources start in free_ids
};

__host__ __device__ inline Lists carve(void* ws, int num_seqs, int num_pages) {
  int32_t* p = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 256);
  Lists l;
  l.claim = p;
  l.src = p + num_seqs;
  l.dst = p + 2LL * num_seqs;
  l.tokens = p + 3LL * num_seqs;
  l.len = p + 4LL * num_seqs;
  l.free_ids = p + 5LL * num_seqs;
  l.map = l.free_ids + num_pages;
  l.count = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 128);
  return l;
}

// Exclusive sum over the CTA's threads in thread order; *total gets the sum of all.
__device__ __forceinline__ int cta_exclusive_sum(int v, int* total) {
  __shared__ int part[kPlanWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) part[w] = incl;
  __syncthreads();
  const int x = part[lane];
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += o;
  }
  const int base = __shfl_sync(0xFFFFFFFFu, s - x, w);
  *total = __shfl_sync(0xFFFFFFFFu, s, 31);
  __syncthreads();  // part is free again
  return base + incl - v;
}

// Counts 4 t .. 4 t + 3 (t = thread) of ids base ..; ids past the pool count as held.
__device__ __forceinline__ int4 load_counts(const Pool& p, int base) {
  const int id = base + 4 * threadIdx.x;
  int4 r = make_int4(1, 1, 1, 1);
  if (id + 3 < p.num_pages && (reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0) {
    r = *reinterpret_cast<const int4*>(p.refs + id);
  } else {
    if (id < p.num_pages) r.x = p.refs[id];
    if (id + 1 < p.num_pages) r.y = p.refs[id + 1];
    if (id + 2 < p.num_pages) r.z = p.refs[id + 2];
    if (id + 3 < p.num_pages) r.w = p.refs[id + 3];
  }
  return r;
}

// The first `want` free pages in id order into free_ids; returns how many there are (at most want).
// `first`: load_counts(p, 0), asked for early.
__device__ inline int find_free(const Pool& p, int want, int32_t* free_ids, int4 first) {
  int found = 0;
  for (int base = 0; base < p.num_pages && found < want; base += 4 * kPlanThreads) {
    const int4 r = base == 0 ? first : load_counts(p, base);
    int total;
    int at = found + cta_exclusive_sum((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), &total);
    const int id = base + 4 * threadIdx.x;
    if (r.x == 0 && at < want) free_ids[at] = id;
    at += r.x == 0;
    if (r.y == 0 && at < want) free_ids[at] = id + 1;
    at += r.y == 0;
    if (r.z == 0 && at < want) free_ids[at] = id + 2;
    at += r.z == 0;
    if (r.w == 0 && at < want) free_ids[at] = id + 3;
    found += total;
  }
  __syncthreads();
  return found < want ? found : want;
}

__device__ __forceinline__ int pages_of(int n) { return (n + kBlock - 1) / kBlock; }
__device__ __forceinline__ bool in(int x, int n) { return x >= 0 && x < n; }
__device__ __forceinline__ bool good_len(const Pool& p, int n) {
  return n >= 0 && n <= static_cast<long long>(p.max_pages) * kBlock;
}

constexpr int kSmemSeqs = 8192;  // sequences whose claims are kept in shared memory

inline msa_status make_pool(const msa_page_pool* a, bool tables, void* ws, size_t ws_bytes, Pool* out) {
  if (a == nullptr || a->num_seqs < 0 || a->num_pages < 1 || a->max_pages_per_seq < 1 || a->num_planes < 0 ||
      a->num_planes > MSA_MAX_PLANES)
    return MSA_ERR_INVALID_ARG;
  if (static_cast<long long>(a->max_pages_per_seq) * kBlock >= (1LL << 31) || a->num_pages > kMaxPages ||
      a->num_seqs > kMaxPages)
    return MSA_ERR_UNSUPPORTED;
  if (tables && (a->ref_counts == nullptr || (a->num_seqs > 0 && (a->seq_lens == nullptr || a->block_table == nullptr))))
    return MSA_ERR_INVALID_ARG;
  Pool p = {};
  p.num_seqs = a->num_seqs;
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages_per_seq;
  p.num_planes = a->num_planes;
  p.seq_lens = a->seq_lens;
  p.table = a->block_table;
  p.refs = a->ref_counts;
  long long chunks = 0;
  for (int k = 0; k < a->num_planes; ++k) {
    const msa_page_plane& s = a->planes[k];
    Plane& d = p.planes[k];
    if (s.data == nullptr || (reinterpret_cast<uintptr_t>(s.data) & 15u) != 0) return MSA_ERR_INVALID_ARG;
    if (s.slot_bytes < 0 || s.slot_bytes % 8 != 0 || s.slot_bytes > (1 << 16)) return MSA_ERR_INVALID_ARG;
    if (s.slot_bytes > 0 ? (s.strips < 1 || s.strips > 1024) : (s.page_bytes < 4 || s.page_bytes % 4 != 0))
      return MSA_ERR_INVALID_ARG;
    d.data = static_cast<uint8_t*>(s.data);
    d.slot_bytes = s.slot_bytes;
    d.strips = s.slot_bytes > 0 ? s.strips : 1;
    d.strip_bytes = s.slot_bytes > 0 ? kBlock * s.slot_bytes : s.page_bytes;
    d.page_bytes = static_cast<long long>(d.strips) * d.strip_bytes;
    d.chunks = s.slot_bytes > 0 ? (d.strip_bytes + kChunk - 1) / kChunk : 1;
    d.first = static_cast<int>(chunks);
    chunks += static_cast<long long>(d.chunks) * d.strips;
  }
  p.chunks = static_cast<int>(chunks);
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MSA_ERR_WORKSPACE;
  size_t need = 0;
  msa_pages_workspace_size(a, &need);
  if (ws_bytes < need) return MSA_ERR_WORKSPACE;
  p.flags = static_cast<uint32_t*>(ws);
  *out = p;
  return MSA_OK;
}

// Launch chained to the kernel before it in the stream: it waits for that kernel's end itself.
template <typename... Args>
msa_status launch_chained(void (*kernel)(Args...), int grid, int threads, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

inline msa_status launched() { return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

}  // namespace
}  // namespace msa
