// Page operators of a pool of cache pages: copy, fork, reserve, free, compact
// (msa_pages_*). Contracts in include/msa.h.
//
// Each operator is a plan over small integer state (lengths, counts, block tables), then the
// movement of page bytes:
//   * the plan runs in one CTA and is bound by its chain of dependent reads (0.6-0.8 us each):
//     list entries are checked, the pages that each one needs are summed in list order, and the
//     free pages are found by one scan of the counts in id order, whose first 4,096 are asked for
//     before anything else. Ranks come from prefix sums, so ids do not depend on timing.
//   * pages move in one grid-wide kernel over (pair, 16 KB chunk): bound by memory, 2 bytes
//     moved for each byte of a page. Four 16-byte loads per thread are in flight before the first
//     store. Block-table rows are copied or remapped by the same launch, which is set up while
//     the plan runs (programmatic dependent launch).
// Measured (graph replays): 1,024 pages of 131 KB copied in 45 us (268 MB, 0.89 of the copy rate);
// 2,048 live pages of 4,096 compacted in 51 us, of which the plan is 6; 256 forks of 16 long parents
// with 256 reservations 23 us (plan 7, tails and rows 10, reservations 5); a fork to 4 children, their
// growth and their end 12.5 us, four launches of about 3 us each.
// Sources are live pages and targets are free ones, so no order among the copies matters.
#include <climits>
#include <cstdint>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kChunk = 16384;   // bytes of a unit of copying: 4 x 16 bytes per thread
constexpr int kCopyCtasPerSm = 4;
constexpr int kTableChunk = 1024;  // block-table entries of a unit
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
__device__ int find_free(const Pool& p, int want, int32_t* free_ids, int4 first) {
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

// claim[s] = the first entry that lists sequence s, for every listed one: in shared memory when the
// pool's sequences fit there.
constexpr int kSmemSeqs = 8192;
__device__ void claim_first(const Pool& p, int32_t* claim, int n, const int32_t* seqs) {
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (in(seqs[i], p.num_seqs)) claim[seqs[i]] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (in(seqs[i], p.num_seqs)) atomicMin(&claim[seqs[i]], i);
  __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const Pool p, const Lists l, int n,
                                                                 const int32_t* parents, const int32_t* children) {
  __shared__ int32_t claim_s[kSmemSeqs];
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int4 counts = load_counts(p, 0);
  int32_t* claim = p.num_seqs <= kSmemSeqs ? claim_s : l.claim;
  claim_first(p, claim, n, children);
  // what each entry needs, in list order; len[i] = the parent's length, src[i] = its tail page
  int need_all = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0;
    if (i < n) {
      const int par = parents[i], ch = children[i];
      int len = -1, tail = -1;
      if (!in(par, p.num_seqs) || !in(ch, p.num_seqs) || claim[ch] != i || p.seq_lens[ch] != 0 || par == ch) {
        set_flag(p.flags, kFlagBadSeq);
      } else {
        len = p.seq_lens[par];
        if (!good_len(p, len)) {
          set_flag(p.flags, kFlagBadLength);
          len = -1;
        } else if (len % kBlock) {
          tail = p.table[static_cast<long long>(par) * p.max_pages + len / kBlock];
          if (!in(tail, p.num_pages)) {
            set_flag(p.flags, kFlagBadPage);
            len = -1;
            tail = -1;
          } else {
            need = 1;
          }
        }
      }
      l.len[i] = len;
      l.src[i] = tail;
    }
    int total;
    const int at = need_all + cta_exclusive_sum(need, &total);
    if (i < n) l.dst[i] = need ? at : -1;  // rank among the pages given out
    need_all += total;
  }
  __syncthreads();
  const int have = find_free(p, need_all, l.free_ids, counts);
  // every length and tail has been read: the children may be written
  for (int i = tid; i < n; i += kPlanThreads) {
    const int rank = l.dst[i], len = l.len[i];
    if (rank >= have) {
      set_flag(p.flags, kFlagNoPage);
      l.len[i] = -1;
      l.src[i] = -1;
      l.dst[i] = -1;
      continue;
    }
    if (len < 0) continue;
    const int ch = children[i];
    if (rank >= 0) {
      const int id = l.free_ids[rank];
      l.dst[i] = id;
      l.tokens[i] = len % kBlock;
      p.refs[id] = 1;
      p.table[static_cast<long long>(ch) * p.max_pages + len / kBlock] = id;
    }
    p.seq_lens[ch] = len;
  }
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const Pool p, const Lists l, int n, const int32_t* seqs,
                                                               const int32_t* new_lens) {
  __shared__ int32_t claim_s[kSmemSeqs];
  const int tid = threadIdx.x;
  const int4 counts = load_counts(p, 0);
  int32_t* claim = p.num_seqs <= kSmemSeqs ? claim_s : l.claim;
  claim_first(p, claim, n, seqs);
  // len[i] = the new length (-1: nothing to do), src[i] = pages needed, dst[i] = rank of the first
  int need_all = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0, to = -1;
    if (i < n) {
      const int s = seqs[i];
      if (!in(s, p.num_seqs) || claim[s] != i) {
        set_flag(p.flags, kFlagBadSeq);
      } else {
        const int len = p.seq_lens[s], want = new_lens[i];
        if (!good_len(p, len) || !good_len(p, want)) {
          set_flag(p.flags, kFlagBadLength);
        } else if (want > len) {
          need = pages_of(want) - pages_of(len);
          to = want;
        }
      }
      // an entry that could not be served even by an empty pool adds no more than the pool to the sum
      need = need < p.num_pages + 1 ? need : p.num_pages + 1;
    }
    int total;
    const int mine = cta_exclusive_sum(need, &total);
    if (i < n) {
      const long long at = static_cast<long long>(need_all) + mine;
      l.src[i] = need;
      l.dst[i] = at < INT_MAX / 2 ? static_cast<int>(at) : INT_MAX / 2;
      l.len[i] = to;
    }
    const long long sum = static_cast<long long>(need_all) + total;
    need_all = sum < INT_MAX / 2 ? static_cast<int>(sum) : INT_MAX / 2;
  }
  __syncthreads();
  const int have = find_free(p, need_all < p.num_pages ? need_all : p.num_pages, l.free_ids, counts);
  // Entries that need a few pages take a thread, the others a warp.
  constexpr int kFew = 4;
  auto serve = [&](int i, int lane, int lanes) {
    const int to = l.len[i], need = l.src[i], at = l.dst[i];
    if (to < 0 || (lanes == 1) != (need <= kFew)) return;
    if (at + need > have && need > 0) {
      if (lane == 0) set_flag(p.flags, kFlagNoPage);
      return;
    }
    const int s = seqs[i], c0 = pages_of(to) - need;
    for (int k = lane; k < need; k += lanes) {
      const int id = l.free_ids[at + k];
      p.refs[id] = 1;
      p.table[static_cast<long long>(s) * p.max_pages + c0 + k] = id;
    }
    if (lane == 0) p.seq_lens[s] = to;
  };
  bool many = false;
  for (int i = tid; i < n; i += kPlanThreads) {
    serve(i, 0, 1);
    many |= l.src[i] > kFew;
  }
  if (__syncthreads_or(many))
    for (int i = tid >> 5; i < n; i += kPlanWarps) serve(i, tid & 31, 32);
}

// One CTA per list entry; the exchange of the length decides which of equal entries frees.
__global__ void __launch_bounds__(128) free_kernel(const Pool p, int n, const int32_t* seqs) {
  __shared__ int len_s;
  const int s = seqs[blockIdx.x];
  if (!in(s, p.num_seqs)) {
    if (threadIdx.x == 0) set_flag(p.flags, kFlagBadSeq);
    return;
  }
  if (threadIdx.x == 0) {
    int len = atomicExch(&p.seq_lens[s], 0);
    if (!good_len(p, len)) {
      set_flag(p.flags, kFlagBadLength);
      len = 0;
    }
    len_s = len;
  }
  __syncthreads();
  const int np = pages_of(len_s);
  for (int c = threadIdx.x; c < np; c += 128) {
    const int id = p.table[static_cast<long long>(s) * p.max_pages + c];
    if (!in(id, p.num_pages)) {
      set_flag(p.flags, kFlagBadPage);
    } else if (atomicSub(&p.refs[id], 1) <= 0) {
      atomicAdd(&p.refs[id], 1);
      set_flag(p.flags, kFlagBadPage);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const Pool p, const Lists l, int32_t* new_refs,
                                                                    int32_t* num_live) {
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  constexpr int kStep = 4 * kPlanThreads;
  const int4 first = load_counts(p, 0);
  auto live4 = [](const int4& r) { return (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0); };
  auto get = [](const int4& r, int k) { return k == 0 ? r.x : k == 1 ? r.y : k == 2 ? r.z : r.w; };
  int mine = 0;
  for (int base = 0; base < p.num_pages; base += kStep) {
    const int4 r = base == 0 ? first : load_counts(p, base);
    const int past = base + 4 * tid + 4 - p.num_pages;  // ids past the pool, which count as held
    mine += live4(r) - (past > 0 ? (past < 4 ? past : 4) : 0);
  }
  int live;
  cta_exclusive_sum(mine, &live);
  // holes below `live` in id order
  int holes = 0;
  for (int base = 0; base < live; base += kStep) {
    const int4 r = base == 0 ? first : load_counts(p, base);
    const int id0 = base + 4 * tid;
    int n = 0, total;
#pragma unroll
    for (int k = 0; k < 4; ++k) n += id0 + k < live && get(r, k) <= 0;
    int at = holes + cta_exclusive_sum(n, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int id = id0 + k;
      if (id >= live) break;
      if (get(r, k) <= 0) {
        l.free_ids[at++] = id;
        l.map[id] = -1;
      } else {
        l.map[id] = id;
        if (new_refs != p.refs) new_refs[id] = get(r, k);
      }
    }
    holes += total;
  }
  __syncthreads();
  // live pages from `live` on: as many as holes; k-th to the k-th. In place this writes counts below
  // `live`, which no later step reads, and a step's own, which its sum's barrier has seen read.
  int moved = 0;
  for (int base = live / kStep * kStep; base < p.num_pages; base += kStep) {
    const int4 r = base == 0 ? first : load_counts(p, base);
    const int id0 = base + 4 * tid;
    int n = 0, total;
#pragma unroll
    for (int k = 0; k < 4; ++k) n += id0 + k >= live && id0 + k < p.num_pages && get(r, k) > 0;
    int at = moved + cta_exclusive_sum(n, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int id = id0 + k, ref = get(r, k);
      if (id < live || id >= p.num_pages) continue;
      new_refs[id] = 0;
      if (ref > 0) {
        const int to = l.free_ids[at];
        l.map[id] = to;
        l.free_ids[live + at] = id;  // sources behind the targets: live + holes <= num_pages
        new_refs[to] = ref;
        ++at;
      } else {
        l.map[id] = -1;
      }
    }
    moved += total;
  }
  if (tid == 0) {
    l.count[0] = moved;
    l.count[1] = live;
    if (num_live != nullptr) *num_live = live;
  }
}

// ---- movement
// Copies chunk c of a page's chunks from page src to page dst, the first `tokens` slots of its strip.
__device__ __forceinline__ void copy_chunk(const Pool& p, int c, int src, int dst, int tokens) {
  int k = 0;
  while (k + 1 < p.num_planes && c >= p.planes[k + 1].first) ++k;
  const Plane& pl = p.planes[k];
  const uint8_t* from = pl.data + pl.page_bytes * src;
  uint8_t* to = pl.data + pl.page_bytes * dst;
  if (pl.slot_bytes == 0) {  // kept once for a page: words
    for (int i = threadIdx.x; i < pl.page_bytes / 4; i += kCopyThreads)
      reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(from)[i];
    return;
  }
  c -= pl.first;
  const int strip = c / pl.chunks, off = (c % pl.chunks) * kChunk;
  int bytes = tokens * pl.slot_bytes - off;
  bytes = bytes < kChunk ? bytes : kChunk;
  if (bytes <= 0) return;
  from += static_cast<long long>(strip) * pl.strip_bytes + off;
  to += static_cast<long long>(strip) * pl.strip_bytes + off;
  constexpr int kIter = kChunk / 16 / kCopyThreads;
  uint4 v[kIter];
  const int n16 = bytes / 16;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int at = i * kCopyThreads + threadIdx.x;
    if (at < n16) v[i] = __ldcs(reinterpret_cast<const uint4*>(from) + at);
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int at = i * kCopyThreads + threadIdx.x;
    if (at < n16) __stcs(reinterpret_cast<uint4*>(to) + at, v[i]);
  }
  if ((bytes & 8) && threadIdx.x == 0)  // slots of 8 bytes: an odd number of them
    reinterpret_cast<uint2*>(to)[2 * n16] = reinterpret_cast<const uint2*>(from)[2 * n16];
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const Pool p, int n, const int32_t* src, const int32_t* dst,
                                                            const int32_t* tokens) {
  const long long work = static_cast<long long>(n) * p.chunks;
  for (long long u = blockIdx.x; u < work; u += gridDim.x) {
    const int i = static_cast<int>(u / p.chunks), c = static_cast<int>(u % p.chunks);
    const int a = src[i], b = dst[i];
    if (a < 0 || b < 0 || a == b) continue;
    int t = tokens == nullptr ? kBlock : tokens[i];
    if (a >= p.num_pages || b >= p.num_pages || t < 0 || t > kBlock) {
      if (threadIdx.x == 0) set_flag(p.flags, a >= p.num_pages || b >= p.num_pages ? kFlagBadPage : kFlagBadLength);
      continue;
    }
    copy_chunk(p, c, a, b, t);
  }
}

// Block-table rows of the children, counts of the shared pages, and the tails.
__global__ void __launch_bounds__(kCopyThreads) fork_move_kernel(const Pool p, const Lists l, int n,
                                                                 const int32_t* parents, const int32_t* children,
                                                                 int row_units) {
  pdl_wait_primary();
  const int per = p.chunks + row_units;
  const long long work = static_cast<long long>(n) * per;
  for (long long u = blockIdx.x; u < work; u += gridDim.x) {
    const int i = static_cast<int>(u / per), c = static_cast<int>(u % per);
    const int len = l.len[i];
    if (len < 0) continue;
    if (c < p.chunks) {
      if (l.dst[i] >= 0) copy_chunk(p, c, l.src[i], l.dst[i], l.tokens[i]);
      continue;
    }
    const long long from = static_cast<long long>(parents[i]) * p.max_pages;
    const long long to = static_cast<long long>(children[i]) * p.max_pages;
    const int c0 = (c - p.chunks) * kTableChunk;
    const int c1 = c0 + kTableChunk < len / kBlock ? c0 + kTableChunk : len / kBlock;
    for (int k = c0 + threadIdx.x; k < c1; k += kCopyThreads) {
      const int id = p.table[from + k];
      p.table[to + k] = id;
      if (in(id, p.num_pages)) atomicAdd(&p.refs[id], 1);
      else set_flag(p.flags, kFlagBadPage);
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const Pool p, const Lists l, int32_t* new_table,
                                                                    int row_units) {
  pdl_wait_primary();
  const int moved = l.count[0], sources = l.count[1];
  const long long rows = static_cast<long long>(p.num_seqs) * row_units;
  const long long work = rows + static_cast<long long>(moved) * p.chunks;
  for (long long u = blockIdx.x; u < work; u += gridDim.x) {
    if (u < rows) {
      const int s = static_cast<int>(u / row_units), c0 = static_cast<int>(u % row_units) * kTableChunk;
      const int len = p.seq_lens[s];
      int np = pages_of(len);
      if (!good_len(p, len)) {
        if (threadIdx.x == 0) set_flag(p.flags, kFlagBadLength);
        np = 0;
      }
      const long long row = static_cast<long long>(s) * p.max_pages;
      const int c1 = c0 + kTableChunk < p.max_pages ? c0 + kTableChunk : p.max_pages;
      for (int c = c0 + threadIdx.x; c < c1; c += kCopyThreads) {
        int id = p.table[row + c];
        if (c < np) {
          const int to = in(id, p.num_pages) ? l.map[id] : -1;  // -1: no page of the pool, or one that nobody counts
          if (to >= 0) id = to;
          else set_flag(p.flags, kFlagBadPage);
        }
        new_table[row + c] = id;
      }
    } else {
      const long long m = (u - rows) / p.chunks;
      copy_chunk(p, static_cast<int>((u - rows) % p.chunks), l.free_ids[sources + m], l.free_ids[m], kBlock);
    }
  }
}

msa_status make_pool(const msa_page_pool* a, bool tables, void* ws, size_t ws_bytes, Pool* out) {
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

int copy_grid(long long work, int sms) {
  const long long cap = static_cast<long long>(sms) * kCopyCtasPerSm;
  return static_cast<int>(work < cap ? work : cap);
}

// Launch chained to the kernel before it in the stream: it waits for that kernel's end itself.
template <typename... Args>
msa_status launch_chained(void (*kernel)(Args...), int grid, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

msa_status launched() { return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_pages_workspace_size(const msa_page_pool* a, size_t* bytes) {
  if (a == nullptr || bytes == nullptr || a->num_seqs < 0 || a->num_pages < 1) return MSA_ERR_INVALID_ARG;
  const size_t n = 256 + 4 * (5 * static_cast<size_t>(a->num_seqs) + 2 * static_cast<size_t>(a->num_pages));
  *bytes = (n + 255) / 256 * 256;
  return MSA_OK;
}

msa_status msa_pages_copy(const msa_page_pool* a, int32_t n, const int32_t* src, const int32_t* dst,
                          const int32_t* tokens, void* ws, size_t ws_bytes, void* stream) {
  Pool p;
  int sms = 0;
  msa_status s = make_pool(a, false, ws, ws_bytes, &p);
  if (s != MSA_OK) return s;
  if (n < 0 || (n > 0 && (src == nullptr || dst == nullptr))) return MSA_ERR_INVALID_ARG;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  if (n == 0 || p.chunks == 0) return MSA_OK;
  copy_kernel<<<copy_grid(static_cast<long long>(n) * p.chunks, sms), kCopyThreads, 0,
                static_cast<cudaStream_t>(stream)>>>(p, n, src, dst, tokens);
  return launched();
}

msa_status msa_pages_fork(const msa_page_pool* a, int32_t n, const int32_t* parents, const int32_t* children, void* ws,
                          size_t ws_bytes, void* stream) {
  Pool p;
  int sms = 0;
  msa_status s = make_pool(a, true, ws, ws_bytes, &p);
  if (s != MSA_OK) return s;
  if (n < 0 || n > p.num_seqs || (n > 0 && (parents == nullptr || children == nullptr))) return MSA_ERR_INVALID_ARG;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  if (n == 0) return MSA_OK;
  const Lists l = carve(ws, p.num_seqs, p.num_pages);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  fork_plan_kernel<<<1, kPlanThreads, 0, st>>>(p, l, n, parents, children);
  if ((s = launched()) != MSA_OK) return s;
  const int row_units = (p.max_pages + kTableChunk - 1) / kTableChunk;
  return launch_chained(fork_move_kernel, copy_grid(static_cast<long long>(n) * (p.chunks + row_units), sms), st, p, l,
                        static_cast<int>(n), parents, children, row_units);
}

msa_status msa_pages_reserve(const msa_page_pool* a, int32_t n, const int32_t* seqs, const int32_t* new_lens, void* ws,
                             size_t ws_bytes, void* stream) {
  Pool p;
  int sms = 0;
  msa_status s = make_pool(a, true, ws, ws_bytes, &p);
  if (s != MSA_OK) return s;
  if (n < 0 || n > p.num_seqs || (n > 0 && (seqs == nullptr || new_lens == nullptr))) return MSA_ERR_INVALID_ARG;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  if (n == 0) return MSA_OK;
  reserve_kernel<<<1, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p, carve(ws, p.num_seqs, p.num_pages), n,
                                                                            seqs, new_lens);
  return launched();
}

msa_status msa_pages_free(const msa_page_pool* a, int32_t n, const int32_t* seqs, void* ws, size_t ws_bytes,
                          void* stream) {
  Pool p;
  int sms = 0;
  msa_status s = make_pool(a, true, ws, ws_bytes, &p);
  if (s != MSA_OK) return s;
  if (n < 0 || (n > 0 && seqs == nullptr)) return MSA_ERR_INVALID_ARG;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  if (n == 0) return MSA_OK;
  free_kernel<<<n, 128, 0, static_cast<cudaStream_t>(stream)>>>(p, n, seqs);
  return launched();
}

msa_status msa_pages_compact(const msa_page_pool* a, int32_t* new_block_table, int32_t* new_ref_counts,
                             int32_t* num_live, void* ws, size_t ws_bytes, void* stream) {
  Pool p;
  int sms = 0;
  msa_status s = make_pool(a, true, ws, ws_bytes, &p);
  if (s != MSA_OK) return s;
  if (new_ref_counts == nullptr || (p.num_seqs > 0 && new_block_table == nullptr)) return MSA_ERR_INVALID_ARG;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  const Lists l = carve(ws, p.num_seqs, p.num_pages);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  compact_plan_kernel<<<1, kPlanThreads, 0, st>>>(p, l, new_ref_counts, num_live);
  if ((s = launched()) != MSA_OK) return s;
  const int row_units = (p.max_pages + kTableChunk - 1) / kTableChunk;
  const long long most = static_cast<long long>(p.num_seqs) * row_units +
                         static_cast<long long>(p.num_pages / 2 + 1) * p.chunks;
  if (most == 0) return MSA_OK;  // neither sequences nor planes: only the counts move
  return launch_chained(compact_move_kernel, copy_grid(most, sms), st, p, l, new_block_table, row_units);
}

}  // extern "C"
