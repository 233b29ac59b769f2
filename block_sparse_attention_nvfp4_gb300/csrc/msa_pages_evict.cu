// Eviction (msa_pages_evict): a sequence cut to its first tokens, its last ones and, head by head, the heaviest
// between, moved to pages of its own in the order of their positions. Two launches:
//   * kv8_evict_select_kernel: its first CTA is the plan (checks, new pages: the lowest free ids in list order); the
//     others take a (sequence, cache, head) each. The weight of the last token kept is found by radix
//     selection: three histograms over 11, 10 and 10 bits of the weights as numbers (non-negative FP32 numbers
//     order like their bits), then one pass that writes the kept positions and weights in order; of equal
//     weights the lowest positions stay. Bound: latency and L2 (the weights are read four times, the first time
//     from memory).
//   * kv8_evict_move_kernel: a CTA per (sequence, cache, head, new page) gathers the codes of 128 kept tokens. The new
//     page's scale is the largest of its tokens' pages'; codes of pages with that scale move as they are, the
//     others are multiplied by the scales' ratio and rounded once (exact between powers of two but for what falls
//     among the subnormals). Bound: memory, 128 bytes read here and there for each K and V row. The last CTA of a
//     sequence rewrites its row of the block table, its length and its old pages' counts.
// Ranks come from sums, so nothing depends on timing.
#include "msa_kv8_pipe.cuh"
#include "msa_pages.cuh"

namespace msa {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMaxCaches = MSA_MAX_PLANES / 4;

struct EvictCache {
  uint8_t* k_data;
  float* k_scale;
  uint8_t* v_data;
  float* v_scale;
  float* weights;
  long long stride;  // elements between the heads' weights
  int heads, first;  // heads, and those of the caches before
};

struct EvictParams {
  int n, keep, sinks, recent;
  int num_caches, heads;  // of all caches together
  int cap;                // kept tokens of any sequence: min(keep, the block table's)
  const int32_t* parents;
  const int32_t* children;
  int32_t* pos;           // [n][heads][cap] kept positions of sequences longer than `keep`
  float* weight;          // [n][heads][cap] their weights
  EvictCache caches[kMaxCaches];
};

// The cache and the head of place x among all caches' heads.
__device__ __forceinline__ int cache_of(const EvictParams& e, int x, int* head) {
  int c = 0;
  while (c + 1 < e.num_caches && x >= e.caches[c + 1].first) ++c;
  *head = x - e.caches[c].first;
  return c;
}

// len[i] = the parent's length (-1: the entry does nothing), src[i] = new pages, dst[i] = rank of the first of them,
// tokens[i] = 0 (counts the CTAs that are done).
__device__ void plan(const Pool& p, const Lists& l, const EvictParams& e, int32_t* claim_s) {
  const int tid = threadIdx.x;
  const int4 counts = load_counts(p, 0);
  int32_t* claim = p.num_seqs <= kSmemSeqs ? claim_s : l.claim;
  // claim[s] = the first entry whose child s is; parents' too, to see whether they are some entry's child
  for (int i = tid; i < e.n; i += kPlanThreads) {
    if (in(e.children[i], p.num_seqs)) claim[e.children[i]] = INT_MAX;
    if (in(e.parents[i], p.num_seqs)) claim[e.parents[i]] = INT_MAX;
  }
  __syncthreads();
  for (int i = tid; i < e.n; i += kPlanThreads)
    if (in(e.children[i], p.num_seqs)) atomicMin(&claim[e.children[i]], i);
  __syncthreads();
  int need_all = 0;
  for (int base = 0; base < e.n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0, len = -1;
    if (i < e.n) {
      const int par = e.parents[i], ch = e.children[i];
      bool good = in(par, p.num_seqs) && in(ch, p.num_seqs) && claim[ch] == i && (par == ch || p.seq_lens[ch] == 0);
      if (good && par != ch) {  // a sequence that is cut where it stands is nobody else's parent
        const int k = claim[par];
        good = k == INT_MAX || e.parents[k] != par;
      }
      if (!good) {
        set_flag(p.flags, kFlagBadSeq);
      } else {
        len = p.seq_lens[par];
        if (!good_len(p, len)) {
          set_flag(p.flags, kFlagBadLength);
          len = -1;
        } else if (len == 0 || (par == ch && len <= e.keep)) {
          len = -1;  // nothing to do
        } else {
          need = pages_of(len < e.keep ? len : e.keep);
          need = need < p.num_pages + 1 ? need : p.num_pages + 1;
        }
      }
    }
    int total;
    const int mine = cta_exclusive_sum(need, &total);
    if (i < e.n) {
      const long long at = static_cast<long long>(need_all) + mine;
      l.len[i] = len;
      l.src[i] = need;
      l.dst[i] = at < INT_MAX / 2 ? static_cast<int>(at) : INT_MAX / 2;
      l.tokens[i] = 0;
    }
    const long long sum = static_cast<long long>(need_all) + total;
    need_all = sum < INT_MAX / 2 ? static_cast<int>(sum) : INT_MAX / 2;
  }
  __syncthreads();
  const int have = find_free(p, need_all < p.num_pages ? need_all : p.num_pages, l.free_ids, counts);
  for (int i = tid; i < e.n; i += kPlanThreads)
    if (l.len[i] >= 0 && l.dst[i] + l.src[i] > have) {
      set_flag(p.flags, kFlagNoPage);
      l.len[i] = -1;
    }
  __syncthreads();
  for (int i = tid >> 5; i < e.n; i += kPlanWarps)
    if (l.len[i] >= 0)
      for (int k = tid & 31; k < l.src[i]; k += 32) p.refs[l.free_ids[l.dst[i] + k]] = 1;
}

__global__ void __launch_bounds__(kPlanThreads) kv8_evict_select_kernel(const Pool p, const Lists l, const EvictParams e) {
  __shared__ int32_t shared[kSmemSeqs];
  __shared__ int s_digit, s_above;
  __shared__ int w_sure[kPlanWarps], w_tie[kPlanWarps];
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    plan(p, l, e, shared);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = (blockIdx.x - 1) / e.heads, x = (blockIdx.x - 1) % e.heads;
  const int par = e.parents[i];
  if (!in(par, p.num_seqs)) return;
  const int N = p.seq_lens[par];
  if (!good_len(p, N) || N <= e.keep) return;
  int head;
  const EvictCache& c = e.caches[cache_of(e, x, &head)];
  const float* w = c.weights + (static_cast<long long>(par) * c.heads + head) * c.stride;
  const int lo = e.sinks, hi = N - e.recent;
  auto key = [](float v) { return v > 0.f ? __float_as_uint(v) : 0u; };  // (negative and NaN: 0)

  // the key of the last of the `m` heaviest in [lo, hi), and how many of the tokens that have it stay
  const int m = e.keep - e.sinks - e.recent;
  uint32_t found = 0u;  // its bits so far
  int rest = m;         // tokens to find among those that share them
  if (m > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 0 ? 11 : 10, shift = 20 - 10 * pass, bins = 1 << bits, above = shift + bits;
      for (int k = tid; k < bins; k += kPlanThreads) shared[k] = 0;
      __syncthreads();
      constexpr int kRun = 8;
      for (int base = lo; base < hi; base += kRun * kPlanThreads) {
        float v[kRun];
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int t = base + k * kPlanThreads + tid;
          v[k] = t < hi ? w[t] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int t = base + k * kPlanThreads + tid;
          const uint32_t u = key(v[k]);
          if (t < hi && (pass == 0 || u >> above == found >> above)) atomicAdd(&shared[u >> shift & (bins - 1)], 1);
        }
      }
      __syncthreads();
      // from the highest digit down: the one where the count reaches `rest`
      const int per = bins / kPlanThreads;  // 2 or 1
      int mine = 0;
      for (int k = 0; k < per; ++k) mine += shared[bins - 1 - (tid * per + k)];
      int total;
      int at = cta_exclusive_sum(mine, &total);
      for (int k = 0; k < per; ++k) {
        const int d = bins - 1 - (tid * per + k), n = shared[d];
        if (at < rest && at + n >= rest) {
          s_digit = d;
          s_above = at;
        }
        at += n;
      }
      __syncthreads();
      found |= static_cast<uint32_t>(s_digit) << shift;
      rest -= s_above;
      __syncthreads();
    }
  }
  const int ties = rest;
  // the kept tokens in order: a warp has 256 in a row, 32 at a time
  int32_t* pos = e.pos + (static_cast<long long>(i) * e.heads + x) * e.cap;
  float* weight = e.weight + (static_cast<long long>(i) * e.heads + x) * e.cap;
  int sure_all = 0, tie_all = 0;
  constexpr int kRows = 8;
  for (int base = 0; base < N; base += kRows * kPlanThreads) {
    float v[kRows];
    unsigned sure[kRows], tie[kRows];
    const int t0 = base + warp * 32 * kRows + lane;
#pragma unroll
    for (int k = 0; k < kRows; ++k) v[k] = t0 + 32 * k < N ? w[t0 + 32 * k] : 0.f;
    int n_sure = 0, n_tie = 0;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int t = t0 + 32 * k;
      const bool fixed = t < lo || t >= hi;
      const uint32_t u = key(v[k]);
      sure[k] = __ballot_sync(0xFFFFFFFFu, t < N && (fixed || (m > 0 && u > found)));
      tie[k] = __ballot_sync(0xFFFFFFFFu, t < N && !fixed && m > 0 && u == found);
      n_sure += __popc(sure[k]);
      n_tie += __popc(tie[k]);
    }
    if (lane == 0) {
      w_sure[warp] = n_sure;
      w_tie[warp] = n_tie;
    }
    __syncthreads();
    const int a = w_sure[lane], b = w_tie[lane];
    int sa = a, sb = b;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int oa = __shfl_up_sync(0xFFFFFFFFu, sa, d), ob = __shfl_up_sync(0xFFFFFFFFu, sb, d);
      if (lane >= d) {
        sa += oa;
        sb += ob;
      }
    }
    int sure_at = sure_all + __shfl_sync(0xFFFFFFFFu, sa - a, warp), tie_at = tie_all + __shfl_sync(0xFFFFFFFFu, sb - b, warp);
    sure_all += __shfl_sync(0xFFFFFFFFu, sa, 31);
    tie_all += __shfl_sync(0xFFFFFFFFu, sb, 31);
    const unsigned below = (1u << lane) - 1u;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int rank = tie_at + __popc(tie[k] & below);
      const bool kept = (sure[k] >> lane & 1u) || ((tie[k] >> lane & 1u) && rank < ties);
      if (kept) {
        const int to = sure_at + __popc(sure[k] & below) + (rank < ties ? rank : ties);
        pos[to] = t0 + 32 * k;
        weight[to] = v[k];
      }
      sure_at += __popc(sure[k]);
      tie_at += __popc(tie[k]);
    }
    __syncthreads();  // the warps' counts are free again
  }
}

// 16 codes times a ratio, rounded once.
__device__ __forceinline__ uint4 rescale(uint4 v, float ratio) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t lo, hi;
    e4m3x4_f16x4(x[k], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[k] = f32x2_e4m3x2(a.x * ratio, a.y * ratio) | f32x2_e4m3x2(b.x * ratio, b.y * ratio) << 16;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

__global__ void __launch_bounds__(kMoveThreads) kv8_evict_move_kernel(const Pool p, const Lists l, const EvictParams e, int pages) {
  __shared__ long long src[kBlock];               // row of the code planes; -1: none
  __shared__ float ratio[2][kBlock], top[2][4];
  __shared__ int s_last;
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j = blockIdx.x % pages, ix = blockIdx.x / pages, i = ix / e.heads, x = ix % e.heads;
  const int len = l.len[i], need = l.src[i];
  if (len < 0 || j >= need) return;
  const int par = e.parents[i], ch = e.children[i], kept = len < e.keep ? len : e.keep;
  const int count = kept - j * kBlock < kBlock ? kept - j * kBlock : kBlock;
  const int id = l.free_ids[l.dst[i] + j];
  int head;
  const EvictCache& c = e.caches[cache_of(e, x, &head)];
  float s[2] = {0.f, 0.f};
  if (tid < kBlock) {
    long long from = -1;
    if (tid < count) {
      const int k = j * kBlock + tid;
      const long long at = (static_cast<long long>(i) * e.heads + x) * e.cap + k;
      const int t = len <= e.keep ? k : e.pos[at];
      float* weights = c.weights + head * c.stride;
      const float w = len <= e.keep ? weights[par * static_cast<long long>(c.heads) * c.stride + t] : e.weight[at];
      weights[ch * static_cast<long long>(c.heads) * c.stride + k] = w;
      const int page = p.table[static_cast<long long>(par) * p.max_pages + t / kBlock];
      if (in(page, p.num_pages)) {
        const long long ph = static_cast<long long>(page) * c.heads + head;
        from = ph * kBlock + t % kBlock;
        s[0] = c.k_scale[ph];
        s[1] = c.v_scale[ph];
      } else {
        set_flag(p.flags, kFlagBadPage);
      }
    }
    src[tid] = from;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if (!(s[z] > 0.f && s[z] <= 3.402823466e38f)) s[z] = 0.f;  // a scale that is none counts as 0
      float big = s[z];
#pragma unroll
      for (int d = 1; d < 32; d *= 2) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, d));
      if (lane == 0) top[z][warp] = big;
    }
  }
  __syncthreads();
  float scale[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) scale[z] = fmaxf(fmaxf(top[z][0], top[z][1]), fmaxf(top[z][2], top[z][3]));
  const long long to = static_cast<long long>(id) * c.heads + head;
  if (tid < kBlock)
#pragma unroll
    for (int z = 0; z < 2; ++z) ratio[z][tid] = scale[z] > 0.f ? s[z] / scale[z] : 0.f;
  if (tid == 0) {
    c.k_scale[to] = scale[0];
    c.v_scale[to] = scale[1];
  }
  __syncthreads();
  // thread: one 16-byte piece of every 32nd row, all loads on their way at once
  constexpr int kRows = kBlock * 8 / kMoveThreads;
  const int piece = tid & 7, row0 = tid >> 3;
  uint4 v[2][kRows];
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long from = src[row0 + 32 * k];
      v[z][k] = make_uint4(0u, 0u, 0u, 0u);
      if (from >= 0) v[z][k] = __ldcs(reinterpret_cast<const uint4*>((z == 0 ? c.k_data : c.v_data) + from * kDim) + piece);
    }
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int row = row0 + 32 * k;
      const float f = ratio[z][row];
      if (f != 1.f) v[z][k] = rescale(v[z][k], f);
      if (row < count)
        reinterpret_cast<uint4*>((z == 0 ? c.k_data : c.v_data) + (to * kBlock + row) * kDim)[piece] = v[z][k];
    }
  // the sequence's last CTA: nobody reads its old row any more
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(&l.tokens[i], 1) == need * e.heads - 1;
  }
  __syncthreads();
  if (!s_last) return;
  int32_t* row = p.table + static_cast<long long>(ch) * p.max_pages;
  if (par == ch)
    for (int k = tid; k < pages_of(len); k += kMoveThreads) {
      const int old = row[k];
      if (!in(old, p.num_pages)) {
        set_flag(p.flags, kFlagBadPage);
      } else if (atomicSub(&p.refs[old], 1) <= 0) {
        atomicAdd(&p.refs[old], 1);
        set_flag(p.flags, kFlagBadPage);
      }
    }
  __syncthreads();
  for (int k = tid; k < need; k += kMoveThreads) row[k] = l.free_ids[l.dst[i] + k];
  if (tid == 0) p.seq_lens[ch] = kept;
}

msa_status check_evict(const msa_page_pool* a, int num_caches, const msa_kv8_evict_cache* caches, int n, int keep, int* heads) {
  if (a == nullptr || a->num_seqs < 0 || a->num_pages < 1 || a->max_pages_per_seq < 1) return MSA_ERR_INVALID_ARG;
  if (num_caches < 1 || num_caches > kMaxCaches || caches == nullptr || n < 0 || n > a->num_seqs || keep < 1) return MSA_ERR_INVALID_ARG;
  *heads = 0;
  for (int c = 0; c < num_caches; ++c) {
    if (caches[c].num_kv_heads < 1 || caches[c].num_kv_heads > kKv8MaxHeads) return MSA_ERR_UNSUPPORTED;
    *heads += caches[c].num_kv_heads;
  }
  return MSA_OK;
}
// Kept tokens of any sequence.
long long kept_cap(const msa_page_pool* a, int keep) {
  const long long most = static_cast<long long>(a->max_pages_per_seq) * kBlock;
  return keep < most ? keep : most;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_pages_evict_scratch_size(const msa_page_pool* a, int32_t num_caches, const msa_kv8_evict_cache* caches,
                                        int32_t n, int32_t keep, size_t* bytes) {
  if (bytes == nullptr) return MSA_ERR_INVALID_ARG;
  int heads = 0;
  const msa_status s = check_evict(a, num_caches, caches, n, keep, &heads);
  if (s != MSA_OK) return s;
  *bytes = 8 * static_cast<size_t>(n) * heads * kept_cap(a, keep);
  return MSA_OK;
}

msa_status msa_pages_evict(const msa_page_pool* a, int32_t n, const int32_t* parents, const int32_t* children,
                           int32_t num_caches, const msa_kv8_evict_cache* caches, int32_t keep, int32_t sinks,
                           int32_t recent, void* scratch, size_t scratch_bytes, void* ws, size_t ws_bytes, void* stream) {
  EvictParams e = {};
  msa_status s = check_evict(a, num_caches, caches, n, keep, &e.heads);
  if (s != MSA_OK) return s;
  Pool p;
  int sms = 0;
  if ((s = make_pool(a, true, ws, ws_bytes, &p)) != MSA_OK) return s;
  if (sinks < 0 || recent < 0 || static_cast<long long>(sinks) + recent > keep) return MSA_ERR_INVALID_ARG;
  if (n > 0 && (parents == nullptr || children == nullptr)) return MSA_ERR_INVALID_ARG;
  auto unaligned = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) != 0; };
  int first = 0;
  for (int c = 0; c < num_caches; ++c) {
    const msa_kv8_evict_cache& f = caches[c];
    if (f.k_data == nullptr || f.k_scale == nullptr || f.v_data == nullptr || f.v_scale == nullptr || f.weights == nullptr ||
        unaligned(f.k_data, 16) || unaligned(f.v_data, 16) || unaligned(f.k_scale, 4) || unaligned(f.v_scale, 4) ||
        unaligned(f.weights, 4) || f.head_stride < static_cast<int64_t>(a->max_pages_per_seq) * kBlock)
      return MSA_ERR_INVALID_ARG;
    e.caches[c] = {f.k_data, f.k_scale, f.v_data, f.v_scale, f.weights, f.head_stride, f.num_kv_heads, first};
    first += f.num_kv_heads;
  }
  e.n = n;
  e.keep = keep;
  e.sinks = sinks;
  e.recent = recent;
  e.num_caches = num_caches;
  e.cap = static_cast<int>(kept_cap(a, keep));
  e.parents = parents;
  e.children = children;
  const size_t half = 4 * static_cast<size_t>(n) * e.heads * e.cap;
  if (n > 0 && (scratch == nullptr || unaligned(scratch, 16) || scratch_bytes < 2 * half)) return MSA_ERR_WORKSPACE;
  e.pos = static_cast<int32_t*>(scratch);
  e.weight = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + half);
  const int pages = (e.cap + kBlock - 1) / kBlock;
  const long long items = static_cast<long long>(n) * e.heads, moves = items * pages;
  if (moves >= (1LL << 31) || items + 1 >= (1LL << 31)) return MSA_ERR_UNSUPPORTED;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  if (n == 0) return MSA_OK;
  const Lists l = carve(ws, p.num_seqs, p.num_pages);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  kv8_evict_select_kernel<<<static_cast<unsigned>(items + 1), kPlanThreads, 0, st>>>(p, l, e);
  if ((s = launched()) != MSA_OK) return s;
  return launch_chained(kv8_evict_move_kernel, static_cast<int>(moves), kMoveThreads, st, p, l, e, pages);
}

}  // extern "C"
