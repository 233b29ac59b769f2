// Eviction (msa_pages_evict): a sequence cut to its first tokens, its last ones and, head by head, the heaviest
// between, moved to pages of its own in the order of their positions. Two launches:
//   * kv8_evict_select_kernel. Its first CTA is the plan: checks, new pages (the lowest free ids in list order). Its
//     others, one for each (sequence, cache, head), select: the weight of the last token kept is found by
//     radix selection, three histograms over 11, 10 and 10 bits of the weights as numbers (non-negative FP32 numbers
//     order like their bits), then the kept positions and weights are written in order; of equal weights the lowest
//     positions stay. The weights are read once where they fit the registers (8,192 tokens), else four times, five
//     when many are equal. A warp has a 32nd of the sequence. Bound: instructions (issue slots 63 % busy over 65,536 tokens,
//     28 us); one CTA a head, whatever its length: a sequence of 524,288 tokens with 4 heads, cut to 65,536, takes 204 us on
//     four SMs. (Over 32 sequences of up to 65,536 tokens: four counts of a digit, by lane, against conflicts: no faster. Warps
//     that take their 128 tokens in turn and meet for their sums: as fast where tokens are counted once more instead. Clusters
//     of two or four CTAs a head, whose histograms were added up through distributed shared memory: no faster and slower, the
//     reading took what the split saved.)
//   * kv8_evict_move_kernel: a CTA per (sequence, cache, head, new page) gathers the codes of 128 kept tokens. The new
//     page's scale is the largest of its tokens' pages'; codes of pages with that scale move as they are, the
//     others are multiplied by the scales' ratio and rounded once (exact between powers of two but for what falls
//     among the subnormals). Bound: memory, 128 bytes read here and there for each K and V row (32 sequences of 4 heads
//     cut to 8,192 tokens: 537 MB in 86 us). The last CTA of a
//     sequence to have read its old row of the block table rewrites it, the length and the old pages' counts.
// Ranks come from sums, so nothing depends on timing.
#include <type_traits>

#include "msa_kv8_pipe.cuh"
#include "msa_pages.cuh"

namespace msa {
namespace {

constexpr int kSelectThreads = 1024, kMoveThreads = 256;
constexpr int kMaxCaches = MSA_MAX_PLANES / 4;
constexpr int kMostPages = (1 << 24) - 256;     // of a sequence: positions past its end, of a whole round, are still ints

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
  int2* kept;             // [n][heads][cap] kept positions of sequences longer than `keep`, their weights' bits
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

// CTA 0: the plan. The others: one per (sequence, cache, head), x among all caches' heads.
__global__ void __launch_bounds__(kSelectThreads) kv8_evict_select_kernel(const Pool p, const Lists l, const EvictParams e) {
  static_assert(kSelectThreads == kPlanThreads, "");
  constexpr int kWarps = kSelectThreads / 32;
  // A warp has a 32nd of the sequence, in whole 128s, and takes kRun of them at once: lanes have 4 tokens in a row.
  constexpr int kRun = 2, kRound = kRun * 128;
  __shared__ int hist[kSmemSeqs];                    // by pass: 2,048, 1,024 and 1,024 digits; the plan's claims
  __shared__ int w_part[kWarps], s_found[3];
  __shared__ int w_sure[kWarps], w_tie[kWarps];      // by warp: tokens kept for sure, and ties
  // The tokens that the last pass counts, when they are few: digit and warp << 16.
  constexpr int kFew = 1024;
  __shared__ int few[kFew], s_few;
  static_assert(kSmemSeqs >= 4096 && kFew <= kSelectThreads, "");
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    plan(p, l, e, hist);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x - 1, i = item / e.heads, x = item % e.heads;
  const int par = e.parents[i];
  const int N = in(par, p.num_seqs) ? p.seq_lens[par] : -1;
  if (!good_len(p, N) || N <= e.keep) return;
  int head;
  const EvictCache& c = e.caches[cache_of(e, x, &head)];
  const float* w = c.weights + (static_cast<long long>(par) * c.heads + head) * c.stride;
  const int lo = e.sinks, hi = N - e.recent;
  auto key = [](float v) { return __float_as_uint(fmaxf(v, 0.f)); };  // (negative and NaN: 0)
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
  const int seg = (N + 128 * kWarps - 1) / (128 * kWarps) * 128, begin = warp * seg, end = min(N, begin + seg);
  // the next round's tokens are on their way while these are looked at (7 us a pass of 65,536 tokens without)
  float4 v[kRun], next[kRun];
  auto load = [&](int base) {
    if (wide && base + kRound <= N) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) next[k] = *reinterpret_cast<const float4*>(w + base + 128 * k + 4 * lane);
      return;
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const int t = base + 128 * k + 4 * lane;
      next[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (wide && t + 3 < N) {
        next[k] = *reinterpret_cast<const float4*>(w + t);
      } else {
        if (t < N) next[k].x = w[t];
        if (t + 1 < N) next[k].y = w[t + 1];
        if (t + 2 < N) next[k].z = w[t + 2];
        if (t + 3 < N) next[k].w = w[t + 3];
      }
    }
  };
  const bool once = seg <= kRound;
  auto step = [&](int base) {
#pragma unroll
    for (int k = 0; k < kRun; ++k) v[k] = next[k];
    if (!once) load(base + kRound < end ? base + kRound : begin);  // (the first again, for the pass that follows)
  };
  load(begin);
  for (int k = tid; k < 4096; k += kSelectThreads) hist[k] = 0;
  __syncthreads();

  // the key of the last of the `m` heaviest in [lo, hi), and how many of the tokens that have it stay
  const int m = e.keep - e.sinks - e.recent;
  uint32_t found = m > 0 ? 0u : ~0u;  // its bits so far (no weight's, when there is none)
  int rest = m;         // tokens to find among those that share them
  // Tokens of the warp that stay for sure: the first, the last, the lane's share of those above all that the last pass
  // counts. Those are listed when they are few, so that no further pass has to look which of them stay (65,536 tokens 31.8 us
  // with one, 28.3 without; of tokens that the registers hold it costs less than the list).
  bool list = false;
  int sure = lane == 0 ? max(min(end, lo) - begin, 0) + max(end - max(begin, hi), 0) : 0;
  if (tid == 0) s_few = 0;
  if (m > 0) {
    // Counts the digits of the tokens whose higher bits are those found so far: key - found is below 2^above then.
    auto count = [&](auto which, int* h, int shift, uint32_t below) {
      constexpr int pass = decltype(which)::value;
      for (int base = begin; base < end; base += kRound) {
        step(base);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int t0 = base + 128 * k, t = t0 + 4 * lane;
          if (t0 >= end) break;
          const float f[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          auto add = [&](int c) {
            const uint32_t d = key(f[c]) - found;
            if (pass == 0 || d < below) {
              atomicAdd(&h[d >> shift], 1);
              if (pass == 2 && list) few[atomicAdd(&s_few, 1)] = static_cast<int>(d) | warp << 16;
            }
            if (pass == 2) sure += static_cast<int>(d) >= static_cast<int>(below);
          };
          if (t0 >= lo && t0 + 127 < hi) {
#pragma unroll
            for (int c = 0; c < 4; ++c) add(c);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (t + c >= lo && t + c < hi) add(c);
          }
        }
      }
    };
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 0 ? 11 : 10, shift = 20 - 10 * pass, bins = 1 << bits, above = shift + bits;
      int* h = hist + (pass == 0 ? 0 : 1024 + 1024 * pass);
      if (pass == 0) count(std::integral_constant<int, 0>{}, h, shift, 0u);
      else if (pass == 1) count(std::integral_constant<int, 1>{}, h, shift, 1u << above);
      else count(std::integral_constant<int, 2>{}, h, shift, 1u << above);
      __syncthreads();
      // from the highest digit down: the one where the count reaches `rest`
      const int per = bins / kSelectThreads;  // 2 or 1
      const int d0 = bins - 1 - tid * per, n0 = h[d0], n1 = per > 1 ? h[d0 - 1] : 0;
      int incl = n0 + n1;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
      }
      if (lane == 31) w_part[warp] = incl;
      __syncthreads();
      const int at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w_part[lane] : 0) + incl - n0 - n1;
      if (at < rest && at + n0 + n1 >= rest) {
        const bool second = at + n0 < rest;
        s_found[0] = second ? d0 - 1 : d0;
        s_found[1] = second ? at + n0 : at;
        s_found[2] = second ? n1 : n0;
      }
      __syncthreads();
      found |= static_cast<uint32_t>(s_found[0]) << shift;
      rest -= s_found[1];
      if (pass == 1) list = !once && s_found[2] <= kFew;
    }
  }
  const int ties = rest;
  // The tokens of 4 in a row that stay for sure, as bits, and above them the ties.
  auto kinds = [&](int k, int t0) {
    const int t = t0 + 4 * lane;
    const float f[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t kind = 0u;
    if (t0 >= end) return kind;
    if (t0 >= lo && t0 + 127 < hi) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t u = key(f[c]);
        kind |= u > found ? 1u << c : u == found ? 16u << c : 0u;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t u = key(f[c]);
        if (t + c < N) kind |= t + c < lo || t + c >= hi || u > found ? 1u << c : u == found ? 16u << c : 0u;
      }
    }
    return kind;
  };
  // how many each warp has, and so where its own begin
  int tie = 0;
  if (m > 0 && !list) {
    sure = 0;
    for (int base = begin; base < end; base += kRound) {
      step(base);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const uint32_t kind = kinds(k, base + 128 * k);
        sure += __popc(kind & 15u);
        tie += __popc(kind >> 4);
      }
    }
  }
  sure = __reduce_add_sync(0xFFFFFFFFu, sure);
  tie = __reduce_add_sync(0xFFFFFFFFu, tie);
  if (lane == 0) {
    w_sure[warp] = sure;
    w_tie[warp] = tie;
  }
  __syncthreads();
  if (list) {
    if (tid < s_few) {
      const int d = few[tid] & 1023, last = s_found[0], of = few[tid] >> 16;
      if (d >= last) atomicAdd(d > last ? &w_sure[of] : &w_tie[of], 1);
    }
    __syncthreads();
  }
  int sure_at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w_sure[lane] : 0);
  int tie_at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w_tie[lane] : 0);
  int2* kept = e.kept + static_cast<long long>(item) * e.cap;
  for (int base = begin; base < end; base += kRound) {
    step(base);
    uint32_t kind[kRun], incl[kRun];  // sums over lanes: sure ones in the low half, ties in the high one
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      kind[k] = kinds(k, base + 128 * k);
      incl[k] = __popc(kind[k] & 15u) | __popc(kind[k] >> 4) << 16;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl[k], d);
        if (lane >= d) incl[k] += o;
      }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const uint32_t all = __shfl_sync(0xFFFFFFFFu, incl[k], 31);
      int s_at = sure_at + (incl[k] & 0xFFFFu) - __popc(kind[k] & 15u);
      const int t = base + 128 * k + 4 * lane;
      const float f[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      if (all >> 16 == 0u) {  // no ties, as a rule
        int2* at = kept + (s_at + min(tie_at, ties));
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (kind[k] >> c & 1u) *at++ = make_int2(t + c, __float_as_int(f[c]));
      } else {
        int t_at = tie_at + (incl[k] >> 16) - __popc(kind[k] >> 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool is_sure = kind[k] >> c & 1u, is_tie = kind[k] >> c & 16u;
          if (is_sure || (is_tie && t_at < ties)) kept[s_at + min(t_at, ties)] = make_int2(t + c, __float_as_int(f[c]));
          s_at += is_sure;
          t_at += is_tie;
        }
      }
      sure_at += all & 0xFFFFu;
      tie_at += all >> 16;
    }
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
      const int2 from_select = len <= e.keep ? make_int2(k, 0) : e.kept[at];
      const int t = from_select.x;
      float* weights = c.weights + head * c.stride;
      const float w = len <= e.keep ? weights[par * static_cast<long long>(c.heads) * c.stride + t] : __int_as_float(from_select.y);
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
    // The last CTA of the sequence to come here: nobody reads its old row any more (the reads' values were used above).
    s_last = atomicAdd(&l.tokens[i], 1) == need * e.heads - 1;
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
  if (a->max_pages_per_seq > kMostPages) return MSA_ERR_UNSUPPORTED;
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
  // a `keep` as long as the block table: no sequence is longer, so none is selected from
  const bool selects = n > 0 && keep < static_cast<long long>(a->max_pages_per_seq) * kBlock;
  if (selects && (scratch == nullptr || unaligned(scratch, 16) || scratch_bytes < sizeof(int2) * static_cast<size_t>(n) * e.heads * e.cap))
    return MSA_ERR_WORKSPACE;
  e.kept = static_cast<int2*>(scratch);
  const int pages = (e.cap + kBlock - 1) / kBlock;
  const long long items = static_cast<long long>(n) * e.heads, moves = items * pages;
  if (moves >= (1LL << 31) || items + 1 >= (1LL << 31)) return MSA_ERR_UNSUPPORTED;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  if (n == 0) return MSA_OK;
  const Lists l = carve(ws, p.num_seqs, p.num_pages);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  kv8_evict_select_kernel<<<static_cast<unsigned>(items + 1), kSelectThreads, 0, st>>>(p, l, e);
  if ((s = launched()) != MSA_OK) return s;
  return launch_chained(kv8_evict_move_kernel, static_cast<int>(moves), kMoveThreads, st, p, l, e, pages);
}

}  // extern "C"
