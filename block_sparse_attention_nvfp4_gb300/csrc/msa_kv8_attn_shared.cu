// msa_kv8_attn_shared: attention over the 8-bit cache for requests whose block tables begin with the same pages, as
// msa_pages_fork leaves them. kv8_groups_kernel finds, per group of requests, the leading pages that all members' rows list
// and that all their query rows see whole. The attention kernel (msa_kv8_attn.cuh) then takes chunks of all members' rows
// together: an item's tiles are the group's pages, for all of its rows, and behind them each member's own, for that member's
// rows alone (the others' weights are 0). So one softmax runs over a row's shared and own keys, shared pages are read once
// for a chunk of 128 / q_per_kv rows (kSharedRows at most) instead of once for each request, and a tile of the tensor cores is
// full of rows instead of copies of a few. (Own pages as items of their own, whose FP32 results a further kernel joined with
// the shared pages', took 5 % longer for 64 rows of one prompt and for 4 prompts of 16 requests: hundreds of items of one or
// two tiles, each of which starts and ends.) Whether that pays is counted in reads of a page by a row chunk (below).
// Floor: the shared pages once a group and the own pages once, or the products: 9 us for 64 beams on 16,384 tokens, 49 for 4 x
// 16 requests of 8 rows on 8,192 .. 32,768 tokens each. Measured 49 and 115 us (msa_kv8_attn, each page read for every request: 173 and 198).
// Bound: of 64 beams, latency: the groups' kernel 7 us, 17 tiles a CTA, the partials 9; of 4 x 16 requests, own tiles, whose
// steps cost as much with 8 rows as with 128.
#include "msa_kv8_attn.cuh"

namespace msa {
namespace {

constexpr int kGroupThreads = 1024;
// The sum over a warp's lanes of numbers from 0 to 2^50.
__device__ __forceinline__ long long warp_sum(long long x) {
  const unsigned low = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(x & 0xFFFFFF));
  return low + (static_cast<long long>(__reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(x >> 24))) << 24);
}
// Reads of a page by a row chunk, over all KV heads and groups, that sharing has to save before it pays. (A request's pages are
// read once for each of its row chunks, a group's once for each of the group's: prompts, whose chunks are full
// already, save next to nothing.) The groups' kernel and more partials an item cost some 8 us against the plain call, which is
// taken where the sizes leave less than kMinSizes to save. Behind the groups' kernel, with tiles laid out for a group's rows, it
// pays sooner: from kMinSaved on. Measured (4 KV heads, BF16, one row a member; shared / behind the groups' kernel but
// alone / the plain call, us):
//     768 saved, 4 members   26.7 / 26.8 / 20.7      1,792, 8 members       26.7 / 32.9 / 26.8
//     896, 8 members         26.4 / 26.8 / 22.6      1,920, 16 members      28.5 / 36.9 / 27.0
//     960, 16 members        27.3 / 30.9 / 22.8      3,360, 4 groups of 4   32.9 / 43.2 / 38.6
//   1,536, 4 groups of 4     28.9 / 32.9 / 26.9      3,840, 16 members      30.8 / 47.4 / 37.0
// The sizes have the table's width, not the lengths, which are on the device: 4 samples on 31 shared pages take 16.6 us, the
// plain call, with a table as wide as they are long, and 22.6 with one of 512 pages, behind the groups' kernel but alone.
constexpr int kMinSizes = 2048, kMinSaved = 768;

// Row chunks whose own tiles the groups' kernel adds up at once, in 32 bits. No more than kStep + kMaxReqs pieces of members'
// rows lie in them, with a table's pages each: the plain call takes tables longer than kLongTable (44.7 million tokens).
constexpr int kStep = 2 * kGroupThreads;
constexpr int kLongTable = static_cast<int>((1LL << 31) / (kStep + kMaxReqs));

// CTA g: group g; the last CTA: the requests outside every group. groups[g] = {shared pages (0: none), first row, rows,
// first member}, skip[b] = shared pages of request b. Bound: latency, a chain of dependent reads (the bounds, the
// lengths, the tables); the members' entries are compared kRun at a time, all on their way at once (one after the other
// 64 members of 128 pages took 9.3 us).
__global__ void __launch_bounds__(kGroupThreads) kv8_groups_kernel(const Kv8AttnParams p, const int32_t* indptr, int4* groups,
                                                                   int32_t* skip, GroupChunk* chunks, long long least) {
  __shared__ int s_limit, s_members, s_pages;
  __shared__ long long s_apart[kGroupThreads / 32];
  static_assert(kGroupThreads == 1024, "");
  pdl_launch_dependents();
  const int tid = threadIdx.x, g = blockIdx.x, n = p.num_groups;
  if (tid == 0) s_limit = s_pages = INT_MAX, s_members = 0;
  const int b0 = g < n ? indptr[g] : 0, b1 = g < n ? indptr[g + 1] : 0;
  bool bad = false;  // one bad entry: no group shares anything (two groups might claim a request)
  for (int i = tid; i <= n; i += kGroupThreads) {
    const int x = indptr[i];
    bad |= x < 0 || x > p.num_reqs || (i < n && indptr[i + 1] < x);
  }
  bad = __syncthreads_or(bad);
  if (bad && g == 0 && tid == 0) set_flag(p.flags, kFlagBadLength);
  if (g == n) {
    const int first = bad ? 0 : indptr[0], last = bad ? 0 : indptr[n];
    for (int b = tid; b < p.num_reqs; b += kGroupThreads)
      if (b < first || b >= last) skip[b] = 0;
    return;
  }
  if (bad) {
    if (tid == 0) groups[g] = make_int4(0, 0, 0, 0);
    return;
  }
  int limit = INT_MAX, members = 0;
  long long apart = 0;  // tiles of the members when they are alone
  bool wrong = false;
  for (int b = b0 + tid; b < b1; b += kGroupThreads) {
    Req q;
    if (!load_req<kAll>(p, b, &q)) {  // (its flag is the attention's to set)
      wrong = true;
    } else if (q.R > 0) {
      limit = min(limit, (q.N - q.R) / kBlock);
      ++members;
      q.pages = 0;
      const int last = chunks_of<kSharedWide>(p, q) - 1;
      apart += tiles_of<kSharedWide>(p, q, last);
      if (last > 0) apart += tiles_before<kSharedWide>(p, q, last);
    }
  }
  apart = warp_sum(apart);
  if ((tid & 31) == 0) s_apart[tid >> 5] = apart;
  limit = __reduce_min_sync(0xFFFFFFFFu, limit);
  members = __reduce_add_sync(0xFFFFFFFFu, members);
  if ((tid & 31) == 0) {
    if (limit != INT_MAX) atomicMin(&s_limit, limit);
    if (members > 0) atomicAdd(&s_members, members);
  }
  wrong = __syncthreads_or(wrong);
  members = s_members;
  const int most = wrong || members < 2 ? 0 : s_limit;
  // the first page that some member's row has different from the first one's (members without rows have nothing to read:
  // they count as equal)
  const int32_t* first = p.block_table + static_cast<long long>(b0) * p.max_pages;
  constexpr int kRun = 8;
  int differs = INT_MAX;
  if (most > 0) {
    // thread tid's entries among all members' pages in a row: tid, tid + kGroupThreads, ..
    const int dm = kGroupThreads / most, dc = kGroupThreads - dm * most;
    int m = tid / most, at = tid - m * most;
    while (m < b1 - b0) {
      int c[kRun], mine[kRun], theirs[kRun], rows[kRun];
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const bool on = m < b1 - b0;
        c[k] = on ? at : 0;
        mine[k] = first[c[k]];
        theirs[k] = on ? first[m * static_cast<long long>(p.max_pages) + c[k]] : mine[k];
        rows[k] = on ? p.q_indptr[b0 + m + 1] - p.q_indptr[b0 + m] : 0;
        m += dm;
        at += dc;
        if (at >= most) at -= most, ++m;
      }
#pragma unroll
      for (int k = 0; k < kRun; ++k)
        if (mine[k] != theirs[k] && rows[k] > 0) differs = min(differs, c[k]);
    }
  }
  differs = __reduce_min_sync(0xFFFFFFFFu, differs);
  if (differs != INT_MAX && (tid & 31) == 0) atomicMin(&s_pages, differs);
  __syncthreads();
  const int pages = min(most, s_pages);
  const int r0 = b0 < b1 ? p.q_indptr[b0] : 0, rows = b0 < b1 ? p.q_indptr[b1] - r0 : 0;
  // What sharing saves: reads of a page by a row chunk. Of the shared pages at most those of all members but one, whose rows
  // have a chunk at least each when they are alone and lie in as many when they are together.
  const bool some = pages > 0 && static_cast<long long>(members - 1) * pages * p.num_kv_heads >= least;
  auto decide = [&](int n) {
    for (int b = b0 + tid; b < b1; b += kGroupThreads) skip[b] = n;
    if (tid == 0) groups[g] = make_int4(n, r0, rows, b0);
  };
  decide(some ? pages : 0);
  if (some) {
    // the row chunks: the members' own tiles in each, places on the line up to its end. (The groups before this one have at
    // most r0 / chunk + g chunks.)
    __shared__ int s_own[kStep], s_part[kGroupThreads / 32];
    const int n_chunks = (rows + p.chunk - 1) >> p.chunk_log2;
    GroupChunk* mine = chunks + (r0 >> p.chunk_log2) + g;
    long long before = 0;  // own tiles of the chunks before
    for (int w0 = 0; w0 < n_chunks; w0 += kStep) {
      for (int i = tid; i < kStep; i += kGroupThreads) s_own[i] = 0;
      __syncthreads();
      for (int base = b0; base < b1; base += kGroupThreads) {  // (whole warps: they exchange)
        const int b = base + tid;
        int s = 0, e = 0, N = 0;
        if (b < b1) s = p.q_indptr[b] - r0, e = p.q_indptr[b + 1] - r0, N = p.context_lens[b];
        // member b's own tiles in its chunks of the rows, every `by`-th from `from` on
        auto add = [&](int b, int s, int e, int N, int from, int by) {
          const int i1 = min((e - 1) >> p.chunk_log2, w0 + kStep - 1);
          for (int i = max(s >> p.chunk_log2, w0) + from; i <= i1; i += by) {
            const int z = min(e, (i + 1) << p.chunk_log2);
            atomicAdd(&s_own[i - w0], ((N - e + z - 1) >> 7) + 1 - pages);
            if (s <= i << p.chunk_log2) mine[i].first = b;
          }
        };
        const bool many = e - s > 32 << p.chunk_log2;  // a prompt: its chunks for the whole warp
        if (s < e && !many) add(b, s, e, N, 0, 1);
        for (unsigned w = __ballot_sync(0xFFFFFFFFu, many); w != 0u; w &= w - 1u) {
          const int k = __ffs(w) - 1;
          add(__shfl_sync(0xFFFFFFFFu, b, k), __shfl_sync(0xFFFFFFFFu, s, k), __shfl_sync(0xFFFFFFFFu, e, k),
              __shfl_sync(0xFFFFFFFFu, N, k), tid & 31, 32);
        }
      }
      __syncthreads();
      const int x = s_own[2 * tid], y = s_own[2 * tid + 1];
      int incl = x + y;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if ((tid & 31) >= d) incl += o;
      }
      if ((tid & 31) == 31) s_part[tid >> 5] = incl;
      __syncthreads();
      const int lane = tid & 31, sum = lane < kGroupThreads / 32 ? s_part[lane] : 0;
      const long long at = before + __reduce_add_sync(0xFFFFFFFFu, lane < tid >> 5 ? sum : 0) + incl - x - y;
      const long long each = kItemCost<kShared> + pages;
      const int i = w0 + 2 * tid;
      if (i < n_chunks) mine[i].places = at + x + (i + 1) * each;
      if (i + 1 < n_chunks) mine[i + 1].places = at + x + y + (i + 2) * each;
      before += __reduce_add_sync(0xFFFFFFFFu, sum);
      __syncthreads();
    }
    const long long together = before + static_cast<long long>(n_chunks) * pages;
    // (each thread rewrites its own)
    if ((warp_sum(s_apart[tid & 31]) - together) * p.num_kv_heads < least) decide(0);
  }
}

// Query rows of a request, or of a group, that the tile is laid out for: the rows of a group, on average and up to kSharedRows;
// or of a request alone, whose items have as many rows as the plain call's.
int layout_rows(const msa_kv8_attn_args* a, int num_groups) {
  const int64_t rows = (static_cast<int64_t>(a->total_rows) + num_groups - 1) / num_groups;
  const int some = rows < kSharedRows ? static_cast<int>(rows) : kSharedRows;
  return some > a->max_rows_per_req ? some : a->max_rows_per_req;
}
// Whether sharing can pay, by the sizes. The row chunks that it saves at most: all members' but one in each group; where a
// request has one chunk, no more than the chunks that its rows do not fill. And where the rows show that all requests are
// prompts (what they have less than max_rows together is less than one has), of four chunks at least, k members of a
// group have more than (k - 1) max_rows rows, so 4 (k - 1) chunks, of which no more than k - 1 are saved, whatever the lengths: what
// the form costs a tile, 6 to 10 % more than the plain call's, and the groups' kernel take that. (2 prompts of 512 rows
// behind 64 pages, 32 x 1 heads: 129 us, 141 with the groups looked at.)
bool may_pay(const msa_kv8_attn_args* a, int num_groups) {
  const int alone = chunk_log2_for(layout_rows(a, num_groups), a->q_per_kv);
  const long long rows = a->total_rows, most = a->max_rows_per_req, chunks = (rows + (1 << alone) - 1) >> alone;
  if (most >= 4LL << alone && rows > (a->num_reqs - 1) * most) return false;
  long long saved = a->num_reqs - num_groups;
  if (most <= 1 << alone && 1 << alone <= kSharedRows && a->num_reqs - chunks < saved) saved = a->num_reqs - chunks;
  return saved * a->max_pages_per_req * a->num_kv_heads >= kMinSizes;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// What the form adds to the workspace: the groups, the requests' shared pages, the groups' row chunks.
size_t groups_bytes(int n) { return up256(static_cast<size_t>(n) * sizeof(int4)); }
size_t skip_bytes(const msa_kv8_attn_args* a) { return up256(static_cast<size_t>(a->num_reqs) * sizeof(int32_t)); }
size_t added_workspace(const msa_kv8_attn_args* a, int n) {
  return groups_bytes(n) + skip_bytes(a) + (static_cast<size_t>(a->total_rows) + n + 1) * sizeof(GroupChunk);
}

msa_status check_groups(const msa_kv8_attn_args* a, int n) {
  const msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  return n < 0 || n > kMaxReqs ? MSA_ERR_INVALID_ARG : MSA_OK;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_kv8_attn_shared_workspace_size(const msa_kv8_attn_args* a, int32_t num_groups, size_t* bytes) {
  if (bytes == nullptr) return MSA_ERR_INVALID_ARG;
  const msa_status s = check_groups(a, num_groups);
  if (s != MSA_OK) return s;
  int sms = 0;
  const msa_status d = check_device(&sms);
  if (d != MSA_OK) return d;
  *bytes = up256(base_workspace(sms)) + added_workspace(a, num_groups);
  return MSA_OK;
}

msa_status msa_kv8_attn_shared(const msa_kv8_attn_args* a, int32_t num_groups, const int32_t* group_indptr,
                               int32_t min_saved, void* ws, size_t ws_bytes, void* stream) {
  msa_status s = check_groups(a, num_groups);
  if (s != MSA_OK) return s;
  if (a->n_block_ids != 0 || (num_groups > 0 && group_indptr == nullptr)) return MSA_ERR_INVALID_ARG;
  const long long saved = min_saved >= 0 ? min_saved : kMinSaved;
  if (num_groups == 0 || (min_saved < 0 && !may_pay(a, num_groups)) || a->max_pages_per_req > kLongTable)
    return msa_kv8_attn(a, ws, ws_bytes, stream);
  Kv8AttnParams p;
  CUtensorMap kmap;
  int sms = 0, copies = 0;
  if ((s = set_params(a, ws, ws_bytes, added_workspace(a, num_groups), layout_rows(a, num_groups), &p, &kmap, &sms, &copies)) != MSA_OK) return s;
  if (a->num_reqs == 0 || a->total_rows == 0) return MSA_OK;
  uint8_t* at = static_cast<uint8_t*>(ws) + up256(base_workspace(sms));
  int4* groups = reinterpret_cast<int4*>(at);
  int32_t* skip = reinterpret_cast<int32_t*>(at + groups_bytes(num_groups));
  p.num_groups = num_groups;
  p.groups = groups;
  p.group_indptr = group_indptr;
  p.skip = skip;
  GroupChunk* chunks = reinterpret_cast<GroupChunk*>(at + groups_bytes(num_groups) + skip_bytes(a));
  p.chunks = chunks;
  p.alone_log2 = p.chunk_log2;
  while (p.chunk > kSharedRows) p.chunk /= 2, --p.chunk_log2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // (each group by itself: its part of what has to be saved)
  kv8_groups_kernel<<<num_groups + 1, kGroupThreads, 0, st>>>(p, group_indptr, groups, skip, chunks,
                                                          (saved + num_groups - 1) / num_groups);
  if (cudaGetLastError() != cudaSuccess) return MSA_ERR_CUDA;
  const bool q_bf16 = a->q_type == MSA_TYPE_BF16;
  const cudaError_t e = p.alone_log2 > p.chunk_log2 ? launch_kv8_attn_shared_wide(kmap, p, copies, q_bf16, sms, st)
                                                    : launch_form<kShared>(kmap, p, copies, q_bf16, sms, st);
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
