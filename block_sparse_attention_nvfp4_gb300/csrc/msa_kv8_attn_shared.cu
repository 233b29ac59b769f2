// msa_kv8_attn_shared: attention over the 8-bit cache for requests whose block tables begin with the same pages, as
// msa_pages_fork leaves them. Per group of requests
//   * kv8_groups_kernel finds the leading pages that all members' rows list and that all their query rows see whole;
//   * the attention kernel (msa_kv8_attn.cuh) has items of two kinds on its line of tiles: a group's shared pages for
//     the rows of all members together, and each request's own pages. With O_i = sum_t 2^(x_t - y_i) v_t and
//     y_i = log2 sum_t 2^(x_t) of half i, both in FP32,
//   * kv8_join_kernel adds them up: out = sum_i 2^(y_i - y) O_i, y = log2(2^y_1 + 2^y_2).
// Shared pages are read once for 128 / q_per_kv rows instead of once for each request, and a tile of the tensor cores
// is full of rows instead of copies of a few.
#include "msa_kv8_attn.cuh"

namespace msa {
namespace {

constexpr int kGroupThreads = 512, kJoinThreads = 256;
// Pages, over all KV heads and groups, that sharing has to save before it pays. The groups' kernel, the second kind of
// items and the joining cost some 8 us against the plain call, which is taken where the sizes leave less than kMinSizes to
// save. Behind the groups' kernel, with tiles laid out for a group's rows, it pays sooner: from kMinSaved on. Measured (4 KV
// heads, BF16, one row a member; shared / behind the groups' kernel but alone / the plain call, us):
//   768 saved, 4 members   28.7 / 24.6 / 20.5      1,536, 4 groups of 4   26.7 / 30.8 / 26.7
//   896, 8 members         24.2 / 26.1 / 20.6      1,792, 8 members       26.4 / 30.7 / 26.7
//   960, 16 members        24.9 / 26.7 / 22.5      3,840, 16 members      29.2 / 43.0 / 36.9
constexpr int kMinSizes = 1536, kMinSaved = 768;

// CTA g: group g; the last CTA: the requests outside every group. groups[g] = {shared pages (0: none), first row, rows,
// first member}, skip[b] = shared pages of request b. Bound: latency, a chain of dependent reads (the bounds, the
// lengths, the tables); the members' entries are compared kRun at a time, all on their way at once (one after the other
// 64 members of 128 pages took 9.3 us).
__global__ void __launch_bounds__(kGroupThreads) kv8_groups_kernel(const Kv8AttnParams p, const int32_t* indptr, int4* groups,
                                                                   int32_t* skip, long long least) {
  __shared__ int s_limit, s_members, s_pages;
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
  bool wrong = false;
  for (int b = b0 + tid; b < b1; b += kGroupThreads) {
    Req q;
    if (!load_req<kAll>(p, b, &q)) {  // (its flag is the attention's to set)
      wrong = true;
    } else if (q.R > 0) {
      limit = min(limit, (q.N - q.R) / kBlock);
      ++members;
    }
  }
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
  int pages = min(most, s_pages);
  if (static_cast<long long>(members - 1) * pages * p.num_kv_heads < least) pages = 0;
  for (int b = b0 + tid; b < b1; b += kGroupThreads) skip[b] = pages;
  if (tid == 0) groups[g] = make_int4(pages, b0 < b1 ? p.q_indptr[b0] : 0, b0 < b1 ? p.q_indptr[b1] - p.q_indptr[b0] : 0, b0);
}

// Joins the halves of the rows of the groups that share pages; CTA (x, g) takes heads of group g's rows, a warp a
// head at a time. Bound: memory (1 KB read and 256 bytes written per head), latency for few rows.
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const Kv8AttnParams p) {
  pdl_wait_primary();
  const int4 g = p.groups[blockIdx.y];
  if (g.x == 0) return;
  const int lane = threadIdx.x & 31, heads = p.num_kv_heads * p.q_per_kv;
  const long long n = static_cast<long long>(g.z) * heads, base = static_cast<long long>(g.y) * heads;
  constexpr int kWarps = kJoinThreads / 32;
  for (long long i = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < n; i += gridDim.x * kWarps) {
    const long long orow = base + i;
    const float4 a = *reinterpret_cast<const float4*>(half_row(p, 1, orow) + 4 * lane);
    const float4 b = *reinterpret_cast<const float4*>(half_row(p, 2, orow) + 4 * lane);
    const float ya = *half_lse(p, 1, orow), yb = *half_lse(p, 2, orow);
    float wa = 0.f, wb = 0.f, y = -INFINITY;
    const float top = fmaxf(ya, yb);
    if (top != -INFINITY) {
      const float ea = ex2(ya - top), eb = ex2(yb - top), inv = 1.f / (ea + eb);
      wa = ea * inv;
      wb = eb * inv;
      y = top + log2f(ea + eb);
    }
    if (isnan(ya) || isnan(yb)) wa = wb = y = __int_as_float(0x7FFFFFFF);
    // (a half of weight 0 counts for nothing, whatever it holds)
    float o[4];
    const float fa[4] = {a.x, a.y, a.z, a.w}, fb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = (wa != 0.f ? wa * fa[u] : 0.f) + (wb != 0.f ? wb * fb[u] : 0.f);
    *reinterpret_cast<uint2*>(p.out + orow * kDim + 4 * lane) = make_uint2(bf16x2_bits(o[0], o[1]), bf16x2_bits(o[2], o[3]));
    if (lane == 0 && p.lse != nullptr) p.lse[orow] = y * 0.69314718055994531f;
  }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// What the form adds to the workspace: the groups, the requests' shared pages, the rows' halves.
size_t groups_bytes(int n) { return up256(static_cast<size_t>(n) * sizeof(int4)); }
size_t skip_bytes(const msa_kv8_attn_args* a) { return up256(static_cast<size_t>(a->num_reqs) * sizeof(int32_t)); }
size_t added_workspace(const msa_kv8_attn_args* a, int n) {
  const size_t rows = static_cast<size_t>(a->total_rows) * a->num_kv_heads * a->q_per_kv;
  return groups_bytes(n) + skip_bytes(a) + 2 * rows * (kDim + 1) * sizeof(float);
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
  // what sharing could save at most, by the sizes
  const long long most_saved = static_cast<long long>(a->num_reqs - num_groups) * a->max_pages_per_req * a->num_kv_heads;
  if (num_groups == 0 || (min_saved < 0 && most_saved < kMinSizes)) return msa_kv8_attn(a, ws, ws_bytes, stream);
  Kv8AttnParams p;
  CUtensorMap kmap;
  int sms = 0, copies = 0;
  // items of the shared pages have the rows of a group, on average
  const int rows = (a->total_rows + num_groups - 1) / num_groups;
  const int most = rows > a->max_rows_per_req ? rows : a->max_rows_per_req;
  if ((s = set_params(a, ws, ws_bytes, added_workspace(a, num_groups), most, &p, &kmap, &sms, &copies)) != MSA_OK) return s;
  if (a->num_reqs == 0 || a->total_rows == 0) return MSA_OK;
  uint8_t* at = static_cast<uint8_t*>(ws) + up256(base_workspace(sms));
  int4* groups = reinterpret_cast<int4*>(at);
  int32_t* skip = reinterpret_cast<int32_t*>(at + groups_bytes(num_groups));
  p.num_groups = num_groups;
  p.groups = groups;
  p.skip = skip;
  p.halves = reinterpret_cast<float*>(at + groups_bytes(num_groups) + skip_bytes(a));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // (each group by itself: its part of what has to be saved)
  kv8_groups_kernel<<<num_groups + 1, kGroupThreads, 0, st>>>(p, group_indptr, groups, skip, (saved + num_groups - 1) / num_groups);
  if (cudaGetLastError() != cudaSuccess) return MSA_ERR_CUDA;
  if (launch_form<kShared>(kmap, p, copies, a->q_type == MSA_TYPE_BF16, sms, st) != cudaSuccess) return MSA_ERR_CUDA;
  const long long heads = static_cast<long long>(a->total_rows) * a->num_kv_heads * a->q_per_kv;
  const long long per = (heads / num_groups + kJoinThreads / 32 - 1) / (kJoinThreads / 32), cap = (4 * sms + num_groups - 1) / num_groups;
  const int x = static_cast<int>(per < 1 ? 1 : per < cap ? per : cap);
  return launch_after(kv8_join_kernel, dim3(x, num_groups), kJoinThreads, 0, st, p) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
