// Attention weights by token (msa_kv8_attn_weights): for token t of request b and KV head h, over the rows and the
// queries of the head that see it,
//   new[t] = (t < N - R ? keep old[t] : 0) + sum 2^(s log2 e - lse log2 e),   s = sm_scale q . k_t,
// lse given by the attention of the same rows, so one pass over the keys is enough and no maximum is kept.
//
// Products. S^T = K Q^T: tokens are the M side, so a thread holds one token's scores against many queries and
// sums them in registers; no sum crosses lanes, and nothing but 4 bytes a token is written. K is multiplied as it is
// in the cache (E4M3); BF16 queries are two E4M3 rows as in the attention (msa_kv8_attn.cuh), which
// kv8_weights_queries_kernel lays out once, with each row's factor and -lse log2 e: a prompt's queries
// meet every page of keys, and would be converted 128 times otherwise. Sums are FP32.
//
// Work. A unit is four pages of keys (a "quad") against a chunk of 128 query rows ("columns"); each of four sets of
// four warps has one of the pages, so the chunk is loaded once for all. A request's quads have as many units as
// chunks see them (one for decode steps). All units form a line that the CTAs (one per SM) take in equal
// contiguous ranges; a quad that is cut leaves its sums in the workspace, and kv8_weights_merge_kernel adds them
// up in order: no atomics, the same bits every time.
//
// Roles: a warp that finds the units and starts the copies (pages and query chunks by tensor copies, two stages
// each), two that issue the products, and the four sets, which exponentiate and sum. A set has one score buffer: its
// next scores are computed while the other sets are at work.
//
// Floors: few rows, memory (128 bytes of a key, 4 read and 4 written per token and head); prompts, exponentials and
// products alike (two E4M3 products of 128 x 128 x 128 cost what 128 x 128 exponentials do).
// Measured (4 KV heads of 8 queries; floor): one row over 4,096 keys 10.3 us (0.3), bound by latency; 64 ragged requests of up
// to 8 rows 67.4 (46.8), memory and the start and end of a CTA; 2,053 rows on 16,421 keys 246 (135). There a unit costs 4,200
// cycles against 2,048 of exponentials and 2,480 of products, with 3,150 wavefronts of shared memory beside the products'
// operands: 1,024 reads of the columns' factors (16 warps, 16 bytes at a time, the same for all lanes), the rest polls of
// barriers, descriptions and what the copies write. What a factor's read costs was not measured by itself; with E4M3
// queries, which have half of them and half of the products, the same rows take 206 us (BF16 243 in that run). (Warps with two pages each read them half as often, but tensor memory has one score buffer a page: half of the
// warps wait for the products then, 297 us in step and 305 with pairs of sets.)
#include <climits>

#include "msa_kv8_pipe.cuh"

namespace msa {
namespace {

constexpr int kSets = 4, kMmaWarp = 4 * kSets, kMmaWarps = 2, kLoadWarp = kMmaWarp + kMmaWarps, kThreads = 32 * (kLoadWarp + 1);
constexpr int kKStages = 2, kQStages = 2, kCStages = 4;  // of quads of keys, of query chunks, of their factors
constexpr int kCols = 128;                    // columns of a chunk
constexpr int kRing = 16;                     // units whose description is kept (fewer are under way)
constexpr uint32_t kTileBytes = kBlock * kDim;
constexpr uint32_t kTmemCols = 512;
static_assert(kSets * kCols <= static_cast<int>(kTmemCols), "TMEM");

struct WeightsParams {
  int num_reqs, total_rows, max_rows, num_pages, max_pages, num_kv_heads, q_per_kv;
  const int32_t* context_lens;
  const int32_t* q_indptr;
  const int32_t* block_table;
  const void* q;
  long long q_stride;
  const float* k_scale;
  const float* lse;
  float sm_scale_log2, keep;
  const float* old_weights;  // or null
  float* new_weights;
  long long stride;          // elements between heads
  uint32_t* flags;
  uint8_t* parts;            // headers, then 2 partials of 512 sums for each CTA
  uint8_t* codes;            // [parts of a query][heads][rows x queries a head][128]
  float* coef;               // [heads][rows x queries a head] factors of the scores (BF16 queries); then a 0
  float* nlse;               // [heads][rows x queries a head] -lse log2 e; then a -inf (-inf counts for nothing)
};

enum : int { kEnd = 1, kNewK = 2, kLastK = 4, kNewQ = 8, kLastQ = 16, kNoQ = 32, kTile0 = 64 };  // kTile0 << e: page e is there
struct alignas(16) Unit {
  int flags, pos0, first, N;  // position of the first token, of the first row; tokens
  int c0, cols, slot, pad;    // first column, columns of the chunk that are there; -1: the whole quad is this CTA's, else
                              // its partial
  float ks[kSets];            // the pages' key scales
  long long off, pad2;        // of the head's weights
};

template <int NP>
struct Smem {
  uint8_t k[kKStages][kSets][kTileBytes];
  uint8_t q[kQStages][NP][kTileBytes];
  float coef[kCStages][kCols], nlse[kCStages][kCols];
  Unit unit[kRing];
  uint64_t told[kRing], k_full[kKStages][kSets], k_empty[kKStages], q_full[kQStages], q_empty[kQStages];
  uint64_t c_full[kCStages], c_empty[kCStages], s_full[kSets], s_empty[kSets], drain[kMmaWarps];
  long long sums[kThreads], part[kThreads / 32];
  uint32_t taddr;
};

struct Header {
  int tail;            // 1: partial 1 starts a quad that goes on in the next CTA's partial 0
  int cont, cont_end;  // partial 0 goes on with an earlier CTA's quad; and ends it
  int pos0, first, N;  // of the quad in partial 1
  long long off;
};
constexpr int kQuadTokens = kSets * kBlock;
__host__ __device__ inline size_t header_bytes(int grid) { return (grid * sizeof(Header) + 255) / 256 * 256; }

__device__ __forceinline__ bool load_req(const WeightsParams& p, int b, int* N, int* R, int* r0) {
  *N = p.context_lens[b];
  *r0 = p.q_indptr[b];
  *R = p.q_indptr[b + 1] - *r0;
  return *N >= 0 && *N <= p.max_pages * static_cast<long long>(kBlock) && *R >= 0 && *R <= p.max_rows && *R <= *N &&
         *r0 >= 0 && *r0 <= p.total_rows - *R;
}
// The quads of a request's head: quad i is seen by the chunks from max(0, 4 G i - a) on, a = ceil((N - R) G / 128)
// (the first column that sees token 512 i is (512 i - (N - R)) G).
struct Quads {
  int count, chunks, step;
  long long a;
  __device__ __forceinline__ Quads(int N, int R, int G)
      : count((N + kQuadTokens - 1) / kQuadTokens), chunks((R * G + kCols - 1) / kCols), step(kSets * G),
        a((static_cast<long long>(N - R) * G + kCols - 1) / kCols) {
    if (chunks == 0) {  // no rows: a unit without columns for each quad, which copies what is kept
      chunks = 1;
      a = LLONG_MAX / 4;
    }
  }
  __device__ __forceinline__ int first_chunk(int i) const {
    const long long j = static_cast<long long>(step) * i - a;
    return j > 0 ? static_cast<int>(j) : 0;
  }
  __device__ __forceinline__ long long before(int i) const {  // units before quad i
    const long long k0 = a / step + 1;                         // the first quad that not all chunks see
    long long n = static_cast<long long>(i) * chunks;
    if (i > k0) n -= step * ((i * (i - 1LL) - k0 * (k0 - 1)) / 2) - a * (i - k0);
    return n;
  }
};
static_assert(kQuadTokens == kSets * kCols, "");

// Query rows as the products take them: E4M3 codes head by head (two parts of a BF16 row, with 2^e), and -lse log2 e.
// Half a warp per row and query head, 8 elements a lane; kRows of them are on their way at once, without which the
// latency of a prompt's 65,696 rows was 15 us of 253. Bound: memory, latency for few rows.
template <int NP>
__global__ void __launch_bounds__(256) kv8_weights_queries_kernel(const WeightsParams p) {
  constexpr int kRows = 4;
  pdl_launch_dependents();
  const int lane = threadIdx.x & 15;
  const uint32_t G = p.q_per_kv, heads = p.num_kv_heads * G, per = p.total_rows * G, n = per * p.num_kv_heads;  // below 2^30
  if (blockIdx.x == 0 && threadIdx.x == 0) {  // columns that are not there
    if constexpr (NP == 2) p.coef[n] = 0.f;
    p.nlse[n] = -INFINITY;
  }
  const uint32_t step = gridDim.x * 16u, half = threadIdx.x >> 4 & 1u;
  for (uint32_t w0 = blockIdx.x * 16u + (threadIdx.x >> 5) * 2u; w0 < n; w0 += kRows * step) {  // (whole warps: they exchange)
    const uint32_t i0 = w0 + half;
    uint4 w[kRows];
    float lse[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const uint32_t i = i0 + k * step < n ? i0 + k * step : n - 1u, row = i / heads;
      const long long at = row * p.q_stride + (i - row * heads) * kDim + 8 * lane;
      lse[k] = p.lse[i];
      if constexpr (NP == 1) {
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.q) + at);
        w[k] = make_uint4(x.x, x.y, 0u, 0u);
      } else {
        w[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at);
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const uint32_t i = i0 + k * step;
      bool odd = !(fabsf(lse[k]) <= 3.402823466e38f);  // -inf, inf, NaN
      uint2 hi, lo = make_uint2(0u, 0u);
      float coef = p.sm_scale_log2;
      if constexpr (NP == 1) {
        hi = make_uint2(w[k].x, w[k].y);
        uint32_t nan = __vcmpeq4(hi.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(hi.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) nan |= __shfl_xor_sync(0xFFFFFFFFu, nan, d);
        odd |= nan != 0u;
      } else {
        const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
        uint32_t big = 0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) big = __vmaxu2(big, x[c] & 0x7FFF7FFFu);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, d));
        const uint32_t amax = max(big & 0xFFFFu, big >> 16);
        odd |= amax >= 0x7F80u;
        // the smallest 2^e with amax <= 448 2^e, not below 2^-120: the attention's split
        int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
        e = e < -120 ? -120 : e;
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        coef *= odd ? 1.f : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        uint32_t hc[4], lc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float a = __uint_as_float(x[c] << 16) * inv, b = __uint_as_float(x[c] & 0xFFFF0000u) * inv;
          hc[c] = f32x2_e4m3x2(a, b);
          const uint32_t hh = e4m3x2_f16x2(hc[c]);
          const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hh));
          lc[c] = f32x2_e4m3x2(a - hv.x, b - hv.y);
        }
        hi = make_uint2(hc[0] | hc[1] << 16, hc[2] | hc[3] << 16);
        lo = make_uint2(lc[0] | lc[1] << 16, lc[2] | lc[3] << 16);
      }
      if (i >= n) continue;
      if (odd) hi = lo = make_uint2(0u, 0u);
      const uint32_t row = i / heads, hd = i - row * heads, kv = hd / G;
      const long long to = kv * per + row * G + (hd - kv * G);
      *reinterpret_cast<uint2*>(p.codes + to * kDim + 8 * lane) = hi;
      if constexpr (NP == 2) *reinterpret_cast<uint2*>(p.codes + (n + to) * kDim + 8 * lane) = lo;
      if (lane == 0) {
        if constexpr (NP == 2) p.coef[to] = coef;
        p.nlse[to] = odd ? -INFINITY : lse[k] * -1.4426950408889634f;
      }
    }
  }
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int NP>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_weights_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap, const WeightsParams p) {
  extern __shared__ uint8_t smem_raw[];
  Smem<NP>& sm = *reinterpret_cast<Smem<NP>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.q_per_kv;
  pdl_launch_dependents();
  {
    auto init = [&](uint64_t* bar, int n, int first, uint32_t count) {
      if (tid >= first && tid < first + n) mbar_init(smem_u32(bar + (tid - first)), count);
    };
    init(sm.told, kRing, 0, 1);
    init(&sm.k_full[0][0], kKStages * kSets, 16, 1);
    init(sm.k_empty, kKStages, 24, kMmaWarps);
    init(sm.q_full, kQStages, 26, 1);
    init(sm.q_empty, kQStages, 28, kMmaWarps);
    init(sm.c_full, kCStages, 30, 32);
    init(sm.c_empty, kCStages, 34, 4 * kSets);
    init(sm.s_full, kSets, 38, 1);
    init(sm.s_empty, kSets, 42, 4);
    init(sm.drain, kMmaWarps, 46, 1);
    if (tid < 64) mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&sm.taddr), kTmemCols);

  // ---- the line: every thread sums a run of requests
  const int per = (p.num_reqs + kThreads - 1) / kThreads;
  {
    const int b0 = tid * per < p.num_reqs ? tid * per : p.num_reqs;
    const int b1 = b0 + per < p.num_reqs ? b0 + per : p.num_reqs;
    long long incl = 0;
    for (int b = b0; b < b1; ++b) {
      int N, R, r0;
      if (load_req(p, b, &N, &R, &r0)) {
        const Quads x(N, R, G);
        incl += p.num_kv_heads * x.before(x.count);
      } else if (blockIdx.x == 0) {
        set_flag(p.flags, kFlagBadLength);
      }
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    sm.sums[tid] = incl;
    if (lane == 31) sm.part[warp] = incl;
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.taddr;

  if (warp == kLoadWarp) {
    // ================= finds the units and loads their keys and queries
    Header hd = {};
    int u = 0;
    bool good = true, waited = false;
    Ring<kKStages> rk;
    Ring<kQStages> rq;
    Ring<kCStages> rc;
    int nk = 0, nq = 0;
    long long left = 0, start = 0;  // units in the range; the first one's offset in request b
    int b = 0;
    {
      constexpr int kWarps = kThreads / 32;
      long long incl = lane < kWarps ? sm.part[lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
      }
      const long long total = __shfl_sync(0xFFFFFFFFu, incl, 31);
      // fewer units than CTAs: the last CTAs have none (a partial's continuation is in the next CTA)
      const long long use = total < gridDim.x ? total : gridDim.x;
      long long lo = 0, hi = 0;
      if (blockIdx.x < use) {
        const long long each = total / use, more = total - each * use;
        lo = each * blockIdx.x + (blockIdx.x < more ? blockIdx.x : more);
        hi = lo + each + (blockIdx.x < more ? 1 : 0);
      }
      left = hi - lo;
      if (left > 0) {
        // the warp whose requests hold place lo, then the thread, then the request
        const int w = __ffs(__ballot_sync(0xFFFFFFFFu, lo < incl)) - 1;
        const long long before = w > 0 ? __shfl_sync(0xFFFFFFFFu, incl, w - 1) : 0;
        const long long mine = before + sm.sums[32 * w + lane];
        const int th = __ffs(__ballot_sync(0xFFFFFFFFu, lo < mine)) - 1;
        long long at = th > 0 ? __shfl_sync(0xFFFFFFFFu, mine, th - 1) : before;
        b = (32 * w + th) * per;
        for (int i = 1; i < per && b + 1 < p.num_reqs; ++i) {
          int N, R, r0;
          long long n = 0;
          if (load_req(p, b, &N, &R, &r0)) {
            const Quads x(N, R, G);
            n = p.num_kv_heads * x.before(x.count);
          }
          if (lo < at + n) break;
          at += n;
          ++b;
        }
        start = lo - at;
      }
    }
    int h = -1;
    while (left > 0 && good) {
      int N, R, r0;
      if (!load_req(p, b, &N, &R, &r0)) {
        if (++b >= p.num_reqs) break;
        continue;
      }
      const Quads x(N, R, G);
      const long long per_head = x.before(x.count);
      if (per_head == 0) {
        if (++b >= p.num_reqs) break;
        continue;
      }
      int i = 0, at = 0;  // the quad, and the CTA's place in it
      if (h < 0) {
        h = static_cast<int>(start / per_head);
        const long long off = start - h * per_head;
        int e = x.count;  // before(i) <= off < before(e)
        while (e - i > 1) {
          const int mid = (i + e) / 2;
          if (x.before(mid) <= off) i = mid;
          else e = mid;
        }
        at = static_cast<int>(off - x.before(i));
      }
      const int32_t* table = p.block_table + static_cast<long long>(b) * p.max_pages;
      const int tiles = (N + kBlock - 1) / kBlock;
      const long long qrow0 = static_cast<long long>(h) * p.total_rows * G + static_cast<long long>(r0) * G;
      const int cols = R * G;
      int base = -32, phys = -1, have_q = -1;  // lanes hold tiles base .. base + 31
      float ks = 0.f;
      for (; i < x.count && left > 0 && good; ++i) {
        if (kSets * i >= base + 32) {
          base = kSets * i;
          phys = -1;
          ks = 0.f;
          if (base + lane < tiles) {
            phys = table[base + lane];
            if (phys < 0 || phys >= p.num_pages) {
              if (cols > 0) set_flag(p.flags, kFlagBadPage);
              phys = -1;
            } else {
              ks = p.k_scale[static_cast<long long>(phys) * p.num_kv_heads + h];
            }
          }
        }
        // lane e < 4: page e of the quad
        const int page = __shfl_sync(0xFFFFFFFFu, phys, kSets * i - base + (lane & (kSets - 1)));
        const float scale = __shfl_sync(0xFFFFFFFFu, ks, kSets * i - base + (lane & (kSets - 1)));
        const int there = __ballot_sync(0xFFFFFFFFu, page >= 0) & ((1 << kSets) - 1);
        const int j0 = x.first_chunk(i), n = x.chunks - j0;
        const int take = n - at < left ? n - at : static_cast<int>(left);
        const bool begin = at == 0, end = at + take == n;
        const int slot = begin && end ? -1 : begin ? 1 : 0;
        const long long off = (static_cast<long long>(b) * p.num_kv_heads + h) * p.stride;
        if (slot == 1) {
          hd.tail = 1;
          hd.pos0 = i * kQuadTokens;
          hd.first = N - R;
          hd.N = N;
          hd.off = off;
        } else if (slot == 0) {
          hd.cont = 1;
          hd.cont_end = end;
        }
        left -= take;
        for (int j = j0 + at; j < j0 + at + take && good; ++j, ++u) {
          int flags = there * kTile0;
          const bool new_k = j == j0 + at, last_k = j + 1 == j0 + at + take;
          const bool new_q = cols > 0 && have_q != j;
          const bool same_next = last_k && i + 1 < x.count && left > 0 && x.first_chunk(i + 1) == j;
          const int here = cols - kCols * j < kCols ? cols - kCols * j : kCols;
          if (new_k) flags |= kNewK;
          if (last_k) flags |= kLastK;
          if (new_q) flags |= kNewQ;
          if (cols == 0) flags |= kNoQ;
          else if (!same_next) flags |= kLastQ;
          if (new_k && nk >= kKStages) good = warp_wait(smem_u32(&sm.k_empty[rk.at]), rk.phase ^ 1u, p.flags);
          if (good && new_q && nq >= kQStages) good = warp_wait(smem_u32(&sm.q_empty[rq.at]), rq.phase ^ 1u, p.flags);
          if (good && new_q && nq >= kCStages) good = warp_wait(smem_u32(&sm.c_empty[rc.at]), rc.phase ^ 1u, p.flags);
          if (!good) break;
          if (lane == 0) {
            Unit& x1 = sm.unit[u % kRing];
            x1.flags = flags;
            x1.pos0 = i * kQuadTokens;
            x1.first = N - R;
            x1.N = N;
            x1.c0 = kCols * j;
            x1.cols = here;
            x1.slot = slot;
            x1.off = off;
          }
          if (lane < kSets) sm.unit[u % kRing].ks[lane] = scale;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.told[u % kRing]));
          if (new_k && lane < kSets) {
            const uint32_t kb = smem_u32(&sm.k_full[rk.at][lane]);
            if (cols > 0 && page >= 0) {
              mbar_arrive_expect_tx(kb, kTileBytes);
              tma_load_2d(smem_u32(sm.k[rk.at][lane]), &kmap, 0, (page * p.num_kv_heads + h) * kBlock, kb);
            } else {
              mbar_arrive(kb);
            }
          }
          __syncwarp();
          if (new_q) {
            if (!waited) pdl_wait_primary();  // (keys, lengths and tables are older than the kernel before)
            waited = true;
            const uint32_t qb = smem_u32(&sm.q_full[rq.at]);
            const long long row = qrow0 + kCols * static_cast<long long>(j);
            const long long all = static_cast<long long>(p.num_kv_heads) * p.total_rows * G;
#pragma unroll
            for (int k = 0; k < kCols / 32; ++k) {
              const int c = 32 * k + lane;
              const long long src = c < here ? row + c : all;
              cp_async4(smem_u32(&sm.nlse[rc.at][c]), p.nlse + src);
              if constexpr (NP == 2) cp_async4(smem_u32(&sm.coef[rc.at][c]), p.coef + src);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.c_full[rc.at])) : "memory");
            if (lane == 0) {
              mbar_arrive_expect_tx(qb, NP * kTileBytes);
#pragma unroll
              for (int part = 0; part < NP; ++part)
                tma_load_2d(smem_u32(sm.q[rq.at][part]), &qmap, 0, static_cast<int>(row + part * all), qb);
            }
            __syncwarp();
            have_q = j;
            ++nq;
            rq.step();
            rc.step();
          }
          if (new_k) {
            ++nk;
            rk.step();
          }
          if (flags & kLastQ) have_q = -1;
        }
        at = 0;
      }
      if (++h == p.num_kv_heads) {
        h = 0;
        if (++b >= p.num_reqs) break;
      }
    }
    if (good && lane == 0) {
      sm.unit[u % kRing].flags = kEnd;
      mbar_arrive(smem_u32(&sm.told[u % kRing]));
    }
    if (!waited) pdl_wait_primary();
    // no copy may still be landing when the CTA leaves
    for (int j = nk - kKStages < 0 ? 0 : nk - kKStages; j < nk; ++j)
      for (int e = 0; e < kSets; ++e)
        if (!wait_bar(smem_u32(&sm.k_full[j % kKStages][e]), (j / kKStages) & 1, p.flags)) break;
    for (int j = nq - kQStages < 0 ? 0 : nq - kQStages; j < nq; ++j)
      if (!wait_bar(smem_u32(&sm.q_full[j % kQStages]), (j / kQStages) & 1, p.flags)) break;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) reinterpret_cast<Header*>(p.parts)[blockIdx.x] = hd;
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // ================= products: set e's scores of unit u into its buffer, each warp for half of the sets (one warp for
    // all took longer to issue them than the tensor cores to compute them)
    const int part0 = (warp - kMmaWarp) * (kSets / kMmaWarps);
    const uint32_t el = elect_one();
    const uint64_t kdesc0 = sdesc_kmajor_sw128(smem_u32(sm.k[0][0])), qdesc0 = sdesc_kmajor_sw128(smem_u32(sm.q[0][0]));
    Ring<kKStages> rk;
    Ring<kQStages> rq;
    Ring<kRing> rt;
    bool any = false, good = true;
    for (int u = 0; good; ++u, rt.step()) {
      if (!warp_wait(smem_u32(&sm.told[rt.at]), rt.phase, p.flags)) break;
      const int flags = sm.unit[rt.at].flags;
      if (flags & kEnd) break;
      const int cols = sm.unit[rt.at].cols;
      if (flags & kNewQ && !warp_wait(smem_u32(&sm.q_full[rq.at]), rq.phase, p.flags)) break;
      // (whole 32 columns: that is what the sets read; rows that are not the request's are finite)
      const uint32_t idesc = idesc_e4m3_f32(kBlock, cols > 0 ? (cols + 31) / 32 * 32 : 32, false, false);
      const uint64_t qdesc = qdesc0 + rq.at * NP * (kTileBytes >> 4);
#pragma unroll 1
      for (int e = part0; e < part0 + kSets / kMmaWarps && good; ++e) {
        if (flags & kNewK) good = warp_wait(smem_u32(&sm.k_full[rk.at][e]), rk.phase, p.flags);
        if (good && u > 0) good = warp_wait(smem_u32(&sm.s_empty[e]), (u - 1) & 1, p.flags);
        if (!good) break;
        tc_fence_after();
        if (!(flags & kNoQ) && flags & (kTile0 << e)) {
          const uint64_t kdesc = kdesc0 + (rk.at * kSets + e) * (kTileBytes >> 4);
#pragma unroll
          for (int part = 0; part < NP; ++part)
#pragma unroll
            for (int kk = 0; kk < kDim / 32; ++kk)
              mma_f8_ss_elect(el, tbase + e * kCols, kdesc + 2 * kk, qdesc + part * (kTileBytes >> 4) + 2 * kk, idesc,
                              part > 0 || kk > 0);
          any = true;
        }
        commit_elect(el, smem_u32(&sm.s_full[e]));
      }
      if (!good) break;
      if (flags & kLastK) {
        commit_elect(el, smem_u32(&sm.k_empty[rk.at]));
        rk.step();
      }
      if (flags & kLastQ) {
        commit_elect(el, smem_u32(&sm.q_empty[rq.at]));
        rq.step();
      }
    }
    if (any) {  // every MMA of this thread has finished before the tensor memory is released
      commit_elect(el, smem_u32(&sm.drain[warp - kMmaWarp]));
      warp_wait(smem_u32(&sm.drain[warp - kMmaWarp]), 0, p.flags);
    }
    __syncwarp();
  } else {
    // ================= set e: exponentials and sums of page 4 i + e, a token per thread
    const int e = warp / 4, quad = warp % 4, l = 32 * quad + lane;
    const uint32_t s_cols = tbase + (static_cast<uint32_t>(32 * quad) << 16) + e * kCols;
    Ring<kCStages> rc;
    Ring<kRing> rt;
    float2 acc = make_float2(0.f, 0.f);
    float old = 0.f;
    for (int u = 0;; ++u, rt.step()) {
      if (!warp_wait(smem_u32(&sm.told[rt.at]), rt.phase, p.flags)) break;
      const int4 x = *reinterpret_cast<const int4*>(&sm.unit[rt.at].flags);
      if (x.x & kEnd) break;
      const int4 y = *reinterpret_cast<const int4*>(&sm.unit[rt.at].c0);
      const float ks = sm.unit[rt.at].ks[e] * (NP == 1 ? p.sm_scale_log2 : 1.f);
      const long long off = sm.unit[rt.at].off;
      const int t = x.y + kBlock * e + l;
      if (x.x & kNewK) {
        acc = make_float2(0.f, 0.f);
        old = 0.f;
        if (y.z < 0 && p.old_weights != nullptr && t < x.z) old = p.keep * p.old_weights[off + t];  // (on its way meanwhile)
      }
      if (x.x & kNewQ && !warp_wait(smem_u32(&sm.c_full[rc.at]), rc.phase, p.flags)) break;
      if (!warp_wait(smem_u32(&sm.s_full[e]), u & 1, p.flags)) break;
      // the scores have been read (in registers): the buffer is free
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[e]));
      };
      if (!(x.x & kNoQ) && x.x & (kTile0 << e)) {
        tc_fence_after();
        const float2 ks2 = make_float2(ks, ks);
        const float* coef = sm.coef[rc.at];
        const float* nlse = sm.nlse[rc.at];
        // the exponents' arguments of 4 columns
        auto args = [&](const uint32_t* v, int c, float2& a, float2& b) {
          const float4 n = *reinterpret_cast<const float4*>(nlse + c);
          a = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
          b = make_float2(__uint_as_float(v[2]), __uint_as_float(v[3]));
          if constexpr (NP == 1) {
            a = __ffma2_rn(a, ks2, make_float2(n.x, n.y));
            b = __ffma2_rn(b, ks2, make_float2(n.z, n.w));
          } else {
            const float4 f = *reinterpret_cast<const float4*>(coef + c);
            a = __ffma2_rn(__fmul2_rn(a, ks2), make_float2(f.x, f.y), make_float2(n.x, n.y));
            b = __ffma2_rn(__fmul2_rn(b, ks2), make_float2(f.z, f.w), make_float2(n.z, n.w));
          }
        };
        // the columns before lo do not see the thread's token; the page's last token decides for all threads
        const long long last = static_cast<long long>(x.y + kBlock * e + kBlock - 1 - x.z) * G - y.x;
        if (last <= 0) {  // (columns that are not there have factors that leave 0)
          const int n = (y.y + 31) / 32;
          // (a sum for the unit first: one running sum of a prompt's thousands of exponentials loses the faint ones)
          float2 unit = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int ch = 0; ch < n; ++ch) {
            uint32_t v[32];
            tmem_ld32(s_cols + 32 * ch, v);
            tc_wait_ld();
            if (ch + 1 == n) release();
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float2 a, b;
              args(v + c, 32 * ch + c, a, b);
              unit = __fadd2_rn(unit, make_float2(ex2(a.x), ex2(a.y)));
              sum = __fadd2_rn(sum, make_float2(ex2(b.x), ex2(b.y)));
            }
            unit = __fadd2_rn(unit, sum);
          }
          acc = __fadd2_rn(acc, unit);
        } else {
          const int ahead = t - x.z;  // of the first row
          const int lo = ahead > 0 ? ahead * G - y.x : 0, n = (y.y + 15) / 16;
          float2 unit = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int ch = 0; ch < n; ++ch) {
            uint32_t v[16];
            tmem_ld16(s_cols + 16 * ch, v);
            tc_wait_ld();
            if (ch + 1 == n) release();
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
              float2 a, b;
              const int at = 16 * ch + c;
              args(v + c, at, a, b);
              unit.x += at >= lo ? ex2(a.x) : 0.f;
              unit.y += at + 1 >= lo ? ex2(a.y) : 0.f;
              unit.x += at + 2 >= lo ? ex2(b.x) : 0.f;
              unit.y += at + 3 >= lo ? ex2(b.y) : 0.f;
            }
          }
          acc = __fadd2_rn(acc, unit);
        }
      } else {
        release();
      }
      if (x.x & kLastQ) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.c_empty[rc.at]));
        rc.step();
      }
      if (x.x & kLastK) {
        float w = acc.x + acc.y;
        if (isnan(w)) w = 0.f;  // a NaN in the key: every row that sees it is NaN and counts for nothing
        if (y.z < 0) {
          if (t < x.w) p.new_weights[off + t] = old + w;
        } else {
          reinterpret_cast<float*>(p.parts + header_bytes(gridDim.x))[(2LL * blockIdx.x + y.z) * kQuadTokens + kBlock * e + l] = w;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// Adds up the sums of a quad that starts in CTA blockIdx.x's range and ends in a later one's, in order.
__global__ void __launch_bounds__(kQuadTokens) kv8_weights_merge_kernel(const WeightsParams p, int grid) {
  pdl_wait_primary();
  const Header* hd = reinterpret_cast<const Header*>(p.parts);
  const Header me = hd[blockIdx.x];
  if (!me.tail) return;
  const float* part = reinterpret_cast<const float*>(p.parts + header_bytes(grid));
  float w = part[(2LL * blockIdx.x + 1) * kQuadTokens + threadIdx.x];
  for (int i = blockIdx.x + 1; i < grid && hd[i].cont; ++i) {
    w += part[2LL * i * kQuadTokens + threadIdx.x];
    if (hd[i].cont_end) break;
  }
  const int t = me.pos0 + threadIdx.x;
  if (t >= me.N) return;
  if (p.old_weights != nullptr && t < me.first) w += p.keep * p.old_weights[me.off + t];
  p.new_weights[me.off + t] = w;
}

template <int NP>
msa_status launch(const CUtensorMap& kmap, const CUtensorMap& qmap, const WeightsParams& p, int sms, cudaStream_t st) {
  const int smem = static_cast<int>(sizeof(Smem<NP>)) + 1024;
  if (cudaFuncSetAttribute(kv8_weights_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return MSA_ERR_CUDA;
  const long long rows = static_cast<long long>(p.total_rows) * p.num_kv_heads * p.q_per_kv, ctas = (rows + 15) / 16, cap = 4LL * sms;
  const int grid = static_cast<int>(ctas < 1 ? 1 : ctas < cap ? ctas : cap);
  kv8_weights_queries_kernel<NP><<<grid, 256, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return MSA_ERR_CUDA;
  if (launch_after(kv8_weights_kernel<NP>, dim3(sms), kThreads, smem, st, kmap, qmap, p) != cudaSuccess) return MSA_ERR_CUDA;
  // (quads of one unit are never cut)
  if (static_cast<long long>(p.max_rows) * p.q_per_kv <= kCols) return MSA_OK;
  return launch_after(kv8_weights_merge_kernel, dim3(sms), kQuadTokens, 0, st, p, sms) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
struct Layout {
  size_t parts, codes, coef, nlse, total;
};
Layout layout(const msa_kv8_attn_args* a, int sms) {
  const size_t rows = static_cast<size_t>(a->total_rows) * a->num_kv_heads * a->q_per_kv;
  const size_t np = a->q_type == MSA_TYPE_BF16 ? 2 : 1;
  Layout l;
  l.parts = 256;
  l.coef = up256(l.parts + header_bytes(sms) + 2 * static_cast<size_t>(sms) * kQuadTokens * sizeof(float));
  l.nlse = up256(l.coef + (np == 2 ? (rows + 1) * sizeof(float) : 0));
  l.codes = up256(l.nlse + (rows + 1) * sizeof(float));
  l.total = up256(l.codes + np * rows * kDim);
  return l;
}

msa_status check_weights(const msa_kv8_attn_args* a) {
  const msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  // rows of the query parts are counted in 32 bits, and so are the positions of a whole quad behind the last token
  if (2LL * a->total_rows * a->num_kv_heads * a->q_per_kv + kBlock >= (1LL << 31)) return MSA_ERR_UNSUPPORTED;
  return a->max_pages_per_req > (1 << 24) - 256 ? MSA_ERR_UNSUPPORTED : MSA_OK;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_kv8_attn_weights_workspace_size(const msa_kv8_attn_args* a, size_t* bytes) {
  if (bytes == nullptr) return MSA_ERR_INVALID_ARG;
  const msa_status s = check_weights(a);
  if (s != MSA_OK) return s;
  int sms = 0;
  const msa_status d = check_device(&sms);
  if (d != MSA_OK) return d;
  *bytes = layout(a, sms).total;
  return MSA_OK;
}

msa_status msa_kv8_attn_weights(const msa_kv8_attn_args* a, const float* lse, float keep, const float* old_weights,
                                float* new_weights, int64_t head_stride, void* ws, size_t ws_bytes, void* stream) {
  msa_status s = check_weights(a);
  if (s != MSA_OK) return s;
  auto unaligned = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) != 0; };
  if (a->num_reqs > 0 && (a->context_lens == nullptr || a->q_indptr == nullptr || a->block_table == nullptr ||
                          new_weights == nullptr))
    return MSA_ERR_INVALID_ARG;
  if (a->n_block_ids != 0 || a->block_ids != nullptr || a->k_data == nullptr || a->k_scale == nullptr) return MSA_ERR_INVALID_ARG;
  if (a->total_rows > 0 && (a->q == nullptr || lse == nullptr)) return MSA_ERR_INVALID_ARG;
  const int q_size = a->q_type == MSA_TYPE_BF16 ? 2 : 1;
  if (unaligned(a->q, 16) || unaligned(a->k_data, 16) || unaligned(a->k_scale, 4) || unaligned(lse, 4) ||
      unaligned(old_weights, 4) || unaligned(new_weights, 4) ||
      a->q_row_stride < static_cast<int64_t>(kDim) * a->num_kv_heads * a->q_per_kv || a->q_row_stride * q_size % 16 != 0)
    return MSA_ERR_INVALID_ARG;
  if (!(keep >= 0.f) || !std::isfinite(keep) || head_stride < static_cast<int64_t>(a->max_pages_per_req) * kBlock)
    return MSA_ERR_INVALID_ARG;
  if (ws == nullptr || unaligned(ws, 256)) return MSA_ERR_WORKSPACE;
  int sms = 0;
  if ((s = check_device(&sms)) != MSA_OK) return s;
  const Layout l = layout(a, sms);
  if (ws_bytes < l.total) return MSA_ERR_WORKSPACE;
  if (a->num_reqs == 0) return MSA_OK;
  uint8_t* base = static_cast<uint8_t*>(ws);
  WeightsParams p = {};
  p.num_reqs = a->num_reqs;
  p.total_rows = a->total_rows;
  p.max_rows = a->max_rows_per_req;
  p.num_pages = a->num_pages;
  p.max_pages = a->max_pages_per_req;
  p.num_kv_heads = a->num_kv_heads;
  p.q_per_kv = a->q_per_kv;
  p.context_lens = a->context_lens;
  p.q_indptr = a->q_indptr;
  p.block_table = a->block_table;
  p.q = a->q;
  p.q_stride = a->q_row_stride;
  p.k_scale = a->k_scale;
  p.lse = lse;
  p.sm_scale_log2 = a->sm_scale * 1.4426950408889634f;
  p.keep = keep;
  p.old_weights = keep == 0.f ? nullptr : old_weights;
  p.new_weights = new_weights;
  p.stride = head_stride;
  p.flags = static_cast<uint32_t*>(ws);
  p.parts = base + l.parts;
  p.codes = base + l.codes;
  p.coef = reinterpret_cast<float*>(base + l.coef);
  p.nlse = reinterpret_cast<float*>(base + l.nlse);
  CUtensorMap kmap, qmap;
  if ((s = encode_kv8_map(&kmap, a->k_data, static_cast<long long>(a->num_pages) * a->num_kv_heads * kBlock)) != MSA_OK) return s;
  const int np = a->q_type == MSA_TYPE_BF16 ? 2 : 1;
  const long long rows = static_cast<long long>(np) * a->total_rows * a->num_kv_heads * a->q_per_kv;
  if ((s = encode_kv8_map(&qmap, p.codes, rows > 0 ? rows : 1)) != MSA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return np == 2 ? launch<2>(kmap, qmap, p, sms, st) : launch<1>(kmap, qmap, p, sms, st);
}

}  // extern "C"
