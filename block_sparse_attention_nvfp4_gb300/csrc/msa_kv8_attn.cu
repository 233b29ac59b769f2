// Attention over the 8-bit cache (msa_kv8_attn): E4M3 keys and values with one FP32 scale for
// each 128-token page and KV head.
//
// For a query row at position p, over the keys t <= p of the listed blocks (or of all), with
// x_t = sm_scale log2(e) k_scale (q . k_t) + log2(v_scale):
//   out = sum_t 2^(x_t - m) v_t / sum_t 2^(x_t - m) / v_scale_t,  m the running maximum of x,
// an online softmax in FP32. The value scale sits in the exponent, so the weights that meet the
// V codes have one range whatever the pages' scales are, and the sum divides it out again. Two pages' scales
// may lie 2^120 apart while their keys count alike in the sum, and FP32 ends at 2^-126: sums are carried
// from reference to reference in two steps, and a tile whose weights lie far below the row's others is
// summed relative to its own maximum.
//
// Products. S = Q K^T is an FP8 product straight from the cache's bytes: K is copied into
// shared memory and never converted. BF16 queries become two E4M3 rows, q = (hi + lo) 2^e (8
// significant bits = two 4-bit significands; exact while lo is a multiple of E4M3's smallest step,
// 2^-9 with the row's largest element in (224, 448], so down to 2^-9.8 of the largest, and within
// half that step, 2^-17.8 of the largest, below), so S costs two FP8 products instead of a
// conversion of K. P V runs in FP16: V codes are widened (exact), P is FP16 (an E4M3 P loses
// 2^-4 of a weight, and two E4M3 parts lose weights below 2^-18 of the largest, which a long
// context's tail adds up to).
//
// Floors: memory for few rows (a token and head is 256 bytes; the MMAs of a 128-token tile take
// less than its copy), tensor and exponential rate for prompts. Measured on a GB300 (graph replays):
//   64 requests of one row over 65,536 keys, 4 x 8 heads, E4M3 queries   669 us   6.4 TB/s
//   64 of one row over 16,384 keys, BF16 / E4M3 queries             190 / 178 us  5.7 / 6.0 TB/s
//   64 ragged requests, 512 .. 65,536 keys, up to 8 rows, BF16 queries   163 us   5.3 TB/s
//   one token over 4,096 keys, E4M3 queries                             14.5 us  (fixed costs)
//   16 requests with 16 listed blocks each, 8 rows, E4M3 queries        24.5 us  1.4 TB/s
//   2,053 rows on 16,421 keys, BF16 / E4M3 queries                  370 / 361 us  1.4 PFLOP/s
// (The figures beside the choices below are replays of this kernel with the one thing changed, in turn
// with it as it is.)
//
// Work. An item is a (request, KV head, chunk of query rows); its tiles are the pages its
// last row sees, or its block ids. All items' tiles form one line that the CTAs (one per SM)
// take in equal contiguous ranges, so ragged lengths balance and one long request uses the whole
// GPU; an item has kItemCost places on the line before its tiles, because starting and finishing
// a part costs a CTA as much as that many tiles. A CTA's part of an item is a segment; segments
// that are not whole items leave (O, m, l) in the workspace and kv8_merge_kernel joins them
// (log-sum-exp), in tile order: no atomics, the same bits every time.
//
// A CTA's M = rows x q_per_kv query rows are repeated C = 4, 2 or 1 times down the 128 rows of
// the MMA tile; copy c takes tokens 128 c / C .. of every tile with its own maximum and sum, so
// that few rows still spread the exponentials over all four SM sub-partitions (P is zero in the
// other copies' columns). Roles, as in the sparse attention over the NVFP4 cache (msa_attn.cu):
//   * K warp: finds the tiles (32 block-table entries and scales at a time, one per lane) and
//     copies their K (16 KB, tensor copies) into a ring; what the others need of a tile or
//     segment goes into small rings beside it;
//   * V warp: copies the tiles' V codes (16-byte asynchronous copies, zeros past the context). K and
//     V come by different paths: tensor and bulk copies alone measured 20-23 bytes a cycle and SM
//     whatever is in flight, a tile's 32 KB then 1,400 cycles even from L2; both paths together 50;
//   * 8 converting warps, four for each 64-token half of a tile: V to FP16 in four buffers that
//     the halves take in turn; at a segment's first tile they also lay out its queries;
//   * S warp (three score buffers in tensor memory) and P V warp (one O);
//   * 8 softmax warps in two sets. With one copy (prompts) a set takes every other tile, and the
//     rows' reference goes from set to set through shared memory. With more copies, where a row
//     has few tokens, both sets share every tile: of the tokens that a copy takes, set 0 has the
//     first half and set 1 the second, and the two threads of a row exchange their maxima.
//     (When both were built in both forms, prompts were 9 % faster in turn and 64 ragged requests of up
//     to 8 rows 6 % slower.)
//
// What bounds it now: long decode, memory (0.96 of the copy rate in the first line above; the same work on
// pages that L2 holds takes 575 us). Prompts, the roles' instruction streams: a tile costs a CTA 1,720
// cycles against 1,024 of tensor work with BF16 queries (62 % by the counter) and 1,700 against 768 with
// E4M3 (47 %), which therefore gain only 2 %; most of it are the dependent instructions of single warps
// between two hand-overs. What the loops hold in registers and how long their code is count for more
// there than the work in them: reading a row's maximum in a loop unrolled twice costs a prompt 4 % (BF16)
// or 6 % (E4M3), four times 29 or 45 %.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "msa_common.cuh"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kSoftWarps = 8;                        // warps 0..7: two sets of 4, one per TMEM lane quadrant
constexpr int kMmaWarp = 8, kPvWarp = 9, kKWarp = 10, kVWarp = 11;
constexpr int kCvWarp0 = 12, kCvWarps = 8;           // two groups of 4
constexpr int kThreads = (kCvWarp0 + kCvWarps) * 32;
constexpr int kVBufs = 4;                            // FP16 halves of V
// A wait on a barrier's parity has to be for its current phase or the one before. Waiters that
// fall behind therefore have barriers that go round 6 tiles or 8 halves (no wait is as far behind), or
// 12 tiles for a tile's description (up to 9 ahead).
constexpr int kBars = 6, kTold = 12;
constexpr int kRing = 16;                            // tiles and segments whose description is kept
constexpr int kRows = 8;                             // segments whose query scales and NaN marks are kept
constexpr uint32_t kTileBytes = kBlock * kDim;       // K or V of a tile
constexpr uint32_t kHalfBytes = 64 * 128;            // FP16 V: 64 tokens x 64 dims
// TMEM columns: three score buffers (128 FP32), O. The weights (FP16 pairs) go over the scores: tokens
// 0 .. 63 of a tile over columns 0 .. 31 of its buffer, tokens 64 .. 127 over columns 64 .. 95.
constexpr int kSBufs = 3;
constexpr uint32_t kColS = 0, kColO = kSBufs * kBlock, kTmemCols = 512;
static_assert(kColO + kDim <= kTmemCols, "TMEM");
// The largest weight of a row is 2^7 when its reference is set and may grow to 2^15 before O is rescaled: the
// upper part of FP16's range, so that weights vanish below 2^-32 of the largest and not below 2^-25 (a
// million keys at the border are then 2^-12 of a row; at 2^-25 they were a few hundredths of it).
constexpr float kStartLog2 = 7.f, kTopLog2 = 15.f;
constexpr float kZeroLog2 = -64.f;                   // stands for the logarithm of a value scale of 0
constexpr float kFaintLog2 = 60.f;                   // a tile's weights below 2^-60 are 0 in FP16 by far
constexpr int kNoPos = 1 << 30;                      // position of a tile that nobody sees
// Exchange between the copies of a row: two copies hand over 16 dims of every lane at a time, four put
// down whole rows, some at a time (floats of a lane or row, padded).
constexpr int kHandStride = 17, kRedRows = 32, kRedStride = 68;
static_assert(128 * kHandStride == kRedRows * kRedStride, "");
constexpr int kMergeThreads = 512, kMergeY = 4;      // CTAs that share an item, 32 dims each

enum : int { kEnd = 1, kFirst = 2, kLast = 4, kPart = 8 };
struct alignas(16) Tile {
  int page;      // physical page x KV heads + head
  int rows;      // V rows to read: tokens inside the context; 0 when its values count for nothing
  int marks;     // kEnd: no tile, the work is over; kFirst, kLast of its segment; kPart: some rows do
                 // not see all of its tokens
  int pos0;      // position of its first token
  float kscale;
  float lv, iv;  // log2 of the value scale, and its inverse
  int pad;
};

struct Seg {
  int last;      // its last tile
  int row0;      // first query row
  int rows;
  int head;      // KV head
  int pos;       // position of row0
  int slot;      // -1: a whole item, else the CTA's partial 0 or 1
};

// Counts round N places; `phase` flips every time round (a barrier's parity), without divisions.
template <int N>
struct Ring {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++at == N) at = 0, phase ^= 1u;
  }
};

template <int NP>
struct Smem {
  static constexpr int kKStages = 3, kVStages = NP == 1 ? 4 : 3;
  uint8_t q[NP][kTileBytes];                         // A of S: copies of the query rows, by part
  uint8_t k[kKStages][kTileBytes];                   // B of S (K-major), 128-byte swizzle
  uint8_t v[kVStages][kTileBytes];                   // V codes as they are in the page
  uint8_t v16[kVBufs][2][kHalfBytes];                // B of O (MN-major): [dim half][token][64 dims]
  float red[2][kRedRows * kRedStride];               // by set: what the copies exchange
  float qscale[kRows][128];                          // 2^e of each tile row (BF16 queries)
  int nanpos[kRows][kDim];                           // first position with a NaN value in a dim, of partly seen tokens
  int nanany[kRows];
  float half_max[2][2][128];                         // by tile parity: each set's maxima, or the reference
  float xm[2][128], xl[2][128], xm2[2][128];
  Tile tile[kRing];
  Seg seg[kRing];
  uint64_t k_full[kKStages], k_empty[kKStages], told[kTold];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t q_full, q_free, s_full[kBars], p_full[kBars], pv_done[kBars], v16_full[kVBufs], v16_free[2 * kVBufs], drain[2];
  uint64_t row_told[4];                              // by quadrant: a tile's maxima or reference are there
  uint64_t sets_met, set_met[2];                     // the softmax warps of both sets, or of one, have come here
  long long part[kThreads / 32];                     // places on the line by warp's requests
  uint32_t taddr;
};
static_assert(sizeof(Smem<2>) + 1024 <= 227 * 1024, "shared memory a CTA may opt into");
static_assert(offsetof(Smem<2>, k) % 1024 == 0 && offsetof(Smem<2>, v16) % 1024 == 0 && offsetof(Smem<1>, k) % 1024 == 0,
              "swizzled tiles");

// What a CTA leaves for the merge: [grid] headers, then 2 partials for each CTA.
struct Header {
  int tail;          // 1: partial 1 starts an item that goes on in the next CTA's partial 0
  int row0, rows, head;
  int cont;          // 1: partial 0 is a part of an item that an earlier CTA started
  int cont_end;      //    and its last one
  int pad[2];
};
constexpr long long kPartFloats = 128LL * kDim + 256;  // O, m, l
// Where dims d .. d + 3 of row l of a partial's O are: 8 rows' 16-byte pieces side by side, so that
// lanes with a row each and lanes with some rows and dims each both move whole lines. (Rows one after
// the other cost the writer 32 lines a store: one token over 4,096 keys 16.4 us instead of 14.4, 16
// requests with 16 listed blocks 26.5 instead of 25.)
__device__ __forceinline__ int part_at(int l, int d) { return (((l >> 3) * (kDim / 4) + (d >> 2)) * 8 + (l & 7)) * 4; }
__host__ __device__ inline size_t headers_bytes(int grid) { return (grid * sizeof(Header) + 255) / 256 * 256; }

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

// ---- the line of tiles
// Places of an item before its tiles. 64 ragged requests / 16 requests with 16 listed blocks each take
// 168 / 24.7 us with 4 places, 164 / 25.0 with 5, 163 / 25.3 with 6.
constexpr int kItemCost = 5;
struct Req {
  int N, R, r0;
};
__device__ __forceinline__ bool load_req(const Kv8AttnParams& p, int b, Req* q) {
  q->N = p.context_lens[b];
  q->r0 = p.q_indptr[b];
  q->R = p.q_indptr[b + 1] - q->r0;
  return q->N >= 0 && q->N <= p.max_pages * static_cast<long long>(kBlock) && q->R >= 0 && q->R <= p.max_rows &&
         q->R <= q->N && q->r0 >= 0 && q->r0 <= p.total_rows - q->R;
}
__device__ __forceinline__ int chunks_of(const Kv8AttnParams& p, int R) { return (R + p.chunk - 1) >> p.chunk_log2; }
// Tiles of row chunk i: the pages up to its last row's position.
__device__ __forceinline__ int tiles_of(const Kv8AttnParams& p, const Req& q, int i) {
  if (p.n_ids) return p.n_ids;
  const int end = (i + 1) << p.chunk_log2;
  const int last = q.N - q.R + (end < q.R ? end : q.R) - 1;
  return (last >> 7) + 1;
}
// Tiles of the chunks before i (i at most the last chunk, so each of them is whole). With
// base = N - R - 1 = 128 a + r0 and u = 128 / chunk chunks to a page, chunk k has
// 1 + a + floor((r0 / chunk + k + 1) / u) tiles; the floors sum in closed form.
__device__ __forceinline__ long long tiles_before(const Kv8AttnParams& p, const Req& q, int i) {
  if (p.n_ids) return static_cast<long long>(i) * p.n_ids;
  const int base = q.N - q.R - 1, a = base >> 7, c0 = (base & 127) >> p.chunk_log2, lu = 7 - p.chunk_log2;
  auto floors = [lu](long long m) {  // sum of j >> lu over j < m
    const long long w = m >> lu, rem = m & ((1LL << lu) - 1);
    return (w * (w - 1) / 2 << lu) + w * rem;
  };
  return static_cast<long long>(i) * (1 + a) + floors(c0 + i + 1LL) - floors(c0 + 1LL);
}
// Places on the line before row chunk i (at most the last one), and of one KV head of the request.
__device__ __forceinline__ long long cost_before(const Kv8AttnParams& p, const Req& q, int i) {
  return i > 0 ? tiles_before(p, q, i) + static_cast<long long>(i) * kItemCost : 0;
}
__device__ __forceinline__ long long head_cost(const Kv8AttnParams& p, const Req& q) {
  if (q.R == 0) return 0;
  const int n = chunks_of(p, q.R);
  return cost_before(p, q, n - 1) + kItemCost + tiles_of(p, q, n - 1);
}

// C copies of the query rows down the MMA tile (128 / C rows each); NP = E4M3 parts of a query.
template <int C, int NP>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap kmap, const Kv8AttnParams p) {
  constexpr int kMpad = 128 / C;
  constexpr bool kTurns = C == 1;  // the softmax sets take tiles in turn; otherwise they share every tile
  constexpr int kStages = Smem<NP>::kKStages, kVStages = Smem<NP>::kVStages;
  extern __shared__ uint8_t smem_raw[];
  Smem<NP>& sm = *reinterpret_cast<Smem<NP>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.q_per_kv;

  pdl_launch_dependents();  // the merge waits for this grid's end; its CTAs may be set up before
  {  // a thread per barrier
    auto init = [&](uint64_t* bar, int n, int first, uint32_t count) {
      if (tid >= first && tid < first + n) mbar_init(smem_u32(bar + (tid - first)), count);
    };
    init(sm.k_full, kStages, 0, 1);
    init(sm.k_empty, kStages, 8, 1);
    init(sm.told, kTold, 16, 1);
    init(sm.v_full, kVStages, 28, 33);
    init(sm.v_empty, kVStages, 32, kCvWarps);
    init(sm.s_full, kBars, 36, 1);
    init(sm.p_full, kBars, 42, kTurns ? kSoftWarps / 2 : kSoftWarps);
    init(sm.pv_done, kBars, 48, 1);
    init(sm.v16_full, kVBufs, 54, kCvWarps / 2);
    init(sm.v16_free, 2 * kVBufs, 58, 1);
    init(sm.drain, 2, 66, 1);
    init(&sm.q_full, 1, 68, kCvWarps);
    init(&sm.q_free, 1, 69, 1);
    init(&sm.sets_met, 1, 70, kSoftWarps);
    init(sm.set_met, 2, 72, kSoftWarps / 2);
    init(sm.row_told, 4, 74, kTurns ? 1 : 2);
    if (tid < 96) mbar_fence_init();
  }
  for (int i = tid; i < kRows * kDim; i += kThreads) (&sm.nanpos[0][0])[i] = INT_MAX;
  if (tid < kRows) sm.nanany[tid] = 0;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&sm.taddr), kTmemCols);
  if (warp == kKWarp && lane == 0)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");

  // ---- the line: every thread sums a run of requests; the K warp finds the CTA's range in the sums
  const int per = (p.num_reqs + kThreads - 1) / kThreads;
  long long* sums = reinterpret_cast<long long*>(sm.red[0]);  // inclusive within a warp (red has no use yet)
  static_assert(sizeof(sm.red) >= kThreads * sizeof(long long), "");
  {
    const int b0 = tid * per < p.num_reqs ? tid * per : p.num_reqs;
    const int b1 = b0 + per < p.num_reqs ? b0 + per : p.num_reqs;
    long long incl = 0;
    for (int b = b0; b < b1; ++b) {
      Req q;
      if (load_req(p, b, &q)) incl += p.num_kv_heads * head_cost(p, q);
      else if (blockIdx.x == 0) set_flag(p.flags, kFlagBadLength);
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    sums[tid] = incl;
    if (lane == 31) sm.part[warp] = incl;
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.taddr;

  if (warp == kKWarp) {
    // ================= K warp
    int t = 0, nseg = 0;
    bool good = true;
    Header hd = {};
    // Waits until tile t's stage is free, writes its description and starts its K copy.
    auto emit = [&](int pos0, int nvalid, int marks, int page, float ks, float lv, float iv, bool vzero) {
      const int st = t % kStages;
      if (t >= kStages) {
        good = warp_wait(smem_u32(&sm.k_empty[st]), ((t / kStages) - 1) & 1, p.flags);
        if (!good) return;
      }
      if (lane == 0) {
        Tile& x = sm.tile[t % kRing];
        *reinterpret_cast<int4*>(&x.page) = make_int4(page, vzero ? 0 : nvalid, marks, pos0);
        *reinterpret_cast<float4*>(&x.kscale) = make_float4(ks, lv, iv, 0.f);
        mbar_arrive(smem_u32(&sm.told[t % kTold]));
        const uint32_t kb = smem_u32(&sm.k_full[st]);
        if (nvalid > 0) {
          mbar_arrive_expect_tx(kb, kTileBytes);
          tma_load_2d(smem_u32(sm.k[st]), &kmap, 0, page * kBlock, kb);
        } else {
          mbar_arrive(kb);
        }
      }
      __syncwarp();
      ++t;
    };

    long long left = 0, start = 0;  // places in the range; the first one's offset in request b
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
      // fewer tiles than CTAs: the last CTAs have none (a partial's continuation is in the next CTA)
      long long lo = 0, hi = 0;
      if (total < (1LL << 31)) {  // 32-bit division: this is on the way of the first copy
        const uint32_t tot = static_cast<uint32_t>(total), use = tot < gridDim.x ? tot : gridDim.x;
        if (blockIdx.x < use) {
          const uint32_t each = tot / use, more = tot - each * use;  // the first `more` CTAs take one more
          lo = each * blockIdx.x + (blockIdx.x < more ? blockIdx.x : more);
          hi = lo + each + (blockIdx.x < more ? 1 : 0);
        }
      } else {
        lo = total * blockIdx.x / gridDim.x;
        hi = total * (blockIdx.x + 1) / gridDim.x;
      }
      left = hi - lo;
      if (left > 0) {
        // the warp whose requests hold place lo, then the thread, then the request
        const int w = __ffs(__ballot_sync(0xFFFFFFFFu, lo < incl)) - 1;
        const long long before = w > 0 ? __shfl_sync(0xFFFFFFFFu, incl, w - 1) : 0;
        const long long mine = before + sums[32 * w + lane];
        const int th = __ffs(__ballot_sync(0xFFFFFFFFu, lo < mine)) - 1;
        long long at = th > 0 ? __shfl_sync(0xFFFFFFFFu, mine, th - 1) : before;
        b = (32 * w + th) * per;
        for (int i = 1; i < per && b + 1 < p.num_reqs; ++i) {
          Req q;
          const long long n = load_req(p, b, &q) ? p.num_kv_heads * head_cost(p, q) : 0;
          if (lo < at + n) break;
          at += n;
          ++b;
        }
        start = lo - at;
      }
    }
    if (left > 0) {
      Req q;
      load_req(p, b, &q);
      int h, ch, at, n_ch = chunks_of(p, q.R);  // at: the CTA's place in the item
      {
        const long long hc = head_cost(p, q);
        h = start < (1LL << 31) && hc < (1LL << 31)
                ? static_cast<int>(static_cast<uint32_t>(start) / static_cast<uint32_t>(hc))
                : static_cast<int>(start / hc);
        const long long off = start - h * hc;
        int a = 0, e = n_ch;  // cost_before(a) <= off < cost_before(e)
        while (e - a > 1) {
          const int mid = (a + e) / 2;
          if (cost_before(p, q, mid) <= off) a = mid;
          else e = mid;
        }
        ch = a;
        at = static_cast<int>(off - cost_before(p, q, a));
      }
      while (left > 0 && good) {
        const int nt = tiles_of(p, q, ch);
        const int j0 = at > kItemCost ? at - kItemCost : 0;
        const long long to = at + left - kItemCost;
        const int j1 = to < nt ? static_cast<int>(to) : nt;
        if (j1 <= j0) break;  // the range ends before the item's first tile
        const int nb = (q.N + kBlock - 1) / kBlock;
        const bool begin = j0 == 0, end = j1 == nt;
        const int row0 = ch << p.chunk_log2, rows = q.R - row0 < p.chunk ? q.R - row0 : p.chunk;
        const int32_t* table = p.block_table + static_cast<long long>(b) * p.max_pages;
        // listed blocks: lane j holds id j; the ones of this segment that count
        int id = -1;
        unsigned use = 0u;
        if (p.n_ids) {
          if (lane < p.n_ids) id = p.block_ids[(static_cast<long long>(b) * p.num_kv_heads + h) * p.n_ids + lane];
          const bool in = id >= 0 && id < nb;
          const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
          const bool twice = in && (__ffs(same) - 1) != lane;
          if (ch == 0 && lane >= j0 && lane < j1 && ((!in && id != -1) || twice)) set_flag(p.flags, kFlagBadIds);
          use = __ballot_sync(0xFFFFFFFFu, in && !twice && lane >= j0 && lane < j1);
        }
        const int count = p.n_ids ? (use ? __popc(use) : 1) : j1 - j0;
        const int first = t, last = t + count - 1, pos = q.N - q.R + row0;
        auto marks = [&]() { return (t == first ? kFirst : 0) | (t == last ? kLast : 0); };
        const int slot = begin && end ? -1 : (begin ? 1 : 0);
        if (lane == 0) {
          Seg& s = sm.seg[nseg % kRing];
          s.last = last;
          s.row0 = q.r0 + row0;
          s.rows = rows;
          s.head = h;
          s.pos = pos;
          s.slot = slot;
        }
        if (slot == 1) {
          hd.tail = 1;
          hd.row0 = q.r0 + row0;
          hd.rows = rows;
          hd.head = h;
        } else if (slot == 0) {
          hd.cont = 1;
          hd.cont_end = end;
        }
        __syncwarp();
        for (int base = p.n_ids ? 0 : j0; base < (p.n_ids ? 1 : j1) && good; base += 32) {
          const int c = p.n_ids ? id : base + lane;
          const bool on = p.n_ids ? (use >> lane) & 1u : c < j1;
          int phys = -1;
          float ks = 1.f, lv = 0.f, iv = 1.f;
          bool vzero = false;
          if (on) {
            phys = table[c];
            if (phys < 0 || phys >= p.num_pages) {
              set_flag(p.flags, kFlagBadPage);
              phys = -1;
            } else {
              const long long ph = static_cast<long long>(phys) * p.num_kv_heads + h;
              ks = p.k_scale[ph];
              const float vs = p.v_scale[ph];
              vzero = vs == 0.f;
              // a page of scale 0 has keys but no values: below every scale, so that its scores do not
              // raise the reference and take the other pages' weights out of FP16's range
              lv = vzero ? kZeroLog2 : log2f(vs);
              iv = vzero ? exp2f(-kZeroLog2) : 1.f / vs;
            }
          }
          for (unsigned m = __ballot_sync(0xFFFFFFFFu, on); m != 0u && good; m &= m - 1u) {
            const int src = __ffs(m) - 1;
            const int cc = __shfl_sync(0xFFFFFFFFu, c, src), pp = __shfl_sync(0xFFFFFFFFu, phys, src);
            const float kk = __shfl_sync(0xFFFFFFFFu, ks, src), ll = __shfl_sync(0xFFFFFFFFu, lv, src);
            const float ii = __shfl_sync(0xFFFFFFFFu, iv, src);
            const bool zz = __shfl_sync(0xFFFFFFFFu, static_cast<int>(vzero), src) != 0;
            const int pos0 = cc * kBlock, nv = q.N - pos0 < kBlock ? q.N - pos0 : kBlock;
            if (pp < 0) emit(kNoPos, 0, marks(), 0, 1.f, 0.f, 1.f, true);
            else emit(pos0, nv, marks() | (pos0 + nv - 1 > pos ? kPart : 0), pp * p.num_kv_heads + h, kk, ll, ii, zz);
          }
        }
        if (p.n_ids && use == 0u && good) emit(kNoPos, 0, marks(), 0, 1.f, 0.f, 1.f, true);
        ++nseg;
        left -= kItemCost + nt - at;
        // the next item
        at = 0;
        if (left > 0 && ++ch == n_ch) {
          ch = 0;
          if (++h == p.num_kv_heads) {
            h = 0;
            do ++b; while (b < p.num_reqs && (!load_req(p, b, &q) || q.R == 0));
            if (b == p.num_reqs) break;  // never, unless the lengths changed meanwhile
            n_ch = chunks_of(p, q.R);
          }
        }
      }
    }
    if (good) emit(kNoPos, 0, kEnd, 0, 1.f, 0.f, 1.f, true);
    // no copy may still be landing when the CTA leaves
    for (int j = t - kStages < 0 ? 0 : t - kStages; j < t; ++j)
      if (!wait_bar(smem_u32(&sm.k_full[j % kStages]), (j / kStages) & 1, p.flags)) break;
    if (lane == 0) reinterpret_cast<Header*>(p.parts)[blockIdx.x] = hd;
    __syncwarp();
  } else if (warp == kVWarp) {
    // ================= V warp: the tiles' V codes by 16-byte asynchronous copies, a lane = one piece of
    // every 4th row; zeros for rows past the context
    const uint32_t dst0 = smem_u32(sm.v[0]) + 16u * lane;
    Ring<kTold> rt;
    Ring<kVStages> rs;
    for (int t = 0;; ++t, rt.step(), rs.step()) {
      if (t >= kVStages && !warp_wait(smem_u32(&sm.v_empty[rs.at]), rs.phase ^ 1u, p.flags)) break;
      if (!warp_wait(smem_u32(&sm.told[rt.at]), rt.phase, p.flags)) break;
      const int4 x = *reinterpret_cast<const int4*>(&sm.tile[t % kRing].page);
      const bool end = x.z & kEnd;
      if (!end) {
        const uint8_t* src = p.v_data + static_cast<long long>(x.x) * kTileBytes + 16 * lane;
        const uint32_t dst = dst0 + rs.at * kTileBytes;
        const int rows = x.y - (lane >> 3);
        if (x.y == kBlock) {
#pragma unroll
          for (int i = 0; i < 32; ++i) cp_async16(dst + 512u * i, src + 512 * i, 16u);
        } else {
#pragma unroll 1
          for (int i = 0; i < 32; ++i) cp_async16(dst + 512u * i, src + 512 * i, rows > 4 * i ? 16u : 0u);
        }
      }
      // 32 arrivals when the copies have landed, and one now that hands the description on
      const uint32_t full = smem_u32(&sm.v_full[rs.at]);
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
      if (lane == 0) mbar_arrive(full);
      if (end) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // none may still be landing when the CTA leaves
    __syncwarp();
  } else if (warp >= kCvWarp0) {
    // ================= converting warps: group h has tokens 64 h .. 64 h + 63 of every tile; thread =
    // one 16-byte piece of every 16th row
    const int h = (warp - kCvWarp0) / 4, r = (tid - kCvWarp0 * 32) & 127;
    // V row (mod 16) and 16-byte piece: 16 codes become two 16-byte pieces of dim half vc / 4. The second
    // half's threads take the row beside, so that 8 neighbours meet 8 different bank groups
    const int vc = r & 7, vr = (r >> 3) ^ (vc >> 2);
    const uint32_t o0 = static_cast<uint32_t>((2 * (vc & 3)) ^ (vr & 7)) << 4, o1 = o0 ^ 16u;
    const uint32_t slot0 = smem_u32(sm.v[0]) + static_cast<uint32_t>(64 * kDim * h + kDim * vr + 16 * vc);
    int k = -1;                        // the segment
    Ring<kVStages> rs;
    for (int t = 0;; ++t, rs.step()) {
      if (!warp_wait(smem_u32(&sm.v_full[rs.at]), rs.phase, p.flags)) break;
      const int4 x = *reinterpret_cast<const int4*>(&sm.tile[t % kRing].page);
      const bool end = x.z & kEnd;
      if (x.z & kFirst) {
        const Seg& sg = sm.seg[++k % kRing];
        // the segment's queries, once the last segment's scores are computed: two threads per row
        if (k > 0 && !warp_wait(smem_u32(&sm.q_free), (k - 1) & 1, p.flags)) break;
        const int rr = 64 * h + (r >> 1), half = r & 1, m = rr % kMpad;
        const bool real = m < G * sg.rows;
        const long long at = real ? static_cast<long long>(sg.row0 + m / G) * p.q_stride + (sg.head * G + m % G) * kDim : 0;
        const uint32_t row = smem_u32(sm.q[0]) + static_cast<uint32_t>(rr) * 128u;
        if constexpr (NP == 1) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) + at) + 4 * half;
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_shared_v4(row + (static_cast<uint32_t>((4 * half + c) ^ (rr & 7)) << 4), v[c].x, v[c].y, v[c].z, v[c].w);
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at) + 8 * half;
          uint4 v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          // largest magnitude by its bits: BF16 pairs, both halves at once
          uint32_t big = 0u;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            big = __vmaxu2(big, __vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu)));
          big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
          const uint32_t amax = max(big & 0xFFFFu, big >> 16);
          const bool odd = amax >= 0x7F80u;  // an infinity or a NaN: the whole row becomes NaN
          // smallest 2^e with amax <= 448 2^e; below 2^-120 nothing a score could show is left
          int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
          e = e < -120 ? -120 : e;
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          if (half == 0) sm.qscale[k % kRows][rr] = odd ? 1.f : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16 elements: 16 code bytes of each part
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t w[4] = {v[2 * c + u].x, v[2 * c + u].y, v[2 * c + u].z, v[2 * c + u].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = __uint_as_float(w[i] << 16) * inv, b2 = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
                const uint32_t hc = f32x2_e4m3x2(a, b2);
                const uint32_t hh = e4m3x2_f16x2(hc);
                const float2 hv = __half22float2(*reinterpret_cast<const __half2*>(&hh));
                const uint32_t lc = f32x2_e4m3x2(a - hv.x, b2 - hv.y);
                if (i & 1) {
                  hi[2 * u + i / 2] |= hc << 16;
                  lo[2 * u + i / 2] |= lc << 16;
                } else {
                  hi[2 * u + i / 2] = hc;
                  lo[2 * u + i / 2] = lc;
                }
              }
            }
            if (odd)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                hi[i] = 0x7F7F7F7Fu;
                lo[i] = 0u;
              }
            const uint32_t o = static_cast<uint32_t>((4 * half + c) ^ (rr & 7)) << 4;
            st_shared_v4(row + o, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(row + kTileBytes + o, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));
      }
      const uint32_t raw = slot0 + rs.at * kTileBytes;
      // a token that some rows of the segment do not see: its weight is 0 there, but 0 x NaN is
      // NaN, so its NaN codes become 0 here and are put back for the rows that see it
      if (x.z & kPart) {
        const int pos = sm.seg[k % kRing].pos;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {  // word i % 4 of the piece of row 16 (i / 4) + vr
          const int token = 64 * h + 16 * (i >> 2) + vr;
          const uint32_t at = raw + 2048u * (i >> 2) + 4u * (i & 3);
          const uint32_t w = lds_u1(at), nan = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          if (nan == 0u || token >= x.y || x.w + token <= pos) continue;
          for (int z = 0; z < 4; ++z)
            if ((nan >> (8 * z)) & 1u) atomicMin(&sm.nanpos[k % kRows][16 * vc + 4 * (i & 3) + z], x.w + token);
          sm.nanany[k % kRows] = 1;
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w & ~nan) : "memory");
        }
      }
      // the half that was in this buffer (four halves ago) has been multiplied (waiting here and not
      // with the converted values in registers: BF16 prompt 392 -> 370 us, 64 ragged requests 168 -> 164)
      const uint32_t u = 2 * t + h, uv = u % kVBufs;
      if (t >= 2 && !warp_wait(smem_u32(&sm.v16_free[(u - kVBufs) % (2 * kVBufs)]), ((u - kVBufs) / (2 * kVBufs)) & 1, p.flags))
        break;
      if (end) {
        if (h == 0 && lane == 0) mbar_arrive(smem_u32(&sm.v16_full[uv]));
        break;
      }
      uint32_t f[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = lds_u4(raw + 2048u * i);
        e4m3x4_f16x4(w.x, f[i][0], f[i][1]);
        e4m3x4_f16x4(w.y, f[i][2], f[i][3]);
        e4m3x4_f16x4(w.z, f[i][4], f[i][5]);
        e4m3x4_f16x4(w.w, f[i][6], f[i][7]);
      }
      const uint32_t dst = smem_u32(sm.v16[uv][vc >> 2]) + static_cast<uint32_t>(vr) * 128u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st_shared_v4(dst + 2048u * i + o0, f[i][0], f[i][1], f[i][2], f[i][3]);
        st_shared_v4(dst + 2048u * i + o1, f[i][4], f[i][5], f[i][6], f[i][7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&sm.v16_full[uv]));
        mbar_arrive(smem_u32(&sm.v_empty[rs.at]));  // (the stores above have used every value)
      }
    }
  } else if (warp == kMmaWarp) {
    // ================= S warp: S_t = Q K_t^T into buffer t % 3
    const uint32_t el = elect_one();
    const uint64_t qdesc = sdesc_kmajor_sw128(smem_u32(sm.q[0])), kdesc0 = sdesc_kmajor_sw128(smem_u32(sm.k[0]));
    const uint32_t idesc = idesc_e4m3_f32(128, kBlock, false, false);
    int seg = -1;
    bool good = true;
    Ring<kStages> rk;
    Ring<kBars> rb;
    static_assert(kBars == 2 * kSBufs, "");
    for (int t = 0;; ++t, rb.step(), rk.step()) {
      const uint32_t sb = rb.at < 3u ? rb.at : rb.at - 3u;
      if (!warp_wait(smem_u32(&sm.k_full[rk.at]), rk.phase, p.flags)) break;
      // the buffer's previous weights (of tile t - 3) have been used
      if (t >= kSBufs)
        good = rb.at < 3u ? warp_wait(smem_u32(&sm.pv_done[rb.at + 3u]), rb.phase ^ 1u, p.flags)
                          : warp_wait(smem_u32(&sm.pv_done[rb.at - 3u]), rb.phase, p.flags);
      if (!good) break;
      const int marks = sm.tile[t % kRing].marks;
      if (marks & kEnd) {
        if (lane == 0) mbar_arrive(smem_u32(&sm.s_full[rb.at]));
        break;
      }
      if (marks & kFirst && !warp_wait(smem_u32(&sm.q_full), ++seg & 1, p.flags)) break;
      tc_fence_after();
      const uint64_t kdesc = kdesc0 + rk.at * (kTileBytes >> 4);
#pragma unroll
      for (int part = 0; part < NP; ++part)
#pragma unroll
        for (int kk = 0; kk < kDim / 32; ++kk)  // 32 bytes along the rows: + 2 in the address field
          mma_f8_ss_elect(el, tbase + kColS + kBlock * sb, qdesc + part * (kTileBytes >> 4) + 2 * kk, kdesc + 2 * kk, idesc,
                          part > 0 || kk > 0);
      commit_elect(el, smem_u32(&sm.s_full[rb.at]));
      commit_elect(el, smem_u32(&sm.k_empty[rk.at]));
      if (marks & kLast) commit_elect(el, smem_u32(&sm.q_free));
    }
    if (seg >= 0) {  // every MMA of this thread has finished before the tensor memory is released
      commit_elect(el, smem_u32(&sm.drain[0]));
      warp_wait(smem_u32(&sm.drain[0]), 0, p.flags);
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ================= P V warp: O (+)= P_t V_t, a half of the tokens at a time
    const uint32_t el = elect_one();
    const uint32_t idesc = idesc_f16_f32(128, kDim, true);
    // 128 dims = two 64-dim halves (the leading offset), 8-token groups 1 KB apart, 16 tokens = 2 KB
    const uint64_t vdesc0 = sdesc_mn_sw128(smem_u32(sm.v16[0][0]), kHalfBytes);
    bool good = true, any = false;
    Ring<kBars> rb;        // tiles
    Ring<2 * kVBufs> ru;   // halves
    Ring<kVBufs> rv;       // the halves' buffers
    for (int t = 0; good; ++t, rb.step()) {
      if (!warp_wait(smem_u32(&sm.v16_full[rv.at]), rv.phase, p.flags)) break;
      const int marks = sm.tile[t % kRing].marks;
      if (marks & kEnd) break;
      if (!warp_wait(smem_u32(&sm.p_full[rb.at]), rb.phase, p.flags)) break;
      const uint32_t pcol = tbase + kColS + kBlock * (rb.at < 3u ? rb.at : rb.at - 3u);
#pragma unroll
      for (int h = 0; h < 2; ++h, rv.step(), ru.step()) {
        if (h == 1) {
          good = warp_wait(smem_u32(&sm.v16_full[rv.at]), rv.phase, p.flags);
          if (!good) break;
        }
        tc_fence_after();
        const uint64_t vdesc = vdesc0 + rv.at * (2 * kHalfBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_tmemA_elect(el, tbase + kColO, pcol + 64 * h + 8 * kk, vdesc + 128 * kk, idesc,
                              !(marks & kFirst) || h > 0 || kk > 0 ? 1u : 0u);
        commit_elect(el, smem_u32(&sm.v16_free[ru.at]));
      }
      any = true;  // (a half may be on its way)
      if (!good) break;
      commit_elect(el, smem_u32(&sm.pv_done[rb.at]));
    }
    if (any) {
      commit_elect(el, smem_u32(&sm.drain[1]));
      warp_wait(smem_u32(&sm.drain[1]), 0, p.flags);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ================= softmax warps of set s: TMEM lane l = query row m of copy c, which takes
    // tokens 128 c / C .. of every tile. With one copy set s takes tiles s, s + 2, ..; with more both sets
    // take every tile, half of a copy's tokens each. A thread has kN tokens from k0 on.
    constexpr int kN = kTurns ? kMpad : kMpad / 2;
    const int s = warp / 4, quad = warp % 4;
    const int l = 32 * quad + lane, m = l % kMpad, c = l / kMpad, k0 = c * kMpad + (kTurns ? 0 : s * kN);
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t p_off = 64u * (k0 / 64) + (k0 % 64) / 2;  // the weights' first column
    const int row = m / G;
    float mref = -INFINITY, lrun = 0.f;  // the row's reference at this set's last tile, this set's sum
    int seg = 0;
    uint32_t met_all = 0, met_set = 0;               // phases of the meeting points
    // A meeting of warps, bounded like every other wait: after a timeout anywhere each warp leaves
    // by itself.
    auto meet = [&](uint64_t* bar, uint32_t& phase) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(bar));
      return warp_wait(smem_u32(bar), phase++ & 1u, p.flags);
    };

    // The segment's output or partial. Both sets take part: set s writes dims 64 s .. 64 s + 63.
    auto finish = [&](int k) -> bool {
      const Seg sg = sm.seg[k % kRing];
      if (!warp_wait(smem_u32(&sm.pv_done[sg.last % kBars]), (sg.last / kBars) & 1, p.flags)) return false;
      sm.xm[s][l] = mref;
      sm.xl[s][l] = lrun;
      if (!meet(&sm.sets_met, met_all)) return false;
      tc_fence_after();
      // reference and sum of row mm over its copies
      auto stats = [&](int mm, float& ref, float& sum) {
        ref = -INFINITY;
#pragma unroll
        for (int i = 0; i < C; ++i) ref = fmaxf(ref, fmaxf(sm.xm[0][i * kMpad + mm], sm.xm[1][i * kMpad + mm]));
        const float r0 = ref == -INFINITY ? 0.f : ref;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i)
          sum += carry(sm.xl[0][i * kMpad + mm], sm.xm[0][i * kMpad + mm], r0) +
                 carry(sm.xl[1][i * kMpad + mm], sm.xm[1][i * kMpad + mm], r0);
      };
      const bool whole = sg.slot < 0;
      const bool nans = sm.nanany[k % kRows] != 0;
      const int M = G * sg.rows;
      float* part = reinterpret_cast<float*>(p.parts + headers_bytes(gridDim.x)) +
                    (2LL * blockIdx.x + (whole ? 0 : sg.slot)) * kPartFloats;
      // 4 N dims from d on of row mm, not yet divided by the sum: to the output, or to the partial.
      auto put = [&](int mm, int d, auto& f, float sum) {
        constexpr int kF = sizeof(f) / sizeof(float);
        const float inv = !whole ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);
#pragma unroll
        for (int u = 0; u < kF; ++u) {
          f[u] *= inv;
          if (nans && sm.nanpos[k % kRows][d + u] <= sg.pos + mm / G) f[u] = __int_as_float(0x7FFFFFFF);
        }
        if (whole) {
          const long long orow = static_cast<long long>(sg.row0 + mm / G) * (p.num_kv_heads * G) + sg.head * G + mm % G;
          uint16_t* to = p.out + orow * kDim + d;
          if constexpr (kF % 8 == 0) {
#pragma unroll
            for (int u = 0; u < kF; u += 8)
              *reinterpret_cast<uint4*>(to + u) = make_uint4(bf16x2_bits(f[u], f[u + 1]), bf16x2_bits(f[u + 2], f[u + 3]),
                                                             bf16x2_bits(f[u + 4], f[u + 5]), bf16x2_bits(f[u + 6], f[u + 7]));
          } else {
            *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]));
          }
        } else {
#pragma unroll
          for (int u = 0; u < kF; u += 4)
            *reinterpret_cast<float4*>(part + part_at(mm, d + u)) = make_float4(f[u], f[u + 1], f[u + 2], f[u + 3]);
        }
      };
      auto put_lse = [&](float ref, float sum) {
        if (p.lse != nullptr)
          p.lse[static_cast<long long>(sg.row0 + row) * (p.num_kv_heads * G) + sg.head * G + m % G] =
              sum == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + log2f(sum)) * 0.69314718055994531f;
      };
      const float copy_ref = fmaxf(sm.xm[0][l], sm.xm[1][l]);  // of this copy's tokens
      if constexpr (C == 1) {  // a thread has 64 dims of its row
        const float r0 = copy_ref == -INFINITY ? 0.f : copy_ref;
        const float sum = carry(sm.xl[0][l], sm.xm[0][l], r0) + carry(sm.xl[1][l], sm.xm[1][l], r0);
#pragma unroll 1
        for (int d = 64 * s; d < 64 * s + 64; d += 16) {
          uint32_t a[16];
          tmem_ld16(tbase + lane_base + kColO + d, a);
          tc_wait_ld();
          float f[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) f[u] = __uint_as_float(a[u]);
          if (m < M) put(m, d, f, sum);
        }
        if (m < M && s == 0) {
          if (whole) {
            put_lse(copy_ref, sum);
          } else {
            part[128 * kDim + m] = copy_ref;
            part[128 * kDim + 128 + m] = sum;
          }
        }
      } else {
        float my_ref, my_sum;
        stats(m, my_ref, my_sum);
        const float w0 = ex2(copy_ref - (my_ref == -INFINITY ? 0.f : my_ref));
        if constexpr (C == 4) {
          // Some rows at a time (one round for a decode step's few): every copy's lane puts its row's 64
          // dims of this set down, then the set's threads add the copies up in a fixed order, 4 dims of
          // a row each.
          constexpr int kG = kRedRows / C;
          float* red = sm.red[s];
#pragma unroll 1
          for (int g = 0; g < M; g += kG) {
            if (g > 0 && !meet(&sm.set_met[s], met_set)) return false;  // the rows before have been read
            const bool mine = m >= g && m < g + kG;
            const uint32_t to = smem_u32(red + (c * kG + m - g) * kRedStride);
#pragma unroll 1
            for (int d = 0; d < 64; d += 16) {
              uint32_t a[16];
              tmem_ld16(tbase + lane_base + kColO + 64 * s + d, a);
              tc_wait_ld();
              if (mine)
#pragma unroll
                for (int u = 0; u < 16; u += 4)
                  st_shared_v4(to + 4u * (d + u), __float_as_uint(w0 * __uint_as_float(a[u])),
                               __float_as_uint(w0 * __uint_as_float(a[u + 1])), __float_as_uint(w0 * __uint_as_float(a[u + 2])),
                               __float_as_uint(w0 * __uint_as_float(a[u + 3])));
            }
            if (!meet(&sm.set_met[s], met_set)) return false;
            static_assert(kG == 8, "");  // a thread has 4 dims of a row
            const int i = l & 7, d = 4 * (l >> 3);
            if (g + i < M) {
              float f[4] = {};
#pragma unroll
              for (int z = 0; z < C; ++z) {
                const float4 o = *reinterpret_cast<const float4*>(red + (z * kG + i) * kRedStride + d);
                f[0] += o.x;
                f[1] += o.y;
                f[2] += o.z;
                f[3] += o.w;
              }
              float ref, sum = 1.f;
              if (whole) stats(g + i, ref, sum);
              put(g + i, 64 * s + d, f, sum);
            }
          }
        } else {
          // Copy c finishes dims kD c .. of this set's 64: in round r every lane hands 16 dims to copy
          // c + r and takes 16 from copy c - r, in a fixed order.
          // (Rows at a time, as above, were 3 % slower here for 64 ragged requests when both were built.)
          constexpr int kD = 64 / C;
          float* red = sm.red[s];
          float y[kD];
#pragma unroll
          for (int ch = 0; ch < kD / 16; ++ch) {
            uint32_t a[16];
            tmem_ld16(tbase + lane_base + kColO + 64 * s + kD * c + 16 * ch, a);
            tc_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; ++u) y[16 * ch + u] = w0 * __uint_as_float(a[u]);
          }
#pragma unroll
          for (int step = 0; step < (C - 1) * (kD / 16); ++step) {
            const int r = 1 + step / (kD / 16), ch = step % (kD / 16), to = (c + r) % C, from = (c + C - r) % C;
            uint32_t a[16];
            tmem_ld16(tbase + lane_base + kColO + 64 * s + kD * to + 16 * ch, a);
            tc_wait_ld();
            if (step > 0 && !meet(&sm.set_met[s], met_set)) return false;  // the last round's values are in y
#pragma unroll
            for (int u = 0; u < 16; ++u) red[l * kHandStride + u] = w0 * __uint_as_float(a[u]);
            if (!meet(&sm.set_met[s], met_set)) return false;
            float z = 0.f;
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              y[16 * ch + u] += red[(from * kMpad + m) * kHandStride + u];
              z = fmaxf(z, y[16 * ch + u]);
            }
            sm.xm2[s][l] = z;  // (a store of what was read: the loads are over when the next meeting is reached)
          }
          if (m < M) put(m, 64 * s + kD * c, y, my_sum);
        }
        if (m < M && s == 0 && c == 0) {
          if (whole) {
            put_lse(my_ref, my_sum);
          } else {
            part[128 * kDim + m] = my_ref;
            part[128 * kDim + 128 + m] = my_sum;
          }
        }
      }
      // O, the exchange and the NaN marks are free again
      tc_fence_before();
      if (!meet(&sm.sets_met, met_all)) return false;
      if (nans) {
        if (s == 0) sm.nanpos[k % kRows][l] = INT_MAX;
        if (tid == 0) sm.nanany[k % kRows] = 0;
      }
      mref = -INFINITY;
      lrun = 0.f;
      return true;
    };

    int pos_max = 0;      // position of the thread's row, and its scores' factor but for the page's
    float coef_q = 0.f;
    Ring<kBars> rb;
    for (int t = 0;; ++t, rb.step()) {
      if (!warp_wait(smem_u32(&sm.s_full[rb.at]), rb.phase, p.flags)) break;
      const int4 x = *reinterpret_cast<const int4*>(&sm.tile[t % kRing].page);
      const float4 y = *reinterpret_cast<const float4*>(&sm.tile[t % kRing].kscale);
      if (x.z & kEnd) break;
      if (x.z & kFirst) {
        pos_max = sm.seg[seg % kRing].pos + row;
        coef_q = p.sm_scale_log2 * (NP == 1 ? 1.f : sm.qscale[seg % kRows][l]);
      }
      if (kTurns && (t & 1) != s) {  // the other set's tile
        if (x.z & kLast && !finish(seg++)) break;
        continue;
      }
      tc_fence_after();
      const float lv = y.y, iv = y.z;
      const bool full_vis = !(x.z & kPart) && x.y == kBlock;  // every token visible to every row
      const int lim = pos_max - x.w - k0;                      // token k0 + n visible iff n <= lim
      // the floor keeps a masked score at -inf when a scale is 0
      const float coef = fmaxf(coef_q * y.x, 1e-30f);
      const uint32_t s_cols = tbase + lane_base + kColS + kBlock * (rb.at < 3u ? rb.at : rb.at - 3u);
      // The loop bodies are short and run several times on purpose: the roles' code together is what
      // an SM's instruction cache has to hold, and fetching it was the bound when they were unrolled.
      constexpr int kStep = kN < 32 ? kN : 32, kCh = kN / kStep;
      uint32_t v[kStep];
      auto load = [&](int ch) {
        if constexpr (kStep == 32) tmem_ld32(s_cols + k0 + 32 * ch, v);
        else tmem_ld16(s_cols + k0, v);
        tc_wait_ld();
      };
      float mx = -INFINITY;
      if (kCh > 1 && full_vis) {
#pragma unroll 1
        for (int ch = 0; ch < kCh; ++ch) {  // the TMEM load reduces (two at a time spill: BF16 prompt 385 us, not 370)
          float m0 = tmem_ld32_max(s_cols + k0 + 32 * ch);
          tc_wait_ld();
          asm volatile("" : "+f"(m0));  // no use moves above the wait
          mx = fmaxf(mx, m0);
        }
      } else {
#pragma unroll 1
        for (int ch = 0; ch < kCh; ++ch) {
          load(ch);
          if (!full_vis) {  // scores of tokens that the row does not see become -inf
#pragma unroll
            for (int u = 0; u < kStep; ++u) v[u] = kStep * ch + u <= lim ? v[u] : __float_as_uint(-INFINITY);
            if constexpr (kCh > 1) tmem_st32(s_cols + k0 + 32 * ch, v);  // in place: they are read again
          }
#pragma unroll
          for (int u = 0; u < kStep; u += 2) mx = fmax3(mx, __uint_as_float(v[u]), __uint_as_float(v[u + 1]));
        }
        if (kCh > 1) tc_wait_st();
      }
      float* hm = &sm.half_max[t & 1][0][0];
      float r_old = mref;
      if constexpr (kTurns) {  // the reference goes from tile to tile and so from set to set
        if (t > 0 && !warp_wait(smem_u32(&sm.row_told[quad]), (t - 1) & 1, p.flags)) break;
        r_old = x.z & kFirst ? -INFINITY : sm.half_max[(t - 1) & 1][0][l];
      } else {
        // the row's maximum over both sets; after the meeting nobody needs the scores that the weights of
        // the other set go over
        hm[128 * s + l] = mx;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.row_told[quad]));
        if (!warp_wait(smem_u32(&sm.row_told[quad]), t & 1, p.flags)) break;
        mx = fmaxf(mx, hm[128 * (s ^ 1) + l]);
      }
      // P is taken relative to a reference that moves only when the maximum passes it by more
      // than kTopLog2 (P stays within FP16); O / l does not depend on it
      const float bmax = fmaf(mx, coef, lv);
      const bool move = bmax > r_old + kTopLog2 || (r_old == -INFINITY && bmax != -INFINITY);
      const float m_new = move ? bmax - kStartLog2 : r_old;
      if constexpr (kTurns) {
        hm[l] = m_new;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.row_told[quad]));
      }
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const bool rescale = move && r_old != -INFINITY;
      // A tile whose weights are all 0 in FP16 may still count in the sum, where its values' scale is far
      // below the row's others: its keys are then summed relative to its own maximum, mxs. With one copy a
      // loop of its own does it, a score at a time: what matters there is how little code it is (E4M3
      // prompts took 2.5 % more with 32 at a time, 5 % with selects among the weights as below, 0.5 % so).
      const bool faint = bmax < m_new - kFaintLog2 && mx != -INFINITY;
      const bool some_faint = __any_sync(0xFFFFFFFFu, faint);
      const float mxs = mx * coef;
      float own = 0.f;
      if constexpr (kTurns) {
        if (some_faint) {
#pragma unroll 1
          for (int n = 0; n < kN; ++n) {
            uint32_t x;
            tmem_ld1(s_cols + n, x);
            tc_wait_ld();
            own += ex2(fmaf(__uint_as_float(x), coef, -mxs));
          }
        }
      }
      const float off = !kTurns && faint ? -mxs : lv - ref;
      const float2 coef2 = make_float2(coef, coef), off2 = make_float2(off, off);
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int ch = 0; ch < kCh; ++ch) {
        if (kCh > 1) load(ch);
#pragma unroll
        for (int u = 0; u < kStep / 2; ++u) {  // scores -> columns of FP16 pairs
          const float2 d = __ffma2_rn(make_float2(__uint_as_float(v[2 * u]), __uint_as_float(v[2 * u + 1])), coef2, off2);
          const float2 e = make_float2(ex2(d.x), ex2(d.y));
          acc = __fadd2_rn(acc, e);
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v[u]) : "f"(e.y), "f"(e.x));
        }
        if (!kTurns && some_faint)
#pragma unroll
          for (int u = 0; u < kStep / 2; ++u) v[u] = faint ? 0u : v[u];
        if constexpr (kTurns) tmem_st16(s_cols + 64 * (ch >> 1) + 16 * (ch & 1), v);
        else if constexpr (kStep == 32) tmem_st16(s_cols + p_off, v);
        else tmem_st8(s_cols + p_off, v);
      }
      // the weights of the tokens of other copies are 0: 16-column blocks (32 tokens each, block z at
      // column 64 (z / 2) + 16 (z % 2)), shared out between the sets
      if constexpr (C == 2) tmem_zero16(s_cols + 64 * (c ^ 1) + 16 * s);
      if constexpr (C == 4) {
#pragma unroll
        for (int i = 1 + s; i < 2 + 2 * s; ++i) tmem_zero16(s_cols + 64 * (((c + i) & 3) >> 1) + 16 * ((c + i) & 1));
      }
      if (__any_sync(0xFFFFFFFFu, rescale)) {
        // O holds the segment's earlier tiles once the P V before is done; this tile's waits for the
        // arrival below
        if (!warp_wait(smem_u32(&sm.pv_done[(t - 1) % kBars]), ((t - 1) / kBars) & 1, p.flags)) break;
        tc_fence_after();
        const float a = rescale ? ex2(r_old - ref) : 1.f;
#pragma unroll 1
        for (int d = kTurns ? 0 : 64 * s; d < (kTurns ? kDim : 64 * s + 64); d += 32)
          tmem_scale32(tbase + lane_base + kColO + d, a);
      }
      const float sum = kTurns && faint ? own : acc.x + acc.y;
      lrun = carry(lrun, mref, ref) + sum * (faint ? ex2(mxs - ref) : iv);  // mref -inf: nothing summed yet
      mref = m_new;
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[rb.at]));
      if (x.z & kLast && !finish(seg++)) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// Joins the partials of an item that starts in CTA blockIdx.x's range and ends in a later one's
// (log-sum-exp), partials in tile order. CTA blockIdx.y has dims 32 y .. 32 y + 31; a warp 8 rows and
// 16 dims, 4 dims of a row per lane. With at most 8 partials the 8 pairs of warps take 8 rows each; with
// more they share 8 rows, every eighth partial each, and the first joins their sums.
// Bound: latency (headers, then all of a run's loads at once) and the time to start 4 CTAs per SM:
// runs of 4 in 64 registers measured best (one token over 4,096 keys: 14.4 us, runs of 8 in 128
// registers 16.5; 64 ragged requests 164 and 167).
__global__ void __launch_bounds__(kMergeThreads, 2) kv8_merge_kernel(const Kv8AttnParams p, int grid) {
  constexpr int kPairs = kMergeThreads / 64;
  __shared__ float4 part_o[kPairs][64];
  __shared__ float part_l[kPairs][64], part_m[kPairs][64];
  pdl_wait_primary();
  const Header* hd = reinterpret_cast<const Header*>(p.parts);
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Header me = hd[cta];
  // partials: this CTA's, then those of the next ones up to the item's last
  auto middle = [&](int i) { return i < grid && hd[i].cont && !hd[i].cont_end; };
  unsigned ends = __ballot_sync(0xFFFFFFFFu, !middle(cta + 1 + lane));
  if (!me.tail) return;
  int n = 1 + (ends ? __ffs(ends) : 32);
  for (int base = cta + 33; ends == 0u && base < grid; base += 32) {
    ends = __ballot_sync(0xFFFFFFFFu, !middle(base + lane));
    n += ends ? __ffs(ends) : 32;
  }
  if (cta + n > grid) n = grid - cta;
  const float* parts = reinterpret_cast<const float*>(p.parts + headers_bytes(grid));
  auto part = [&](int i) { return parts + (i == 0 ? 2LL * cta + 1 : 2LL * (cta + i)) * kPartFloats; };
  const int rows = me.rows * p.q_per_kv;
  // (one token over 4,096 keys: 14.4 us shared, 18.5 not; 16 requests with 16 listed blocks: 32 and 25)
  const bool shared = n > kPairs;
  const int pair = warp >> 1, d = 32 * blockIdx.y + 16 * (warp & 1) + 4 * (lane >> 3);
  const int first = shared ? pair : 0, step = shared ? kPairs : 1;
  for (int m0 = shared ? 0 : 8 * pair; m0 < rows; m0 += shared ? 8 : 8 * kPairs) {
    const int m = m0 + (lane & 7);
    const bool on = m < rows;
    constexpr int kRun = 4;  // partials whose loads are in flight at once
    float ref = -INFINITY, lt = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float m, float m_to, const float4& x, float l) {
      const float h = ex2(0.5f * (m - m_to)), w = h * h;  // the sum in two steps: see carry()
      lt += l * h * h;
      if (w != 0.f) {
        o.x += w * x.x;
        o.y += w * x.y;
        o.z += w * x.z;
        o.w += w * x.w;
      }
    };
    auto lower = [&](float to) {  // everything so far relative to a larger reference
      const float l = lt;
      const float4 x = o;
      lt = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      add(ref == to ? 0.f : ref, ref == to ? 0.f : to, x, l);
      ref = to;
    };
    if (on)
#pragma unroll 1
      for (int e0 = first; e0 < n; e0 += kRun * step) {
        float4 x[kRun];
        float mm[kRun], ll[kRun], top = ref;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
          const int e = e0 + j * step;
          mm[j] = -INFINITY;
          if (e < n) {
            const float* q = part(e);
            x[j] = *reinterpret_cast<const float4*>(q + part_at(m, d));
            mm[j] = q[128 * kDim + m];
            ll[j] = q[128 * kDim + 128 + m];
          }
        }
#pragma unroll
        for (int j = 0; j < kRun; ++j) top = fmaxf(top, mm[j]);
        lower(top);
        const float base = top == -INFINITY ? 0.f : top;  // nothing seen (a NaN sum still counts)
#pragma unroll
        for (int j = 0; j < kRun; ++j)
          if (e0 + j * step < n) add(mm[j], base, x[j], ll[j]);
      }
    if (shared) {
      const int at = 32 * (warp & 1) + lane;
      part_o[pair][at] = o;
      part_l[pair][at] = lt;
      part_m[pair][at] = ref;
      __syncthreads();
      if (pair == 0) {
        float top = ref;
#pragma unroll
        for (int i = 1; i < kPairs; ++i) top = fmaxf(top, part_m[i][at]);
        lower(top);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 1; i < kPairs; ++i) add(part_m[i][at], base, part_o[i][at], part_l[i][at]);
      }
    }
    if (first == 0 && on) {
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      const long long orow = static_cast<long long>(me.row0 + m / p.q_per_kv) * (p.num_kv_heads * p.q_per_kv) +
                             me.head * p.q_per_kv + m % p.q_per_kv;
      *reinterpret_cast<uint2*>(p.out + orow * kDim + d) =
          make_uint2(bf16x2_bits(o.x * inv, o.y * inv), bf16x2_bits(o.z * inv, o.w * inv));
      if (d == 0 && p.lse != nullptr) p.lse[orow] = lt == 0.f ? -INFINITY : (ref + log2f(lt)) * 0.69314718055994531f;
    }
    if (shared) __syncthreads();
  }
}

template <int C, int NP>
cudaError_t launch(const CUtensorMap& kmap, const Kv8AttnParams& prm, int grid, cudaStream_t st) {
  const int smem = static_cast<int>(sizeof(Smem<NP>)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kv8_attn_kernel<C, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kv8_attn_kernel<C, NP><<<grid, kThreads, smem, st>>>(kmap, prm);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, kMergeY);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel, prm, grid);
}

// Copies of the query rows that a request of max_rows rows (taken as a power of two) leaves room
// for, and the rows of a chunk. At 8 query rows (one token, 8 queries a head) 16 requests over 16,384
// keys take 60.3 us with four copies, 61.6 with two, 63.4 with one, and one token over 4,096 keys 14.4,
// 14.4 and 16.3; at up to 64 rows 64 ragged requests 164 us with two and 168 with one.
int copies_for(int max_rows, int q_per_kv) {
  long long r = 1;
  while (r < max_rows && r < 128) r *= 2;
  const long long m = r * q_per_kv;
  return m <= 32 ? 4 : m <= 64 ? 2 : 1;
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

cudaError_t launch_kv8_attn(const CUtensorMap& kmap, const Kv8AttnParams& prm, bool q_bf16, int grid,
                            cudaStream_t st) {
  const int c = copies_for(prm.max_rows, prm.q_per_kv);
  if (q_bf16)
    return c == 4 ? launch<4, 2>(kmap, prm, grid, st)
           : c == 2 ? launch<2, 2>(kmap, prm, grid, st) : launch<1, 2>(kmap, prm, grid, st);
  return c == 4 ? launch<4, 1>(kmap, prm, grid, st)
         : c == 2 ? launch<2, 1>(kmap, prm, grid, st) : launch<1, 1>(kmap, prm, grid, st);
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_kv8_attn_workspace_size(const msa_kv8_attn_args* a, size_t* bytes) {
  if (bytes == nullptr) return MSA_ERR_INVALID_ARG;
  const msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  int sms = 0;
  const msa_status d = check_device(&sms);
  if (d != MSA_OK) return d;
  // flags, the CTAs' headers, two partials for each CTA
  *bytes = 256 + headers_bytes(sms) + 2 * static_cast<size_t>(sms) * kPartFloats * sizeof(float);
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
  p.parts = static_cast<uint8_t*>(ws) + 256;
  p.out = a->out;
  p.lse = a->lse;
  const int room = 128 / copies_for(p.max_rows, p.q_per_kv) / p.q_per_kv;
  p.chunk = 1;
  while (2 * p.chunk <= room) p.chunk *= 2, ++p.chunk_log2;
  CUtensorMap kmap;
  const long long token_rows = static_cast<long long>(a->num_pages) * a->num_kv_heads * kBlock;
  if ((s = encode_kv8_map(&kmap, a->k_data, token_rows)) != MSA_OK) return s;
  return launch_kv8_attn(kmap, p, a->q_type == MSA_TYPE_BF16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MSA_OK
             : MSA_ERR_CUDA;
}

}  // extern "C"
