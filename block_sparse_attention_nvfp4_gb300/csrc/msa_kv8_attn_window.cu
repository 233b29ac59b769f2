// msa_kv8_attn_window: attention over the 8-bit cache to a window of the last tokens and to the first ones (sinks).
// A row at position p sees t <= p with t > p - window or t < sinks. The kernel is msa_kv8_attn.cuh's: a chunk's tiles
// are the sinks' pages and those from its first row's window to its last row, so the pages between are neither looked
// up nor read, and the line of tiles that the CTAs share counts what is left. A chunk has at most `window` rows, so
// that a token which its last row has left is never one that its first row does not see yet: what a NaN value
// reaches is then a prefix or a suffix of the rows.
// Floor: the codes of the tokens seen, or their products. Measured (4 KV heads of 8 queries; floor): one token at 32,768 with a
// window of 4,096, 16.4 us (0.6); 64 ragged requests of up to 8 rows, 65 (33); 2,053 rows on 16,421 keys, 148 (72).
// Bound: one token, latency, as over 4,096 keys without a window; 64 requests, the start and end of 2 or 3 parts a CTA (memory 49 %
// busy); prompts, the roles' instruction streams (the tensor pipe 43 %): a set of warps takes 2,150 cycles for a tile, 3,500 for one of the two
// or three of an item's 34 that are masked, and 6,800 at an item's end. (Masked tiles taken 32 tokens at a time, all, none or some
// seen, have less to do but more code: 159 us.)
#include "msa_kv8_attn.cuh"

using namespace msa;

extern "C" {

msa_status msa_kv8_attn_window(const msa_kv8_attn_args* a, int32_t window, int32_t sinks, void* ws, size_t ws_bytes,
                               void* stream) {
  msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  if (window < 1 || sinks < 0 || a->n_block_ids != 0) return MSA_ERR_INVALID_ARG;
  Kv8AttnParams p;
  CUtensorMap kmap;
  int sms = 0, copies = 0;
  if ((s = set_params(a, ws, ws_bytes, 0, a->max_rows_per_req, &p, &kmap, &sms, &copies)) != MSA_OK) return s;
  if (a->num_reqs == 0 || a->total_rows == 0) return MSA_OK;
  const int most = a->max_pages_per_req * kBlock;  // (no request is longer)
  p.window = window < most ? window : most;
  p.sinks = sinks < most ? sinks : most;
  p.sink_pages = (p.sinks + kBlock - 1) / kBlock;
  while (p.chunk > p.window) p.chunk /= 2, --p.chunk_log2;
  const cudaError_t e =
      launch_form<kWindow>(kmap, p, copies, a->q_type == MSA_TYPE_BF16, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
