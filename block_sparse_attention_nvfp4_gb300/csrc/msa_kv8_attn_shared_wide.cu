// The attention kernel of msa_kv8_attn_shared for one to three queries a KV head, where the row chunks of a request that
// shares nothing have up to 128 rows, as in the plain call, and those of a group 32: a form of its own because its
// NaN marks and chunk sizes, a few more instructions in the roles' loops, took 2 % of the time of 4 prompts of 16 requests
// with 8 queries a head (115.0 us, 117.5 with them).
#include "msa_kv8_attn.cuh"

namespace msa {

cudaError_t launch_kv8_attn_shared_wide(const CUtensorMap& kmap, const Kv8AttnParams& prm, int copies, bool q_bf16, int grid,
                                        cudaStream_t st) {
  // (four copies leave room for 32 rows at most)
  if (q_bf16) return copies == 2 ? launch<2, 2, kSharedWide>(kmap, prm, grid, st) : launch<1, 2, kSharedWide>(kmap, prm, grid, st);
  return copies == 2 ? launch<2, 1, kSharedWide>(kmap, prm, grid, st) : launch<1, 1, kSharedWide>(kmap, prm, grid, st);
}

}  // namespace msa
