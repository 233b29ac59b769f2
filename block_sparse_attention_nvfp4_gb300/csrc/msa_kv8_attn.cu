// msa_kv8_attn: attention over the 8-bit cache, of all blocks or of listed ones. The kernel: msa_kv8_attn.cuh.
#include "msa_kv8_attn.cuh"

using namespace msa;

extern "C" {

msa_status msa_kv8_attn_workspace_size(const msa_kv8_attn_args* a, size_t* bytes) {
  if (bytes == nullptr) return MSA_ERR_INVALID_ARG;
  const msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  int sms = 0;
  const msa_status d = check_device(&sms);
  if (d != MSA_OK) return d;
  *bytes = base_workspace(sms);
  return MSA_OK;
}

msa_status msa_kv8_attn(const msa_kv8_attn_args* a, void* ws, size_t ws_bytes, void* stream) {
  msa_status s = check_args(a);
  if (s != MSA_OK) return s;
  Kv8AttnParams p;
  CUtensorMap kmap;
  int sms = 0, copies = 0;
  if ((s = set_params(a, ws, ws_bytes, 0, a->max_rows_per_req, &p, &kmap, &sms, &copies)) != MSA_OK) return s;
  if (a->num_reqs == 0 || a->total_rows == 0) return MSA_OK;
  const cudaError_t e = launch_form<kAll>(kmap, p, copies, a->q_type == MSA_TYPE_BF16, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
