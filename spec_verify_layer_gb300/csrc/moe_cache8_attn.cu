// moe_tree_attention8: the attention of drafted rows over a paged cache of 8 bits, codes with a
// scale for each block of tokens and head.
#include "moe_tree_attn.cuh"

using namespace moe;

extern "C" size_t moe_tree_attention8_workspace_bytes(const moe_tree_attention8_args* args) {
  return check(args) == MOE_OK ? layout(*args).total : 0;
}

extern "C" int moe_tree_attention8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream) {
  Plan p{};
  int sms = 0;
  const int rc = prepare(args, ws, ws_bytes, p, sms);
  if (rc != MOE_OK || args->n_rows == 0) return rc;
  using A = moe_tree_attention8_args;
  const A& a = *args;
  p.flip = 0;  // the sign of the scale goes with the rows' factors
  p.c = 1.f;
  p.score = a.scale * 1.4426950408889634f * (a.cache.format == MOE_E4M3 ? 256.f : 1.f);
  while ((1 << p.block_shift) < a.cache.block_size) ++p.block_shift;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // products are of fp16 numbers whatever the type of q and out
  switch (a.head_dim) {
    case 64: return launch<A, MOE_F16, 64>(a, p, sms, st);
    case 128: return launch<A, MOE_F16, 128>(a, p, sms, st);
    default: return launch<A, MOE_F16, 256>(a, p, sms, st);
  }
}
