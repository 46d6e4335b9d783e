// moe_tree_attention8: the attention of drafted rows over a paged cache of 8 bits, codes with a
// scale for each block of tokens and head.
#include "moe_cache8_attn.cuh"

using namespace moe;

extern "C" size_t moe_tree_attention8_workspace_bytes(const moe_tree_attention8_args* args) {
  return check(args) == MOE_OK ? layout(*args).total : 0;
}

extern "C" int moe_tree_attention8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream) {
  if (args && args->cache.format == MOE_I8) return attention8_i8(args, ws, ws_bytes, stream);
  return attention8<MOE_E4M3>(args, ws, ws_bytes, stream);
}
