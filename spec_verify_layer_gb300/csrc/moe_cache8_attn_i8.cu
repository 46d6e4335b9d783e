// moe_tree_attention8 over int8 codes.
#include "moe_cache8_attn.cuh"

int moe::attention8_i8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream) {
  return attention8<MOE_I8>(args, ws, ws_bytes, stream);
}
