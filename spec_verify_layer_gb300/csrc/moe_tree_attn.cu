// moe_tree_attention: the attention of drafted rows over a paged cache of 16-bit elements.
#include "moe_tree_attn.cuh"

using namespace moe;

extern "C" size_t moe_tree_attention_workspace_bytes(const moe_tree_attention_args* args) {
  return check(args) == MOE_OK ? layout(*args).total : 0;
}

extern "C" int moe_set_attention_wait_limit_ns(uint64_t ns) {
  g_attention_wait_ns.store(ns ? ns : kWaitNs, std::memory_order_relaxed);
  return MOE_OK;
}

extern "C" int moe_tree_attention(const moe_tree_attention_args* args, void* ws, size_t ws_bytes, void* stream) {
  Plan p{};
  int sms = 0;
  const int rc = prepare(args, ws, ws_bytes, p, sms);
  if (rc != MOE_OK || args->n_rows == 0) return rc;
  using A = moe_tree_attention_args;
  const A& a = *args;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = a.dtype == MOE_BF16;
  switch (a.head_dim) {
    case 64: return bf ? launch<A, MOE_BF16, 64>(a, p, sms, st) : launch<A, MOE_F16, 64>(a, p, sms, st);
    case 128: return bf ? launch<A, MOE_BF16, 128>(a, p, sms, st) : launch<A, MOE_F16, 128>(a, p, sms, st);
    default: return bf ? launch<A, MOE_BF16, 256>(a, p, sms, st) : launch<A, MOE_F16, 256>(a, p, sms, st);
  }
}
