// moe_tree_attention8: the attention of drafted rows over a paged cache of 8 bits, codes with a
// scale for each block of tokens and head.
#include "moe_tree_attn.cuh"

using namespace moe;

namespace {

constexpr int kFewRows = 32;

template <int FMT>
int choose(const moe_tree_attention8_args& a, const Plan& p, int sms, cudaStream_t st) {
  using A = moe_tree_attention8_args;
  // Few query rows a head: products of codes in registers, in groups of up to 32 query rows (heads of 256: 16).
  const int rows = a.max_tree * p.group, nt = rows > kFewRows ? 0 : rows <= 8 ? 1 : rows <= 16 || a.head_dim == 256 ? 2 : 4;
  if (nt) {
    const auto few = [&](auto d, auto n) { return launch<A, FMT, decltype(d)::value, false, decltype(n)::value>(a, p, sms, st); };
    using I = std::integral_constant<int, 64>;
    using J = std::integral_constant<int, 128>;
    using K = std::integral_constant<int, 256>;
    std::integral_constant<int, 1> one;
    std::integral_constant<int, 2> two;
    std::integral_constant<int, 4> four;
    if (a.head_dim == 64) return nt == 1 ? few(I{}, one) : nt == 2 ? few(I{}, two) : few(I{}, four);
    if (a.head_dim == 128) return nt == 1 ? few(J{}, one) : nt == 2 ? few(J{}, two) : few(J{}, four);
    return nt == 1 ? few(K{}, one) : few(K{}, two);
  }
  // Blocks of 16 tokens and more have one scale for each run of 16 keys of a tile; smaller ones are taken key by key.
  const bool coarse = a.cache.block_size >= 16;
  switch (a.head_dim) {
    case 64: return coarse ? launch<A, FMT, 64, true>(a, p, sms, st) : launch<A, FMT, 64, false>(a, p, sms, st);
    case 128: return coarse ? launch<A, FMT, 128, true>(a, p, sms, st) : launch<A, FMT, 128, false>(a, p, sms, st);
    default: return coarse ? launch<A, FMT, 256, true>(a, p, sms, st) : launch<A, FMT, 256, false>(a, p, sms, st);
  }
}

}  // namespace

extern "C" size_t moe_tree_attention8_workspace_bytes(const moe_tree_attention8_args* args) {
  return check(args) == MOE_OK ? layout(*args).total : 0;
}

extern "C" int moe_tree_attention8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream) {
  Plan p{};
  int sms = 0;
  const int rc = prepare(args, ws, ws_bytes, p, sms);
  if (rc != MOE_OK || args->n_rows == 0) return rc;
  const moe_tree_attention8_args& a = *args;
  p.flip = 0;
  p.c = 1.f;
  p.score = a.scale * 1.4426950408889634f;
  while ((1 << p.block_shift) < a.cache.block_size) ++p.block_shift;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.cache.format == MOE_E4M3 ? choose<MOE_E4M3>(a, p, sms, st) : choose<MOE_I8>(a, p, sms, st);
}
