// moe_tree_attention8: the attention of drafted rows over a paged cache of 8 bits, codes with a
// scale for each block of tokens and head.
#include "moe_tree_attn.cuh"

using namespace moe;

namespace {

using Encode = decltype(&cuTensorMapEncodeTiled);

// The driver's function, without a link to its library; NULL if there is none.
Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  return fn;
}

// Codes as [page][head][slot][D] bytes, or [page][slot][head][D] where a head's stride is the smaller one;
// false where the strides make no tensor map.
bool encode(CUtensorMap* map, void* base, const moe_tree_attention8_args& a, int box, bool head_first) {
  const moe_kv_cache8& c = a.cache;
  const cuuint64_t slots = (cuuint64_t)c.page_size, heads = (cuuint64_t)a.kv_heads;
  const cuuint64_t slot_stride = (cuuint64_t)c.slot_stride, head_stride = (cuuint64_t)c.head_stride;
  const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, head_first ? heads : slots, head_first ? slots : heads, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {head_first ? head_stride : slot_stride, head_first ? slot_stride : head_stride, (cuuint64_t)c.page_stride};
  const cuuint32_t rows[4] = {(cuuint32_t)a.head_dim, head_first ? 1u : (cuuint32_t)box, head_first ? (cuuint32_t)box : 1u, 1u};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  const Encode fn = encoder();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, rows, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of 16 tokens and more have one scale for each run of 16 keys of a tile, smaller ones are taken key
// by key.  Pages that are a multiple of 8 rows come in boxes, as far as their strides make a tensor map.
template <int FMT>
int choose(const moe_tree_attention8_args& a, Plan p, int sms, cudaStream_t st) {
  using A = moe_tree_attention8_args;
  Maps maps = {};
  const bool coarse = a.cache.block_size >= 16;
  if (a.cache.page_size % 8 == 0) {
    p.box = 8;
    while (2 * p.box <= (a.head_dim == 256 ? 64 : 128) && a.cache.page_size % (2 * p.box) == 0) p.box *= 2;
    p.head_first = a.cache.head_stride < a.cache.slot_stride;
    if (!encode(&maps.k, a.cache.k, a, p.box, p.head_first) || !encode(&maps.v, a.cache.v, a, p.box, p.head_first)) p.box = 0;
  }
  // Few query rows a head: products of codes in registers.  (64 requests of one row and 8 heads a key, up to
  // 8,192 keys: FEW_A us against FEW_B.)
  const int rows = a.max_tree * p.group, nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 && a.head_dim < 256 ? 4 : 0;
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
  switch (a.head_dim) {
    case 64: return coarse ? launch<A, FMT, 64, true>(a, p, sms, st, maps) : launch<A, FMT, 64, false>(a, p, sms, st, maps);
    case 128: return coarse ? launch<A, FMT, 128, true>(a, p, sms, st, maps) : launch<A, FMT, 128, false>(a, p, sms, st, maps);
    default: return coarse ? launch<A, FMT, 256, true>(a, p, sms, st, maps) : launch<A, FMT, 256, false>(a, p, sms, st, maps);
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
