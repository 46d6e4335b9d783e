// Attention of drafted rows over a paged cache of 8 bits (moe_tree_attention8): a block for each
// query row and head, a warp for every fourth key, sums in 32 bits throughout.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kTree = 64, kThreads = 128, kWarps = kThreads / 32;

template <int D>
__global__ void __launch_bounds__(kThreads) k_tree_attn8(const __grid_constant__ moe_tree_attention8_args a) {
  constexpr int E = D / 32;  // elements of a lane
  __shared__ float m_of[kWarps], l_of[kWarps], acc_of[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x, head = blockIdx.y, kv = head / (a.q_heads / a.kv_heads);
  const int b = last_not_above_warp(a.row_start, a.n_req, row);
  const int s = __ldg(a.row_start + b), e = __ldg(a.row_start + b + 1), ctx = __ldg(a.ctx_len + b), i = row - s;
  unsigned flags = 0;
  if (s < 0 || i < 0 || row >= e || e > a.n_rows) return;
  const bool ok = e - s <= a.max_tree && ctx >= 0 &&
                  (long long)ctx + e - s <= min((long long)a.table_width * a.cache.page_size, 0x7fffffffll - 256);
  if (!ok) flags |= MOE_DEV_LENGTH;
  const uint64_t tree = a.tree_mask ? __ldg(a.tree_mask + row) : i >= 63 ? ~0ull : (2ull << i) - 1;
  const bool bf = a.dtype == MOE_BF16, i8 = a.cache.format == MOE_I8;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + row * a.q_stride + head * D;
  const auto wide = [&](uint32_t w) { return bf ? unpack2<MOE_BF16>(w).x : unpack2<MOE_F16>(w).x; };
  const auto code = [&](const void* base, long long at) {
    const int c = static_cast<const int8_t*>(base)[at];
    return i8 ? (float)c : __uint_as_float(((uint32_t)c & 0x80000000u) | ((uint32_t)(c & 0x7f) << 20)) * 1.329227995784916e36f;
  };
  float m = -INFINITY, l = 0.f, acc[E] = {}, x[E];
  for (int j = 0; j < E; ++j) x[j] = wide(q[lane + 32 * j]);
  for (int pos = warp; ok && pos < ctx + e - s; pos += kWarps) {
    if (pos >= ctx && !(tree >> (pos - ctx) & 1)) continue;
    const int col = pos / a.cache.page_size, slot = pos - col * a.cache.page_size;
    const int page = __ldg(a.block_table + (long long)b * a.table_width + col);
    if (page < 0 || page >= a.cache.n_pages) {
      flags |= MOE_DEV_INDEX;
      continue;
    }
    const long long at = page * a.cache.page_stride + slot * a.cache.slot_stride + kv * a.cache.head_stride;
    const long long sc = page * a.cache.scale_page_stride + slot / a.cache.block_size * a.cache.scale_block_stride +
                         kv * a.cache.scale_head_stride;
    const float ks = scale_of(a.cache.k_scale[sc], flags), vs = scale_of(a.cache.v_scale[sc], flags);
    float dot = 0.f;
    for (int j = 0; j < E; ++j) dot = fmaf(x[j], code(a.cache.k, at + lane + 32 * j), dot);
    for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float t = dot * ks * a.scale, top = fmaxf(m, t), f = m == -INFINITY ? 0.f : expf(m - top), w = expf(t - top);
    m = top;
    l = fmaf(l, f, w);
    for (int j = 0; j < E; ++j) acc[j] = fmaf(acc[j], f, w * (code(a.cache.v, at + lane + 32 * j) * vs));
  }
  if (lane == 0) {
    m_of[warp] = m;
    l_of[warp] = l;
  }
  for (int j = 0; j < E; ++j) acc_of[warp][lane + 32 * j] = acc[j];
  __syncthreads();
  m = -INFINITY;
  l = 0.f;
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, m_of[w]);
  for (int w = 0; w < kWarps; ++w) l += m_of[w] == -INFINITY ? 0.f : l_of[w] * expf(m_of[w] - m);
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w) sum += m_of[w] == -INFINITY ? 0.f : acc_of[w][c] * expf(m_of[w] - m);
    sum = l == 0.f ? 0.f : sum / l;
    const uint32_t h = bf ? pack2<MOE_BF16>(sum, 0.f) : pack2<MOE_F16>(sum, 0.f);
    static_cast<uint16_t*>(a.out)[row * a.out_stride + head * D + c] = (uint16_t)h;
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(long long)row * a.q_heads + head] = l == 0.f ? -INFINITY : m + logf(l);
  if (flags) atomicOr(a.dev_status, flags);
}

int check(const moe_tree_attention8_args* p) {
  if (!p) return MOE_EINVAL;
  const moe_tree_attention8_args& a = *p;
  if (a.n_req < 1 || a.n_rows < 0 || a.max_tree < 1 || a.table_width < 1 || a.q_heads < 1 || a.kv_heads < 1 ||
      a.head_dim < 1 || a.q_heads % a.kv_heads || !std::isfinite(a.scale))
    return MOE_EINVAL;
  if (a.dtype != MOE_BF16 && a.dtype != MOE_F16) return a.dtype == MOE_F32 ? MOE_EUNSUPPORTED : MOE_EINVAL;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return MOE_EUNSUPPORTED;
  if (a.max_tree > kTree || a.q_heads / a.kv_heads > 64 || a.q_heads > 1024 || a.n_req > 16384 || a.n_rows > (1 << 20))
    return MOE_EUNSUPPORTED;
  const int rc = check_cache(a.cache, a.kv_heads);
  if (rc != MOE_OK) return rc;
  if (!stride_ok(a.q_stride) || !stride_ok(a.out_stride)) return MOE_EINVAL;
  if (!rows_ok(a.n_rows, a.q_stride) || !rows_ok(a.n_rows, a.out_stride)) return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.ctx_len, 4) || !ptr_ok(a.block_table, 4) ||
      !opt_ok(a.lse, 4) || !opt_ok(a.tree_mask, 8))
    return MOE_EINVAL;
  if (a.n_rows > 0 && (!ptr_ok(a.q, 16) || !ptr_ok(a.out, 16))) return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_tree_attention8_workspace_bytes(const moe_tree_attention8_args* args) {
  return check(args) == MOE_OK ? kCounterBytes : 0;
}

extern "C" int moe_tree_attention8(const moe_tree_attention8_args* args, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  if (!ptr_ok(ws, 16)) return MOE_EINVAL;
  if (ws_bytes < kCounterBytes) return MOE_EWORKSPACE;
  if (args->n_rows == 0) return MOE_OK;
  const auto fn = args->head_dim == 64 ? k_tree_attn8<64> : args->head_dim == 128 ? k_tree_attn8<128> : k_tree_attn8<256>;
  fn<<<dim3(args->n_rows, args->q_heads), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(*args);
  return launch_status(cudaGetLastError());
}
