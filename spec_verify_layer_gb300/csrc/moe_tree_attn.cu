// Attention of drafted rows over a paged cache (moe_tree_attention).
//
// First form: a block per (row, query head); its warps take every eighth position, hold
// the row's query in registers, and keep a running maximum and sum of the softmax each;
// the warps are joined through shared memory at the end.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kAttnThreads = 256, kAttnWarps = 8;
constexpr int kTree = 64;

template <int DT, int D>
__global__ void __launch_bounds__(kAttnThreads) k_tree_attn(const __grid_constant__ moe_tree_attention_args a) {
  constexpr int E = D / 32;
  __shared__ float sm_m[kAttnWarps], sm_l[kAttnWarps], sm_o[kAttnWarps][D];
  const int row = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.row_start[0] != 0 && tid == 0 && row == 0 && head == 0) atomicOr(a.dev_status, MOE_DEV_LENGTH);
  // the request of the row: the last that starts at or before it
  int lo = 0, hi = a.n_req;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.row_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  const int b = lo, s = a.row_start[b], e = a.row_start[b + 1];
  if (row < s || row >= e) return;
  const int i = row - s, n = e - s, ctx = a.ctx_len[b];
  const int P = a.cache.page_size;
  unsigned flags = 0;
  bool ok = s >= 0 && e <= a.n_rows && n <= a.max_tree && ctx >= 0 &&
            (long long)ctx + n <= (long long)a.table_width * P;
  if (!ok) flags |= MOE_DEV_LENGTH;
  const int kvh = head / (a.q_heads / a.kv_heads);
  const uint64_t seen = a.tree_mask ? a.tree_mask[row] : (i >= 63 ? ~0ull : (2ull << i) - 1);
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (long long)row * a.q_stride + (long long)head * D;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    const float2 v = unpack2<DT>(reinterpret_cast<const uint32_t*>(q)[lane * (E / 2) + j]);
    qv[2 * j] = v.x;
    qv[2 * j + 1] = v.y;
    o[2 * j] = o[2 * j + 1] = 0.f;
  }
  const int total = ok ? ctx + n : 0;
  for (int p = warp; p < total; p += kAttnWarps) {
    if (p >= ctx && !((seen >> (p - ctx)) & 1)) continue;
    const int page = a.block_table[(long long)b * a.table_width + p / P];
    if (page < 0 || page >= a.cache.n_pages) {
      flags |= MOE_DEV_INDEX;
      continue;
    }
    const long long at = page * a.cache.page_stride + (p % P) * a.cache.slot_stride + kvh * a.cache.head_stride;
    const uint32_t* k = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.cache.k) + at) + lane * (E / 2);
    const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.cache.v) + at) + lane * (E / 2);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 x = unpack2<DT>(k[j]);
      dot = fmaf(qv[2 * j], x.x, fmaf(qv[2 * j + 1], x.y, dot));
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
    dot *= a.scale;
    const float top = fmaxf(m, dot), c = expf(m - top), w = expf(dot - top);
    m = top;
    l = l * c + w;
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 x = unpack2<DT>(v[j]);
      o[2 * j] = fmaf(w, x.x, o[2 * j] * c);
      o[2 * j + 1] = fmaf(w, x.y, o[2 * j + 1] * c);
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) sm_o[warp][lane * E + j] = o[j];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sm_m[w]);
  const float shift = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int w = 0; w < kAttnWarps; ++w) sum += sm_l[w] * expf(sm_m[w] - shift);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int d = 2 * tid; d < D; d += 2 * kAttnThreads) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < kAttnWarps; ++w) {
      const float c = expf(sm_m[w] - shift);
      x = fmaf(c, sm_o[w][d], x);
      y = fmaf(c, sm_o[w][d + 1], y);
    }
    uint16_t* out = static_cast<uint16_t*>(a.out) + (long long)row * a.out_stride + (long long)head * D;
    *reinterpret_cast<uint32_t*>(out + d) = pack2<DT>(x * inv, y * inv);
  }
  if (tid == 0 && a.lse) a.lse[(long long)row * a.q_heads + head] = top + logf(sum);
  if (flags) atomicOr(a.dev_status, flags);
}

template <int DT>
cudaError_t launch(const moe_tree_attention_args& a, cudaStream_t st) {
  const dim3 grid(a.n_rows, a.q_heads);
  switch (a.head_dim) {
    case 64: k_tree_attn<DT, 64><<<grid, kAttnThreads, 0, st>>>(a); break;
    case 128: k_tree_attn<DT, 128><<<grid, kAttnThreads, 0, st>>>(a); break;
    default: k_tree_attn<DT, 256><<<grid, kAttnThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

int check(const moe_tree_attention_args* p) {
  if (!p) return MOE_EINVAL;
  const moe_tree_attention_args& a = *p;
  if (a.n_req < 1 || a.n_rows < 0 || a.max_tree < 1 || a.table_width < 1 || a.q_heads < 1 || a.kv_heads < 1 ||
      a.head_dim < 1 || a.q_heads % a.kv_heads || !std::isfinite(a.scale))
    return MOE_EINVAL;
  if (a.dtype != MOE_BF16 && a.dtype != MOE_F16) return a.dtype == MOE_F32 ? MOE_EUNSUPPORTED : MOE_EINVAL;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return MOE_EUNSUPPORTED;
  if (a.max_tree > kTree || a.q_heads / a.kv_heads > 64 || a.q_heads > 1024 || a.n_req > 16384 ||
      a.n_rows > (1 << 20))
    return MOE_EUNSUPPORTED;
  const int rc = check_cache(a.cache);
  if (rc != MOE_OK) return rc;
  if (!stride_ok(a.q_stride) || !stride_ok(a.out_stride)) return MOE_EINVAL;
  if (!ptr_ok(a.dev_status, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.ctx_len, 4) || !ptr_ok(a.block_table, 4) ||
      !opt_ok(a.lse, 4) || !opt_ok(a.tree_mask, 8))
    return MOE_EINVAL;
  if (a.n_rows > 0 && (!ptr_ok(a.q, 16) || !ptr_ok(a.out, 16))) return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_tree_attention_workspace_bytes(const moe_tree_attention_args* args) {
  return check(args) == MOE_OK ? 256 : 0;
}

extern "C" int moe_tree_attention(const moe_tree_attention_args* args, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  if (!ptr_ok(ws, 16)) return MOE_EINVAL;
  if (ws_bytes < moe_tree_attention_workspace_bytes(args)) return MOE_EWORKSPACE;
  if (args->n_rows == 0) return MOE_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(args->dtype == MOE_BF16 ? launch<MOE_BF16>(*args, st) : launch<MOE_F16>(*args, st));
}
