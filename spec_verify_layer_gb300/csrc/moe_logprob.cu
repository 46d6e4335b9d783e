// Log probabilities of given tokens, entropies, ranks and top alternatives
// (moe_token_logprobs), one launch and one pass over the logits.
//
// A block takes a slice of one row, a chunk at a time: a thread holds four 16-byte vectors
// of the chunk in registers and updates its own running maximum m (of the logits), sum
// s = sum 2^u and w = sum 2^u u with u = (x - m) / T * log2(e); no thread waits for another
// until the slice ends.  Entropy is ln s - ln 2 * w / s, log probabilities (x - m) / T - ln s.
//
// Top entries: 64-bit keys (logit order, ~id) make the order total.  A chunk's entries that
// may be among the first k are those at or above the k-th largest of 32 group maxima (each
// of 16 threads), and above the k-th so far; they are few (about 30 of 16384 for k = 20),
// go to shared memory, and each finds its place by counting the larger ones.
//
// With few rows a row is cut into 2^i slices, up to 32; the block that ends last joins the
// slices' partials in their order, so the result does not depend on which one that is.
#include "moe_common.cuh"
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kLpVecs = 4;      // 16-byte vectors a thread holds of a chunk
constexpr int kLpMaxK = 32, kLpMaxSlices = 32;
constexpr int kLpCand = 1024;   // entries at or above the threshold that are kept
using Key = unsigned long long;

struct LpPartial {  // a slice's result in the workspace
  float m, s, w;
  int rank;
  Key top[kLpMaxK];
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ Key key_of(float x, int id) { return ((Key)order_key(x) << 32) | (uint32_t)~id; }
__device__ __forceinline__ float key_logit(Key k) { return key_value((unsigned)(k >> 32)); }
__device__ __forceinline__ int key_id(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ Key max_key(Key a, Key b) { return a > b ? a : b; }

// 32 keys of a warp in descending order over the lanes
__device__ __forceinline__ Key sort_desc(Key v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const Key x = __shfl_xor_sync(0xffffffffu, v, o);
      const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
      v = keep_max ? (v > x ? v : x) : (v < x ? v : x);
    }
  return v;
}

template <int DT>
struct Vec {
  static constexpr int N = DT == MOE_F32 ? 4 : 8;
  static constexpr uint32_t kNone = DT == MOE_F32 ? 0xff800000u : DT == MOE_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  uint4 raw;
  __device__ __forceinline__ float at(int e) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (DT == MOE_F32) {
      return __uint_as_float(w[e]);
    } else {
      const float2 p = unpack2<DT>(w[e >> 1]);
      return (e & 1) ? p.y : p.x;
    }
  }
};

template <int DT>
__device__ __forceinline__ float logit_at(const void* base, long long i) {
  if constexpr (DT == MOE_F32) {
    return static_cast<const float*>(base)[i];
  } else {
    const uint32_t w = static_cast<const uint16_t*>(base)[i];
    return unpack2<DT>(w).x;
  }
}

// A vector whose first element is entry `first` of the row; entries outside [0, vocab) -infinity.
template <int DT>
__device__ __forceinline__ Vec<DT> load_vec(const void* row, int first, int vocab) {
  Vec<DT> v;
  constexpr int N = Vec<DT>::N, size = 16 / N;
  if (first >= 0 && first + N <= vocab) {
    v.raw = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(row) + (long long)first * size));
    return v;
  }
  uint32_t w[4] = {Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone};
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int i = first + e;
    if (i < 0 || i >= vocab) continue;
    if constexpr (DT == MOE_F32) {
      w[e] = static_cast<const uint32_t*>(row)[i];
    } else {
      const uint32_t x = static_cast<const uint16_t*>(row)[i];
      w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (x << 16) : (w[e >> 1] & 0xffff0000u) | x;
    }
  }
  v.raw = make_uint4(w[0], w[1], w[2], w[3]);
  return v;
}

struct LpShared {
  Key list[2][kLpMaxK];
  Key group[kLpWarps * 2];
  Key cand[kLpCand + kLpMaxK];
  Key best[kLpWarps];
  float m[kLpWarps], s[kLpWarps], w[kLpWarps];
  int rank[kLpWarps];
  int count;
  int last;
};

// sm.cand[0 .. n) -> the first k of them in order, in `out` (0 where there are fewer).
__device__ __forceinline__ void place(LpShared& sm, int n, int k, Key* out) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const Key mine = sm.cand[i];
    int before = 0;
    for (int j = 0; j < n; ++j) before += sm.cand[j] > mine;
    if (before < k) out[before] = mine;
  }
  if ((int)threadIdx.x < k && (int)threadIdx.x >= n) out[threadIdx.x] = 0;
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads, 2) k_token_logprobs(const __grid_constant__ moe_logprob_args a, int slices,
                                                                  int slice_vecs, unsigned* counters,
                                                                  LpPartial* partials) {
  constexpr int N = Vec<DT>::N;
  __shared__ LpShared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.top_k;
  const int row = blockIdx.x / slices, slice = blockIdx.x - row * slices;
  const char* base = static_cast<const char*>(a.logits) + (long long)row * a.stride * (16 / N);
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15) / (16 / N));
  const int vecs = (a.vocab + lead + N - 1) / N;
  const int v0 = slice * slice_vecs, v1 = min(v0 + slice_vecs, vecs);

  const int token = a.tokens ? a.tokens[row] : -1;
  const bool has_token = token >= 0 && token < a.vocab;
  const float xt = has_token ? logit_at<DT>(base, token) : INFINITY;
  const float above = nextafterf(xt, INFINITY);  // entries behind the token have to exceed it
  const float c2 = a.inv_temperature * 1.4426950408889634f;
  float m = -INFINITY, s = 0.f, w = 0.f;
  int rank = 0, cur = 0;
  if (tid < kLpMaxK) sm.list[0][tid] = 0;
  __syncthreads();

  for (int c = v0; c < v1; c += kLpThreads * kLpVecs) {
    Vec<DT> x[kLpVecs];
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      const int v = c + j * kLpThreads + tid;
      if (v < v1) x[j] = load_vec<DT>(base, v * N - lead, a.vocab);
      else x[j].raw = make_uint4(Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone);
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) top = fmaxf(top, x[j].at(e));
    if (top > m) {
      if (m > -INFINITY) {
        const float d = (m - top) * c2, f = exp2_fast(d);
        w = f * fmaf(d, s, w);
        s *= f;
      }
      m = top;
    }
    const float shift = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      const int v = c + j * kLpThreads + tid, first = v * N - lead;
      const bool full = v < v1 && first >= 0 && first + N <= a.vocab;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float u = (x[j].at(e) - shift) * c2, p = exp2_fast(u);
        s += p;
        w = fmaf(p, fmaxf(u, -300.f), w);  // 0 * -infinity is 0 here; p carries a NaN
      }
      if (full && (token < first || token >= first + N)) {
        const float thr = token < first ? above : xt;
#pragma unroll
        for (int e = 0; e < N; ++e) rank += x[j].at(e) >= thr;
      } else if (v < v1) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int i = first + e;
          if (i >= 0 && i < a.vocab) rank += x[j].at(e) > xt || (x[j].at(e) == xt && i < token);
        }
      }
    }
    if (k == 0) continue;

    const Key floor_key = sm.list[cur][k - 1];
    Key mine = 0;
    if (top > -INFINITY && order_key(top) >= (unsigned)(floor_key >> 32)) {
      int id = 0;
#pragma unroll
      for (int j = kLpVecs - 1; j >= 0; --j)
#pragma unroll
        for (int e = N - 1; e >= 0; --e)
          if (x[j].at(e) == top) id = (c + j * kLpThreads + tid) * N - lead + e;
      mine = key_of(top, id);
      if (mine <= floor_key) mine = 0;
    }
    if (!__syncthreads_or(mine != 0)) continue;
    Key g = mine;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) g = max_key(g, __shfl_xor_sync(0xffffffffu, g, o));
    if ((lane & 15) == 0) sm.group[2 * warp + (lane >> 4)] = g;
    if (tid == 0) sm.count = 0;
    __syncthreads();
    const Key sorted = sort_desc(sm.group[lane], lane);
    const Key thr = max_key(__shfl_sync(0xffffffffu, sorted, k - 1), floor_key + 1);
    if (mine >= thr) {
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float f = x[j].at(e);
          if (f > -INFINITY) {
            const Key key = key_of(f, (c + j * kLpThreads + tid) * N - lead + e);
            if (key >= thr) {
              const int at = atomicAdd(&sm.count, 1);
              if (at < kLpCand) sm.cand[at] = key;
            }
          }
        }
    }
    __syncthreads();
    int n = sm.count;
    if (n > kLpCand) {
      // many equal or ordered logits: the k largest one after the other
      __syncthreads();
      Key prev = ~0ull;
      for (int r = 0; r < k; ++r) {
        Key b = 0;
#pragma unroll
        for (int j = 0; j < kLpVecs; ++j)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float f = x[j].at(e);
            if (f > -INFINITY) {
              const Key key = key_of(f, (c + j * kLpThreads + tid) * N - lead + e);
              if (key < prev) b = max_key(b, key);
            }
          }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) b = max_key(b, __shfl_xor_sync(0xffffffffu, b, o));
        if (lane == 0) sm.best[warp] = b;
        __syncthreads();
        prev = sm.best[0];
        for (int q = 1; q < kLpWarps; ++q) prev = max_key(prev, sm.best[q]);
        if (tid == 0) sm.cand[r] = prev;
        __syncthreads();
      }
      n = k;
    }
    // the list so far joins the candidates: its entries are other ids than the chunk's
    if (tid < k) sm.cand[n + tid] = sm.list[cur][tid];
    __syncthreads();
    int total = n;
    for (int j = 0; j < k; ++j) total += sm.cand[n + j] != 0;
    place(sm, total, k, sm.list[cur ^ 1]);
    cur ^= 1;
    __syncthreads();
  }

  // the block's sums, in a fixed order
  {
    float top = m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sm.m[warp] = top;
    __syncthreads();
    top = sm.m[0];
    for (int q = 1; q < kLpWarps; ++q) top = fmaxf(top, sm.m[q]);
    const float d = m == -INFINITY ? 0.f : (m - top) * c2, f = exp2_fast(d);
    w = f * fmaf(d, s, w);
    s *= f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    if (lane == 0) {
      sm.s[warp] = s;
      sm.w[warp] = w;
      sm.rank[warp] = rank;
    }
    __syncthreads();
    m = top;
    s = w = 0.f;
    rank = 0;
    for (int q = 0; q < kLpWarps; ++q) {
      s += sm.s[q];
      w += sm.w[q];
      rank += sm.rank[q];
    }
  }

  if (slices > 1) {
    LpPartial* mine = partials + (size_t)row * slices + slice;
    if (tid == 0) {
      mine->m = m;
      mine->s = s;
      mine->w = w;
      mine->rank = rank;
    }
    if (tid < k) mine->top[tid] = sm.list[cur][tid];
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const bool last = atomicAdd(counters + row, 1u) == (unsigned)slices - 1;
      if (last) counters[row] = 0;  // ready for the next call
      sm.last = last;
      sm.count = 0;
    }
    __syncthreads();
    if (!sm.last) return;
    __threadfence();
    const LpPartial* all = partials + (size_t)row * slices;
    // every warp joins the sums alike: lane = slice
    float pm = -INFINITY, ps = 0.f, pw = 0.f;
    int pr = 0;
    if (lane < slices) {
      pm = __ldcg(&all[lane].m);
      ps = __ldcg(&all[lane].s);
      pw = __ldcg(&all[lane].w);
      pr = __ldcg(&all[lane].rank);
    }
    m = pm;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float d = pm == -INFINITY ? 0.f : (pm - m) * c2, f = exp2_fast(d);
    w = f * fmaf(d, ps, pw);
    s = f * ps;
    rank = pr;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    if (k > 0) {
      // the lists are in order: the first 32 / slices of each are group maxima
      const int each = 32 / slices;
      Key head = lane / each < slices && lane % each < k ? __ldcg(&all[lane / each].top[lane % each]) : 0;
      head = sort_desc(head, lane);
      const Key thr = max_key(__shfl_sync(0xffffffffu, head, k - 1), 1);
      for (int i = tid; i < slices * k; i += kLpThreads) {
        const Key key = __ldcg(&all[i / k].top[i % k]);
        if (key >= thr) sm.cand[atomicAdd(&sm.count, 1)] = key;  // at most 32 * 32
      }
      __syncthreads();
      place(sm, sm.count, k, sm.list[0]);
      cur = 0;
      __syncthreads();
    }
  }

  const bool empty = m == -INFINITY && s == 0.f;
  const float log_s = empty ? 0.f : logf(s);
  if (tid == 0) {
    if (a.logp) {
      float v = -INFINITY;
      if (has_token && !empty) v = (xt - m) * a.inv_temperature - log_s;
      a.logp[row] = v;
    }
    if (a.entropy) a.entropy[row] = empty ? 0.f : log_s - 0.6931471805599453f * (w / s);
    if (a.rank) a.rank[row] = has_token ? rank : -1;
    if (a.tokens && !has_token && token != -1) atomicOr(a.dev_status, MOE_DEV_INDEX);
  }
  if (tid < k) {
    const Key key = sm.list[cur][tid];
    a.top_ids[(long long)row * k + tid] = key ? key_id(key) : -1;
    a.top_logp[(long long)row * k + tid] = key ? (key_logit(key) - m) * a.inv_temperature - log_s : -INFINITY;
  }
}

int check(const moe_logprob_args* p) {
  if (!p) return MOE_EINVAL;
  const moe_logprob_args& a = *p;
  if (a.n_rows < 0 || a.vocab < 1 || a.top_k < 0 || a.stride < 0) return MOE_EINVAL;
  if (!(a.inv_temperature > 0.f) || !std::isfinite(a.inv_temperature)) return MOE_EINVAL;
  if (a.dtype != MOE_BF16 && a.dtype != MOE_F16 && a.dtype != MOE_F32) return MOE_EINVAL;
  if (a.vocab > (1 << 24) || a.top_k > kLpMaxK || a.n_rows > (1 << 24) || a.stride >= ((int64_t)1 << 40))
    return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4)) return MOE_EINVAL;
  if (a.n_rows == 0) return MOE_OK;
  if (!ptr_ok(a.logits, a.dtype == MOE_F32 ? 4 : 2)) return MOE_EINVAL;
  if (!opt_ok(a.tokens, 4) || !opt_ok(a.logp, 4) || !opt_ok(a.entropy, 4) || !opt_ok(a.rank, 4)) return MOE_EINVAL;
  if (!a.tokens && (a.logp || a.rank)) return MOE_EINVAL;
  if (a.top_k > 0 ? !ptr_ok(a.top_ids, 4) || !ptr_ok(a.top_logp, 4) : false) return MOE_EINVAL;
  return MOE_OK;
}

// Slices of a row: while there are SMs to spare (two blocks each) and every thread of a
// slice still has a vector.
int slices_of(const moe_logprob_args& a) {
  constexpr int kBlocks = 304;
  const int per = a.dtype == MOE_F32 ? 4 : 8;
  int s = 1;
  while (s < kLpMaxSlices && (int64_t)a.n_rows * s * 2 <= kBlocks && a.vocab / per / (2 * s) >= kLpThreads) s *= 2;
  return s;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_token_logprobs_workspace_bytes(const moe_logprob_args* args) {
  if (check(args) != MOE_OK) return 0;
  const int s = slices_of(*args);
  if (s == 1) return 256;
  return up256((size_t)args->n_rows * 4) + (size_t)args->n_rows * s * sizeof(LpPartial);
}

extern "C" int moe_token_logprobs(const moe_logprob_args* args, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  if (!ptr_ok(ws, 16)) return MOE_EINVAL;
  if (ws_bytes < moe_token_logprobs_workspace_bytes(args)) return MOE_EWORKSPACE;
  const moe_logprob_args& a = *args;
  if (a.n_rows == 0) return MOE_OK;
  const int s = slices_of(a), per = a.dtype == MOE_F32 ? 4 : 8;
  const int vecs = (a.vocab + 2 * per - 2) / per;  // wherever a row starts
  const int slice_vecs = (vecs + s - 1) / s;
  unsigned* counters = static_cast<unsigned*>(ws);
  LpPartial* partials = reinterpret_cast<LpPartial*>(static_cast<char*>(ws) + up256((size_t)a.n_rows * 4));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)a.n_rows * s;
  if (a.dtype == MOE_F32) k_token_logprobs<MOE_F32><<<grid, kLpThreads, 0, st>>>(a, s, slice_vecs, counters, partials);
  else if (a.dtype == MOE_BF16) k_token_logprobs<MOE_BF16><<<grid, kLpThreads, 0, st>>>(a, s, slice_vecs, counters, partials);
  else k_token_logprobs<MOE_F16><<<grid, kLpThreads, 0, st>>>(a, s, slice_vecs, counters, partials);
  return launch_status(cudaGetLastError());
}
