// Which drafted tokens stand and which token follows (moe_verify_drafts), three launches, each of
// which starts while the one before it ends.
//
// k_sums: one pass over the logits of the rows that drafts hang on (greedy: of all rows); a block
// takes a slice of a row, a thread running maximum m and sum s = sum 2^((x - m) c), c = log2(e) / T
// (greedy: the largest logit's key).  Rows without drafts behind them need no sums and are
// left out.
//
// k_walk: a block a request joins its rows' sums and walks down its drafts, a few dozen numbers, in 64
// bits.  (Done by each of the last launch's blocks for itself: 70 us of the 90 that 64 chains took.)
//
// k_draw: a request's blocks each scan a slice of the row where the walk ended for the largest
// rest(x) / noise(x): an exponential race, so the draw needs one pass, no prefix sums, and no
// order between slices.  The request's block that ends last joins the slices, by (ratio, lower id), so
// it does not matter which one that is.
//
// Five rows of 32,003 in fp32 (one request) 16.4 us: latency of three launches in a chain, each of which
// waits for the one before.  64 chains of up to 8 rows of 131,072 in bf16, with draft probabilities (101
// MB), 45.5 us: by themselves sums 18, walk 10, draws 24, the draws bound by what an entry costs (logit,
// noise and draft probability each unpacked, compared in products).  24 trees of 8 to 48 rows of 129,283
// in fp32, 80.8 us: sums 47 (224 MB, 4.7 TB/s), walk 14, draws 18.  The draws wait for the walk before they read
// anything, the noise too; where rows of noise and of logits begin apart (an odd vocabulary) its elements are loaded
// one by one: the 64 chains over 131,071 entries 50 us.
// Greedy, which reads every row and draws nothing: the five rows 8.7 us, 64 such chains 20.3 (68 MB, 3.4 TB/s),
// in fp32 30.9 (4.4 TB/s), the 24 trees 69.2 (342 MB, 4.95 TB/s, 73 % of measured).
//
// The exponent (x - m) c is taken with c in two parts (c >= hi, lo > 0, so that -infinity stays
// what it is): with c rounded to 32 bits probabilities far from the maximum would be off by
// some 1e-6, and a decision lies that near its border far more often than by the 1e-7 of the
// rounded sums.
#include <algorithm>

#include "moe_vocab.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTree = 64;
constexpr int kVecs = 4;         // vectors a thread has on their way
constexpr int kMaxSlices = 32;
// Rows (of sums, most blocks of which have none to take) are cut into slices up to about so many blocks, requests
// (of draws) while the blocks stay within the 608 that run at once (64 chains, 512 blocks, 52.7 us with the 456
// of three blocks an SM and 45.5 with 608; 24 trees 84 with 768 blocks and 80.6 with 384); slices have so
// many entries at least.
// Long slices (in bytes) of rows are cut once more, since the last of them to begin end alone: 24 trees of
// fp32 rows 88.4 us without, 84.0 so; 64 chains of bf16 rows, whose slices would be 16 KB then, 52.5 and 55.9.
// Looked-up chains of 8, us as it is / never / always cut once more, in fp32: 96 rows of 262,144 49 / 49 / 48, 640 of
// 131,072 94 / 90 / 94, 400 of 262,144 113 / 126 / 112, 760 of 200,000 160 / 183 / 160; in bf16: 200 of 262,144
// 49 / 49 / 51, 400 of 262,144 73 / 74 / 73, 512 of 131,072 56 / 56 / 59.
constexpr int kSumBlocks = 1500, kDrawBlocks = 304, kSliceMin = 2048, kLongSlice = 48 << 10;
constexpr int kCounters = (int)(kCounterBytes / sizeof(unsigned));

// Ratios and ids of candidates as keys: the larger ratio, of equal ones the lower id; 0: none.
struct Drawn {  // a slice's: of the rest, and of p for where nothing of the rest is left
  Key best, best_p;
  float m;  // that the ratios are taken from
  int bad;
};
__device__ __forceinline__ Key ratio_key(float ratio, int id) { return ratio > 0.f ? (Key)__float_as_uint(ratio) << 32 | (uint32_t)~id : 0; }
__device__ __forceinline__ Key warp_max(Key k) {
  const unsigned hi = (unsigned)(k >> 32), top = __reduce_max_sync(0xffffffffu, hi);
  return (Key)top << 32 | __reduce_max_sync(0xffffffffu, hi == top ? (unsigned)k : 0u);
}
__device__ __forceinline__ float warp_max(float x) { return key_value(__reduce_max_sync(0xffffffffu, order_key(x))); }

struct End {  // of a request's walk, in the workspace
  double S;
  float m;
  int last, child, n_out, inner;  // last < 0: nothing to draw
  int out[kTree];                 // tokens that were rejected behind the last row
};

struct Plan {
  int row_slices, row_vecs;    // slices of a row in k_sums, vectors of a slice
  int draw_slices, draw_vecs;  // of the row that is drawn from
  float hi, lo;                // c
  double inv_t;
  float2* sums;    // [rows][row_slices]: m, s
  Key* keys;       // greedy: [rows][row_slices]
  Drawn* drawn;    // [requests][draw_slices]
  End* end;        // [requests]
  unsigned* left;  // [requests]
};

__device__ __forceinline__ float2 exponent(float2 x, float m, const Plan& p) {
  const Pair d = add2(pair(x), pair(-m, -m));
  return split(fma2(d, pair(p.hi, p.hi), mul2(d, pair(p.lo, p.lo))));
}
__device__ __forceinline__ float factor(float from, float to, const Plan& p) {  // of sums that go from one maximum to a larger
  const float d = from - to;
  return exp2_fast(fmaf(d, p.hi, d * p.lo));
}
__device__ __forceinline__ float element(const void* base, int dt, long long i) {
  return dt == MOE_F32 ? logit_at<MOE_F32>(base, i) : dt == MOE_BF16 ? logit_at<MOE_BF16>(base, i) : logit_at<MOE_F16>(base, i);
}

template <int DT>
struct Row {  // a row of logits in vectors
  static constexpr int N = Vec<DT>::N;
  const char* base;
  int lead, vecs;
  __device__ __forceinline__ Row(const moe_verify_args& a, int row) {
    base = static_cast<const char*>(a.logits) + (long long)row * a.stride * (16 / N);
    lead = (int)((reinterpret_cast<uintptr_t>(base) & 15) / (16 / N));
    vecs = (a.vocab + lead + N - 1) / N;
  }
};

template <int DT, bool GREEDY>
__global__ void __launch_bounds__(kThreads) k_sums(const __grid_constant__ moe_verify_args a, const __grid_constant__ Plan p) {
  constexpr int N = Vec<DT>::N;
  __shared__ float m_of[kWarps], s_of[kWarps];
  __shared__ Key k_of[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.row_slices, slice = blockIdx.x - row * p.row_slices;
  asm volatile("griddepcontrol.launch_dependents;");  // k_walk's blocks may take their places; they wait for this launch's end
  {
    // every warp finds the row's request and looks for its children
    const int b = last_not_above_warp(a.row_start, a.n_req, row);
    const int s = __ldg(a.row_start + b), e = __ldg(a.row_start + b + 1), n = e - s, i = row - s;
    if (s < 0 || i < 0 || row >= e || e > a.n_rows || n > kTree) return;  // k_draw says so
    if (!GREEDY) {
      bool child = false;
      for (int j = i + 1 + lane; j < n; j += 32) child |= a.parents ? __ldg(a.parents + s + j) == i : j == i + 1;
      if (!__any_sync(0xffffffffu, child)) return;
    }
  }
  const Row<DT> r(a, row);
  const int v0 = slice * p.row_vecs, v1 = min(v0 + p.row_vecs, r.vecs);
  float m = -INFINITY, s = 0.f;
  int id = 0;
  bool bad = false;
  for (int v = v0 + tid; v < v1; v += kThreads * kVecs) {
    Vec<DT> x[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      x[j].raw = make_uint4(Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone);
      if (v + j * kThreads < v1) x[j] = load_vec<DT>(r.base, (v + j * kThreads) * N - r.lead, a.vocab);
    }
    if constexpr (GREEDY) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float f = x[j].at(e);
          bad |= !(f < INFINITY);
          if (f > m) {
            m = f;
            id = (v + j * kThreads) * N - r.lead + e;
          }
        }
    } else {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) top = fmaxf(top, x[j].at(e));
      if (top > m) {
        if (m > -INFINITY) s *= factor(m, top, p);
        m = top;
      }
      const float shift = m == -INFINITY ? 0.f : m;
      Pair sum = 0;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 u = exponent(make_float2(x[j].at(e), x[j].at(e + 1)), shift, p);
          sum = add2(sum, pair(exp2_fast(u.x), exp2_fast(u.y)));
        }
      const float2 both = split(sum);
      s += both.x + both.y;
    }
  }
  if constexpr (GREEDY) {
    Key key = bad ? ~0ull : m == -INFINITY ? 0 : key_of(m, id);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) key = max_key(key, __shfl_xor_sync(0xffffffffu, key, o));
    if (lane == 0) k_of[warp] = key;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w) key = max_key(key, k_of[w]);
      p.keys[blockIdx.x] = key;
    }
  } else {
    const auto join = [&](float om, float os) {
      const float to = fmaxf(m, om);
      if (m < to) s = m == -INFINITY ? s : s * factor(m, to, p);  // (nothing so far: 0, or NaN that has to stay)
      if (om < to) os = om == -INFINITY ? os : os * factor(om, to, p);
      s += os;
      m = to;
    };
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
      join(om, os);
    }
    if (lane == 0) {
      m_of[warp] = m;
      s_of[warp] = s;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w) join(m_of[w], s_of[w]);
      p.sums[blockIdx.x] = make_float2(m, s);
    }
  }
}

struct Walk {  // of one request, in shared memory
  double prob[kTree], S[kTree], border[kTree];
  float m[kTree], u[kTree];
  int parent[kTree], token[kTree], best[kTree], inner[kTree], order[kTree];
};

// N consecutive entries of a row from `first` on, in 32 bits; `other` outside [0, n).
template <int N>
__device__ __forceinline__ void entries(const void* row, int dt, int first, int n, float other, float* x) {
  const int size = dt == MOE_F32 ? 4 : 2;
  const char* at = static_cast<const char*>(row) + (long long)first * size;
  if (first >= 0 && first + N <= n && (reinterpret_cast<uintptr_t>(at) & (N * size >= 16 ? 15 : 7)) == 0) {
    if (dt == MOE_F32) {
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(at) + j);
        x[4 * j] = v.x;
        x[4 * j + 1] = v.y;
        x[4 * j + 2] = v.z;
        x[4 * j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(at) + j);
        const float2 lo = dt == MOE_BF16 ? unpack2<MOE_BF16>(w.x) : unpack2<MOE_F16>(w.x);
        const float2 hi = dt == MOE_BF16 ? unpack2<MOE_BF16>(w.y) : unpack2<MOE_F16>(w.y);
        x[4 * j] = lo.x;
        x[4 * j + 1] = lo.y;
        x[4 * j + 2] = hi.x;
        x[4 * j + 3] = hi.y;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) x[j] = first + j >= 0 && first + j < n ? element(row, dt, first + j) : other;
}

// A block a request: joins its rows' sums, a warp a row, and goes down its drafts.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_walk(const __grid_constant__ moe_verify_args a, const __grid_constant__ Plan p) {
  __shared__ Walk w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const bool greedy = isinf(a.inv_temperature);
  const int s = __ldg(a.row_start + b), e = __ldg(a.row_start + b + 1);
  unsigned flags = 0;
  if (b == 0 && tid == 0 && s != 0) flags |= MOE_DEV_LENGTH;
  const bool ok = s >= 0 && e >= s && e <= a.n_rows && e - s <= kTree;
  const int n = ok ? e - s : 0;
  if (n == 0) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the workspace may be in use)
    if (tid == 0) {
      if (!ok) flags |= MOE_DEV_LENGTH;
      a.accepted[b] = 0;
      a.next_token[b] = -1;
      if (!greedy) p.end[b].last = -1;
      if (flags) atomicOr(a.dev_status, flags);
    }
    return;
  }
  // what does not wait for the sums
  if (tid < n) {
    const int i = tid;
    int up = i - 1, token = i ? __ldg(a.tokens + s + i) : -1;
    if (a.parents && i) {
      up = __ldg(a.parents + s + i);
      if (up < -1 || up >= i) {
        flags |= MOE_DEV_INDEX;
        up = -1;
      }
    }
    if (token < -1 || token >= a.vocab) {
      flags |= MOE_DEV_INDEX;
      token = -1;
    }
    w.parent[i] = up;
    w.token[i] = token;
    w.u[i] = greedy || !i ? 0.f : __ldg(a.uniform + s + i);
    w.inner[i] = 0;
  }
  __syncthreads();
  if (tid < n && w.parent[tid] >= 0) w.inner[w.parent[tid]] = 1;
  float x = 0.f, q = 0.f;
  bool tried = false, again = false;
  if (tid < n) {
    const int up = w.parent[tid], token = w.token[tid];
    tried = up >= 0 && token >= 0;
    if (tried && !greedy) {
      x = logit_at<DT>(static_cast<const char*>(a.logits), (long long)(s + up) * a.stride + token);
      if (a.draft_probs) q = element(a.draft_probs, a.draft_dtype, (long long)(s + tid) * a.draft_stride + token);
      else
        for (int j = 0; j < tid; ++j) again |= w.parent[j] == up && w.token[j] == token;
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");  // k_draw's blocks may take their places; they wait for this launch's end
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = warp; i < n; i += kWarps) {
    if (greedy) {
      Key top = lane < p.row_slices ? p.keys[(long long)(s + i) * p.row_slices + lane] : 0;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = max_key(top, __shfl_xor_sync(0xffffffffu, top, o));
      // (requests that overlap, of which one may have no sums, must not bring tokens that are none)
      if (lane == 0) w.best[i] = top == ~0ull ? -2 : top == 0 || (unsigned)key_id(top) >= (unsigned)a.vocab ? -1 : key_id(top);
    } else if (w.inner[i]) {
      const float2 part = lane < p.row_slices ? p.sums[(long long)(s + i) * p.row_slices + lane] : make_float2(-INFINITY, 0.f);
      float m = part.x;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double S = part.x == -INFINITY ? (double)part.y : (double)part.y * factor(part.x, m, p);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
      if (lane == 0) {
        w.m[i] = m;
        w.S[i] = S;
      }
    }
  }
  __syncthreads();
  if (tid < n) {
    double prob = 0., border = 1.;
    if (tried) {
      const int up = w.parent[tid];
      if (greedy) {
        prob = w.best[up] == w.token[tid] ? 1. : 0.;
        border = 0.;
      } else {
        if (w.S[up] != 0. && !again) prob = exp(((double)x - (double)w.m[up]) * p.inv_t) / w.S[up];
        border = (double)w.u[tid] * (double)q;
      }
    }
    w.prob[tid] = prob;
    w.border[tid] = border;
  }
  __syncthreads();
  if (warp == 0) {
    // the walk itself, by all lanes alike: the children of `last` one after the other
    const int up0 = lane < n ? w.parent[lane] : -1, up1 = lane + 32 < n ? w.parent[lane + 32] : -1;
    const auto children = [&](int i) {
      return (unsigned long long)__ballot_sync(0xffffffffu, up0 == i) | (unsigned long long)__ballot_sync(0xffffffffu, up1 == i) << 32;
    };
    int last = 0, stands = 0;
    double rest = 1.;
    const bool chain = greedy || a.draft_probs;
    for (unsigned long long left = children(0); left;) {
      const int i = __ffsll((long long)left) - 1;
      left &= left - 1;
      const double prob = w.prob[i], border = chain ? w.border[i] : (double)w.u[i] * rest;
      if (prob > 0. && border < prob) {
        last = i;
        rest = 1.;
        ++stands;
        if (lane == 0) w.order[stands] = i;
        left = children(i);
      } else {
        rest -= prob;
      }
    }
    if (lane == 0) w.order[0] = 0;
    __syncwarp();
    for (int i = lane; i < n; i += 32) a.path[s + i] = i <= stands ? w.order[i] : -1;
    if (lane == 0) a.accepted[b] = stands;
    if (greedy) {
      if (lane == 0) {
        a.next_token[b] = max(w.best[last], -1);
        if (w.best[last] == -2) flags |= MOE_DEV_VALUE;
      }
    } else {
      End& end = p.end[b];
      const bool inner = w.inner[last] != 0, none = inner && !(w.S[last] > 0.);  // nothing to draw from
      // its children with tokens, all of them rejected
      const bool r0 = up0 == last && lane < n && w.token[lane] >= 0, r1 = up1 == last && lane + 32 < n && w.token[lane + 32] >= 0;
      const unsigned m0 = __ballot_sync(0xffffffffu, r0), m1 = __ballot_sync(0xffffffffu, r1), before = (1u << lane) - 1;
      if (r0) end.out[__popc(m0 & before)] = w.token[lane];
      if (r1) end.out[__popc(m0) + __popc(m1 & before)] = w.token[lane + 32];
      if (lane == 0) {
        end.last = none ? -1 : last;
        end.inner = inner;
        end.S = inner ? w.S[last] : 0.;
        end.m = inner ? w.m[last] : 0.f;
        end.child = m1 ? 63 - __clz(m1) : m0 ? 31 - __clz(m0) : -1;
        end.n_out = __popc(m0) + __popc(m1);
        if (none) {
          a.next_token[b] = -1;
          if (w.S[last] != 0.) flags |= MOE_DEV_VALUE;
        }
      }
    }
  }
  if (flags) atomicOr(a.dev_status, flags);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) k_draw(const __grid_constant__ moe_verify_args a, const __grid_constant__ Plan p) {
  constexpr int N = Vec<DT>::N;
  __shared__ Drawn all[kWarps];
  __shared__ int out[kTree], ends;
  __shared__ unsigned bound[2];  // what the block's warps have reached, of the rest and of p (a known maximum)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.draw_slices, slice = blockIdx.x - b * p.draw_slices;
  const int s = __ldg(a.row_start + b);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const End* const end = p.end + b;
  const int last = __ldcg(&end->last), child = __ldcg(&end->child), rejected = __ldcg(&end->n_out);
  const bool inner = __ldcg(&end->inner) != 0;
  const double S = __ldcg(&end->S);
  const float m = __ldcg(&end->m);
  if (last < 0) return;
  if (tid < 2) bound[tid] = 0;
  if (tid < rejected) out[tid] = __ldcg(&end->out[tid]);
  __syncthreads();

  const Row<DT> r(a, s + last);
  const float* noise = a.noise + b * a.noise_stride;
  const int n_out = a.draft_probs ? 0 : rejected;
  const char* q = a.draft_probs && child >= 0
                      ? static_cast<const char*>(a.draft_probs) + (long long)(s + child) * a.draft_stride * (a.draft_dtype == MOE_F32 ? 4 : 2)
                      : nullptr;
  const bool residual = q || n_out > 0;
  const float inv_S = inner ? (float)(1. / S) : 1.f;
  struct { float m, best, best_p; int id, id_p, bad; } d = {inner ? m : -INFINITY, 0.f, 0.f, 0, 0, 0};
  const int v0 = slice * p.draw_vecs, v1 = min(v0 + p.draw_vecs, r.vecs);
  // Ratios are compared as products with the best so far; only where one of a warp's lanes has a larger
  // one, which is some ln(entries) times, they are divided and looked at one by one.  (With a best
  // of each lane's own that was nearly every time: 41 us for 64 chains.)
  constexpr int VECS = N == 8 ? 1 : 2;
  float least = 0.f, least_p = 0.f;
#pragma unroll 1
  for (int vw = v0 + warp * 32; vw < v1; vw += VECS * kThreads) {
    const int v = vw + lane;
    Vec<DT> x[VECS];
    float race[VECS][N], from[VECS][N];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int at = v + j * kThreads, first = at < v1 ? at * N - r.lead : a.vocab;
      x[j] = load_vec<DT>(r.base, first, a.vocab);
      entries<N>(noise, MOE_F32, first, a.vocab, 0.f, race[j]);
      if (q) entries<N>(q, a.draft_dtype, first, a.vocab, 0.f, from[j]);
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VECS; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float f = x[j].at(i);
        d.bad |= !(f < INFINITY);
        top = fmaxf(top, f);
      }
    if (!inner) {  // the maximum is not known: the warp's so far
      top = warp_max(top);
      if (top > d.m) {
        if (d.m > -INFINITY) {
          const float f = factor(d.m, top, p);
          d.best_p *= f;
          least_p *= f;
        }
        d.m = top;
      }
    }
    if (inner) {
      least = fmaxf(least, __uint_as_float(*(volatile unsigned*)&bound[0]));
      least_p = fmaxf(least_p, __uint_as_float(*(volatile unsigned*)&bound[1]));
    }
    const float shift = d.m == -INFINITY ? 0.f : d.m;
    float mass[VECS][N];
    bool larger = false;
#pragma unroll
    for (int j = 0; j < VECS; ++j)
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 u = exponent(make_float2(x[j].at(i), x[j].at(i + 1)), shift, p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float y = exp2_fast(h ? u.y : u.x) * inv_S;
          mass[j][i + h] = y;
          larger |= y > least_p * race[j][i + h];
          if (residual) larger |= (q ? y - fmaxf(from[j][i + h], 0.f) : y) > least * race[j][i + h];
        }
      }
    if (!__any_sync(0xffffffffu, larger)) continue;
    // A bound that the largest of these reach, from reciprocals that may be off by 2^-22; then those above it.
    float most = 0.f, most_p = 0.f;
    int most_id = -1;
#pragma unroll
    for (int j = 0; j < VECS; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float noisy = race[j][i], y = mass[j][i];
        float inv;
        asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(noisy));
        inv = noisy > 0.f ? fminf(inv, 3e38f) : 0.f;  // (of the smallest numbers it is infinite)
        most_p = fmaxf(most_p, y * inv);
        const float left = (q ? y - fmaxf(from[j][i], 0.f) : y) * inv;
        if (left > most) {
          most = left;
          most_id = (v + j * kThreads) * N - r.lead + i;
        }
      }
    for (int k = 0; k < n_out; ++k)
      if (out[k] == most_id) most = 0.f;
    least_p = fmaxf(least_p, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most_p))) * 0.99999f);
    least = fmaxf(least, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most))) * 0.99999f);
    if (inner && lane == 0) {
      atomicMax(&bound[0], __float_as_uint(least));
      atomicMax(&bound[1], __float_as_uint(least_p));
    }
#pragma unroll
    for (int j = 0; j < VECS; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = (v + j * kThreads) * N - r.lead + i;
        const float noisy = race[j][i], y = mass[j][i], rest = q ? y - fmaxf(from[j][i], 0.f) : y;
        if (y > least_p * noisy && noisy > 0.f) {
          const float ratio = y / noisy;
          if (ratio > d.best_p) {
            d.best_p = ratio;
            d.id_p = id;
          }
        }
        if (residual && rest > least * noisy && noisy > 0.f && rest > 0.f) {
          const float ratio = rest / noisy;
          bool gone = !(ratio > d.best);
          for (int k = 0; k < n_out; ++k) gone |= out[k] == id;
          if (!gone) {
            d.best = ratio;
            d.id = id;
          }
        }
      }
  }
  // The block's, taken from its largest maximum.  (A NaN is in `bad` already.)
  const auto scaled = [&](float from, float to) { return from < to && from > -INFINITY ? factor(from, to, p) : 1.f; };
  const float warp_top = warp_max(d.m);
  const Key best = warp_max(ratio_key(d.best, d.id)), best_p = warp_max(ratio_key(d.best_p * scaled(d.m, warp_top), d.id_p));
  const int bad = __any_sync(0xffffffffu, d.bad);
  if (lane == 0) all[warp] = {best, best_p, warp_top, bad};
  __syncthreads();
  if (warp != 0) return;
  const auto joined = [&](const Drawn& x) {  // over the warp's lanes
    const float top = warp_max(x.m);
    return Drawn{warp_max(x.best), warp_max(ratio_key(__uint_as_float((unsigned)(x.best_p >> 32)) * scaled(x.m, top), key_id(x.best_p))),
                 top, __any_sync(0xffffffffu, x.bad)};
  };
  const Drawn none{0, 0, -INFINITY, 0};
  Drawn own = joined(lane < kWarps ? all[lane] : none);
  if (p.draw_slices > 1) {
    if (lane == 0) {
      p.drawn[blockIdx.x] = own;
      unsigned before;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.left + b) : "memory");
      ends = before == (unsigned)p.draw_slices - 1;
    }
    __syncwarp();
    if (!ends) return;
    Drawn part = none;
    if (lane < p.draw_slices) {
      const Drawn* o = p.drawn + (long long)b * p.draw_slices + lane;
      part = Drawn{__ldcg(&o->best), __ldcg(&o->best_p), __ldcg(&o->m), __ldcg(&o->bad)};
    }
    own = joined(part);
    if (lane == 0) p.left[b] = 0;  // ready for the next call
  }
  if (lane == 0) {
    a.next_token[b] = own.bad ? -1 : own.best ? key_id(own.best) : own.best_p ? key_id(own.best_p) : -1;
    if (own.bad) atomicOr(a.dev_status, MOE_DEV_VALUE);
  }
}

// The descriptor without what a greedy call does not read, which may be anything.
moe_verify_args read_by(const moe_verify_args& args) {
  moe_verify_args a = args;
  if (std::isinf(a.inv_temperature)) {
    a.draft_probs = nullptr;
    a.uniform = a.noise = nullptr;
  }
  return a;
}

int check(const moe_verify_args* args) {
  if (!args) return MOE_EINVAL;
  const moe_verify_args a = read_by(*args);
  if (a.n_req < 1 || a.n_rows < 0 || a.vocab < 1 || !(a.inv_temperature > 0.f)) return MOE_EINVAL;
  const auto type_ok = [](int t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_F32; };
  if (!type_ok(a.dtype) || (a.draft_probs && !type_ok(a.draft_dtype))) return MOE_EINVAL;
  const auto count_ok = [](int64_t s) { return s >= 0 && s < ((int64_t)1 << 40); };
  if (!count_ok(a.stride) || (a.draft_probs && !count_ok(a.draft_stride)) || (a.noise && !count_ok(a.noise_stride))) return MOE_EINVAL;
  if (a.n_req > 16384 || a.n_rows > (1 << 20) || a.vocab > (1 << 24)) return MOE_EUNSUPPORTED;
  if (a.draft_probs && a.parents) return MOE_EUNSUPPORTED;
  if (!rows_ok(a.n_rows, a.stride) || (a.draft_probs && !rows_ok(a.n_rows, a.draft_stride)) ||
      (a.noise && !rows_ok(a.n_req, a.noise_stride)))
    return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.accepted, 4) || !ptr_ok(a.next_token, 4)) return MOE_EINVAL;
  if (!opt_ok(a.parents, 4) || !opt_ok(a.uniform, 4) || !opt_ok(a.noise, 4)) return MOE_EINVAL;
  if (a.n_rows > 0) {
    const bool greedy = std::isinf(a.inv_temperature);
    if (!ptr_ok(a.logits, a.dtype == MOE_F32 ? 4 : 2) || !ptr_ok(a.tokens, 4) || !ptr_ok(a.path, 4)) return MOE_EINVAL;
    if (!greedy && (!a.uniform || !a.noise)) return MOE_EINVAL;
    if (!opt_ok(a.draft_probs, a.draft_dtype == MOE_F32 ? 4 : 2)) return MOE_EINVAL;
  }
  return MOE_OK;
}

// The most that slices_for may give for rows of this vocabulary.
int most_slices(int vocab) {
  int n = 1;
  while (n < kMaxSlices && vocab / (2 * n) >= kSliceMin) n *= 2;
  return n;
}
int slices_for(int64_t rows, int vocab, int size, int blocks) {
  const int most = most_slices(vocab);
  int n = 1;
  while (n < most && (rows * n < blocks || (rows * n < 2 * blocks && (int64_t)vocab / (2 * n) * size >= kLongSlice))) n *= 2;
  return n;
}
// A bound on rows * slices_for(...), whatever the size of an element, that does not fall as rows or vocab grow: rows
// are cut once more while there are fewer than 2 * blocks slices, so there are fewer than 4 * blocks then.
size_t places_for(int64_t rows, int vocab, int blocks) {
  return (size_t)std::min(rows * most_slices(vocab), std::max(rows, (int64_t)4 * blocks));
}
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
  int row_slices, draw_slices;
  size_t sums, drawn, end, total;
};
// Sized by n_req, n_rows and vocab alone, so that what serves a program's largest round serves its others.
Workspace layout(const moe_verify_args& a) {
  Workspace w{};
  w.row_slices = slices_for(a.n_rows, a.vocab, a.dtype == MOE_F32 ? 4 : 2, kSumBlocks);
  w.draw_slices = a.n_req <= kCounters ? slices_for(a.n_req, a.vocab, 0, kDrawBlocks) : 1;
  w.sums = kCounterBytes;
  w.drawn = w.sums + up256(places_for(a.n_rows, a.vocab, kSumBlocks) * sizeof(Key));
  w.end = w.drawn + up256(places_for(a.n_req, a.vocab, kDrawBlocks) * sizeof(Drawn));
  w.total = w.end + up256((size_t)a.n_req * sizeof(End));
  return w;
}

// A launch whose blocks may start while the one before it ends.
template <typename F>
cudaError_t after(F fn, unsigned grid, bool overlap, cudaStream_t st, const moe_verify_args& a, const Plan& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, a, p);
}

template <int DT>
cudaError_t launch(const moe_verify_args& a, const Plan& p, bool greedy, cudaStream_t st) {
  if (a.n_rows > 0) {
    const auto fn = greedy ? k_sums<DT, true> : k_sums<DT, false>;
    const cudaError_t e = launch_kernel(fn, (unsigned)a.n_rows * p.row_slices, kThreads, 0, st, a, p);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = after(k_walk<DT>, (unsigned)a.n_req, a.n_rows > 0, st, a, p);
  if (e != cudaSuccess || greedy || a.n_rows == 0) return e;
  return after(k_draw<DT>, (unsigned)a.n_req * p.draw_slices, true, st, a, p);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_verify_drafts_workspace_bytes(const moe_verify_args* args) {
  return check(args) == MOE_OK ? layout(*args).total : 0;
}

extern "C" int moe_verify_drafts(const moe_verify_args* args, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  const moe_verify_args a = read_by(*args);
  if (!ptr_ok(ws, 16)) return MOE_EINVAL;
  const Workspace w = layout(a);
  if (ws_bytes < w.total) return MOE_EWORKSPACE;
  const bool greedy = std::isinf(a.inv_temperature);
  char* base = static_cast<char*>(ws);
  Plan p{};
  const int N = a.dtype == MOE_F32 ? 4 : 8, vecs = (a.vocab + 2 * N - 2) / N;  // a row that begins off a vector's start has one more
  p.row_slices = w.row_slices;
  p.row_vecs = (vecs + w.row_slices - 1) / w.row_slices;
  p.draw_slices = w.draw_slices;
  p.draw_vecs = (vecs + w.draw_slices - 1) / w.draw_slices;
  const double c = (double)a.inv_temperature * 1.4426950408889634;
  float hi = c < 3.0e38 ? (float)c : 3.0e38f;
  if ((double)hi > c) hi = std::nextafter(hi, 0.f);
  const float lo = greedy || hi >= 3.0e38f ? 0.f : (float)(c - (double)hi);
  p.hi = hi;
  p.lo = lo > 0.f ? lo : 1.4e-45f;  // the smallest number: of no weight beside any c
  p.inv_t = (double)a.inv_temperature;
  p.left = reinterpret_cast<unsigned*>(base);
  p.sums = reinterpret_cast<float2*>(base + w.sums);
  p.keys = reinterpret_cast<Key*>(base + w.sums);
  p.drawn = reinterpret_cast<Drawn*>(base + w.drawn);
  p.end = reinterpret_cast<End*>(base + w.end);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(a.dtype == MOE_BF16  ? launch<MOE_BF16>(a, p, greedy, st)
                       : a.dtype == MOE_F16 ? launch<MOE_F16>(a, p, greedy, st)
                                            : launch<MOE_F32>(a, p, greedy, st));
}
