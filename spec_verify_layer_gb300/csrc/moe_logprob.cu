// Log probabilities of given tokens, entropies, ranks and top alternatives
// (moe_token_logprobs), one launch and one pass over the logits.
//
// A block takes a slice of one row, a chunk at a time: a thread takes three 16-byte vectors
// of the chunk, asked for two chunks ahead into shared memory (a thread reads only what it
// asked for itself, so nothing else has to wait), and updates its own running maximum m (of the logits), sum
// s = sum 2^u and w = sum 2^u u with u = (x - m) / T * log2(e), two elements an instruction;
// nothing waits for another warp until the slice ends.  Entropy is ln s - ln 2 * w / s, log
// probabilities (x - m) / T - ln s.
//
// Top entries: 64-bit keys (logit order, ~id) make the order total; a block keeps its first k
// in shared memory.  Of the first chunk it takes what is not below a bound that k entries
// are known to reach (from the threads' maxima); from then on an entry only counts if it is
// above the k-th, which few are (k of each doubling of what was seen), so threads append
// such entries to a buffer and the block merges it in after 1, 4, 16 ... chunks, each
// entry counting the larger ones for its place.  A buffer that runs over (logits that rise along
// the row, or a masked or low start of it) has its chunks gone through again, one maximum after
// the other: k times up to three quarters of the row (2,000 rows of 129,283, k = 8: 178 us as
// they come, 331 with the first 6,200 entries masked, 1,635 with the first half, 2,310 where
// all rise).  The lists of slices are joined alike: their first entries give the bound.
//
// With few rows a row is cut into 2^i slices, up to 32; the block that ends last joins the
// slices' partials in their order, so the result does not depend on which one that is.
//
// What bounds it (GB300): 2,000 rows of 129,283 logits in 32 bits (1.03 GB) take 173 to 177 us by machine,
// 5.85 to 5.95 TB/s of the 6.8 that a large copy reaches; what is missing is the last wave of rows (a row a
// block, four blocks an SM) and the first list of each.  With the vectors loaded straight
// into registers, five blocks an SM, 191 us; one chunk ahead 183; three of two
// vectors a thread 182; three blocks an SM 185; more slices a row than the SMs need cost a
// first list each (201 cut in two, 246 in four).  16 rows of 131,072 in 16 bits take 11.8
// us in a graph and 5 of 32,003 7.1: a chunk's latency, the first list, and the join one
// after the other.
#include <type_traits>

#include "moe_common.cuh"
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpBlocks = 4;    // of an SM
constexpr int kLpVecs = 3;      // 16-byte vectors a thread holds of a chunk
constexpr int kLpStages = 3;    // chunks in shared memory, asked for ahead of their turn
constexpr int kLpMaxK = 32, kLpMaxSlices = 32;
constexpr int kLpPend = 480;    // entries that wait to be merged
constexpr int kLpSliced = 304;  // blocks up to which rows are cut into slices
using Key = unsigned long long;

struct LpPartial {  // a slice's result in the workspace
  float m, s, w;
  int rank;
  Key top[kLpMaxK];
};

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

__device__ __forceinline__ float one_if_ge(float x, float y) {
  float r;
  asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// The exponent that takes sums from a maximum to a larger one.  A maximum of the type's lowest
// numbers (masked entries) is so far below that the difference may be -infinity; bounded, the
// factor 2^d is 0 all the same, and d itself times a sum stays a number.  (A NaN is in the
// sums already when it is one here.)
__device__ __forceinline__ float lower(float from, float to, float c2) { return fmaxf((from - to) * c2, -300.f); }

struct LpShared {
  Key list[kLpMaxSlices * kLpMaxK];  // what waits to be merged; candidates of the join of slices
  Key top[kLpMaxK];                  // the block's first k so far, in order; 0 where there are fewer
  Key best[kLpWarps];
  float m[kLpWarps], s[kLpWarps], w[kLpWarps];
  int rank[kLpWarps];
  unsigned kth[kLpWarps], part[kLpWarps];
  int count, last;
};

// sm.list[0 .. n) -> the first k of them in order in sm.top, 0 where there are fewer.  (All
// threads call, behind a barrier; ends with one.)
__device__ __forceinline__ void place(LpShared& sm, int n, int k) {
  const int tid = threadIdx.x;
  if (tid < k) sm.top[tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kLpThreads) {
    const Key mine = sm.list[i];
    int before = 0;
    for (int j = 0; j < n; ++j) before += sm.list[j] > mine;
    if (before < k && mine) sm.top[before] = mine;
  }
  __syncthreads();
}

// The first k entries of the slices' lists (descending, 2^i of them, 32 at most) into sm.top.
// The 32 / n first entries of each are maxima of 32 groups, so nothing below the k-th largest
// of them is among the first k.  All threads make one and call; what is read is asked for
// when it is made.
struct LpLists {
  static constexpr int kPer = kLpMaxSlices * kLpMaxK / kLpThreads;
  Key head, mine[kPer];
  __device__ __forceinline__ LpLists(int n, int k, const LpPartial* all) {
    const int tid = threadIdx.x, lane = tid & 31, each = 32 / n;
    head = lane % each < k ? __ldcg(&all[lane / each].top[lane % each]) : 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid + j * kLpThreads;
      mine[j] = i < n * k ? __ldcg(&all[i / k].top[i % k]) : 0;
    }
  }
  __device__ __forceinline__ void join(LpShared& sm, int k) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) sm.count = 0;
    const Key thr = max_key(__shfl_sync(0xffffffffu, sort_desc(head, lane), k - 1), 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (mine[j] >= thr) sm.list[atomicAdd(&sm.count, 1)] = mine[j];
    __syncthreads();
    place(sm, sm.count, k);
  }
};

template <int DT>
__global__ void __launch_bounds__(kLpThreads, kLpBlocks)
    k_token_logprobs(const __grid_constant__ moe_logprob_args a, int slices, int slice_vecs, unsigned* counters,
                     LpPartial* partials) {
  constexpr int N = Vec<DT>::N;
  __shared__ LpShared sm;
  __shared__ uint4 ring[kLpStages][kLpVecs][kLpThreads];  // chunks to come; a thread reads what it asked for itself
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.top_k;
  const int row = blockIdx.x / slices, slice = blockIdx.x - row * slices;
  const char* base = static_cast<const char*>(a.logits) + (long long)row * a.stride * (16 / N);
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15) / (16 / N));
  const int vecs = (a.vocab + lead + N - 1) / N;
  const int v0 = slice * slice_vecs, v1 = min(v0 + slice_vecs, vecs);

  const int token = a.tokens ? a.tokens[row] : -1;
  const bool has_token = token >= 0 && token < a.vocab;
  const float xt = has_token ? logit_at<DT>(base, token) : INFINITY;
  const float above = nextafterf(xt, INFINITY);  // what entries behind the token have to reach
  // (finite: 0 times an infinity would be NaN)
  const float c2 = fminf(a.inv_temperature * 1.4426950408889634f, 3.402823466e38f);
  float m = -INFINITY, s = 0.f, w = 0.f;
  int rank = 0;
  float kth = -INFINITY;  // the k-th logit so far: later entries have to be above it
  if (tid < kLpMaxK) sm.top[tid] = 0;
  if (tid == 0) sm.count = 0;

  constexpr int kStep = kLpThreads * kLpVecs;
  const auto full = [&](int c) {  // every vector of the chunk lies in the slice and in the row
    const int first = c * N - lead;
    return c + kStep <= v1 && first >= 0 && first + kStep * N <= a.vocab;
  };
  int stage = 0;
  const auto ask = [&](int c, int to) {
    if (full(c)) {
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(&ring[to][j][tid])),
                     "l"(base + (long long)((c + j * kLpThreads + tid) * N - lead) * (16 / N))
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kLpStages - 1; ++i) ask(v0 + i * kStep, i);
  __syncthreads();
  const auto chunk = [&](int c, auto inner) {  // inner: every vector is there in full, the token in none
    Vec<DT> x[kLpVecs];
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      const int v = c + j * kLpThreads + tid;
      if constexpr (inner.value)
        x[j].raw = ring[stage][j][tid];
      else if (v < v1) x[j] = load_vec<DT>(base, v * N - lead, a.vocab);
      else x[j].raw = make_uint4(Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone, Vec<DT>::kNone);
    }
    float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j)
#pragma unroll
      for (int e = 0; e < N; e += 2) tops[j & 1] = fmaxf(fmaxf(tops[j & 1], x[j].at(e)), x[j].at(e + 1));
    const float top = fmaxf(tops[0], tops[1]);
    if (top > m) {
      if (m > -INFINITY) {
        const float d = lower(m, top, c2), f = exp2_fast(d);
        w = f * fmaf(d, s, w);
        s *= f;
      }
      m = top;
    }
    const float shift = m == -INFINITY ? 0.f : m;
    const Pair less = pair(-shift, -shift), scale = pair(c2, c2);
    Pair s2 = 0, w2 = 0, r2 = 0;
    const float ahead = token < c * N - lead ? above : xt;
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      const int v = c + j * kLpThreads + tid, first = v * N - lead;
      // entries before the token count from its logit on, those behind it above that
      float thr = ahead;
      bool apart = false;
      if constexpr (!inner.value) {
        thr = v >= v1 ? INFINITY : token < first ? above : xt;
        apart = v < v1 && ((token >= first && token < first + N) ||
                           (xt == -INFINITY && (first < 0 || first + N > a.vocab)));
      }
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float x0 = x[j].at(e), x1 = x[j].at(e + 1);
        const float2 u = split(mul2(add2(pair(x0, x1), less), scale));
        const Pair p = pair(exp2_fast(u.x), exp2_fast(u.y));
        s2 = add2(s2, p);
        w2 = fma2(p, pair(fmaxf(u.x, -300.f), fmaxf(u.y, -300.f)), w2);  // 0 * -infinity is 0 here; p carries a NaN
        r2 = add2(r2, pair(one_if_ge(x0, thr), one_if_ge(x1, thr)));
      }
      if (apart) {  // the token's own vector, or one with filled places under a token of -infinity
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int i = first + e;
          const float f = x[j].at(e);
          rank -= f >= thr;
          if (i >= 0 && i < a.vocab) rank += f > xt || (f == xt && i < token);
        }
      }
    }
    {
      const float2 sv = split(s2), wv = split(w2), rv = split(r2);
      s += sv.x + sv.y;
      w += wv.x + wv.y;
      rank += (int)(rv.x + rv.y);
    }
    if (k == 0) return;
    float least = kth;  // entries above it are appended; for the first chunk, from it on
    if (c == v0) {
      // each warp's k-th of its lanes' maxima is a bound that k entries reach, and so is the
      // least of what every warp has its part of the k of
      unsigned sorted = order_key(top);
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
          const unsigned y = __shfl_xor_sync(0xffffffffu, sorted, o);
          sorted = ((lane & o) == 0) == ((lane & size) == 0) ? max(sorted, y) : min(sorted, y);
        }
      if (lane == k - 1) sm.kth[warp] = sorted;
      if (lane == (k + kLpWarps - 1) / kLpWarps - 1) sm.part[warp] = sorted;
      __syncthreads();
      unsigned bound = 0, all = 0xffffffffu;
#pragma unroll
      for (int q = 0; q < kLpWarps; ++q) {
        bound = max(bound, sm.kth[q]);
        all = min(all, sm.part[q]);
      }
      // the key below the bound's, so that "above" means from the bound on (-0 has no key of its own)
      const unsigned below = max(max(bound, all), 0x00800000u) - 1u;
      least = key_value(below == 0x7fffffffu ? below - 1u : below);
    }
    if (top > least) {
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) {
        float most = x[j].at(0);
#pragma unroll
        for (int e = 1; e < N; ++e) most = fmaxf(most, x[j].at(e));
        if (!(most > least)) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float f = x[j].at(e);
          if (f > least) {
            const int at = atomicAdd(&sm.count, 1);
            if (at < kLpPend) sm.list[at] = key_of(f, (c + j * kLpThreads + tid) * N - lead + e);
          }
        }
      }
    }
  };
  // What waits is merged with the list so far; chunks [from, to) are where it came from.
  const auto merge = [&](int from, int to) {
    __syncthreads();
    int n = sm.count;
    if (n > kLpPend) {
      // rising logits, or many equal ones: the chunks' first k, one maximum after the other
      Key prev = ~0ull;
#pragma unroll 1
      for (n = 0; n < k; ++n) {
        Key b = 0;
#pragma unroll 1
        for (int v = from + tid; v < min(to, v1); v += kLpThreads) {
          const Vec<DT> x = load_vec<DT>(base, v * N - lead, a.vocab);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const Key key = x.at(e) > -INFINITY ? key_of(x.at(e), v * N - lead + e) : 0;
            if (key < prev) b = max_key(b, key);
          }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) b = max_key(b, __shfl_xor_sync(0xffffffffu, b, o));
        __syncthreads();
        if (lane == 0) sm.best[warp] = b;
        __syncthreads();
        for (int q = 0; q < kLpWarps; ++q) b = max_key(b, sm.best[q]);
        prev = b;
        if (tid == 0) sm.list[n] = b;
      }
    }
    if (tid < k) sm.list[n + tid] = sm.top[tid];
    __syncthreads();
    place(sm, n + k, k);
    if (tid == 0) sm.count = 0;
    const Key last = sm.top[k - 1];
    kth = last ? key_logit(last) : -INFINITY;
    __syncthreads();
  };
  int merged = v0, next = v0 + kStep;
  for (int c = v0; c < v1; c += kStep) {
    const int first = c * N - lead, last = first + kStep * N;
    asm volatile("cp.async.wait_group %0;" ::"n"(kLpStages - 2) : "memory");
    ask(c + (kLpStages - 1) * kStep, stage == 0 ? kLpStages - 1 : stage - 1);
    if (full(c) && (token < first || token >= last)) chunk(c, std::true_type{});
    else chunk(c, std::false_type{});
    stage = stage == kLpStages - 1 ? 0 : stage + 1;
    if (k > 0 && (c + kStep == next || c + kStep >= v1)) {
      merge(merged, c + kStep);
      merged = c + kStep;
      next = v0 + 4 * (merged - v0);
    }
  }

  // the block's sums, in a fixed order
  {
    float top = m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float d = m == -INFINITY ? 0.f : lower(m, top, c2), f = exp2_fast(d);
    w = f * fmaf(d, s, w);
    s *= f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    if (lane == 0) {
      sm.m[warp] = top;
      sm.s[warp] = s;
      sm.w[warp] = w;
      sm.rank[warp] = rank;
    }
    __syncthreads();
    m = sm.m[0];
    for (int q = 1; q < kLpWarps; ++q) m = fmaxf(m, sm.m[q]);
    s = w = 0.f;
    rank = 0;
    for (int q = 0; q < kLpWarps; ++q) {
      const float e = sm.m[q] == -INFINITY ? 0.f : lower(sm.m[q], m, c2), g = exp2_fast(e);
      s = fmaf(g, sm.s[q], s);
      w = fmaf(g, fmaf(e, sm.s[q], sm.w[q]), w);
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
    if (tid < k) mine->top[tid] = sm.top[tid];
    __syncthreads();
    if (tid == 0) {
      // releases what the block wrote before the barrier, acquires what the others did
      unsigned before;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counters + row) : "memory");
      const bool last = before == (unsigned)slices - 1;
      if (last) counters[row] = 0;  // ready for the next call
      sm.last = last;
    }
    __syncthreads();
    if (!sm.last) return;
    const LpPartial* all = partials + (size_t)row * slices;
    // every warp joins the sums alike: lane = slice
    LpLists lists(slices, max(k, 1), all);
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
    const float d = pm == -INFINITY ? 0.f : lower(pm, m, c2), f = exp2_fast(d);
    w = f * fmaf(d, ps, pw);
    s = f * ps;
    rank = pr;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    if (k > 0) lists.join(sm, k);
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
    const Key key = sm.top[tid];
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
  if (a.vocab > (1 << 24) || a.top_k > kLpMaxK || a.n_rows > (1 << 24) || a.stride >= ((int64_t)1 << 40) ||
      !rows_ok(a.n_rows, a.stride))
    return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4)) return MOE_EINVAL;
  if (a.n_rows == 0) return MOE_OK;
  if (!ptr_ok(a.logits, a.dtype == MOE_F32 ? 4 : 2)) return MOE_EINVAL;
  if (!opt_ok(a.tokens, 4) || !opt_ok(a.logp, 4) || !opt_ok(a.entropy, 4) || !opt_ok(a.rank, 4)) return MOE_EINVAL;
  if (!a.tokens && (a.logp || a.rank)) return MOE_EINVAL;
  if (a.top_k > 0 ? !ptr_ok(a.top_ids, 4) || !ptr_ok(a.top_logp, 4) : false) return MOE_EINVAL;
  return MOE_OK;
}

// Slices of a row: while there are SMs to spare (kLpSliced blocks, two for each of 152) and every
// thread of a slice has a vector.  More slices cost more than the last round of blocks: 2,000 rows of 129,283
// take 174 us uncut, 201 cut in two, 246 in four.
int slices_of(const moe_logprob_args& a) {
  const int vecs = a.vocab / (a.dtype == MOE_F32 ? 4 : 8);
  int s = 1;
  while (s < kLpMaxSlices && (int64_t)a.n_rows * s * 2 <= kLpSliced && vecs / (2 * s) >= kLpThreads) s *= 2;
  return s;
}

// Counters of the rows that are cut (at most kLpSliced / 2), partials of their slices (at most kLpSliced).
constexpr size_t kLpWorkspace = kCounterBytes + kLpSliced * sizeof(LpPartial);
static_assert(kLpSliced / 2 * sizeof(unsigned) <= kCounterBytes && kCounterBytes % alignof(LpPartial) == 0, "counters");

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_token_logprobs_workspace_bytes(const moe_logprob_args* args) {
  return check(args) == MOE_OK ? kLpWorkspace : 0;
}

extern "C" int moe_token_logprobs(const moe_logprob_args* args, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  if (!ptr_ok(ws, 16)) return MOE_EINVAL;
  if (ws_bytes < kLpWorkspace) return MOE_EWORKSPACE;
  const moe_logprob_args& a = *args;
  if (a.n_rows == 0) return MOE_OK;
  const int s = slices_of(a), per = a.dtype == MOE_F32 ? 4 : 8;
  const int vecs = (a.vocab + 2 * per - 2) / per;  // wherever a row starts
  const int slice_vecs = (vecs + s - 1) / s;
  unsigned* counters = static_cast<unsigned*>(ws);
  LpPartial* partials = reinterpret_cast<LpPartial*>(static_cast<char*>(ws) + kCounterBytes);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)a.n_rows * s;
  const auto fn = a.dtype == MOE_F32    ? k_token_logprobs<MOE_F32>
                  : a.dtype == MOE_BF16 ? k_token_logprobs<MOE_BF16>
                                        : k_token_logprobs<MOE_F16>;
  return launch_status(launch_kernel(fn, grid, kLpThreads, 0, st, a, s, slice_vecs, counters, partials));
}
