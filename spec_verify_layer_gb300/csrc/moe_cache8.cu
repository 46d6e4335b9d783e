// Rows into a paged cache of 8 bits and out of it (moe_cache8_append, moe_cache8_read), one
// launch each: each row is read once and written once.
//
// Append.  A task is one block of tokens of one head, of keys or of values: its largest magnitude a, the
// least power of two with a <= Q 2^e, the codes of x / 2^e.  With powers of two x / 2^e is exact, so a
// row is rounded once, and for e4m3, which has the same relative precision at every scale, they cost
// one binade of range and no precision; what a block holds from before is carried to a larger scale
// with half a step of its own there (e4m3: only where its code falls below the smallest normal one), and
// to a smaller one exactly.  The rows of a block lie next to each
// other in the call, so a thread block takes up to 64 consecutive rows, a thread looks up the page of each,
// and it works through the blocks that begin among them; a group of 8, 16 or 32 lanes takes a task, in
// 16-byte loads.  A lane keeps what it has read for the maximum in registers (64 elements; more is read
// again, out of the L2).
//   The maximum is taken over the bits of the elements' magnitudes, two of 16 bits at a time; only where
// that says that something is not finite are the rows looked at again one by one (78.6 -> 69.0 us for
// the prompts below, 89.1 -> 69.6 with int8, whose rounding is one addition, all with three thread
// blocks an SM).
//   One token into a block of 16 that is half full 6.6 us: latency (lengths, page, row, one after the other).
// 200 requests of up to 9 rows, 8 heads of 64, blocks of 8, 18.6 us: the same, and groups that look for the blocks
// of ragged rows.  A begun block is walked by its one group, 8 bytes a lane and step, twice where the scale
// moves: one token into a block that is full but for it takes, with blocks of 16, 64 and 128, 8.2, 14.3 and 22.3 us
// with heads of 128, 9.1, 20.5 and 36.2 with heads of 256.
//   Prompts of 20,011 to 32,768 rows, 4 heads of 128 (243 MB), blocks of 16, 63.5 to 65 us, 3.8 TB/s, 56 % of
// measured: a group holds one task's 4 KB at a time and waits for it before it stores, and two thread blocks an SM
// hold as many tasks as registers allow.  Three with the spills that they bring 69.0 us, four with half as many
// elements kept and the rest read again 81.8; fp32 rows 76 (88 with half of them kept).  That size of a task is what
// the registers just hold.  Larger ones are read twice: blocks of 32, 64 and 128 take 69.9, 77.0 and 94.1 us, heads of
// 256 in blocks of 16 69.6.  Smaller ones leave less on its way: blocks of 8, 4, 2 and 1 take 99, 173, 254 and 244,
// 8 heads of 64 in blocks of 16 106.
//
// Read.  A thread takes 16 codes of four rows at a time; a row's request, page and scale's place are looked
// up once a thread block.  1,500 rows, 4 heads of 128, 6.6 us: latency.  Five contexts of 1,001 to 65,536 rows, 8
// heads of 64 (511 MB), 98.0 us, 5.2 TB/s, 76 % of measured, two thirds of it written; 122 with a look-up a warp.  The same
// rows as 2 heads of 256 in e4m3 to bf16 100 us, in int8 88, e4m3 to fp32 182 (4.7 TB/s); blocks of 1 and of 32 alike.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 64;  // of a thread block, at most

struct Request {
  int s, n, ctx;  // first row, rows, context; n < 0: not a request that can be worked on
};

__device__ __forceinline__ Request request(const moe_cache8_args& a, int b) {
  Request q;
  q.s = __ldg(a.row_start + b);
  const int e = __ldg(a.row_start + b + 1);
  q.ctx = __ldg(a.ctx_len + b);
  const bool ok = q.s >= 0 && e >= q.s && e <= a.n_rows && q.ctx >= 0 &&
                  (long long)q.ctx + (e - q.s) <= min((long long)a.table_width * a.cache.page_size, 0x7fffffffll - 256);
  q.n = ok ? e - q.s : -1;
  return q;
}

// The request of a row: the last that begins at or before it.
__device__ __forceinline__ int request_of(const moe_cache8_args& a, int row) { return last_not_above(a.row_start, a.n_req, row); }

// Is the row one of the request's?  (Of a request that can be worked on, first: the difference to a row_start of any
// value may pass 32 bits and come round.)
__device__ __forceinline__ bool holds(const Request& q, int row) { return q.n > 0 && row >= q.s && row - q.s < q.n; }

__device__ __forceinline__ unsigned bad_requests(const moe_cache8_args& a) {
  unsigned flags = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(a.row_start) != 0) flags |= MOE_DEV_LENGTH;
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.n_req; b += gridDim.x * kThreads)
    if (request(a, b).n < 0) flags |= MOE_DEV_LENGTH;
  return flags;
}

// A row's eight elements in 32 bits.
template <int DT>
struct Row8 {
  uint4 raw[DT == MOE_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, long long element) {
    if constexpr (DT == MOE_F32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + element);
      raw[0] = p[0];
      raw[1] = p[1];
    } else {
      raw[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + element);
    }
  }
  __device__ __forceinline__ void floats(float* x) const {
    if constexpr (DT == MOE_F32) {
      const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
    } else {
      const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2<DT>(w[j]);
        x[2 * j] = v.x;
        x[2 * j + 1] = v.y;
      }
    }
  }
  // The larger of `most` and the elements' magnitudes, as bits of the type (two elements a word for 16-bit types).
  __device__ __forceinline__ uint32_t larger(uint32_t most) const {
#pragma unroll
    for (int i = 0; i < (DT == MOE_F32 ? 2 : 1); ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) most = DT == MOE_F32 ? max(most, w[j] & 0x7fffffffu) : __vmaxu2(most, w[j] & 0x7fff7fffu);
    }
    return most;
  }
  static __device__ __forceinline__ float magnitude(uint32_t most) {  // what `larger` found
    if constexpr (DT == MOE_F32) return __uint_as_float(most);
    return unpack2<DT>(max(most & 0xffffu, most >> 16)).x;
  }
};

// The values of four codes.
__device__ __forceinline__ void decode4(uint32_t w, bool i8, float* x) {
  if (i8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = (float)(int8_t)(w >> (8 * j));
    return;
  }
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = unpack2<MOE_F16>(lo), b = unpack2<MOE_F16>(hi);
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

// Codes of four numbers times a power of two.  ODD: there may be infinities, which become the largest code,
// and NaN, which becomes 0; otherwise all are within the codes' range.
template <bool ODD>
__device__ __forceinline__ uint32_t encode4(const float* x, float inv, bool i8) {
  if (i8) {
    // x inv is exact, so adding 1.5 * 2^23 rounds it once, to the nearest integer, ties to even, in the last bits
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = ODD ? (x[j] == x[j] ? fminf(fmaxf(x[j] * inv, -127.f), 127.f) : 0.f) : 0.f;
      w[j] = __float_as_uint(ODD ? y + 12582912.f : fmaf(x[j], inv, 12582912.f));
    }
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  }
  float2 lo2 = make_float2(x[0], x[1]), hi2 = make_float2(x[2], x[3]);
  if (ODD) {
    lo2 = make_float2(x[0] == x[0] ? x[0] : 0.f, x[1] == x[1] ? x[1] : 0.f);
    hi2 = make_float2(x[2] == x[2] ? x[2] : 0.f, x[3] == x[3] ? x[3] : 0.f);
  }
  const Pair by = pair(inv, inv);
  lo2 = split(mul2(pair(lo2), by));
  hi2 = split(mul2(pair(hi2), by));
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(lo2.y), "f"(lo2.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(hi2.y), "f"(hi2.x));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// e of the least power of two 2^e, e >= -126, with most <= Q 2^e: most = 1.f * 2^E is at most
// 448 * 2^(E - 8) where 1.f <= 1.75, at most 127 * 2^(E - 6) where 1.f <= 127 / 64.
__device__ __forceinline__ int scale_exponent(float most, bool i8) {
  const uint32_t bits = __float_as_uint(most), f = bits & 0x7fffffu;
  const int E = (int)(bits >> 23) - 127, e = i8 ? E - 6 + (f > 0x7e0000u) : E - 8 + (f > 0x600000u);
  return max(e, -126);
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 2) k_append(const __grid_constant__ moe_cache8_args a, PageDivide pd, int lanes, int rows) {
  constexpr int CPR = D / 8;  // chunks of eight elements of a row
  constexpr int kHold = 8;
  struct Begin {              // a block of tokens that begins among these rows
    long long codes, scales;  // of its first slot, and of its scale, head 0
    int row, held, rows;      // first row, slots before it, rows
  };
  // In the order of rows within a warp.  Thread blocks beside each other deal out the same tasks, so they have to have
  // them in the same order; they have 16 rows, the first warp's (with more there are enough blocks without).
  __shared__ Begin begin[kRows];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, B = a.cache.block_size;
  const bool i8 = a.cache.format == MOE_I8;
  unsigned flags = blockIdx.y == 0 ? bad_requests(a) : 0;
  if (tid == 0) count = 0;
  __syncthreads();
  if (tid < kRows) {
    const int r = blockIdx.x * rows + tid;  // a thread a row
    Begin own;
    bool begins = false;
    if (tid < rows && r < a.n_rows) {
      const int b = request_of(a, r);
      const Request q = request(a, b);
      const int pos = holds(q, r) ? q.ctx + (r - q.s) : -1, in_block = pos & (B - 1);
      if (pos >= 0 && (r == q.s || !in_block)) {
        const int col = (int)(((unsigned long long)(unsigned)pos * pd.mul) >> pd.shift);
        const int page = __ldg(a.block_table + (long long)b * a.table_width + col);
        if (page < 0 || page >= a.cache.n_pages) {
          flags |= MOE_DEV_INDEX;
        } else {
          const int slot = pos - in_block - col * a.cache.page_size;
          begins = true;
          own = {page * a.cache.page_stride + slot * a.cache.slot_stride,
                 page * a.cache.scale_page_stride + slot / B * a.cache.scale_block_stride,
                 r, in_block, min(B - in_block, q.n - (r - q.s))};
        }
      }
    }
    const unsigned all = __ballot_sync(0xffffffffu, begins);
    const int first = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(&count, __popc(all)) : 0, 0);
    if (begins) begin[first + __popc(all & ((1u << lane) - 1))] = own;
  }
  __syncthreads();
  const int heads = a.kv_heads, tasks = count * 2 * heads, at = tid & (lanes - 1);
  const int group = blockIdx.y * (kThreads / lanes) + tid / lanes, groups = gridDim.y * (kThreads / lanes);
  const unsigned members = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u) << (lane & ~(lanes - 1));
  for (int t = group; t < tasks; t += groups) {
    const int head = t % heads, kv = t / heads & 1;
    const Begin g = begin[t / (2 * heads)];
    const void* x = kv ? a.v : a.k;
    const long long x0 = g.row * (kv ? a.v_stride : a.k_stride) + head * D, x_stride = kv ? a.v_stride : a.k_stride;
    uint8_t* codes = static_cast<uint8_t*>(kv ? a.cache.v : a.cache.k) + g.codes + head * a.cache.head_stride;
    float* scale = (kv ? a.cache.v_scale : a.cache.k_scale) + g.scales + head * a.cache.scale_head_stride;
    const float old = g.held ? scale_of(*scale, flags) : 0.f;
    float most = 0.f;  // of what is held and of the rows
    uint32_t top = 0;
    for (int c = at; c < g.held * CPR; c += lanes) {
      const uint2 w = *reinterpret_cast<const uint2*>(codes + c / CPR * a.cache.slot_stride + c % CPR * 8);
      float v[8];
      decode4(w.x, i8, v);
      decode4(w.y, i8, v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // (a NaN counts as an infinity here)
        const float m = fabsf(v[j] * old);
        most = m < INFINITY ? fmaxf(most, m) : INFINITY;
      }
    }
    // the first kHold of a lane's chunks stay in registers, what is more is read again
    Row8<DT> kept[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int c = at + i * lanes;
      if (c < g.rows * CPR) kept[i].load(x, x0 + c / CPR * x_stride + c % CPR * 8);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (at + i * lanes < g.rows * CPR) top = kept[i].larger(top);
    const auto again = [&](int c) {
      Row8<DT> y;
      y.load(x, x0 + c / CPR * x_stride + c % CPR * 8);
      return y;
    };
#pragma unroll 4
    for (int c = at + kHold * lanes; c < g.rows * CPR; c += lanes) top = again(c).larger(top);
    const float rows_most = Row8<DT>::magnitude(top);
    most = rows_most < INFINITY ? fmaxf(most, rows_most) : INFINITY;
    for (int o = lanes >> 1; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(members, most, o));
    const bool odd = !(most < INFINITY);
    if (odd) {  // some are not finite: the largest of those that are
      flags |= MOE_DEV_VALUE;
      most = 0.f;
      const auto look = [&](const float* v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fabsf(v[j]) < INFINITY ? fmaxf(most, fabsf(v[j])) : most;
      };
      float v[8];
#pragma unroll 1
      for (int c = at; c < g.held * CPR; c += lanes) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + c / CPR * a.cache.slot_stride + c % CPR * 8);
        decode4(w.x, i8, v);
        decode4(w.y, i8, v + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= old;
        look(v);
      }
#pragma unroll 1
      for (int c = at; c < g.rows * CPR; c += lanes) {
        again(c).floats(v);
        look(v);
      }
      for (int o = lanes >> 1; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(members, most, o));
    }
    const int e = scale_exponent(most, i8);
    const float now = __uint_as_float((uint32_t)(e + 127) << 23), inv = __uint_as_float((uint32_t)(127 - e) << 23);
    const auto carry = [&]() {  // what is held, under the new scale
#pragma unroll 1
      for (int c = at; c < g.held * CPR; c += lanes) {
        uint2* p = reinterpret_cast<uint2*>(codes + c / CPR * a.cache.slot_stride + c % CPR * 8);
        const uint2 w = *p;
        float v[8];
        decode4(w.x, i8, v);
        decode4(w.y, i8, v + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= old;
        *p = make_uint2(encode4<true>(v, inv, i8), encode4<true>(v + 4, inv, i8));
      }
    };
    const auto place = [&](int c) { return reinterpret_cast<uint2*>(codes + (g.held + c / CPR) * a.cache.slot_stride + c % CPR * 8); };
    float v[8];
    if (odd) {
      carry();  // under a scale that stays, too: a NaN code becomes 0
#pragma unroll 1
      for (int c = at; c < g.rows * CPR; c += lanes) {
        again(c).floats(v);
        __stcs(place(c), make_uint2(encode4<true>(v, inv, i8), encode4<true>(v + 4, inv, i8)));
      }
    } else {
      if (now != old) carry();
#pragma unroll
      for (int i = 0; i < kHold; ++i)
        if (at + i * lanes < g.rows * CPR) {
          kept[i].floats(v);
          __stcs(place(at + i * lanes), make_uint2(encode4<false>(v, inv, i8), encode4<false>(v + 4, inv, i8)));
        }
#pragma unroll 4
      for (int c = at + kHold * lanes; c < g.rows * CPR; c += lanes) {
        again(c).floats(v);
        __stcs(place(c), make_uint2(encode4<false>(v, inv, i8), encode4<false>(v + 4, inv, i8)));
      }
    }
    if (at == 0) *scale = now;
  }
  if (flags) atomicOr(a.dev_status, flags);
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) k_read(const __grid_constant__ moe_cache8_args a, PageDivide pd, int rows_most) {
  constexpr int CPR = D / 16;
  __shared__ long long from[kRows], scales[kRows];  // -1: not a row of a request, -2: nothing cached
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool i8 = a.cache.format == MOE_I8;
  unsigned flags = bad_requests(a);
  const int r0 = blockIdx.x * rows_most, rows = min(rows_most, a.n_rows - r0);
  if (tid < rows) {  // a thread a row
    const int r = r0 + tid, b = request_of(a, r);
    const Request q = request(a, b);
    long long at = -1, scale = 0;
    if (holds(q, r)) {
      const int pos = q.ctx + (r - q.s), col = (int)(((unsigned long long)(unsigned)pos * pd.mul) >> pd.shift);
      const int page = __ldg(a.block_table + (long long)b * a.table_width + col), slot = pos - col * a.cache.page_size;
      if (page < 0 || page >= a.cache.n_pages) {
        flags |= MOE_DEV_INDEX;
        at = -2;
      } else {
        at = page * a.cache.page_stride + slot * a.cache.slot_stride;
        scale = page * a.cache.scale_page_stride + slot / a.cache.block_size * a.cache.scale_block_stride;
      }
    }
    from[tid] = at;
    scales[tid] = scale;
  }
  __syncthreads();
  const int per_row = 2 * a.kv_heads * CPR;
  for (int t = lane; t < per_row; t += 32) {
    const int h2 = t / CPR, c = t % CPR, kv = h2 >= a.kv_heads, head = h2 - (kv ? a.kv_heads : 0);
    const uint8_t* const codes = static_cast<const uint8_t*>(kv ? a.cache.v : a.cache.k) + head * a.cache.head_stride + c * 16;
    const float* const scale = (kv ? a.cache.v_scale : a.cache.k_scale) + head * a.cache.scale_head_stride;
    const long long stride = kv ? a.v_stride : a.k_stride, to0 = (long long)r0 * stride + head * D + c * 16;
    constexpr int kAhead = 4;  // rows on their way
    for (int i0 = warp; i0 < rows; i0 += kWarps * kAhead) {
      uint4 w[kAhead];
      float s[kAhead];
      bool there[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kWarps;
        there[u] = i < rows && from[i] != -1;
        w[u] = make_uint4(0, 0, 0, 0);
        s[u] = 0.f;
        if (there[u] && from[i] >= 0) {
          w[u] = __ldcs(reinterpret_cast<const uint4*>(codes + from[i]));
          s[u] = __ldg(scale + scales[i]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!there[u]) continue;
        const float f = scale_of(s[u], flags);
        const long long to = to0 + (i0 + u * kWarps) * stride;
        float x[16];
        decode4(w[u].x, i8, x);
        decode4(w[u].y, i8, x + 4);
        decode4(w[u].z, i8, x + 8);
        decode4(w[u].w, i8, x + 12);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= f;
        if constexpr (DT == MOE_F32) {
          float4* out = reinterpret_cast<float4*>(static_cast<float*>(kv ? a.v : a.k) + to);
#pragma unroll
          for (int j = 0; j < 4; ++j) __stcs(out + j, make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
        } else {
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? a.v : a.k) + to);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            __stcs(out + j, make_uint4(pack2<DT>(x[8 * j], x[8 * j + 1]), pack2<DT>(x[8 * j + 2], x[8 * j + 3]),
                                       pack2<DT>(x[8 * j + 4], x[8 * j + 5]), pack2<DT>(x[8 * j + 6], x[8 * j + 7])));
        }
      }
    }
  }
  if (flags) atomicOr(a.dev_status, flags);
}

int check(const moe_cache8_args* p) {
  if (!p) return MOE_EINVAL;
  const moe_cache8_args& a = *p;
  if (a.n_req < 1 || a.n_rows < 0 || a.table_width < 1 || a.kv_heads < 1 || a.head_dim < 1) return MOE_EINVAL;
  if (a.dtype != MOE_BF16 && a.dtype != MOE_F16 && a.dtype != MOE_F32) return MOE_EINVAL;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return MOE_EUNSUPPORTED;
  if (a.n_req > 16384 || a.n_rows > (1 << 24) || a.kv_heads > 256) return MOE_EUNSUPPORTED;
  const int rc = check_cache(a.cache, a.kv_heads);
  if (rc != MOE_OK) return rc;
  if (!stride_ok(a.k_stride) || !stride_ok(a.v_stride)) return MOE_EINVAL;
  if (!rows_ok(a.n_rows, a.k_stride) || !rows_ok(a.n_rows, a.v_stride)) return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.ctx_len, 4) || !ptr_ok(a.block_table, 4)) return MOE_EINVAL;
  if (a.n_rows > 0 && (!ptr_ok(a.k, 16) || !ptr_ok(a.v, 16))) return MOE_EINVAL;
  return MOE_OK;
}

// May an append write this cache?  Each block of tokens and head has to have a scale and codes of its own; strides of 0,
// as of a cache that is read under one scale for all, give several the same.
bool own_places(const moe_cache8_args& a) {
  const moe_kv_cache8& c = a.cache;
  if (c.k_scale == c.v_scale) return false;
  if (c.n_pages > 1 && (c.page_stride == 0 || c.scale_page_stride == 0)) return false;
  if (c.page_size > 1 && c.slot_stride == 0) return false;
  if (c.page_size > c.block_size && c.scale_block_stride == 0) return false;
  return a.kv_heads == 1 || (c.head_stride != 0 && c.scale_head_stride != 0);
}

// Rows of a thread block: as many as leave blocks for every SM, 16 at least.
int block_rows(int n_rows) {
  int rows = kRows;
  while (rows > 16 && n_rows / rows < 600) rows /= 2;
  return rows;
}

template <int DT>
cudaError_t append(const moe_cache8_args& a, cudaStream_t st) {
  // lanes of a task: no more than it has chunks of eight elements
  const int chunks = a.cache.block_size * a.head_dim / 8, lanes = chunks >= 32 ? 32 : chunks;
  const auto fn = a.head_dim == 64 ? k_append<DT, 64> : a.head_dim == 128 ? k_append<DT, 128> : k_append<DT, 256>;
  // few rows (16 a block, see k_append): their tasks over several thread blocks
  const int rows = block_rows(a.n_rows);
  const unsigned across = (a.n_rows + rows - 1) / rows;
  unsigned down = 1;
  while (across * down < 600 && down * kThreads / lanes < 2u * a.kv_heads) down *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(across, down);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, fn, a, page_divide(a.cache.page_size), lanes, rows);
}
template <int DT>
cudaError_t read(const moe_cache8_args& a, cudaStream_t st) {
  const auto fn = a.head_dim == 64 ? k_read<DT, 64> : a.head_dim == 128 ? k_read<DT, 128> : k_read<DT, 256>;
  const int rows = block_rows(a.n_rows);
  return launch_kernel(fn, (a.n_rows + rows - 1) / rows, kThreads, 0, st, a, page_divide(a.cache.page_size), rows);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_cache8_append(const moe_cache8_args* args, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  if (!own_places(*args)) return MOE_EINVAL;
  if (args->n_rows == 0) return MOE_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(args->dtype == MOE_BF16  ? append<MOE_BF16>(*args, st)
                       : args->dtype == MOE_F16 ? append<MOE_F16>(*args, st)
                                                : append<MOE_F32>(*args, st));
}

extern "C" int moe_cache8_read(const moe_cache8_args* args, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK || args->n_rows == 0) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(args->dtype == MOE_BF16  ? read<MOE_BF16>(*args, st)
                       : args->dtype == MOE_F16 ? read<MOE_F16>(*args, st)
                                                : read<MOE_F32>(*args, st));
}
