// Shared by the attention-side operators of a verify round (moe_round_map.cu,
// moe_qk_rope.cu, moe_tree_attn.cu, moe_logprob.cu): argument checks and the element
// types.  Internal; not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe_verify.h"

namespace moe {

inline bool ptr_ok(const void* p, unsigned align) { return p && (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }
// NULL, or aligned
inline bool opt_ok(const void* p, unsigned align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

// strides in elements: multiples of 8, not negative
inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < ((int64_t)1 << 40); }

// Offsets in elements, products of counts and strides: in 128 bits, since a descriptor may hold
// any, and far enough below 2^63 for bytes.
using Wide = __int128;
constexpr Wide kMaxOffset = (Wide)1 << 60;
inline bool rows_ok(int64_t rows, int64_t stride) { return (Wide)(rows - 1) * stride < kMaxOffset; }
// of the first element of the last head of the last slot
inline Wide cache_span(const moe_kv_cache& c, int heads) {
  return (Wide)(c.n_pages - 1) * c.page_stride + (Wide)(c.page_size - 1) * c.slot_stride + (Wide)(heads - 1) * c.head_stride;
}

inline int check_cache(const moe_kv_cache& c, int heads) {
  if (!ptr_ok(c.k, 16) || !ptr_ok(c.v, 16)) return MOE_EINVAL;
  if (c.n_pages < 1 || c.page_size < 1) return MOE_EINVAL;
  if (!stride_ok(c.page_stride) || !stride_ok(c.slot_stride) || !stride_ok(c.head_stride)) return MOE_EINVAL;
  if (c.page_size > 65536 || (int64_t)c.n_pages * c.page_size >= ((int64_t)1 << 31) || cache_span(c, heads) >= kMaxOffset)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// The current device's SM count; 0 if there is no usable device.
inline int current_sms() {
  int dev = -1, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// A workspace begins with its call's counters, which are zero between calls, in an area of one size
// whatever the arguments are; what lies behind it is written before it is read.  So one buffer
// serves calls of any shape, one after the other, and of either call that takes one.
constexpr size_t kCounterBytes = 1280;

// What the launch itself reported; a failed launch leaves no error behind for the caller's next call.
inline int launch_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ECUDA;
}

#ifdef __CUDACC__

// A launch and its own status (the runtime's last error may be that of an earlier call).
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*fn)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// A 32-bit word of two elements <-> two floats.
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (DT == MOE_BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == MOE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Two floats in one register pair: an instruction for both.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ Pair pair(float2 v) { return pair(v.x, v.y); }
__device__ __forceinline__ float2 split(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// 2^x, results below the smallest normal number 0
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < a ? 0xffffffffu : s;
}

// Largest b in [0, n) with start[b] <= x, for start ascending with start[0] <= x.
template <typename T>
__device__ __forceinline__ int last_not_above(const T* start, int n, T x) {
  int lo = 0, hi = n;  // start[lo] <= x, start[hi] > x or hi == n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

#endif  // __CUDACC__

}  // namespace moe
