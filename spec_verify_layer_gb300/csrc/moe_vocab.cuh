// Rows over a vocabulary (moe_logprob.cu, moe_verify_drafts.cu): their elements in vectors of 16
// bytes wherever a row begins, and 64-bit keys that order entries by (logit descending, id
// ascending).  Internal; not part of the public ABI.
#pragma once

#include "moe_common.cuh"
#include "moe_round_ops.cuh"

namespace moe {

using Key = unsigned long long;

__device__ __forceinline__ Key key_of(float x, int id) { return ((Key)order_key(x) << 32) | (uint32_t)~id; }
__device__ __forceinline__ float key_logit(Key k) { return key_value((unsigned)(k >> 32)); }
__device__ __forceinline__ int key_id(Key k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ Key max_key(Key a, Key b) { return a > b ? a : b; }

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

}  // namespace moe
