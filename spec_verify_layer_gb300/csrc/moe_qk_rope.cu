// Norm and rotation of queries and keys with the cache write (moe_qk_rope_cache), one
// launch: each element is read once and written once.
//
// A group of D / 8 lanes takes one head of one row; a lane holds two chunks of four
// elements (8-byte loads and stores) chosen so that both elements of each of its rotation
// pairs are its own: chunks (p, p + rot / 8) for halves, (2p, 2p + 1) side by side.  The
// sum of squares is a shuffle reduction inside the group.  The angles of a row are shared
// by all its heads, so a block first writes its rows' cosines and sines to shared memory.
//
// Angles: a position turns pair i by pos * f_i turns, f_i = inv_freq_i / 2 pi.  Only the
// fraction of a turn matters, so f_i is held as a 64-bit fixed-point fraction F_i (one
// conversion in double per pair and block) and pos * F_i is one integer product whose
// overflow drops the whole turns; its error is at most |pos| * 2^-52 turns for f_i < 1,
// 1.4e-9 rad at 10^6 and 3e-6 rad at 2^31.  The top 32 bits go to float as half turns in
// [-1, 1).
#include <type_traits>

#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;    // rows of a block's step
constexpr int kRopeUnroll = 4;  // heads a group has in flight

__device__ __forceinline__ unsigned long long turn_fraction(double inv_freq) {
  const double f = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
  return (unsigned long long)((f - floor(f)) * 18446744073709551616.0);  // NaN and 1.0 saturate
}

template <int DT, int D>
__global__ void __launch_bounds__(kRopeThreads) k_qk_rope(const __grid_constant__ moe_qk_rope_args a) {
  constexpr int L = D / 8, kGroups = kRopeThreads / L;
  __shared__ unsigned long long frac[D / 2];
  __shared__ __align__(16) float2 trig[2][kRopeRows][D / 2];
  __shared__ long long where[2][kRopeRows];  // element offset of the row's slot in the cache, or -1
  const int tid = threadIdx.x, p = tid % L, group = tid / L;
  const int half = a.rot_dim / 2;
  const bool turns = p < a.rot_dim / 8;
  int c0, c1;  // this lane's chunks of four elements
  if (a.interleaved) {
    c0 = 2 * p;
    c1 = 2 * p + 1;
  } else if (turns) {
    c0 = p;
    c1 = p + a.rot_dim / 8;
  } else {
    c0 = a.rot_dim / 4 + 2 * (p - a.rot_dim / 8);
    c1 = c0 + 1;
  }
  const unsigned members = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((tid & 31) / L * L);
  for (int i = tid; i < half; i += kRopeThreads) frac[i] = turn_fraction(a.inv_freq[i]);
  __syncthreads();

  // Heads [row][head] of one kind, U of them in flight in a group.  (n: rows of the step)
  const auto heads = [&](auto kind, int n, int row0, int buf, int count, const void* from, int64_t stride,
                         const void* gain) {
    constexpr int kQuery = 0, kValue = 2, KIND = decltype(kind)::value;
    const unsigned mul = ((1u << 20) + count - 1) / count;  // w / count for w < 1024 + 3 * 32
    float g[8];
    if (gain) {
      const uint2 x = static_cast<const uint2*>(gain)[c0], y = static_cast<const uint2*>(gain)[c1];
      const float2 v[4] = {unpack2<DT>(x.x), unpack2<DT>(x.y), unpack2<DT>(y.x), unpack2<DT>(y.y)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[2 * j] = v[j].x;
        g[2 * j + 1] = v[j].y;
      }
    }
    constexpr int U = KIND == kQuery ? kRopeUnroll : 1;
    for (int w0 = group; w0 < n * count; w0 += kGroups * U) {
      uint2 x[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int w = w0 + u * kGroups, r = (int)(w * mul >> 20), h = w - r * count;
        if (w >= n * count) break;
        const uint16_t* src = static_cast<const uint16_t*>(from) + (row0 + r) * stride + h * D;
        x[u][0] = __ldcs(reinterpret_cast<const uint2*>(src + 4 * c0));
        x[u][1] = __ldcs(reinterpret_cast<const uint2*>(src + 4 * c1));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int w = w0 + u * kGroups, r = (int)(w * mul >> 20), h = w - r * count;
        if (w >= n * count) break;  // a group's lanes agree on w: the shuffles below stay inside the group
        uint2 y0 = x[u][0], y1 = x[u][1];
        if constexpr (KIND != kValue) {
          float2 v[4] = {unpack2<DT>(y0.x), unpack2<DT>(y0.y), unpack2<DT>(y1.x), unpack2<DT>(y1.y)};
          if (gain) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fmaf(v[j].x, v[j].x, fmaf(v[j].y, v[j].y, ss));
#pragma unroll
            for (int o = L / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(members, ss, o);
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);  // within 2 units in the last place
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_float2(v[j].x * inv * g[2 * j], v[j].y * inv * g[2 * j + 1]);
          }
          if (turns) {
            const float4* t = reinterpret_cast<const float4*>(trig[buf][r] + 4 * p);  // cosine, sine, cosine, sine
            const float4 ta = t[0], tb = t[1];
            if (a.interleaved) {
              v[0] = make_float2(v[0].x * ta.x - v[0].y * ta.y, v[0].y * ta.x + v[0].x * ta.y);
              v[1] = make_float2(v[1].x * ta.z - v[1].y * ta.w, v[1].y * ta.z + v[1].x * ta.w);
              v[2] = make_float2(v[2].x * tb.x - v[2].y * tb.y, v[2].y * tb.x + v[2].x * tb.y);
              v[3] = make_float2(v[3].x * tb.z - v[3].y * tb.w, v[3].y * tb.z + v[3].x * tb.w);
            } else {
              const float2 a0 = v[0], a1 = v[1], b0 = v[2], b1 = v[3];
              v[0] = make_float2(a0.x * ta.x - b0.x * ta.y, a0.y * ta.z - b0.y * ta.w);
              v[1] = make_float2(a1.x * tb.x - b1.x * tb.y, a1.y * tb.z - b1.y * tb.w);
              v[2] = make_float2(b0.x * ta.x + a0.x * ta.y, b0.y * ta.z + a0.y * ta.w);
              v[3] = make_float2(b1.x * tb.x + a1.x * tb.y, b1.y * tb.z + a1.y * tb.w);
            }
          }
          y0 = make_uint2(pack2<DT>(v[0].x, v[0].y), pack2<DT>(v[1].x, v[1].y));
          y1 = make_uint2(pack2<DT>(v[2].x, v[2].y), pack2<DT>(v[3].x, v[3].y));
        }
        uint16_t* dst;
        if constexpr (KIND == kQuery) {
          dst = static_cast<uint16_t*>(a.q_out) + (row0 + r) * a.q_out_stride + h * D;
        } else {
          const long long at = where[buf][r];
          if (at < 0) continue;
          dst = static_cast<uint16_t*>(KIND == kValue ? a.cache.v : a.cache.k) + at + h * a.cache.head_stride;
        }
        *reinterpret_cast<uint2*>(dst + 4 * c0) = y0;
        *reinterpret_cast<uint2*>(dst + 4 * c1) = y1;
      }
    }
  };

  unsigned flags = 0;
  int buf = 0;
  for (int row0 = blockIdx.x * kRopeRows; row0 < a.n_rows; row0 += gridDim.x * kRopeRows, buf ^= 1) {
    const int rows = min(kRopeRows, a.n_rows - row0);
    for (int e = tid; e < rows * half; e += kRopeThreads) {
      const int r = e / half, i = e - r * half;
      const long long pos = a.row_pos[row0 + r];
      const int turn = (int)(((unsigned long long)pos * frac[i]) >> 32);
      float s, c;
      sincospif((float)turn * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
      trig[buf][r][i] = make_float2(c * a.rot_scale, s * a.rot_scale);
    }
    if (tid < rows) {
      const int slot = a.row_slot[row0 + tid];
      long long at = -1;
      if (slot >= 0 && slot < a.cache.n_pages * a.cache.page_size) {
        const int page = slot / a.cache.page_size;
        at = page * a.cache.page_stride + (slot - page * a.cache.page_size) * a.cache.slot_stride;
      } else if (slot != -1) {
        flags |= MOE_DEV_INDEX;
      }
      where[buf][tid] = at;
    }
    __syncthreads();  // one a step: the next step writes the other buffer
    heads(std::integral_constant<int, 0>{}, rows, row0, buf, a.q_heads, a.q, a.q_stride, a.q_gain);
    heads(std::integral_constant<int, 1>{}, rows, row0, buf, a.kv_heads, a.k, a.k_stride, a.k_gain);
    heads(std::integral_constant<int, 2>{}, rows, row0, buf, a.kv_heads, a.v, a.v_stride, nullptr);
  }
  if (flags) atomicOr(a.dev_status, flags);
}

template <int DT>
cudaError_t launch(const moe_qk_rope_args& a, int grid, cudaStream_t st) {
  switch (a.head_dim) {
    case 64: k_qk_rope<DT, 64><<<grid, kRopeThreads, 0, st>>>(a); break;
    case 128: k_qk_rope<DT, 128><<<grid, kRopeThreads, 0, st>>>(a); break;
    default: k_qk_rope<DT, 256><<<grid, kRopeThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_qk_rope_cache(const moe_qk_rope_args* p, void* stream) {
  if (!p) return MOE_EINVAL;
  const moe_qk_rope_args& a = *p;
  if (a.n_rows < 0 || a.q_heads < 1 || a.kv_heads < 1 || a.head_dim < 1 || a.rot_dim < 0 || a.rot_dim > a.head_dim)
    return MOE_EINVAL;
  if (!(a.eps >= 0.f) || std::isinf(a.eps) || !std::isfinite(a.rot_scale)) return MOE_EINVAL;
  if (a.dtype != MOE_BF16 && a.dtype != MOE_F16) return a.dtype == MOE_F32 ? MOE_EUNSUPPORTED : MOE_EINVAL;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return MOE_EUNSUPPORTED;
  if (a.rot_dim % 16 || a.q_heads > 256 || a.kv_heads > 256 || a.n_rows > (1 << 24)) return MOE_EUNSUPPORTED;
  const int rc = check_cache(a.cache);
  if (rc != MOE_OK) return rc;
  if (!stride_ok(a.q_stride) || !stride_ok(a.k_stride) || !stride_ok(a.v_stride) || !stride_ok(a.q_out_stride))
    return MOE_EINVAL;
  if (!ptr_ok(a.dev_status, 4) || !opt_ok(a.q_gain, 16) || !opt_ok(a.k_gain, 16)) return MOE_EINVAL;
  if (a.rot_dim > 0 && !ptr_ok(a.inv_freq, 8)) return MOE_EINVAL;
  if (a.n_rows == 0) return MOE_OK;
  if (!ptr_ok(a.q, 16) || !ptr_ok(a.k, 16) || !ptr_ok(a.v, 16) || !ptr_ok(a.q_out, 16) || !ptr_ok(a.row_pos, 4) ||
      !ptr_ok(a.row_slot, 4))
    return MOE_EINVAL;
  if (a.q_out == a.q && a.q_out_stride != a.q_stride) return MOE_EINVAL;
  const int sms = current_sms();
  if (sms < 1) return MOE_ECUDA;
  const int steps = (a.n_rows + kRopeRows - 1) / kRopeRows, most = 6 * sms;
  const int grid = steps < most ? steps : most;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(a.dtype == MOE_BF16 ? launch<MOE_BF16>(a, grid, st) : launch<MOE_F16>(a, grid, st));
}
