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
  __shared__ float2 trig[2][kRopeRows][D / 2];
  __shared__ long long where[2][kRopeRows];  // element offset of the row's slot in the cache, or -1
  const int tid = threadIdx.x, p = tid % L, group = tid / L;
  const int half = a.rot_dim / 2, hq = a.q_heads, hkv = a.kv_heads, heads = hq + 2 * hkv;
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
  for (int i = tid; i < half; i += kRopeThreads) frac[i] = turn_fraction(a.inv_freq[i]);
  const uint2* gq = static_cast<const uint2*>(a.q_gain);
  const uint2* gk = static_cast<const uint2*>(a.k_gain);
  uint2 gain_q[2] = {}, gain_k[2] = {};
  if (gq) {
    gain_q[0] = gq[c0];
    gain_q[1] = gq[c1];
  }
  if (gk) {
    gain_k[0] = gk[c0];
    gain_k[1] = gk[c1];
  }
  unsigned flags = 0;
  int buf = 0;
  for (int row0 = blockIdx.x * kRopeRows; row0 < a.n_rows; row0 += gridDim.x * kRopeRows, buf ^= 1) {
    const int rows = min(kRopeRows, a.n_rows - row0);
    if (row0 == (int)blockIdx.x * kRopeRows) __syncthreads();  // frac
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
    for (int w0 = group; w0 < rows * heads; w0 += kGroups * kRopeUnroll) {
      uint2 x[kRopeUnroll][2];
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int w = w0 + u * kGroups;
        if (w >= rows * heads) continue;
        const int r = w / heads, h = w - r * heads;
        const long long row = row0 + r;
        const uint16_t* src =
            h < hq ? static_cast<const uint16_t*>(a.q) + row * a.q_stride + h * D
            : h < hq + hkv ? static_cast<const uint16_t*>(a.k) + row * a.k_stride + (h - hq) * D
                           : static_cast<const uint16_t*>(a.v) + row * a.v_stride + (h - hq - hkv) * D;
        x[u][0] = *reinterpret_cast<const uint2*>(src + 4 * c0);
        x[u][1] = *reinterpret_cast<const uint2*>(src + 4 * c1);
      }
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int w = w0 + u * kGroups;
        // a group's lanes agree on w; the shuffles below stay inside the group
        if (w >= rows * heads) continue;
        const int r = w / heads, h = w - r * heads;
        const bool is_q = h < hq, is_v = h >= hq + hkv;
        uint2 y0 = x[u][0], y1 = x[u][1];
        if (!is_v) {
          float2 v[4] = {unpack2<DT>(y0.x), unpack2<DT>(y0.y), unpack2<DT>(y1.x), unpack2<DT>(y1.y)};
          if (is_q ? gq != nullptr : gk != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fmaf(v[j].x, v[j].x, fmaf(v[j].y, v[j].y, ss));
            const unsigned members = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((tid & 31) / L * L);
#pragma unroll
            for (int o = L / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(members, ss, o);
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            const uint2 g0 = is_q ? gain_q[0] : gain_k[0], g1 = is_q ? gain_q[1] : gain_k[1];
            const float2 g[4] = {unpack2<DT>(g0.x), unpack2<DT>(g0.y), unpack2<DT>(g1.x), unpack2<DT>(g1.y)};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_float2(v[j].x * inv * g[j].x, v[j].y * inv * g[j].y);
          }
          if (turns) {
            const float2* t = trig[buf][r] + 4 * p;
            if (a.interleaved) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                v[j] = make_float2(v[j].x * t[j].x - v[j].y * t[j].y, v[j].y * t[j].x + v[j].x * t[j].y);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float2 t0 = t[2 * j], t1 = t[2 * j + 1], lo = v[j], hi = v[j + 2];
                v[j] = make_float2(lo.x * t0.x - hi.x * t0.y, lo.y * t1.x - hi.y * t1.y);
                v[j + 2] = make_float2(hi.x * t0.x + lo.x * t0.y, hi.y * t1.x + lo.y * t1.y);
              }
            }
          }
          y0 = make_uint2(pack2<DT>(v[0].x, v[0].y), pack2<DT>(v[1].x, v[1].y));
          y1 = make_uint2(pack2<DT>(v[2].x, v[2].y), pack2<DT>(v[3].x, v[3].y));
        }
        uint16_t* dst;
        if (is_q) {
          dst = static_cast<uint16_t*>(a.q_out) + (long long)(row0 + r) * a.q_out_stride + h * D;
        } else {
          const long long at = where[buf][r];
          if (at < 0) continue;
          dst = static_cast<uint16_t*>(is_v ? a.cache.v : a.cache.k) + at +
                (is_v ? h - hq - hkv : h - hq) * a.cache.head_stride;
        }
        *reinterpret_cast<uint2*>(dst + 4 * c0) = y0;
        *reinterpret_cast<uint2*>(dst + 4 * c1) = y1;
      }
    }
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
