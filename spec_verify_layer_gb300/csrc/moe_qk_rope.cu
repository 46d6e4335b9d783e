// Norm and rotation of queries and keys with the cache write (moe_qk_rope_cache), one
// launch: each element is read once and written once.
//
// A block works through (row, run of heads) tasks in the order of memory: the task's queries,
// keys and values come into a ring of shared-memory stages by asynchronous copies, two
// tasks ahead, while the present one is worked on; the loads in flight that the memory
// needs (some 40 KB an SM) would not fit in registers beside the arithmetic.  A group of
// D / 16 lanes takes one head; a lane holds two 16-byte chunks of eight elements chosen so
// that both elements of each of its rotation pairs are its own: chunks (p, p + rot / 16) for
// halves, (2p, 2p + 1) side by side.  The sum of squares is a shuffle reduction inside the group.
// The angles of a row are shared by its heads: cosines and sines of the next task are
// written to shared memory while this one is worked on, one barrier a task.
//
// Angles: a position turns pair i by pos * f_i turns, f_i = inv_freq_i / 2 pi.  Only the
// fraction of a turn matters, so f_i is held as a 64-bit fixed-point fraction F_i (one
// conversion in double per pair and block) and pos * F_i is one integer product whose
// overflow drops the whole turns; its error is at most |pos| * 2^-52 turns for f_i < 1,
// 1.4e-9 rad at 10^6 and 3e-6 rad at 2^31.  The top 32 bits go to float as half turns in
// [-1, 1).
//
// What bounds it (GB300): memory.  16,384 rows of 32 + 2 * 4 heads of 128 (336 MB) take 57.4 us,
// 5.85 TB/s of the 6.80 that a large copy reaches; a plain copy of this size takes 55.4.  A
// warp a row took 103 us, values in registers instead of the ring 79.8.  Few rows are
// bound by latency: one row 3.0 us in a graph, 701 rows of 24 + 2 * 8 heads of 64 (14.4 MB) 4.3.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 64;
constexpr int kRopeStages = 3;
constexpr int kRopeStage = 10240;  // bytes of a stage at most: six blocks of an SM then fit
constexpr int kRopeBlocks = 6;     // of an SM

__device__ __forceinline__ unsigned long long turn_fraction(double inv_freq) {
  const double f = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
  return (unsigned long long)((f - floor(f)) * 18446744073709551616.0);  // NaN and 1.0 saturate
}

// The run of heads of a task: heads [h0, h1) of a row's queries, keys and values in a line.
struct Runs {
  int length, count;  // heads of a run (the last may be shorter), runs of a row
  int rows_on, runs_on;  // from a block's task to its next one: whole rows, and runs
  unsigned page_mul;     // n / page_size = (n * page_mul) >> page_shift for n below 2^31
  int page_shift;
};

struct Task {  // a place in the list of (row, run)
  int row, run;
  __device__ __forceinline__ void next(const Runs& r) {
    row += r.rows_on;
    run += r.runs_on;
    if (run >= r.count) {
      run -= r.count;
      ++row;
    }
  }
};

template <int DT, int D>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    k_qk_rope(const __grid_constant__ moe_qk_rope_args a, const Runs runs) {
  constexpr int L = D / 16, kGroups = kRopeThreads / L, CPH = D / 8;  // 16-byte chunks of a head
  extern __shared__ __align__(16) unsigned char stages[];
  __shared__ unsigned long long frac[D / 2];
  __shared__ __align__(16) float cosines[2][D / 2], sines[2][D / 2];
  const int tid = threadIdx.x, p = tid % L, group = tid / L;
  const int half = a.rot_dim / 2, hq = a.q_heads, hk = hq + a.kv_heads, heads = hk + a.kv_heads;
  const int stage_bytes = runs.length * D * 2;
  const bool turns = p < a.rot_dim / 16;
  int c0, c1;  // this lane's chunks of eight elements
  if (a.interleaved) {
    c0 = 2 * p;
    c1 = 2 * p + 1;
  } else if (turns) {
    c0 = p;
    c1 = p + a.rot_dim / 16;
  } else {
    c0 = a.rot_dim / 8 + 2 * (p - a.rot_dim / 16);
    c1 = c0 + 1;
  }
  const unsigned members = ((1u << L) - 1u) << ((tid & 31) / L * L);
  const uint32_t stage0 = (uint32_t)__cvta_generic_to_shared(stages);

  const uint4* const q = static_cast<const uint4*>(a.q) + tid;
  const uint4* const k = static_cast<const uint4*>(a.k) - hq * CPH + tid;
  const uint4* const v = static_cast<const uint4*>(a.v) - hk * CPH + tid;
  const auto fetch = [&](Task t, int stage) {
    if (t.row < a.n_rows) {
      const int from = t.run * runs.length * CPH, to = min(from + runs.length * CPH, heads * CPH);
      const uint4* const q_row = q + t.row * (a.q_stride >> 3);
      const uint4* const k_row = k + t.row * (a.k_stride >> 3);
      const uint4* const v_row = v + t.row * (a.v_stride >> 3);
      uint32_t at = stage0 + stage * stage_bytes + tid * 16;
#pragma unroll 4
      for (int c = from; c + tid < to; c += kRopeThreads, at += kRopeThreads * 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at),
                     "l"((c + tid < hq * CPH ? q_row : c + tid < hk * CPH ? k_row : v_row) + c)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const auto angles = [&](int pos, int buf) {
    for (int i = tid; i < half; i += kRopeThreads) {
      const int turn = (int)(((unsigned long long)(long long)pos * frac[i]) >> 32);
      float sine, cosine;
      sincospif((float)turn * 4.656612873077393e-10f, &sine, &cosine);  // 2^-31 half turns
      cosines[buf][i] = cosine * a.rot_scale;
      sines[buf][i] = sine * a.rot_scale;
    }
  };
  const auto position = [&](Task t) { return t.row < a.n_rows ? a.row_pos[t.row] : 0; };

  Task task{(int)blockIdx.x / runs.count, (int)blockIdx.x % runs.count}, ahead = task;
  for (int n = 0; n < kRopeStages - 1; ++n) {
    fetch(ahead, n);
    ahead.next(runs);
  }
  Task second = task;
  second.next(runs);
  int pos = position(second);
  for (int i = tid; i < half; i += kRopeThreads) frac[i] = turn_fraction(a.inv_freq[i]);
  uint4 q_gain[2] = {}, k_gain[2] = {};
  if (a.q_gain) {
    q_gain[0] = static_cast<const uint4*>(a.q_gain)[c0];
    q_gain[1] = static_cast<const uint4*>(a.q_gain)[c1];
  }
  if (a.k_gain) {
    k_gain[0] = static_cast<const uint4*>(a.k_gain)[c0];
    k_gain[1] = static_cast<const uint4*>(a.k_gain)[c1];
  }
  angles(position(task), 0);  // (frac: each thread's own entries)
  unsigned flags = 0;
  int stage = 0, buf = 0;
  for (; task.row < a.n_rows; task.next(runs)) {
    const int h0 = task.run * runs.length, h1 = min(h0 + runs.length, heads);
    const int slot = a.row_slot[task.row];
    second.next(runs);
    const int next_pos = position(second);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRopeStages - 2) : "memory");
    __syncthreads();  // the stage is there, the one before is free, and so are the angles before
    fetch(ahead, stage == 0 ? kRopeStages - 1 : stage - 1);
    ahead.next(runs);
    angles(pos, buf ^ 1);  // the next task's
    pos = next_pos;
    long long at = -1;  // element offset of the row's slot in the cache
    if (slot >= 0 && slot < a.cache.n_pages * a.cache.page_size) {
      const int page = (int)(((unsigned long long)(unsigned)slot * runs.page_mul) >> runs.page_shift);
      at = page * a.cache.page_stride + (slot - page * a.cache.page_size) * a.cache.slot_stride;
    } else if (slot != -1 && h1 > hq) {
      flags |= MOE_DEV_INDEX;
    }
    const uint4* const x = reinterpret_cast<const uint4*>(stages + stage * stage_bytes) - h0 * CPH;
    // a lane's eight pairs: their cosines and sines
    Pair co[4], si[4];
    if (turns) {
      const float4* const c = reinterpret_cast<const float4*>(cosines[buf] + 8 * p);
      const float4* const t = reinterpret_cast<const float4*>(sines[buf] + 8 * p);
      const float4 ca = c[0], cb = c[1], ta = t[0], tb = t[1];
      co[0] = pair(ca.x, ca.y);
      co[1] = pair(ca.z, ca.w);
      co[2] = pair(cb.x, cb.y);
      co[3] = pair(cb.z, cb.w);
      si[0] = pair(ta.x, ta.y);
      si[1] = pair(ta.z, ta.w);
      si[2] = pair(tb.x, tb.y);
      si[3] = pair(tb.z, tb.w);
    }
    // a group's lanes agree on h: the shuffles stay inside the group
    const auto turned = [&](int from, int to, bool norm, const uint4 (&g)[2], uint16_t* dst, int64_t head_stride) {
#pragma unroll 1
      for (int h = from + group; h < to; h += kGroups) {
        const uint4 y0 = x[h * CPH + c0], y1 = x[h * CPH + c1];
        Pair v[8] = {pair(unpack2<DT>(y0.x)), pair(unpack2<DT>(y0.y)), pair(unpack2<DT>(y0.z)), pair(unpack2<DT>(y0.w)),
                     pair(unpack2<DT>(y1.x)), pair(unpack2<DT>(y1.y)), pair(unpack2<DT>(y1.z)), pair(unpack2<DT>(y1.w))};
        if (norm) {
          Pair sq = mul2(v[0], v[0]), sr = mul2(v[1], v[1]);
#pragma unroll
          for (int j = 2; j < 8; j += 2) {
            sq = fma2(v[j], v[j], sq);
            sr = fma2(v[j + 1], v[j + 1], sr);
          }
          const float2 sum = split(add2(sq, sr));
          float ss = sum.x + sum.y;
#pragma unroll
          for (int o = L / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(members, ss, o);
          const float inv = rsqrtf(ss * (1.0f / D) + a.eps);  // within 2 units in the last place
          const Pair inv2 = pair(inv, inv);
          const uint32_t gw[8] = {g[0].x, g[0].y, g[0].z, g[0].w, g[1].x, g[1].y, g[1].z, g[1].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mul2(mul2(v[j], inv2), pair(unpack2<DT>(gw[j])));
        }
        if (turns) {
          if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 e = split(v[j]), c = split(co[j / 2]), t = split(si[j / 2]);
              const float cj = j & 1 ? c.y : c.x, tj = j & 1 ? t.y : t.x;
              v[j] = fma2(pair(-e.y, e.x), pair(tj, tj), mul2(v[j], pair(cj, cj)));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const Pair lo = v[j], hi = v[j + 4];
              const float2 t = split(si[j]);
              v[j] = fma2(hi, pair(-t.x, -t.y), mul2(lo, co[j]));
              v[j + 4] = fma2(lo, si[j], mul2(hi, co[j]));
            }
          }
        }
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 e = split(v[j]);
          w[j] = pack2<DT>(e.x, e.y);
        }
        uint4* const to_head = reinterpret_cast<uint4*>(dst + h * head_stride);
        __stcs(to_head + c0, make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(to_head + c1, make_uint4(w[4], w[5], w[6], w[7]));
      }
    };
    if (h0 < hq)
      turned(h0, min(h1, hq), a.q_gain != nullptr, q_gain, static_cast<uint16_t*>(a.q_out) + task.row * a.q_out_stride, D);
    if (at >= 0) {
      const int64_t hs = a.cache.head_stride;
      if (h1 > hq && h0 < hk)
        turned(max(h0, hq), min(h1, hk), a.k_gain != nullptr, k_gain, static_cast<uint16_t*>(a.cache.k) + at - hq * hs, hs);
      for (int c = max(h0, hk) * CPH + tid; c < h1 * CPH; c += kRopeThreads) {  // values: as they are
        const int h = c / CPH;
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.cache.v) + at + (h - hk) * hs) + c % CPH, x[c]);
      }
    }
    if (++stage == kRopeStages) stage = 0;
    buf ^= 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (flags) atomicOr(a.dev_status, flags);
}

template <int DT>
cudaError_t launch(const moe_qk_rope_args& a, int sms, cudaStream_t st) {
  const int heads = a.q_heads + 2 * a.kv_heads, groups = kRopeThreads * 16 / a.head_dim;
  Runs runs;
  runs.length = kRopeStage / (a.head_dim * 2);
  if (runs.length > heads) runs.length = heads;
  runs.count = (heads + runs.length - 1) / runs.length;
  // shorter runs while there are few rows and a run keeps a head for every group
  while (a.n_rows * runs.count * 2 <= 2 * sms && runs.length >= 2 * groups) {
    runs.length = (runs.length + 1) / 2;
    runs.count = (heads + runs.length - 1) / runs.length;
  }
  runs.length = (heads + runs.count - 1) / runs.count;  // about equal ones
  const int64_t tasks = (int64_t)a.n_rows * runs.count, blocks = (int64_t)sms * kRopeBlocks;
  const int grid = (int)(tasks < blocks ? tasks : blocks);
  runs.rows_on = grid / runs.count;
  runs.runs_on = grid % runs.count;
  int bits = 0;
  while ((1 << bits) < a.cache.page_size) ++bits;
  runs.page_shift = 31 + bits;
  runs.page_mul = (unsigned)((1ull << runs.page_shift) / (unsigned)a.cache.page_size + 1);
  const size_t smem = (size_t)kRopeStages * runs.length * a.head_dim * 2;
  const auto fn = a.head_dim == 64 ? k_qk_rope<DT, 64> : a.head_dim == 128 ? k_qk_rope<DT, 128> : k_qk_rope<DT, 256>;
  return launch_kernel(fn, grid, kRopeThreads, smem, st, a, runs);
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
  const int rc = check_cache(a.cache, a.kv_heads);
  if (rc != MOE_OK) return rc;
  if (!stride_ok(a.q_stride) || !stride_ok(a.k_stride) || !stride_ok(a.v_stride) || !stride_ok(a.q_out_stride))
    return MOE_EINVAL;
  if (!rows_ok(a.n_rows, a.q_stride) || !rows_ok(a.n_rows, a.k_stride) || !rows_ok(a.n_rows, a.v_stride) ||
      !rows_ok(a.n_rows, a.q_out_stride))
    return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4) || !opt_ok(a.q_gain, 16) || !opt_ok(a.k_gain, 16)) return MOE_EINVAL;
  if (a.rot_dim > 0 && !ptr_ok(a.inv_freq, 8)) return MOE_EINVAL;
  if (a.n_rows == 0) return MOE_OK;
  if (!ptr_ok(a.q, 16) || !ptr_ok(a.k, 16) || !ptr_ok(a.v, 16) || !ptr_ok(a.q_out, 16) || !ptr_ok(a.row_pos, 4) ||
      !ptr_ok(a.row_slot, 4))
    return MOE_EINVAL;
  if (a.q_out == a.q && a.q_out_stride != a.q_stride) return MOE_EINVAL;
  const int sms = current_sms();
  if (sms < 1) return MOE_ECUDA;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(a.dtype == MOE_BF16 ? launch<MOE_BF16>(a, sms, st) : launch<MOE_F16>(a, sms, st));
}
