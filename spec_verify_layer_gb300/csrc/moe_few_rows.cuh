// Attention over codes for few query rows a key/value head (moe_tree_attention8): up to 8 NT of them.
//
// Mathematics, as in moe_tree_attn.cuh: scores times the key's scale, weights with the value's scale in
// them, their sum from weight / scale; running maximum and sum a warp, joined when a head's share ends.
//
// Here the memory is the bound (with one row of 8 heads a tile of 128 keys of 128 elements takes
// 1,420 cycles of an SM's share of it), and turning codes into fp16 through shared memory for the
// tensor memory path costs more than that: some 4,200 warp instructions a tile, 176 to 240 us for 64
// requests of one row over up to 8,192 keys in several forms.  So codes go straight into the registers
// of mma.sync, 1,500 instructions a tile: S^T = K Q^T with keys as rows, O^T += V^T P^T with elements
// of V as rows; both of a product's operands then have the query rows as their 8 columns.  A lane's
// 16 bytes of a key are pairs along the product's depth as they lie (any order of elements does, if
// the queries have the same); values are paired key by key with a byte permutation; P comes out of S
// by an 8 x 8 transpose.  Eight or twelve warps take steps of 32 keys in turn, each with a ring of
// stages and a softmax of its own, so that no barrier stands between a warp's loads and its products.
//
// 64 requests of one row over 4,096 to 8,192 keys, 32/4 heads of 128 (403 MB): 82.5 us, 4.9 TB/s, 71 %
// of measured (the bytes take 59 us); 88 with eight warps.  Bound: instructions issued and the latency of
// a warp's own chain (copy, scores, weights, products), 12 warps being all that registers allow.  Page, scales,
// logarithm and reciprocal are taken key by key, so blocks of 1, 4, 16 and 64 tokens take the same (83.7, 81.2, 81.0,
// 82.5).  16/2 heads of 256 82.7, 64/8 heads of 64, twice as many keys of half the size, 135.
// One row over up to 1,000 keys 12.3 us: latency, as for the 16-bit cache.  Six groups of 8 rows for
// heads of 64 (33 ragged requests of up to 48 query rows) 108 us against 89 through tensor memory: sums of
// that many rows leave registers for steps of 16 keys only.
#pragma once

#include "moe_attn_parts.cuh"

namespace moe {
namespace {

template <int D, int NT>
struct FewShape {
  // Twelve warps (and two stages each, if three are too large) where a warp's sums leave the registers
  // for it, else eight and three.
  static constexpr int W = D / 16 * NT <= 8 ? 12 : 8, STAGES = W == 12 && D > 64 ? 2 : 3;
  static constexpr int KS = D == 256 ? 16 : 32;  // keys of a step
  static constexpr int kStage = 2 * KS * D;      // codes of keys and values
  static constexpr int kRing = W * STAGES * kStage;
  static constexpr int ROWS = 8 * NT, kPitch = D + 4;
  static constexpr int kScales = W * STAGES * 2 * KS * 4;  // of keys and values
  static constexpr int kPages = W * 4 * KS * 4, kHoles = W * 4 * 4;
  static constexpr int kQuery = NT * (D / 16) * 32 * 8, kRowBytes = ROWS * 4, kMl = W * ROWS * 8;
  static constexpr int kBytes = kRing + kScales + kPages + kHoles + kQuery + kRowBytes + kMl;
  static_assert(W * ROWS * kPitch * 4 <= kRing, "the ring holds the warps' sums");
};

template <int D, int NT>
constexpr int kFewThreads = FewShape<D, NT == 0 ? 1 : NT>::W * 32;

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // of an 8 x 8 matrix of 16-bit elements
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Four codes as two pairs of fp16.
template <int FMT>
__device__ __forceinline__ void pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == MOE_I8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), off), q = __hsub2(*reinterpret_cast<const __half2*>(&y), off);
    lo = *reinterpret_cast<const uint32_t*>(&p);
    hi = *reinterpret_cast<const uint32_t*>(&q);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// A block's share of the list, unit after unit; all W warps.
template <typename A, int FMT, int D, int NT>
__device__ __forceinline__ void few_rows(const A& a, const Plan& p, Control& ct, unsigned char* smem, Walk<A, D>& wk, int member, unsigned& flags) {
  using F = FewShape<D, NT>;
  constexpr int W = F::W, STAGES = F::STAGES;
  constexpr int KT = kKeyTile<D>, KS = F::KS, MT = KS / 16, CC = D / 16, STEPS = D / 16, OT = D / 16, RPI = 32 / CC, COPIES = KS / RPI;
  constexpr uint32_t kNone = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3, G = p.group;
  unsigned char* const ring = smem + warp * STAGES * F::kStage;
  float* const scales = reinterpret_cast<float*>(smem + F::kRing) + warp * STAGES * 2 * KS;  // [stage][keys, values][KS]
  volatile int* const pages = reinterpret_cast<int*>(smem + F::kRing + F::kScales) + warp * 4 * KS;
  volatile unsigned* const holes = reinterpret_cast<unsigned*>(smem + F::kRing + F::kScales + F::kPages) + warp * 4;
  uint2* const query = reinterpret_cast<uint2*>(smem + F::kRing + F::kScales + F::kPages + F::kHoles);  // [NT][STEPS][32]
  float* const row_factor = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(query) + F::kQuery);
  float2* const ml = reinterpret_cast<float2*>(reinterpret_cast<unsigned char*>(row_factor) + F::kRowBytes);  // [warp][ROWS]
  float* const sums = reinterpret_cast<float*>(smem);  // [warp][ROWS][kPitch], when the ring is done with
  const uint32_t ring0 = smem_u32(ring), scales0 = smem_u32(scales), pages0 = smem_u32(const_cast<int*>(pages));
  const auto column = [&](int pos) { return (int)(__umulhi((unsigned)pos << 1, p.page_mul) >> (p.page_shift - 31)); };
  // places of 16-byte chunks, such that eight lanes of a load meet eight different banks: of keys four chunks
  // of two rows, of values two chunks (D = 64: halves of two) of every other of eight rows
  const auto key_at = [](int r, int c) { return (D == 64 ? r * 4 + c : r * CC + (c ^ (r & 1) << 2)) * 16; };
  const auto value_at = [](int r, int c) {
    return (D == 64 ? (r >> 1) * 8 + ((r ^ r >> 1) & 1) * 4 + (c ^ (r >> 2 & 1) << 1) : r * CC + (c ^ (r >> 1 & 3) << 1)) * 16;
  };
  const uint32_t page_units = (uint32_t)(a.cache.page_stride >> 4), slot_units = (uint32_t)(a.cache.slot_stride >> 4);

  for (int seq = 0; wk.more(); wk.next(a)) {
    const int m0 = member * F::ROWS, rows = min(F::ROWS, wk.q.n * G - m0);  // of the request's query rows
    if (rows <= 0 || wk.t0 == wk.t1) continue;
    const int len = wk.q.ctx + wk.q.n, k0 = wk.t0 * KT, k1 = min(len, wk.t1 * KT);
    const int32_t* table = a.block_table + (long long)wk.b * a.table_width;
    const bool whole = wk.t0 == 0 && wk.t1 == wk.q.tiles;
    if (tid == 0) {
      ct.bad[seq & 7] = 0;
      if (!whole) {  // who shares this head
        const int at = ct.w1 - wk.left - wk.p0 + kUnit;
        const int first = gang_of(ct.total, ct.gangs, at), last = gang_of(ct.total, ct.gangs, at + wk.q.tiles - 1);
        ct.split[wk.t0 == 0] = {wk.q.s, wk.q.n, wk.h, first, last - first + 1};
      }
    }
    const int steps = (k1 - k0 + KS - 1) / KS, mine = steps > warp ? (steps - warp + W - 1) / W : 0;
    const uint32_t head_units = (uint32_t)(wk.h * a.cache.head_stride >> 4);
    const long long scale_at = wk.h * a.cache.scale_head_stride;
    const auto key0 = [&](int j) { return k0 + (warp + j * W) * KS; };
    const auto look = [&](int j) {  // the pages of this warp's step j
      const int pos = key0(j) + lane;
      const bool there = j < mine && lane < KS && pos < k1;
      if (lane < KS) copy4(pages0 + ((j & 3) * KS + lane) * 4, table + (there ? column(pos) : 0), there);
    };
    const auto ask = [&](int j, int stage) {  // step j, whose pages are there; and the pages of the second next
      if (j < mine) {
        const int pos = key0(j) + lane, in_page = pos - column(pos) * a.cache.page_size;
        const int page = lane < KS ? pages[(j & 3) * KS + lane] : -1;
        const bool there = lane < KS && pos < k1, good = there && page >= 0 && page < a.cache.n_pages;
        const uint32_t at = good ? (uint32_t)page * page_units + (uint32_t)in_page * slot_units + head_units : kNone;
        const unsigned hole = __ballot_sync(0xffffffffu, there && !good);
        if (lane == 0) holes[j & 3] = hole;
        if (lane < KS) {
          const long long sc = good ? page * a.cache.scale_page_stride + (in_page >> p.block_shift) * a.cache.scale_block_stride + scale_at : 0;
          copy4(scales0 + (stage * 2 * KS + lane) * 4, a.cache.k_scale + sc, good);
          copy4(scales0 + (stage * 2 * KS + KS + lane) * 4, a.cache.v_scale + sc, good);
        }
        const int c = lane % CC;
        const uint32_t dst = ring0 + stage * F::kStage;
        uint32_t from[COPIES];
#pragma unroll
        for (int i = 0; i < COPIES; ++i) from[i] = __shfl_sync(0xffffffffu, at, i * RPI + lane / CC);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int r = i * RPI + lane / CC;
          const bool ok = from[i] != kNone;
          const uint32_t src = ok ? from[i] + c : 0;
          copy16(dst + key_at(r, c), static_cast<const uint4*>(a.cache.k) + src, ok);
          copy16(dst + KS * D + value_at(r, c), static_cast<const uint4*>(a.cache.v) + src, ok);
        }
      }
      look(j + 2);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look(0);
    look(1);
    asm volatile("cp.async.commit_group;" ::: "memory");

    // The queries as the products take them, fp16 whatever their type: each row times the power of two
    // that brings its largest element to 2^14 .. 2^15, which the row's factor takes back.  An n-tile a warp.
    if (warp < NT) {
      const int mi = m0 + min(warp * 8 + g, rows - 1), n = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi;
      const bool there = warp * 8 + g < rows, bf = a.dtype == MOE_BF16;
      const uint16_t* const src = static_cast<const uint16_t*>(a.q) + (long long)(wk.q.s + n) * a.q_stride + (wk.h * G + mi - n * G) * D + t * 16;
      uint4 x[D / 64][2];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[i][u] = there ? *reinterpret_cast<const uint4*>(src + i * 64 + u * 8) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x[i][u].x, x[i][u].y, x[i][u].z, x[i][u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) most = max(most, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
        }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int k = min(126, 14 - (bf ? (int)(most >> 7) - 127 : (int)(most >> 10) - 15));
      const float by = __uint_as_float((uint32_t)(k + 127) << 23 | (p.score < 0.f ? 0x80000000u : 0u));
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w[4] = {x[i][u].x, x[i][u].y, x[i][u].z, x[i][u].w};
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = bf ? unpack2<MOE_BF16>(w[e]) : unpack2<MOE_F16>(w[e]);
            y[e] = pack2<MOE_F16>(v.x * by, v.y * by);
          }
          query[(warp * STEPS + i * 4 + u * 2) * 32 + lane] = make_uint2(y[0], y[1]);
          query[(warp * STEPS + i * 4 + u * 2 + 1) * 32 + lane] = make_uint2(y[2], y[3]);
        }
      if (t == 0) row_factor[warp * 8 + g] = fabsf(p.score) * __uint_as_float((uint32_t)(127 - k) << 23);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    ask(0, 0);
    ask(1, 1);
    __syncthreads();  // the queries

    float m[NT][2], l[NT][2], factor[NT][2], o[OT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
        factor[nt][e] = row_factor[nt * 8 + 2 * t + e];
      }
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }
    int stage = 0;
#pragma unroll 1
    for (int j = 0; j < mine; ++j) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // this step; the next is on its way
      __syncwarp();
      if (STAGES == 3) ask(j + 2, stage == 0 ? STAGES - 1 : stage - 1);  // into the stage before, which is done with
      const unsigned char* const keys = ring + stage * F::kStage;
      unsigned char* const values = ring + stage * F::kStage + KS * D;
      const float* const sc = scales + stage * 2 * KS;
      const int pos0 = key0(j);
      const unsigned hole = holes[j & 3];
      if (hole) flags |= MOE_DEV_INDEX;
      const bool all = pos0 + KS <= wk.q.ctx && !hole;
      if (FMT == MOE_E4M3 && pos0 + KS > wk.q.ctx) {
        // drafted rows' values: codes that are NaN are noted and taken out, and added at the end to the rows
        // that see them
        const int r = lane, node = pos0 + r - wk.q.ctx;
        if (r < KS && node >= 0 && node < wk.q.n) {
          bool found = false;
#pragma unroll 1
          for (int c = 0; c < CC; ++c) {
            uint4* const v = reinterpret_cast<uint4*>(values + value_at(r, c));
            const uint4 x = *v, n = make_uint4(nan_codes(x.x), nan_codes(x.y), nan_codes(x.z), nan_codes(x.w));
            if (n.x | n.y | n.z | n.w) {
              *v = make_uint4(x.x & ~n.x, x.y & ~n.y, x.z & ~n.z, x.w & ~n.w);
              found = true;
            }
          }
          if (found) atomicOr(&ct.bad[seq & 7], 1ull << node);
        }
        __syncwarp();
      }
      // scores: keys 16 mt + g and + 8, query rows 8 nt + 2 t and + 1
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint4 x[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) x[mt][h] = *reinterpret_cast<const uint4*>(keys + key_at(16 * mt + 8 * h + g, i * 4 + t));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint2 b[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) b[nt] = query[(nt * STEPS + i * 4 + w) * 32 + lane];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t w0 = w == 0 ? x[mt][0].x : w == 1 ? x[mt][0].y : w == 2 ? x[mt][0].z : x[mt][0].w;
            const uint32_t w1 = w == 0 ? x[mt][1].x : w == 1 ? x[mt][1].y : w == 2 ? x[mt][1].z : x[mt][1].w;
            uint32_t a0, a1, a2, a3;
            pairs<FMT>(w0, a0, a2);
            pairs<FMT>(w1, a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16x8x16(s[mt][nt], a0, a1, a2, a3, b[nt].x, b[nt].y);
          }
        }
      }
      // powers of two with the value's scale in them (the tensor memory kernel's softmax says how)
      float inv[MT][2], top[NT][2];
      bool no_value[MT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * mt + 8 * h + g;
          const float ks = scale_of(sc[r], flags), vs = value_scale(sc[KS + r], flags);
          float log;
          asm("lg2.approx.f32 %0, %1;" : "=f"(log) : "f"(vs));
          asm("rcp.approx.f32 %0, %1;" : "=f"(inv[mt][h]) : "f"(vs));
          no_value[mt][h] = vs == 0.f;  // such values are zeros (and NaN, where a code is: 0 times it)
          if (vs == 0.f) log = kNoValueLog, inv[mt][h] = kNoValueInverse;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[mt][nt][2 * h + e] = fmaf(s[mt][nt][2 * h + e], ks * factor[nt][e], log);
          if (!all) {
            const int pos = pos0 + r, node = pos - wk.q.ctx;
            const bool there = pos < k1 && !(hole >> r & 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int mi = m0 + min(nt * 8 + 2 * t + e, rows - 1), n = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi;
                const bool seen = there && (node < 0 || (a.tree_mask ? (__ldg(a.tree_mask + wk.q.s + n) >> (node & 63) & 1) != 0 : node <= n));
                if (!seen) s[mt][nt][2 * h + e] = -INFINITY;
              }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) top[nt][e] = fmaxf(top[nt][e], s[mt][nt][2 * h + e]);
        }
      bool far = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) far |= top[nt][e] > -INFINITY && !(top[nt][e] - m[nt][e] <= kRescale<MOE_F16>);
      if (__any_sync(0xffffffffu, far)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], x));
            // row by row: what the rows beside it do leaves a row's bits as they are
            if (m[nt][e] == -INFINITY) {
              m[nt][e] = top[nt][e];  // every weight so far was 0
            } else if (top[nt][e] - m[nt][e] > kRescale<MOE_F16>) {
              const float f = exp2_fast(m[nt][e] - top[nt][e]);
              m[nt][e] = top[nt][e];
              l[nt][e] *= f;
#pragma unroll
              for (int i = 0; i < OT; ++i) {
                o[i][nt][e] *= f;
                o[i][nt][2 + e] *= f;
              }
            }
          }
      }
      uint32_t b[MT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float shift0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kBias<MOE_F16>;
        const float shift1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kBias<MOE_F16>;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float e0 = exp2_fast(s[mt][nt][2 * h] - shift0), e1 = exp2_fast(s[mt][nt][2 * h + 1] - shift1);
            l[nt][0] = fmaf(e0, inv[mt][h], l[nt][0]);
            l[nt][1] = fmaf(e1, inv[mt][h], l[nt][1]);
            b[mt][nt][h] = transposed(no_value[mt][h] ? 0u : pack2<MOE_F16>(e0, e1));
          }
      }
      // sums: elements (g + 8 i) 16 + 4 w + 2 u and the next (D = 64: 8 g + 4 w + 2 u), rows as above
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        constexpr int WORDS = D == 64 ? 2 : 4;
#pragma unroll
        for (int i = 0; i < (D == 64 ? 1 : D / 128); ++i) {
          uint32_t y[4][WORDS];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * mt + 2 * t + (r & 1) + (r >> 1) * 8;
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(values + value_at(row, g >> 1) + (g & 1) * 8);
              y[r][0] = v.x;
              y[r][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(values + value_at(row, g + 8 * i));
              y[r][0] = v.x;
              y[r][1] = v.y;
              y[r][2 % WORDS] = v.z;
              y[r][3 % WORDS] = v.w;
            }
          }
#pragma unroll
          for (int w = 0; w < WORDS; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const unsigned sel = u ? 0x7362 : 0x5140;
              uint32_t a0, a1, a2, a3;
              pairs<FMT>(__byte_perm(y[0][w], y[1][w], sel), a0, a1);
              pairs<FMT>(__byte_perm(y[2][w], y[3][w], sel), a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16x8x16(o[i * 8 + w * 2 + u][nt], a0, a1, a2, a3, b[mt][nt][0], b[mt][nt][1]);
            }
        }
      }
      if (STAGES == 2) {
        __syncwarp();
        ask(j + 2, stage);
      }
      if (++stage == STAGES) stage = 0;
    }

    // ---- the warps' parts together
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
        if (g == 0) ml[warp * F::ROWS + nt * 8 + 2 * t + e] = make_float2(m[nt][e], l[nt][e]);
      }
    __syncthreads();  // every warp is done with its stages
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        const int d = D == 64 ? 8 * g + 2 * i : (g + (i >> 3) * 8) * 16 + 2 * (i & 7);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(sums + (warp * F::ROWS + nt * 8 + 2 * t + e) * F::kPitch + d) = make_float2(o[i][nt][e], o[i][nt][2 + e]);
      }
    __syncthreads();
    const unsigned long long bad = FMT == MOE_E4M3 ? *(volatile unsigned long long*)&ct.bad[seq & 7] : 0;
    const int part = wk.t0 == 0;
    const long long slot = (long long)blockIdx.x * 2 + part;
#pragma unroll 1
    for (int i = tid; i < rows * (D / 4); i += W * 32) {
      const int r = i / (D / 4), c4 = i % (D / 4), mi = m0 + r, n = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi, head = wk.h * G + mi - n * G;
      float top = -INFINITY, total = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * F::ROWS + r].x);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 v = ml[w * F::ROWS + r];
        const float f = v.x == -INFINITY ? 1.f : exp2_fast(v.x - top);  // nothing seen: zeros, or NaN that has to stay
        const float4 y = *reinterpret_cast<const float4*>(sums + (w * F::ROWS + r) * F::kPitch + c4 * 4);
        total = fmaf(v.y, f, total);
        x[0] = fmaf(y.x, f, x[0]);
        x[1] = fmaf(y.y, f, x[1]);
        x[2] = fmaf(y.z, f, x[2]);
        x[3] = fmaf(y.w, f, x[3]);
      }
      const uint64_t tree = a.tree_mask ? __ldg(a.tree_mask + wk.q.s + n) : n >= 63 ? ~0ull : (2ull << n) - 1;
      if (bad & tree) {
#pragma unroll 1
        for (int nd = 0; nd < kTree; ++nd) {
          if (!((bad & tree) >> nd & 1)) continue;
          const int pos = wk.q.ctx + nd, pc = pos / a.cache.page_size, page = __ldg(table + pc);
          const uint32_t w = nan_codes(*reinterpret_cast<const uint32_t*>(
              static_cast<const uint8_t*>(a.cache.v) + page * a.cache.page_stride + (pos - pc * a.cache.page_size) * a.cache.slot_stride +
              wk.h * a.cache.head_stride + c4 * 4));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (w >> (8 * e) & 1) x[e] = __uint_as_float(0x7fffffffu);
        }
      }
      if (whole) {
        const float div = total == 0.f ? 0.f : 1.f / total;
        const auto result2 = [&](float y, float z) { return a.dtype == MOE_BF16 ? pack2<MOE_BF16>(y, z) : pack2<MOE_F16>(y, z); };
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (long long)(wk.q.s + n) * a.out_stride + (long long)head * D + c4 * 4) =
            make_uint2(result2(x[0] * div, x[1] * div), result2(x[2] * div, x[3] * div));
        if (c4 == 0 && a.lse)
          a.lse[(long long)(wk.q.s + n) * a.q_heads + head] = total == 0.f ? -INFINITY : (top - kBias<MOE_F16> + log2f(total)) * 0.6931471805599453f;
      } else {
        __stcg(p.part + (slot * (D / 4) + c4) * p.part_rows + r, make_float4(x[0], x[1], x[2], x[3]));
        if (c4 == 0) __stcg(p.part_ml + slot * p.part_rows + r, make_float2(top, total));
      }
    }
    __syncthreads();
    if (!whole && tid == 0)  // releases what the block wrote before the barrier
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.arrive + ct.split[part].first * ct.groups + member) : "memory");
    ++seq;
  }
}

}  // namespace
}  // namespace moe
