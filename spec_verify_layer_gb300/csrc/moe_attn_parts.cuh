// Parts that the attention kernels over a paged cache share (moe_tree_attn.cuh, moe_few_rows.cuh): barriers,
// the list of work and its shares, the plan, codes of a cache in 8 bits.
#pragma once

#include <atomic>
#include <type_traits>

#include "moe_round_ops.cuh"

namespace moe {

inline std::atomic<unsigned long long> g_attention_wait_ns{2000000000ull};

namespace {

constexpr int kTree = 64;
constexpr int kThreads = 384;  // 8 softmax warps, 3 producer warps, 1 issuing warp: 168 registers a thread
constexpr int kSoftmaxThreads = 256, kProducers = 3;
constexpr int kMaxBlocks = 160;         // workspace sizing; the launch takes min(SM count, this)
constexpr int kMaxSlots = 10;
// Weights are 2^(score - maximum + kBias), and a maximum may lag 2^kRescale behind.  fp16 has few
// places below 1: a weight under 2^-14 loses bits and one under 2^-25 would be 0, while the sum,
// in 32 bits, holds it, so a long flat tail beside one strong key would vanish from the result
// alone.  The places above 1 are used for it (2^15 at most, then): what is lost are weights under
// 2^-32 of the largest.  (A smaller lag leaves room for a larger bias, but more tiles are gone
// through again: 33 ragged requests 55.6 us with 8 and 7, 57.3 with 7 and 8, 62.1 with 5 and
// 10; 55.0 with 14 and none.)  bf16 has the exponents of 32 bits and needs no bias.
template <int DT>
constexpr float kBias = DT == MOE_F16 ? 7.0f : 0.0f;
template <int DT>
constexpr float kRescale = DT == MOE_F16 ? 8.0f : 14.0f;
constexpr unsigned long long kWaitNs = 2000000000ull;  // a wait gives up after 2 s
constexpr long long kCyclesPerNs = 2;  // waits count SM cycles: ns at 2 GHz, a few times ns at lower clocks

template <int D>
constexpr int kKeyTile = D == 256 ? 64 : 128;  // keys of a tile in shared memory

// A is the call's descriptor: moe_tree_attention_args (a cache of 16-bit elements, which the tensor
// cores take as they are) or moe_tree_attention8_args (codes, which producers turn into fp16).
template <typename A>
constexpr bool kQ8 = std::is_same_v<A, moe_tree_attention8_args>;

template <typename A, int D>
struct Shape {
  static constexpr int KT = kKeyTile<D>;
  static constexpr int NS = D == 256 ? 1 : 2;          // streams (tensor memory holds 512 columns)
  static constexpr int PARTS = KT / 64;                // the weights are handed over 64 keys at a time
  static constexpr int MG = 128 * NS;                  // query rows of a group
  static constexpr int kSlot = KT * D * 2;             // bytes of a key or value tile
  static constexpr int kQ = 128 * D * 2;               // bytes of a query tile
  static constexpr int CPR = D / 8;                    // 16-byte chunks of a query row
  static constexpr int CC = kQ8<A> ? D / 16 : D / 8;   // and of a cached row
  static constexpr int RPI = 32 / CC;                  // rows that a warp copies with one instruction
  static constexpr int STEPS = (KT / RPI + kProducers - 1) / kProducers;  // instructions of a producer for a tile
  // Codes: scale of the key, logarithm and reciprocal of the value's scale, of each key of kRing tiles (a
  // tile's are written when its slot of keys is free, up to half the slots ahead of the softmax); a
  // factor a query row; page and scales of the rows that a producer's lane looks up, twice; codes on
  // their way, a stage for a tile's keys or values.
  static constexpr int LOOKS = (STEPS * RPI + 31) / 32;  // rows of a producer that a lane looks up
  static constexpr int kRing = D == 64 ? 8 : 4;
  static constexpr int kRaw = KT * D, kRawStages = 3;
  static constexpr int kLooked = kProducers * 2 * 3 * LOOKS * 32;
  static constexpr int kScales = kQ8<A> ? (kRing * 3 * KT + 256 + kLooked) * 4 + kRawStages * kRaw : 0;
  // Columns of tensor memory.  Scores: a buffer for each stream (or two that take turns where
  // there is one stream); the weights, in 16 bits, go over the second half of their scores.
  __host__ __device__ static constexpr int s_col(int buf) { return NS == 2 ? 256 * buf : 64 * buf; }
  __host__ __device__ static constexpr int p_col(int buf) { return s_col(buf) + KT / 2; }
  __host__ __device__ static constexpr int o_col(int s) { return NS == 2 ? 256 * s + 128 : 256; }
};

struct Plan {  // host-computed, the same for every block
  int nq;      // query tiles held
  int nslot;
  int group;   // query heads of a key/value head
  int part_rows;
  unsigned group_mul;  // n / group = umulhi(n, group_mul); 0: group is 1
  unsigned page_mul;
  int page_shift;
  int flip;    // of the queries: 1 negated (a negative scale), 2 taken as 0 (a scale of 0)
  float c;     // |scale| * log2(e); codes: 1 (scores are made powers of two key by key)
  float score; // codes: scale * log2(e), times what a code's fp16 number has to be multiplied with
  int block_shift;  // codes: log2 of the tokens of a block
  float4* part;      // [blocks][2: as Control::split][D / 4][part_rows]: a warp's rows side by side
  float2* part_ml;   // [blocks][2][part_rows]: maximum, sum
  unsigned* arrive;  // [blocks]
  unsigned* done;    // [blocks]
  long long wait_cycles;  // bound of a wait
};

struct Split {  // a head that is split over blocks: its request's rows, its first block, how many
  int s, n, h, first, parts;
};

struct Control {
  unsigned long long full[kMaxSlots], empty[kMaxSlots];
  unsigned long long s_full[2], p_full[4], o_done[2], q_ready, drain;  // p_full: [buffer][part]
  unsigned long long bad[8];          // per unit: tree rows with values that are not finite
  __align__(16) unsigned hole[8][8];  // per tile: rows without a page, two words for each producer's rows (codes: a bit a run)
  int red[kThreads / 32], redn[kThreads / 32];
  // the block's share of the list: places [w0, w1) of total, from start_off of request start_b on
  int total, w0, w1, start_off;
  int start_b, gangs, groups, gang, member;
  Split split[2];  // of the share's units: one that began in a share before, one that goes on in the next
  unsigned tmem;
  int abort;
  long long wait_cycles;  // as the plan's
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(unsigned long long* b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase of `parity` to end; false once any wait of the block gave up.
__device__ __forceinline__ bool bar_wait_slow(uint32_t b, uint32_t parity, Control& ct, unsigned* status) {
  const long long t0 = clock64();
  while (!bar_try(b, parity)) {
    if (*(volatile int*)&ct.abort) return false;
    if (clock64() - t0 > *(volatile long long*)&ct.wait_cycles) {
      *(volatile int*)&ct.abort = 1;
      atomicOr(status, MOE_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool bar_wait(unsigned long long* b, uint32_t parity, Control& ct, unsigned* status) {
  if (bar_try(smem_u32(b), parity)) return true;
  return bar_wait_slow(smem_u32(b), parity, ct, status);
}
// The last wait, for products in flight: they end by themselves, whatever other waits of the block
// gave up, and until they have the block may neither free tensor memory nor leave.
__device__ __forceinline__ void bar_drain(unsigned long long* b, unsigned* status) {
  const long long t0 = clock64();
  while (!bar_try(smem_u32(b), 0)) {
    if (clock64() - t0 > (long long)kWaitNs * kCyclesPerNs) {
      atomicOr(status, MOE_DEV_TIMEOUT);
      return;
    }
  }
}
// Barrier of the softmax warps; true if all of them said so.
__device__ __forceinline__ bool named_all(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand in the 128-byte swizzle: address, bytes between 64-element blocks
// (read where the operand is stored along its M or N), bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t block_bytes) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)((block_bytes >> 4) & 0x3fff) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
template <int DT>
__host__ __device__ constexpr uint32_t instruction(int n, bool b_along_n) {
  const uint32_t fmt = DT == MOE_BF16 ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (b_along_n ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned long long* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
// One lane of a warp whose lanes are all here.
__device__ __forceinline__ bool elected() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// The registers of a load are ready after tm_wait; `ready` makes their users wait for it
// (a volatile statement alone would not keep plain arithmetic behind it).
__device__ __forceinline__ void tm_load(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void ready(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tm_read(uint32_t* r, uint32_t addr) {
  tm_load(r, addr);
  tm_wait();
  ready(r);
}
__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_store2(uint32_t addr, float x, float y) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(addr), "r"(__float_as_uint(x)),
               "r"(__float_as_uint(y))
               : "memory");
}
__device__ __forceinline__ float2 tm_load2(uint32_t addr) {
  uint32_t x, y;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(x), "=r"(y)
               : "r"(addr)
               : "memory");
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ void tm_read16(float* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// ---- the list of work -----------------------------------------------------------------

struct Req {
  int s, n, ctx, tiles;  // first row, rows, context; tiles 0: nothing to do
};

template <int D, typename A>
__device__ __forceinline__ Req request(const A& a, int b) {
  Req q;
  q.s = __ldg(a.row_start + b);
  const int e = __ldg(a.row_start + b + 1);
  q.ctx = __ldg(a.ctx_len + b);
  const bool rows_ok = q.s >= 0 && e >= q.s && e <= a.n_rows;
  q.n = rows_ok ? e - q.s : -1;
  q.tiles = 0;
  if (q.n > 0 && q.n <= a.max_tree && q.ctx >= 0 &&
      (long long)q.ctx + q.n <= min((long long)a.table_width * a.cache.page_size, 0x7fffffffll - 256))
    q.tiles = (q.ctx + q.n + kKeyTile<D> - 1) / kKeyTile<D>;
  return q;
}

// Taking up a head costs about as long as a few tiles (its queries, the first scores, the end
// of its sums), so in the list each head has kUnit places ahead of those of its tiles: with
// 0 a ragged batch of 33 requests took 100.5 us, with 2 68.8, with 3 60.8, with 5 60.0; one
// row over 1,000 keys 14.2 with 3, 13.3 with 4.
constexpr int kUnit = 4;

template <typename A, int D>
struct Walk {  // a block's share, unit (stretch of one head's tiles) after unit
  Req q;
  int b, h, p0, p1;  // places of the head
  int t0, t1;        // its tiles; none where the share has only the head's first places
  int left;          // places left in the share, this unit's among them
  __device__ __forceinline__ void tiles() {
    p1 = min(q.tiles + kUnit, p0 + left);
    t0 = max(0, p0 - kUnit);
    t1 = max(0, p1 - kUnit);
  }
  __device__ __forceinline__ void begin(const A& a, int b_, int off, int left_) {
    left = left_;
    b = b_;
    if (left <= 0) return;
    q = request<D>(a, b);
    h = off / (q.tiles + kUnit);
    p0 = off - h * (q.tiles + kUnit);
    tiles();
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const A& a) {
    left -= p1 - p0;
    if (left <= 0) return;
    p0 = 0;
    if (++h == a.kv_heads) {
      h = 0;
      do {
        if (++b >= a.n_req) {  // not while the lengths stay as they were
          left = 0;
          return;
        }
        q = request<D>(a, b);
      } while (q.tiles == 0);
    }
    tiles();
  }
};

// Shares of the list: floor(total * g / gangs) to floor(total * (g + 1) / gangs); where equal
// heads divide the blocks no share crosses from one head to the next.
__device__ __forceinline__ int share(int total, int gangs, int g) {
  const int each = total / gangs;
  return each * g + (total - each * gangs) * g / gangs;
}
__device__ __forceinline__ int gang_of(int total, int gangs, int x) {
  return (int)((((unsigned long long)x + 1) * gangs - 1) / (unsigned)total);
}

// ---- codes ------------------------------------------------------------------------------

// Eight codes (two words) as fp16 numbers, exactly.  int8: 1024 + (code + 128) has the code in its
// last bits; 1152 is taken off again.
template <int FMT>
__device__ __forceinline__ uint4 codes_to_half(uint32_t a, uint32_t b) {
  uint32_t r[4];
  const uint32_t w[2] = {a, b};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (FMT == MOE_I8) {
      const uint32_t u = w[j] ^ 0x80808080u;
      const __half2 off = __half2half2(__ushort_as_half(0x6480));
      const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
      const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&lo), off), y = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
      r[2 * j] = *reinterpret_cast<const uint32_t*>(&x);
      r[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
          : "=r"(r[2 * j]), "=r"(r[2 * j + 1])
          : "r"(w[j]));
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Values whose scale counts as 0 are zeros of the smallest scale, so that their weights, which count in the
// sum, stay below those of any other.
constexpr float kNoValueLog = -48.f, kNoValueInverse = 281474976710656.f;
// A value's scale: 2^-48 .. 2^48.  The weights' sum is taken from the weights with the scales in them, so
// these may not lie further apart than 32-bit exponents reach; smaller ones count as 0 (their
// values are below 1.6e-12), larger ones too and are reported.
__device__ __forceinline__ float value_scale(float s, unsigned& flags) {
  s = scale_of(s, flags);
  if (s > 281474976710656.f) flags |= MOE_DEV_VALUE;
  return s >= 3.552713678800501e-15f && s <= 281474976710656.f ? s : 0.f;
}
// Bytes of four e4m3 codes that are NaN, as 0xff.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  const uint32_t high = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (high >> 7) * 0xffu;
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

}  // namespace
}  // namespace moe
