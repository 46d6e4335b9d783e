// Attention of drafted rows over a paged cache (moe_tree_attention), one cooperative
// launch of one block per SM.
//
// Work.  The n rows of a request and the G query heads of one key/value head make n * G
// query rows that read the same keys: one group of up to 256 (two tensor-core tiles of
// 128 rows), so each key and value is read once a group.  The keys are cut into tiles of
// kKT; (request, head, tile) in that order is one list, and every block takes an equal,
// contiguous share of it, computed by each block from the lengths (no host plan, nothing
// to synchronise, ragged lengths balance).  More than 256 query rows: that many groups
// share each stretch of the list, in blocks side by side that read the same tiles at the
// same time, the second out of L2.
//
// In a block, four roles meet at mbarriers:
//   - three producer warps copy key and value rows (cp.async, 16 bytes a lane, page table
//     looked up per row) into a ring of shared-memory slots in the 128-byte swizzle that
//     the tensor cores read;
//   - one warp issues the products: S = Q K^T into tensor memory, and O += P V with P
//     read from tensor memory and V from its slot as it lies (no transpose is stored);
//   - two warpgroups do the softmax, a thread per query row: S out of tensor memory,
//     running maximum and sum in registers, P back over S as 16-bit weights.
// Two streams (S, P, O of their own) keep the tensor cores and the exponentials busy at
// once: two row tiles of 128 over the same keys, or, with up to 128 rows, even and odd
// key tiles over the same rows, joined when the share of the head ends.  A head's keys
// split over blocks leave unnormalised sums with their maximum in the workspace; when the
// last of its blocks has arrived, each of them joins some of the rows, in block order.
//
// Running maximum: it is the largest of the first scores seen, and moves only when a score is
// above it by more than 2^14 (bf16) or 2^8 (fp16, see kBias).  So a tile's weights need no pass
// over its scores for the maximum first (full trees 302 us with such a pass, 280 without;
// 296 with 2^8 as the threshold); a tile that moves a row's maximum is gone through again, with O rescaled.
//
// What it takes (GB300, one launch in a stream of them): full trees (40 and 64 rows of 32/4 heads
// of 128 over 131,071 and 200,001 keys) 258 us, 1,090 TFLOP/s of the 1,975 that a large library
// product reaches, 2.7 TB/s; the same of 16/2 heads of 256, 322 us; 64 requests of one row over
// 8,192 keys each 177.6 us, 6.0 TB/s; 16 rows of one request over 32,768 keys 26.7 us, 2.5
// TB/s; 33 ragged requests of 16/8 heads of 64 in fp16, 55.9 us, 3.7 TB/s; one row over 1,000
// keys 12.3 us (10.4 in a graph).
// Full trees are bound by the chain of a stream (of the 3,110 cycles of a tile in both streams:
// scores out to weights back 1,700 to 1,900, products and scores of the next 1,200 to 1,400).
// The tensor cores work 2,048 of them, 64 for each product of 128 x 128 x 16, which is their
// full rate (8,192 operations a cycle); in the rest no product is in flight, since a stream's
// softmax, which waits for its own loads, maxima and exponentials one after the other, takes
// longer than the 1,024 cycles of the other stream's products.  Ragged batches pay for 128 rows
// where a group has 48 at most and 24 on average.  The others are bound by latency: some 6 us
// from the launch to the first weights (lengths, page table, keys and, on the same barrier,
// values: one after the other from memory, and code that is fetched for the first time), and
// 3.5 us for the join of a split head.
//
// Tried and slower: scores of 64 keys in two buffers a stream (full trees 507 us against 372
// of that time: the tensor cores read a query tile for each product, whatever its width);
// two threads a row, 16 softmax warps (377 against 304); the softmax unrolled over a whole
// tile (393: it spills); looking at the next barriers between two products (340 against 283:
// products are issued as they are done, and what stands between them is added to the
// chain) or at all that a stream waits for in one go (267 against 260); the first half's
// weights handed over in the middle of the second half's exponentials (263 against 256).
//
// What is not seen gets the weight 0, but 0 times a cached NaN would still be NaN in the
// product: slots past the last position are zero-filled, and the values of drafted rows
// are looked over on their way: what is not finite becomes 0 in the slot and is added at
// the end to the rows that see it.
#include <atomic>

#include "moe_round_ops.cuh"

namespace moe {
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
std::atomic<unsigned long long> g_wait_ns{kWaitNs};

template <int D>
struct Shape {
  static constexpr int KT = D == 256 ? 64 : 128;       // keys of a tile in shared memory
  static constexpr int NS = D == 256 ? 1 : 2;          // streams (tensor memory holds 512 columns)
  static constexpr int PARTS = KT / 64;                // the weights are handed over 64 keys at a time
  static constexpr int MG = 128 * NS;                  // query rows of a group
  static constexpr int kSlot = KT * D * 2;             // bytes of a key or value tile
  static constexpr int kQ = 128 * D * 2;               // bytes of a query tile
  static constexpr int CPR = D / 8;                    // 16-byte chunks of a row
  static constexpr int RPI = 32 / CPR;                 // rows that a warp copies with one instruction
  static constexpr int STEPS = (KT / RPI + kProducers - 1) / kProducers;  // instructions of a producer for a tile
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
  float c;     // |scale| * log2(e)
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
  __align__(16) unsigned hole[8][8];  // per tile: rows without a page, two words for each producer's rows
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

template <int D>
__device__ __forceinline__ Req request(const moe_tree_attention_args& a, int b) {
  Req q;
  q.s = __ldg(a.row_start + b);
  const int e = __ldg(a.row_start + b + 1);
  q.ctx = __ldg(a.ctx_len + b);
  const bool rows_ok = q.s >= 0 && e >= q.s && e <= a.n_rows;
  q.n = rows_ok ? e - q.s : -1;
  q.tiles = 0;
  if (q.n > 0 && q.n <= a.max_tree && q.ctx >= 0 &&
      (long long)q.ctx + q.n <= min((long long)a.table_width * a.cache.page_size, 0x7fffffffll - 256))
    q.tiles = (q.ctx + q.n + Shape<D>::KT - 1) / Shape<D>::KT;
  return q;
}

// Taking up a head costs about as long as a few tiles (its queries, the first scores, the end
// of its sums), so in the list each head has kUnit places ahead of those of its tiles: with
// 0 a ragged batch of 33 requests took 100.5 us, with 2 68.8, with 3 60.8, with 5 60.0; one
// row over 1,000 keys 14.2 with 3, 13.3 with 4.
constexpr int kUnit = 4;

template <int D>
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
  __device__ __forceinline__ void begin(const moe_tree_attention_args& a, int b_, int off, int left_) {
    left = left_;
    b = b_;
    if (left <= 0) return;
    q = request<D>(a, b);
    h = off / (q.tiles + kUnit);
    p0 = off - h * (q.tiles + kUnit);
    tiles();
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const moe_tree_attention_args& a) {
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

// ---- the kernel -------------------------------------------------------------------------

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_tree_attn(const __grid_constant__ moe_tree_attention_args a, const __grid_constant__ Plan p) {
  using Sh = Shape<D>;
  constexpr int KT = Sh::KT, NS = Sh::NS, CPR = Sh::CPR, RPI = Sh::RPI;
  constexpr uint32_t kBlk = KT * 128;  // bytes of a 64-element block of a key or value tile
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sm_q = smem;
  unsigned char* sm_kv = smem + (size_t)p.nq * Sh::kQ;
  Control& ct = *reinterpret_cast<Control*>(sm_kv + (size_t)p.nslot * Sh::kSlot);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group;

  // total work, the widest request, and the request that holds this block's first place
  unsigned flags = 0;
  int total = 0, maxn = 0, lo, mine;
  Req first{0, 0, 0, 0};
  if (tid < a.n_req) first = request<D>(a, tid);
  if (tid == 0 && __ldg(a.row_start) != 0) flags |= MOE_DEV_LENGTH;
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 11) {
    if (lane < p.nslot) {
      bar_init(&ct.full[lane], 33 * kProducers);  // a warp's copies, and what its first lane wrote
      bar_init(&ct.empty[lane], 1);
    }
    if (lane < 4) bar_init(&ct.p_full[lane], 4);
    if (lane < 2) {
      bar_init(&ct.s_full[lane], 1);
      bar_init(&ct.o_done[lane], 1);
    }
    if (lane == 0) {
      bar_init(&ct.q_ready, kSoftmaxThreads / 32);
      bar_init(&ct.drain, 1);
      ct.abort = 0;
      ct.wait_cycles = p.wait_cycles;
      ct.split[0].parts = ct.split[1].parts = 0;
    }
    if (lane < 8) ct.bad[lane] = 0;
    (&ct.hole[0][0])[lane] = (&ct.hole[0][0])[lane + 32] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const auto scan = [&](int b0, const Req& q) {  // lo: places before request b0 + tid, mine: its own
    mine = q.tiles ? (q.tiles + kUnit) * a.kv_heads : 0;
    int incl = mine;
    const int widest = __reduce_max_sync(0xffffffffu, q.tiles ? q.n : 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (b0) __syncthreads();  // red is read below
    if (lane == 31) {
      ct.red[warp] = incl;
      ct.redn[warp] = widest;
    }
    __syncthreads();
    lo = total + incl - mine;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      const int x = ct.red[i];
      if (i < warp) lo += x;
      total += x;
      maxn = max(maxn, ct.redn[i]);
    }
  };
  scan(0, first);
  for (int b0 = kThreads; b0 < a.n_req; b0 += kThreads) {
    Req q{0, 0, 0, 0};
    if (b0 + tid < a.n_req) q = request<D>(a, b0 + tid);
    scan(b0, q);
  }
  {
    const int groups = max(1, (maxn * G + Sh::MG - 1) / Sh::MG);
    const int gangs = min(total, max(1, (int)gridDim.x / groups));
    const int gang = (int)blockIdx.x / groups;
    const bool works = gang < gangs && groups <= (int)gridDim.x;
    const int w0 = works ? share(total, gangs, gang) : 0, w1 = works ? share(total, gangs, gang + 1) : 0;
    if (tid == 0) {
      ct.total = total;
      ct.w0 = w0;
      ct.w1 = w1;
      ct.groups = groups;
      ct.gangs = gangs;
      ct.gang = gang;
      ct.member = (int)blockIdx.x - gang * groups;
    }
    if (works && a.n_req > kThreads) {  // the sums again, up to that request
      total = 0;
      for (int b0 = 0; b0 < a.n_req && total <= w0; b0 += kThreads) {
        __syncthreads();
        Req q{0, 0, 0, 0};
        if (b0 + tid < a.n_req) q = request<D>(a, b0 + tid);
        scan(b0, q);
        if (w0 >= lo && w0 < lo + mine) {
          ct.start_b = b0 + tid;
          ct.start_off = w0 - lo;
        }
      }
    } else if (works && w0 >= lo && w0 < lo + mine) {
      ct.start_b = tid;
      ct.start_off = w0 - lo;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ct.tmem;
  Walk<D> wk;
  const int member = ct.member;
  wk.begin(a, ct.start_b, ct.start_off, ct.w1 - ct.w0);

  if (warp == 8 || warp == 9 || warp == 11) {
    // ---------------- producers: step k of a warp copies the rows [g RPI, (g + 1) RPI) of a tile,
    // g = k * kProducers + its number
    const int pw = warp == 11 ? 2 : warp - 8, chunk = lane % CPR, sub = lane / CPR;
    constexpr int LOOKS = (Sh::STEPS * RPI + 31) / 32;  // rows of a warp that a lane looks up
    constexpr uint32_t kNone = 0xffffffffu;
    const uint32_t kv0 = smem_u32(sm_kv);
    int slot = 0, tile_seq = 0;
    uint32_t phase = 1;  // the slots start empty
    bool ok = true;
    for (int seq = 0; ok && wk.more(); wk.next(a)) {
      if (wk.q.n * G <= member * Sh::MG || wk.t0 == wk.t1) continue;
      const int len = wk.q.ctx + wk.q.n;
      const int32_t* table = a.block_table + (long long)wk.b * a.table_width;
      const long long head_at = wk.h * a.cache.head_stride;
      if (pw == 2 && !(wk.t0 == 0 && wk.t1 == wk.q.tiles)) {  // who shares this head: read when the unit ends
        const int at = ct.w1 - wk.left - wk.p0 + kUnit;       // the place of the head's first tile
        const int first = gang_of(ct.total, ct.gangs, at), last = gang_of(ct.total, ct.gangs, at + wk.q.tiles - 1);
        if (lane == 0) ct.split[wk.t0 == 0] = {wk.q.s, wk.q.n, wk.h, first, last - first + 1};
      }
      // the table entries of this lane's rows, a tile ahead of their use
      int page[LOOKS];
      const auto look = [&](int t) {
#pragma unroll
        for (int j = 0; j < LOOKS; ++j) {
          const int mine = 32 * j + lane, r = (mine / RPI * kProducers + pw) * RPI + mine % RPI, pos = t * KT + r;
          page[j] = 0;
          if (r < KT && pos < len) page[j] = __ldg(table + (int)(((unsigned long long)(unsigned)pos * p.page_mul) >> p.page_shift));
        }
      };
      look(wk.t0);
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++tile_seq) {
        uint32_t at[LOOKS];  // places in the cache in units of 16 bytes
        unsigned hole[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < LOOKS; ++j) {
          const int mine = 32 * j + lane, r = (mine / RPI * kProducers + pw) * RPI + mine % RPI, pos = t * KT + r;
          const bool there = r < KT && pos < len, good = there && page[j] >= 0 && page[j] < a.cache.n_pages;
          const int col = (int)(((unsigned long long)(unsigned)pos * p.page_mul) >> p.page_shift);
          at[j] = good ? (uint32_t)((page[j] * a.cache.page_stride + (pos - col * a.cache.page_size) * a.cache.slot_stride +
                                     head_at) >> 3)
                       : kNone;
          hole[j] = __ballot_sync(0xffffffffu, there && !good);
        }
        if (hole[0] | hole[1]) flags |= MOE_DEV_INDEX;
        if (t + 1 < wk.t1) look(t + 1);
        // a row's place to the lanes that copy it; all of them ahead of the copies, which would
        // otherwise each wait for their own exchange
        uint32_t from[Sh::STEPS];
#pragma unroll
        for (int k = 0; k < Sh::STEPS; ++k)
          from[k] = __shfl_sync(0xffffffffu, LOOKS > 1 && k * RPI >= 32 ? at[LOOKS - 1] : at[0], (k * RPI + sub) & 31);
        const int v_slot = slot + 1 < p.nslot ? slot + 1 : 0;
        ok = bar_wait(&ct.empty[slot], phase, ct, a.dev_status) &&
             bar_wait(&ct.empty[v_slot], phase ^ (v_slot == 0), ct, a.dev_status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        {
          const uint4* k_src = static_cast<const uint4*>(a.cache.k) + chunk;
          const uint4* v_src = static_cast<const uint4*>(a.cache.v) + chunk;
          const uint32_t k_dst = kv0 + slot * Sh::kSlot + (chunk >> 3) * kBlk;
          const uint32_t v_dst = kv0 + v_slot * Sh::kSlot + (chunk >> 3) * kBlk;
#pragma unroll
          for (int k = 0; k < Sh::STEPS; ++k) {
            const int g = k * kProducers + pw, r = g * RPI + sub;
            const uint32_t to = r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
            const bool there = from[k] != kNone;
            const uint32_t off = there ? from[k] : 0;
            if ((k + 1) * kProducers <= KT / RPI || g < KT / RPI) {
              copy16(k_dst + to, k_src + off, there);
              copy16(v_dst + to, v_src + off, there);
            }
          }
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const int node0 = wk.q.ctx - t * KT;  // the tile's row of the first drafted one
          if (kv == 1 && node0 < KT) {
            // drafted rows' values: what is not finite is noted and taken out (a thread
            // looks over what it copied itself)
            asm volatile("cp.async.wait_all;" ::: "memory");
            const int from = max(node0, 0), to = min(KT, node0 + wk.q.n);
#pragma unroll 1
            for (int k = max(0, (from / RPI - pw) / kProducers); k < Sh::STEPS; ++k) {
              const int r = (k * kProducers + pw) * RPI + sub;
              if (r - sub >= to) break;
              if (r < from || r >= to) continue;
              uint4* v = reinterpret_cast<uint4*>(sm_kv + (size_t)slot * Sh::kSlot + (chunk >> 3) * kBlk + r * 128 +
                                                  (((chunk & 7) ^ (r & 7)) << 4));
              const uint4 x = *v;
              uint32_t w[4] = {x.x, x.y, x.z, x.w};
              constexpr uint32_t kExp = DT == MOE_BF16 ? 0x7f80u : 0x7c00u;
              bool found = false;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if ((w[j] & kExp) == kExp) {
                  w[j] &= 0xffff0000u;
                  found = true;
                }
                if ((w[j] >> 16 & kExp) == kExp) {
                  w[j] &= 0xffffu;
                  found = true;
                }
              }
              if (found) {
                *v = make_uint4(w[0], w[1], w[2], w[3]);
                atomicOr(&ct.bad[seq & 7], 1ull << (r - node0));
              }
            }
            __syncwarp();
            fence_async();
            bar_arrive(&ct.full[slot]);
          } else {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&ct.full[slot])) : "memory");
          }
          if (lane == 0) {
            if (kv == 0) *reinterpret_cast<uint2*>(&ct.hole[tile_seq & 7][2 * pw]) = make_uint2(hole[0], hole[1]);
            bar_arrive(&ct.full[slot]);  // behind what this lane wrote
          }
          __syncwarp();
          if (++slot == p.nslot) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      ++seq;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 10) {
    // ---------------- issue of the products.  The warp goes through the loop as one and one lane
    // of it issues, so that the operands, which are the same for all lanes, can be held as
    // such (issued by a thread on its own: full trees 283 us against 258).
    const auto same = [](auto v) { return __shfl_sync(0xffffffffu, v, 0); };
    {
      constexpr uint32_t id_s = instruction<DT>(KT, false), id_o = instruction<DT>(D, true);
      const uint64_t kv0 = operand(smem_u32(sm_kv), kBlk), q0 = operand(smem_u32(sm_q), 0);
      const uint32_t tm = same(tmem);
      int k_slot = 0, v_slot = 1;       // slots of the next key and value tile
      uint32_t k_ph = 0, v_ph = 0, p_par = 0, q_ph = 0;
      bool ok = true;
      const auto wait = [&](unsigned long long* b, uint32_t parity) {
        return __all_sync(0xffffffffu, bar_wait(b, parity, ct, a.dev_status)) != 0;
      };
      const auto commit = [&](unsigned long long* b) {
        if (elected()) mma_commit(b);
        __syncwarp();
      };
      const auto take = [&](int& s, uint32_t& ph) {  // key and value tiles take turns in the ring
        s += 2;
        if (s >= p.nslot) {
          s -= p.nslot;
          ph ^= 1;
        }
      };
      const auto wait_p = [&](int buf) {
        if (!wait(&ct.p_full[buf], p_par >> buf & 1)) return false;
        p_par ^= 1u << buf;
        fence_after();
        return true;
      };
      // (addresses in descriptors are in units of 16 bytes)
      const auto scores = [&](int buf, int qt) {  // S_buf = Q_qt K^T
        const uint64_t qa = q0 + qt * (Sh::kQ >> 4), kb = kv0 + k_slot * (Sh::kSlot >> 4);
        if (elected()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tm + Sh::s_col(buf), qa + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2,
                   kb + (k >> 2) * (kBlk >> 4) + (k & 3) * 2, id_s, k > 0);
          mma_commit(&ct.s_full[buf]);
        }
        __syncwarp();
      };
      const auto values = [&](int buf, int s, bool first, bool last) {  // O_s += P_buf V, as the parts come, the last keys first
        const uint64_t vb = kv0 + v_slot * (Sh::kSlot >> 4);
#pragma unroll
        for (int part = Sh::PARTS - 1; part >= 0; --part) {
          if (!wait_p(2 * buf + part)) return false;
          if (elected()) {
#pragma unroll
            for (int k = 4 * part; k < 4 * part + 4; ++k)
              mma_ts(tm + Sh::o_col(s), tm + Sh::p_col(buf) + k * 8, vb + k * (2048 >> 4), id_o,
                     !(first && k == 4 * (Sh::PARTS - 1)));
            if (part == 0 && (NS == 1 || last)) mma_commit(&ct.o_done[s]);
          }
          __syncwarp();
        }
        return true;
      };
      const auto wait_tile = [&](int slot, uint32_t ph) {
        if (!wait(&ct.full[slot], ph)) return false;
        fence_async();  // the copies were ordinary writes: order them before the tensor cores' reads
        return true;
      };
      const auto free_tile = [&](int& slot, uint32_t& ph) {
        commit(&ct.empty[slot]);
        take(slot, ph);
      };
      for (; ok && wk.more(); wk.next(a)) {
        const int rows = same(min(Sh::MG, wk.q.n * G - member * Sh::MG)), nt = same(wk.t1 - wk.t0);
        if (rows <= 0 || nt == 0) continue;
        const bool two = NS == 2 && rows > 128;
        if (!(ok = wait(&ct.q_ready, q_ph))) break;
        q_ph ^= 1;
        fence_after();
        if (two) {
          // both streams, tile after tile
          for (int t = 0; ok && t <= nt; ++t) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (t > 0) {
                ok = (s == 1 || wait_tile(v_slot, v_ph)) && values(s, s, t == 1, t == nt);
                if (!ok) break;
                if (s == 1) free_tile(v_slot, v_ph);
              }
              if (t < nt) {
                if (s == 0 && !(ok = wait_tile(k_slot, k_ph))) break;
                scores(s, s);
                if (s == 1) free_tile(k_slot, k_ph);
              }
            }
          }
        } else {
          // tiles take turns between the streams (or the score buffers of one)
          for (int t = 0; ok && t <= nt; ++t) {
            if (t < nt) {
              if (!(ok = wait_tile(k_slot, k_ph))) break;
              scores(t & 1, 0);
              free_tile(k_slot, k_ph);
            }
            if (t > 0) {
              ok = wait_tile(v_slot, v_ph) && values((t - 1) & 1, NS == 2 ? (t - 1) & 1 : 0, t <= NS, t >= nt - 1);
              if (!ok) break;
              free_tile(v_slot, v_ph);
            }
          }
        }
      }
      commit(&ct.drain);  // nothing runs on when the block ends, also where a wait gave up
      bar_drain(&ct.drain, a.dev_status);
      __syncwarp();
    }
  } else {
    // ---------------- softmax
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes of tensor memory
    const uint32_t q0 = smem_u32(sm_q);
    const float c = p.c;
    uint32_t s_par = 0, o_cnt = 0;  // phases of the scores' barriers, products behind this warp
    int tile_seq = 0;
    bool ok = true;
    for (int seq = 0; ok && wk.more(); wk.next(a)) {
      const int m0 = member * Sh::MG, rows = min(Sh::MG, wk.q.n * G - m0);
      if (rows <= 0 || wk.t0 == wk.t1) continue;
      const bool two = NS == 2 && rows > 128;
      // the group's queries into the swizzle, zeros in the rows of nobody (a rolled loop: it runs
      // once a unit, and its instructions have to come from memory the first time)
      const auto q_at = [&](int i) {
        const int r = i / CPR, ch = i % CPR;
        return q0 + (r >> 7) * Sh::kQ + (ch >> 3) * (128 * 128) + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4);
      };
#pragma unroll 1
      for (int i = tid; i < (two ? 256 : 128) * CPR; i += kSoftmaxThreads) {
        const int mi = min(m0 + i / CPR, m0 + rows - 1), n = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi, g = mi - n * G;
        copy16(q_at(i), static_cast<const uint16_t*>(a.q) + (long long)(wk.q.s + n) * a.q_stride + (wk.h * G + g) * D + i % CPR * 8,
               i < rows * CPR);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (p.flip) {
#pragma unroll 1
        for (int i = tid; i < rows * CPR; i += kSoftmaxThreads) {
          uint4* x = reinterpret_cast<uint4*>(smem + (q_at(i) - q0));
          *x = p.flip == 2 ? make_uint4(0, 0, 0, 0)
                           : make_uint4(x->x ^ 0x80008000u, x->y ^ 0x80008000u, x->z ^ 0x80008000u, x->w ^ 0x80008000u);
        }
      }
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&ct.q_ready);

      const int mr = (two ? wg * 128 : 0) + row;       // row of the group
      const bool live = (two ? wg * 128 : 0) + (warp & 3) * 32 < rows;  // any row of this warp
      uint64_t tree = 0;  // rows of the request that this one sees
      if (mr < rows) {
        const int mi = m0 + mr, i = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi;
        tree = a.tree_mask ? __ldg(a.tree_mask + wk.q.s + i) : i >= 63 ? ~0ull : (2ull << i) - 1;
      }
      const int len = wk.q.ctx + wk.q.n, nt = wk.t1 - wk.t0;
      float m = -INFINITY, l = 0.f;
      const bool mine_all = two || NS == 1;
      const int o = NS == 2 ? wg : 0;  // this warpgroup's stream
      if (NS == 2 || wg == 0) {
        const int step = mine_all ? 1 : 2, ti0 = mine_all ? 0 : wg;
        for (int ti = ti0; ok && ti < nt; ti += step) {
          const int buf = NS == 2 ? wg : ti & 1;
          ok = __all_sync(0xffffffffu, bar_wait(&ct.s_full[buf], s_par >> buf & 1, ct, a.dev_status));
          if (!ok) break;
          s_par ^= 1u << buf;
          fence_after();
          const auto hand_over = [&](int part) {
            if (live) tm_wait_store();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&ct.p_full[2 * buf + part]);
          };
          // The scores' barrier covers the stream's products up to this tile, except with one
          // stream, where the last one may still run: waited for here it is never two behind.
          const auto last_product = [&]() {
            if (NS == 1 && o_cnt > 0) {
              ok = __all_sync(0xffffffffu, bar_wait(&ct.o_done[0], (o_cnt - 1) & 1, ct, a.dev_status));
              if (ok) fence_after();
            }
            return ok;
          };
          if (live) {
            const int base = (wk.t0 + ti) * KT;
            // which of the tile's keys this row sees, unless it is all
            const unsigned* hole = ct.hole[(tile_seq + ti) & 7];
            const uint4 hole_a = *reinterpret_cast<const uint4*>(hole);
            const uint2 hole_b = *reinterpret_cast<const uint2*>(hole + 4);
            const bool holes = (hole_a.x | hole_a.y | hole_a.z | hole_a.w | hole_b.x | hole_b.y) != 0;
            const bool all = base + KT <= wk.q.ctx && !holes;
            const auto seen = [&](int w) {  // of keys 32 w .. 32 w + 31
              const int k = wk.q.ctx - base - 32 * w;  // context keys of the word
              unsigned bits = k >= 32 ? 0xffffffffu : k > 0 ? (1u << k) - 1 : 0u;
              if (k < 32) bits |= (unsigned)(k > 0 ? tree << k : k > -64 ? tree >> -k : 0ull);
              const int v = len - base - 32 * w;  // positions of the word
              bits = v >= 32 ? bits : v > 0 ? bits & ((1u << v) - 1) : 0u;
              if (holes) {
#pragma unroll 1
                for (int j = 0; j < 32; ++j) {
                  const int r = 32 * w + j, g = r / RPI, q = g / kProducers * RPI + r % RPI;
                  if (hole[2 * (g % kProducers) + (q >> 5)] >> (q & 31) & 1) bits &= ~(1u << j);
                }
              }
              return bits;
            };
            // 64 scores of a row in registers at a time, the last keys first (the weights go where
            // scores were that are read already).  Weights are taken from the running maximum as
            // it stands, or from the first scores seen; only when a score is above it by more
            // than the threshold, which the last scores' maximum tells before any weight is
            // handed over, the tile is gone through again.  The halves are a rolled loop and the
            // mask a branch inside: this code is fetched anew by every launch, and its length
            // shows in the short ones.
            uint32_t x[64];
            const auto fetch = [&](int half) {
              const uint32_t at = lanes + Sh::s_col(buf) + 64 * half;
              tm_load(x, at);
              tm_load(x + 32, at + 32);
              tm_wait();
              ready(x);
              ready(x + 32);
              if (!all) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  const unsigned bits = seen(2 * half + w);
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (!(bits >> j & 1)) x[32 * w + j] = 0xff800000u;
                }
              }
            };
            const Pair c2 = pair(c, c);
            Pair sums[2] = {0, 0};
            float top = -INFINITY;
            uint32_t y[32];
#pragma unroll 1
            for (int half = Sh::PARTS - 1; half >= 0; --half) {
              fetch(half);
              float tops[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int j = 0; j < 64; ++j) tops[j & 3] = fmaxf(tops[j & 3], __uint_as_float(x[j]));
              top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
              if (m == -INFINITY) m = top;  // every weight so far was 0
              if (half == 0) {
                const bool far = mr < rows && (top - m) * c > kRescale<DT>;
                if (__any_sync(0xffffffffu, far)) {
                  // row by row: what the rows beside it do leaves a row's bits as they are
                  const float f = far ? exp2_fast((m - top) * c) : 1.f;
                  if (ti > ti0) {  // O holds something
                    if (!last_product()) break;
#pragma unroll 1
                    for (int w = 0; w < D / 32; ++w) {
                      tm_read(y, lanes + Sh::o_col(o) + 32 * w);
#pragma unroll
                      for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                      tm_store32(lanes + Sh::o_col(o) + 32 * w, y);
                    }
                    tm_wait_store();
                  }
                  l *= f;
                  if (far) m = top;
                  sums[0] = sums[1] = 0;
                  half = Sh::PARTS;
                  continue;
                }
                if (Sh::PARTS > 1) {
                  tm_store32(lanes + Sh::p_col(buf) + 32, y);
                  hand_over(1);
                }
              }
              const float shift = m == -INFINITY ? 0.f : fmaf(m, c, -kBias<DT>);
              const Pair shift2 = pair(-shift, -shift);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float2 z = split(fma2(pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), c2, shift2));
                const float e0 = exp2_fast(z.x), e1 = exp2_fast(z.y);
                sums[j & 1] = add2(sums[j & 1], pair(e0, e1));
                y[j] = pack2<DT>(e0, e1);
              }
            }
            if (!ok) break;
            tm_store32(lanes + Sh::p_col(buf), y);
            const float2 sum = split(add2(sums[0], sums[1]));
            l += sum.x + sum.y;
          } else if (KT == 128) {
            hand_over(1);
          }
          if (!last_product()) break;
          if (NS == 1) ++o_cnt;
          hand_over(0);
        }
      }
      tile_seq += nt;
      // every product of the unit is done when the last of each stream is
      const bool used = NS == 1 ? wg == 0 : two || nt > wg;
      if (NS == 2 && used) ++o_cnt;  // (the issuing warp says so once a unit)
      if (ok && used)
        ok = __all_sync(0xffffffffu, bar_wait(&ct.o_done[o], (o_cnt - 1) & 1, ct, a.dev_status));
      fence_after();
      if (!two && ok && (NS == 2 || wg == 0)) {  // maxima and sums change hands where the scores were
        tm_store2(lanes + Sh::o_col(o) - 128, m, l);
        tm_wait_store();
      }
      fence_before();
      ok = named_all(1, kSoftmaxThreads, ok);
      if (!ok) break;
      fence_after();
      if (tid == 0) ct.bad[(seq - 1) & 7] = 0;  // every warp is past the unit before
      // two row tiles: each warpgroup ends its own; one: both take half of the columns
      float f0 = 1.f, f1 = 0.f;
      bool add = false;
      if (!two) {
        const float2 x = tm_load2(lanes + Sh::o_col(0) - 128);
        const float2 y = NS == 2 ? tm_load2(lanes + Sh::o_col(1) - 128) : make_float2(-INFINITY, 0.f);
        add = NS == 2 && nt > 1;
        m = fmaxf(x.x, y.x);
        f0 = x.x == -INFINITY ? 1.f : exp2_fast((x.x - m) * c);  // nothing seen: sums of zeros, or NaN that has to stay
        f1 = y.x == -INFINITY ? 1.f : exp2_fast((y.x - m) * c);
        l = x.y * f0 + y.y * f1;
      }
      const bool whole = wk.t0 == 0 && wk.t1 == wk.q.tiles;
      const unsigned long long bad = *(volatile unsigned long long*)&ct.bad[seq & 7];
      if (live) {
        const int c0 = two ? 0 : wg * (D / 2), c1 = two ? D : c0 + D / 2;
        const int part = wk.t0 == 0;
        const long long slot = (long long)blockIdx.x * 2 + part;
        const int mi = m0 + mr, i = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi, head = wk.h * G + mi - i * G;
        const long long orow = wk.q.s + i;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* out = static_cast<uint16_t*>(a.out) + orow * a.out_stride + (long long)head * D;
        float4* to = p.part + slot * (D / 4) * p.part_rows + mr;
        const unsigned long long own_bad = mr < rows ? bad & tree : 0;
        if (whole && !two) f0 *= inv, f1 *= inv;  // (rows of two tiles: f0 is 1)
        if (whole && two) f0 = inv;
#pragma unroll 1
        for (int col = c0; col < c1; col += 16) {
          __syncwarp();
          float x[16];
          tm_read16(x, lanes + Sh::o_col(two ? wg : 0) + col);
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] *= f0;
          if (add) {
            float y[16];
            tm_read16(y, lanes + Sh::o_col(1 % NS) + col);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = fmaf(y[j], f1, x[j]);
          }
          if (own_bad) {
#pragma unroll 1
            for (int nd = 0; nd < kTree; ++nd) {
              if (!(own_bad >> nd & 1)) continue;
              const int pos = wk.q.ctx + nd, pc = pos / a.cache.page_size;
              const int page = __ldg(a.block_table + (long long)wk.b * a.table_width + pc);
              const uint32_t* v = reinterpret_cast<const uint32_t*>(
                  static_cast<const uint16_t*>(a.cache.v) + page * a.cache.page_stride +
                  (pos - pc * a.cache.page_size) * a.cache.slot_stride + wk.h * a.cache.head_stride + col);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 e = unpack2<DT>(v[j]);
                if (!(fabsf(e.x) < INFINITY)) x[2 * j] += e.x;
                if (!(fabsf(e.y) < INFINITY)) x[2 * j + 1] += e.y;
              }
            }
          }
          if (mr < rows) {
            if (whole) {
#pragma unroll
              for (int j = 0; j < 16; j += 8)
                *reinterpret_cast<uint4*>(out + col + j) =
                    make_uint4(pack2<DT>(x[j], x[j + 1]), pack2<DT>(x[j + 2], x[j + 3]), pack2<DT>(x[j + 4], x[j + 5]),
                               pack2<DT>(x[j + 6], x[j + 7]));
            } else {
#pragma unroll
              for (int j = 0; j < 16; j += 4)
                __stcg(to + (col + j) / 4 * p.part_rows, make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]));
            }
          }
        }
        if (mr < rows && c0 == 0) {
          if (!whole) __stcg(p.part_ml + slot * p.part_rows + mr, make_float2(m, l));
          else if (a.lse) a.lse[orow * a.q_heads + head] = l == 0.f ? -INFINITY : (fmaf(m, c, -kBias<DT>) + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (!whole) {
        named_sync(1, kSoftmaxThreads);
        if (tid == 0)  // releases what the block wrote before the barrier
          asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.arrive + ct.split[wk.t0 == 0].first * ct.groups + member)
                       : "memory");
      }
      ++seq;
    }
    // ---------------- heads that are split over blocks: each of these joins some rows
#pragma unroll 1
    for (int which = 0; ok && which < 2; ++which) {
      const Split sp = ct.split[which];
      const int m0 = member * Sh::MG, rows = min(Sh::MG, sp.n * G - m0);
      if (sp.parts == 0 || rows <= 0) continue;
      unsigned* arrive = p.arrive + sp.first * ct.groups + member;
      if (tid == 0) {
        const long long t0 = clock64();
        unsigned v;
        do {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrive) : "memory");
          if (v < (unsigned)sp.parts && clock64() - t0 > p.wait_cycles) {
            atomicOr(a.dev_status, MOE_DEV_TIMEOUT);
            *(volatile int*)&ct.abort = 1;
            break;
          }
        } while (v < (unsigned)sp.parts);
      }
      ok = named_all(1, kSoftmaxThreads, !*(volatile int*)&ct.abort || tid != 0);
      if (!ok) break;
      // items: four columns of 32 rows, a lane per row; as many warps of a block to an item as
      // there are to spare, each with every tw-th part
      const int row_blocks = (rows + 31) >> 5, items = row_blocks * (D / 4);
      int tw_log = 3;
      while (tw_log > 0 && sp.parts << (3 - tw_log) < items) --tw_log;
      const int tw = 1 << tw_log, teams = 8 >> tw_log, mine_k = warp & (tw - 1);
      const int stride = 2 * ct.groups * (D / 4) * p.part_rows;  // from a block's part to the next one's
      float4* sm_acc = reinterpret_cast<float4*>(smem);          // [8][32]
      float2* sm_ml = reinterpret_cast<float2*>(smem + 8 * 32 * 16);
#pragma unroll 1
      for (int it0 = (ct.gang - sp.first) * teams; it0 < items; it0 += sp.parts * teams) {
        const int it = it0 + (warp >> tw_log), c4 = it & (D / 4 - 1), r = it / (D / 4) * 32 + lane;
        const bool here = it < items && r < rows;
        float top = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const auto join = [&](float2 ml, float4 v) {
          const float to = fmaxf(top, ml.x);
          const float f = top == -INFINITY ? 1.f : exp2_fast((top - to) * p.c);  // (nothing so far: zeros, or NaN)
          const float g = ml.x == -INFINITY ? 1.f : exp2_fast((ml.x - to) * p.c);
          top = to;
          l = fmaf(l, f, ml.y * g);
          acc = make_float4(fmaf(acc.x, f, v.x * g), fmaf(acc.y, f, v.y * g), fmaf(acc.z, f, v.z * g),
                            fmaf(acc.w, f, v.w * g));
        };
        // the first block's part lies in its second place
        const int block0 = (sp.first * ct.groups + member) * 2;
        const float4* from = p.part + ((long long)block0 * (D / 4) + c4) * p.part_rows + r;
        const float2* from_ml = p.part_ml + (long long)block0 * p.part_rows + r;
        constexpr int kAhead = 4;  // parts of a lane on their way (10: 53.3 us for the ragged batch against 51.9)
#pragma unroll 1
        for (int k0 = mine_k; k0 < sp.parts && here; k0 += tw * kAhead) {
          float2 ml[kAhead];
          float4 v[kAhead];
          int k = k0;
#pragma unroll
          for (int j = 0; j < kAhead; ++j, k += tw) {
            ml[j] = make_float2(-INFINITY, 0.f);
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < sp.parts) {
              ml[j] = __ldcg(from_ml + (k ? k * (stride / (D / 4)) : p.part_rows));
              v[j] = __ldcg(from + (k ? k * stride : (D / 4) * p.part_rows));
            }
          }
          float2 all = ml[0];
#pragma unroll
          for (int j = 1; j < kAhead; ++j) all.x = fmaxf(all.x, ml[j].x);
          all.y = 0.f;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const float g = ml[j].x == -INFINITY ? 1.f : exp2_fast((ml[j].x - all.x) * p.c);
            all.y = fmaf(ml[j].y, g, all.y);
            sum = make_float4(fmaf(v[j].x, g, sum.x), fmaf(v[j].y, g, sum.y), fmaf(v[j].z, g, sum.z),
                              fmaf(v[j].w, g, sum.w));
          }
          join(all, sum);
        }
        __syncwarp();
        if (tw > 1) {
          named_sync(1, kSoftmaxThreads);
          sm_acc[warp * 32 + lane] = acc;
          sm_ml[warp * 32 + lane] = make_float2(top, l);
          named_sync(1, kSoftmaxThreads);
#pragma unroll 1
          for (int q = 1; q < tw && mine_k == 0; ++q) join(sm_ml[(warp + q) * 32 + lane], sm_acc[(warp + q) * 32 + lane]);
        }
        if (here && mine_k == 0) {
          const int mi = m0 + r, i = p.group_mul ? (int)__umulhi((unsigned)mi, p.group_mul) : mi, head = sp.h * G + mi - i * G;
          const long long orow = sp.s + i;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * a.out_stride + (long long)head * D + 4 * c4) =
              make_uint2(pack2<DT>(acc.x * inv, acc.y * inv), pack2<DT>(acc.z * inv, acc.w * inv));
          if (c4 == 0 && a.lse)
            a.lse[orow * a.q_heads + head] = l == 0.f ? -INFINITY : (fmaf(top, p.c, -kBias<DT>) + log2f(l)) * 0.6931471805599453f;
        }
      }
      named_sync(1, kSoftmaxThreads);
      if (tid == 0) {
        unsigned* done = p.done + sp.first * ct.groups + member;
        if (atomicAdd(done, 1u) == (unsigned)sp.parts - 1) {  // all have seen the count: ready for the next call
          *arrive = 0;
          *done = 0;
        }
      }
    }
    __syncwarp();
    tm_wait_store();  // (a wait that gave up leaves some on their way)
  }
  __syncthreads();
  __syncwarp();
  if (warp == 10) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  // requests that are left out: their rows, where they are rows at all, get nothing seen
  for (int b = (int)blockIdx.x * kThreads + tid; b < a.n_req; b += (int)gridDim.x * kThreads) {
    const Req q = request<D>(a, b);
    if (q.n == 0 || q.tiles) continue;
    flags |= MOE_DEV_LENGTH;
    for (int r = q.s; r < q.s + q.n; ++r) {
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (long long)r * a.out_stride);
      for (int i = 0; i < a.q_heads * CPR; ++i) to[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = 0; i < a.q_heads; ++i) a.lse[(long long)r * a.q_heads + i] = -INFINITY;
    }
  }
  if (flags) atomicOr(a.dev_status, flags);
}

// ---- host -----------------------------------------------------------------------------

int check(const moe_tree_attention_args* p) {
  if (!p) return MOE_EINVAL;
  const moe_tree_attention_args& a = *p;
  if (a.n_req < 1 || a.n_rows < 0 || a.max_tree < 1 || a.table_width < 1 || a.q_heads < 1 || a.kv_heads < 1 ||
      a.head_dim < 1 || a.q_heads % a.kv_heads || !std::isfinite(a.scale))
    return MOE_EINVAL;
  if (a.dtype != MOE_BF16 && a.dtype != MOE_F16) return a.dtype == MOE_F32 ? MOE_EUNSUPPORTED : MOE_EINVAL;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return MOE_EUNSUPPORTED;
  if (a.max_tree > kTree || a.q_heads / a.kv_heads > 64 || a.q_heads > 1024 || a.n_req > 16384 ||
      a.n_rows > (1 << 20))
    return MOE_EUNSUPPORTED;
  const int rc = check_cache(a.cache, a.kv_heads);
  if (rc != MOE_OK) return rc;
  // offsets in the cache travel in units of 16 bytes, in 32 bits
  if (cache_span(a.cache, a.kv_heads) >= ((int64_t)8 << 32) - 256) return MOE_EUNSUPPORTED;
  // the list of (request, head, tile) is numbered in 32 bits
  if ((Wide)(((int64_t)a.table_width * a.cache.page_size + 63) / 64 + kUnit) * a.n_req * a.kv_heads >= ((int64_t)1 << 31))
    return MOE_EUNSUPPORTED;
  if (!stride_ok(a.q_stride) || !stride_ok(a.out_stride)) return MOE_EINVAL;
  if (!rows_ok(a.n_rows, a.q_stride) || !rows_ok(a.n_rows, a.out_stride)) return MOE_EUNSUPPORTED;
  if (!ptr_ok(a.dev_status, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.ctx_len, 4) || !ptr_ok(a.block_table, 4) ||
      !opt_ok(a.lse, 4) || !opt_ok(a.tree_mask, 8))
    return MOE_EINVAL;
  if (a.n_rows > 0 && (!ptr_ok(a.q, 16) || !ptr_ok(a.out, 16))) return MOE_EINVAL;
  return MOE_OK;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int group_rows(const moe_tree_attention_args& a) {  // query rows of a group, as the workspace holds them
  const int rows = a.max_tree * (a.q_heads / a.kv_heads), most = a.head_dim == 256 ? 128 : 256;
  return ((rows < most ? rows : most) + 31) & ~31;
}

struct Workspace {
  size_t ml, part, total;
};
Workspace layout(const moe_tree_attention_args& a) {
  Workspace w{};
  const size_t rows = (size_t)kMaxBlocks * 2 * group_rows(a);
  static_assert(2 * kMaxBlocks * sizeof(unsigned) <= kCounterBytes && kCounterBytes % 256 == 0, "counters");
  w.ml = kCounterBytes;
  w.part = w.ml + up256(rows * 8);
  w.total = w.part + up256(rows * a.head_dim * 4);
  return w;
}

template <int DT, int D>
int launch(const moe_tree_attention_args& a, Plan p, int sms, cudaStream_t st) {
  using Sh = Shape<D>;
  constexpr int kSmem = 227 * 1024;
  const int need = a.max_tree * p.group;
  p.nq = Sh::NS == 2 && need > 128 ? 2 : 1;
  p.nslot = (kSmem - 1024 - (int)sizeof(Control) - p.nq * Sh::kQ) / Sh::kSlot;
  if (p.nslot > kMaxSlots) p.nslot = kMaxSlots;
  static_assert((kSmem - 1024 - (int)sizeof(Control) - Sh::NS * Sh::kQ) / Sh::kSlot >= 4, "ring");
  static thread_local int ready = -1;  // device whose shared-memory limit this thread has set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && ready != dev) {
    e = cudaFuncSetAttribute(k_tree_attn<DT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return launch_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms < kMaxBlocks ? sms : kMaxBlocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // blocks that share a head wait for each other
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_status(cudaLaunchKernelEx(&cfg, k_tree_attn<DT, D>, a, p));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_tree_attention_workspace_bytes(const moe_tree_attention_args* args) {
  return check(args) == MOE_OK ? layout(*args).total : 0;
}

extern "C" int moe_set_attention_wait_limit_ns(uint64_t ns) {
  g_wait_ns.store(ns ? ns : kWaitNs, std::memory_order_relaxed);
  return MOE_OK;
}

extern "C" int moe_tree_attention(const moe_tree_attention_args* args, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check(args);
  if (rc != MOE_OK) return rc;
  const moe_tree_attention_args& a = *args;
  if (!ptr_ok(ws, 16)) return MOE_EINVAL;
  const Workspace w = layout(a);
  if (ws_bytes < w.total) return MOE_EWORKSPACE;
  if (a.n_rows == 0) return MOE_OK;
  const int sms = current_sms();
  if (sms < 1) return MOE_ECUDA;
  char* base = static_cast<char*>(ws);
  Plan p{};
  p.group = a.q_heads / a.kv_heads;
  p.part_rows = group_rows(a);
  p.group_mul = p.group == 1 ? 0u : (unsigned)((1ull << 32) / (unsigned)p.group + 1);
  // n / page_size = (n * mul) >> shift for every n below 2^31
  int bits = 0;
  while ((1 << bits) < a.cache.page_size) ++bits;
  p.page_shift = 31 + bits;
  p.page_mul = (unsigned)((1ull << p.page_shift) / (unsigned)a.cache.page_size + 1);
  p.flip = a.scale < 0.f ? 1 : a.scale == 0.f ? 2 : 0;
  p.c = (a.scale == 0.f ? 1.f : std::fabs(a.scale)) * 1.4426950408889634f;
  p.arrive = reinterpret_cast<unsigned*>(base);
  p.done = p.arrive + kMaxBlocks;
  const unsigned long long ns = g_wait_ns.load(std::memory_order_relaxed);
  p.wait_cycles = (long long)(ns < (1ull << 40) ? ns : 1ull << 40) * kCyclesPerNs;
  p.part_ml = reinterpret_cast<float2*>(base + w.ml);
  p.part = reinterpret_cast<float4*>(base + w.part);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = a.dtype == MOE_BF16;
  switch (a.head_dim) {
    case 64: return bf ? launch<MOE_BF16, 64>(a, p, sms, st) : launch<MOE_F16, 64>(a, p, sms, st);
    case 128: return bf ? launch<MOE_BF16, 128>(a, p, sms, st) : launch<MOE_F16, 128>(a, p, sms, st);
    default: return bf ? launch<MOE_BF16, 256>(a, p, sms, st) : launch<MOE_F16, 256>(a, p, sms, st);
  }
}
