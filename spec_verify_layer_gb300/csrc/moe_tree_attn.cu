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
//   - four producer warps copy key and value rows (cp.async, 16 bytes a lane, page table
//     looked up per row) into a ring of shared-memory slots in the 128-byte swizzle that
//     the tensor cores read;
//   - one thread issues the products: S = Q K^T into tensor memory, and O += P V with P
//     read from tensor memory and V from its slot as it lies (no transpose is stored);
//   - two warpgroups do the softmax, a thread per query row: S out of tensor memory,
//     running maximum and sum in registers, P back over S as 16-bit weights.
// Two streams (S, P, O of their own) keep the tensor cores and the exponentials busy at
// once: two row tiles of 128 over the same keys, or, with up to 128 rows, even and odd
// key tiles over the same rows, joined when the share of the head ends.  A head's keys
// split over blocks leave unnormalised sums with their maximum in the workspace; when the
// last of its blocks has arrived, each of them joins some of the rows, in block order.
//
// Running maximum: O is rescaled only when a row's maximum rises by more than 2^8 (the
// weights then stay below 2^8 and the sums are exact in relative terms), so the pass over
// O in tensor memory is rare after the first tiles.
//
// What is not seen gets the weight 0, but 0 times a cached NaN would still be NaN in the
// product: slots past the last position are zero-filled, and the values of drafted rows
// are looked over on their way: what is not finite becomes 0 in the slot and is added at
// the end to the rows that see it.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kTree = 64;
constexpr int kThreads = 512;           // 8 softmax warps, 4 producer warps, 1 issuing warp (3 idle: warpgroups)
constexpr int kSoftmaxThreads = 256, kProducers = 128;
constexpr int kMaxBlocks = 160;         // workspace sizing; the launch takes min(SM count, this)
constexpr int kMaxSlots = 10;
constexpr float kRescale = 8.0f;        // log2 of how far a maximum may lag behind
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s

template <int D>
struct Shape {
  static constexpr int KT = D == 256 ? 64 : 128;       // keys of a tile
  static constexpr int NS = D == 256 ? 1 : 2;          // streams (tensor memory holds 512 columns)
  static constexpr int MG = 128 * NS;                  // query rows of a group
  static constexpr int kSlot = KT * D * 2;             // bytes of a key or value tile
  static constexpr int kQ = 128 * D * 2;               // bytes of a query tile
  static constexpr int CPR = D / 8;                    // 16-byte chunks of a row
  static constexpr int RPP = kProducers / CPR;         // rows a pass of the producers copies
  static constexpr int PASSES = KT / RPP;
  __host__ __device__ static constexpr int s_col(int s) { return NS == 2 ? 256 * s : 64 * s; }
  __host__ __device__ static constexpr int o_col(int s) { return NS == 2 ? 256 * s + 128 : 256; }
};

struct Plan {  // host-computed, the same for every block
  int nq;      // query tiles held
  int nslot;
  int group;   // query heads of a key/value head
  int part_rows;
  unsigned page_mul;
  int page_shift;
  int flip;    // scale is negative: the queries are negated
  float c;     // |scale| * log2(e)
  float* part;       // [blocks][2][part_rows][D]
  float2* part_ml;   // [blocks][2][part_rows]
  unsigned* arrive;  // [blocks]
  unsigned* done;    // [blocks]
};

struct Control {  // the start of dynamic shared memory
  unsigned long long full[kMaxSlots], empty[kMaxSlots];
  unsigned long long s_full[2], p_full[2], o_done[2], q_ready, drain;
  unsigned long long bad[8];          // per unit: tree rows with values that are not finite
  __align__(16) unsigned short hole[8][16];  // per tile: rows without a page, by pass
  long long total, red[16];
  int redn[16];
  int maxn, start_b;
  long long start_off;
  unsigned tmem;
  int abort;
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
__device__ __noinline__ bool bar_wait_slow(uint32_t b, uint32_t parity, int* abort_flag, unsigned* status) {
  const long long t0 = clock64();
  while (!bar_try(b, parity)) {
    if (*(volatile int*)abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *(volatile int*)abort_flag = 1;
      atomicOr(status, MOE_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool bar_wait(unsigned long long* b, uint32_t parity, Control& ct, unsigned* status) {
  if (bar_try(smem_u32(b), parity)) return true;
  return bar_wait_slow(smem_u32(b), parity, &ct.abort, status);
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
// A load and its wait are one statement: the registers are not ready in between.
__device__ __forceinline__ void tm_load(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_store32(uint32_t addr, const uint32_t (&r)[32]) {
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
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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

template <int D>
struct Walk {  // a block's share, unit (stretch of one head's tiles) after unit
  Req q;
  int b, h, t0, t1;
  long long w, end;  // place in the list, end of the share
  int seq;           // units so far that have rows for this block
  __device__ __forceinline__ void begin(const moe_tree_attention_args& a, int b_, long long off, long long w_,
                                        long long end_) {
    w = w_;
    end = end_;
    b = b_;
    seq = -1;
    if (w >= end) return;
    q = request<D>(a, b);
    h = (int)(off / q.tiles);
    t0 = (int)(off - (long long)h * q.tiles);
    t1 = (int)min((long long)q.tiles, t0 + (end - w));
  }
  __device__ __forceinline__ bool more() const { return w < end; }
  __device__ __forceinline__ void next(const moe_tree_attention_args& a) {
    w += t1 - t0;
    if (w >= end) return;
    t0 = 0;
    if (++h == a.kv_heads) {
      h = 0;
      if (b + 1 >= a.n_req) {
        w = end;
        return;
      }
      do q = request<D>(a, ++b);
      while (q.tiles == 0 && b + 1 < a.n_req);
      if (q.tiles == 0) {  // not while the lengths stay as they were
        w = end;
        return;
      }
    }
    t1 = (int)min((long long)q.tiles, end - w);
  }
};

__device__ __forceinline__ long long share(long long total, int gangs, int g) { return total * g / gangs; }
__device__ __forceinline__ int gang_of(long long total, int gangs, long long x) {
  return (int)(((x + 1) * gangs - 1) / total);
}

// ---- the kernel -------------------------------------------------------------------------

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_tree_attn(const __grid_constant__ moe_tree_attention_args a, const __grid_constant__ Plan p) {
  using Sh = Shape<D>;
  constexpr int KT = Sh::KT, NS = Sh::NS, CPR = Sh::CPR, RPP = Sh::RPP, PASSES = Sh::PASSES;
  constexpr uint32_t kBlk = KT * 128;  // bytes of a 64-element block of a key or value tile
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sm_q = smem;
  unsigned char* sm_kv = smem + (size_t)p.nq * Sh::kQ;
  Control& ct = *reinterpret_cast<Control*>(sm_kv + (size_t)p.nslot * Sh::kSlot);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.group;

  if (tid == 0) {
    for (int i = 0; i < p.nslot; ++i) {
      bar_init(&ct.full[i], kProducers);
      bar_init(&ct.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&ct.s_full[i], 1);
      bar_init(&ct.p_full[i], 4);
      bar_init(&ct.o_done[i], 1);
    }
    bar_init(&ct.q_ready, kSoftmaxThreads / 32);
    bar_init(&ct.drain, 1);
    ct.abort = 0;
    ct.start_b = 0;
    ct.start_off = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 8) ct.bad[tid] = 0;
  if (tid < 128) (&ct.hole[0][0])[tid] = 0;
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ct.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // total work and the widest request
  unsigned flags = 0;
  {
    long long sum = 0;
    int maxn = 0;
    for (int b = tid; b < a.n_req; b += kThreads) {
      const Req q = request<D>(a, b);
      sum += (long long)q.tiles * a.kv_heads;
      if (q.tiles) maxn = max(maxn, q.n);
      if (q.n != 0 && q.tiles == 0) {
        flags |= MOE_DEV_LENGTH;
        if (q.n > 0 && b % (int)gridDim.x == (int)blockIdx.x) {
          for (int r = q.s; r < q.s + q.n; ++r) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (long long)r * a.out_stride);
            for (int i = 0; i < a.q_heads * CPR; ++i) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse)
              for (int i = 0; i < a.q_heads; ++i) a.lse[(long long)r * a.q_heads + i] = -INFINITY;
          }
        }
      }
    }
    if (tid == 0 && __ldg(a.row_start) != 0) flags |= MOE_DEV_LENGTH;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    maxn = __reduce_max_sync(0xffffffffu, maxn);
    if (lane == 0) {
      ct.red[warp] = sum;
      ct.redn[warp] = maxn;
    }
    __syncthreads();
    if (tid == 0) {
      long long t = 0;
      int m = 0;
      for (int i = 0; i < kThreads / 32; ++i) {
        t += ct.red[i];
        m = max(m, ct.redn[i]);
      }
      ct.total = t;
      ct.maxn = m;
    }
    __syncthreads();
  }
  const long long total = ct.total;
  const int groups = max(1, (ct.maxn * G + Sh::MG - 1) / Sh::MG);
  const int gangs = (int)min(total, (long long)max(1, (int)gridDim.x / groups));
  const int gang = (int)blockIdx.x / groups, member = (int)blockIdx.x - gang * groups;
  const bool works = gang < gangs && groups <= (int)gridDim.x;
  const long long w0 = works ? share(total, gangs, gang) : 0, w1 = works ? share(total, gangs, gang + 1) : 0;
  // the request that holds place w0
  if (works) {
    long long before = 0;
    for (int b0 = 0; b0 < a.n_req; b0 += kThreads) {
      const int b = b0 + tid;
      const long long mine = b < a.n_req ? (long long)request<D>(a, b).tiles * a.kv_heads : 0;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) ct.red[warp] = incl;
      __syncthreads();
      long long lo = before;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) lo += ct.red[i];
        before += ct.red[i];
      }
      lo += incl - mine;
      if (w0 >= lo && w0 < lo + mine) {
        ct.start_b = b;
        ct.start_off = w0 - lo;
      }
      if (before > w0) break;  // the same for every thread
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ct.tmem;
  Walk<D> wk;
  wk.begin(a, ct.start_b, ct.start_off, w0, w1);

  if (warp >= 8 && warp < 12) {
    // ---------------- producers
    const int pt = tid - kSoftmaxThreads, chunk = pt % CPR, rr = pt / CPR;
    const uint32_t kv0 = smem_u32(sm_kv);
    int slot = 0, tile_seq = 0;
    unsigned holes = 0;  // entries of ct.hole that this thread left set
    uint32_t phase = 1;  // the slots start empty
    bool ok = true;
    for (int seq = 0; ok && wk.more(); wk.next(a)) {
      if (wk.q.n * G <= member * Sh::MG) continue;
      const int len = wk.q.ctx + wk.q.n;
      const int32_t* table = a.block_table + (long long)wk.b * a.table_width;
      const long long head_at = wk.h * a.cache.head_stride + chunk * 8;
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++tile_seq) {
        long long at[PASSES];
        unsigned hole = 0;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const int pos = t * KT + i * RPP + rr;
          at[i] = -1;
          if (pos < len) {
            const int col = (int)(((unsigned long long)(unsigned)pos * p.page_mul) >> p.page_shift);
            const int page = __ldg(table + col);
            if (page >= 0 && page < a.cache.n_pages)
              at[i] = page * a.cache.page_stride + (pos - col * a.cache.page_size) * a.cache.slot_stride + head_at;
            else
              hole |= 1u << i;
          }
        }
        if (hole) flags |= MOE_DEV_INDEX;
        const bool noted = chunk == 0 && (hole != 0 || (holes >> (tile_seq & 7) & 1));
        if (noted) {
          ct.hole[tile_seq & 7][rr] = (unsigned short)hole;
          holes = (holes & ~(1u << (tile_seq & 7))) | (hole ? 1u << (tile_seq & 7) : 0u);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!(ok = ok && bar_wait(&ct.empty[slot], phase, ct, a.dev_status))) break;
          const uint16_t* src = static_cast<const uint16_t*>(kv ? a.cache.v : a.cache.k);
          const uint32_t dst = kv0 + slot * Sh::kSlot + (chunk >> 3) * kBlk;
#pragma unroll
          for (int i = 0; i < PASSES; ++i) {
            const int r = i * RPP + rr;
            copy16(dst + r * 128 + (((chunk & 7) ^ (r & 7)) << 4), src + max(at[i], 0ll), at[i] >= 0);
          }
          const bool drafted = kv == 1 && (t + 1) * KT > wk.q.ctx;
          if (drafted) {
            // drafted rows' values: what is not finite is noted and taken out (a thread
            // looks over what it copied itself)
            asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
            for (int i = 0; i < PASSES; ++i) {
              const int r = i * RPP + rr, node = t * KT + r - wk.q.ctx;
              if (node < 0 || node >= wk.q.n) continue;
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
                atomicOr(&ct.bad[seq & 7], 1ull << node);
              }
            }
          }
          if (drafted || (kv == 0 && noted)) {
            // what this thread wrote itself goes ahead of its arrival
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async();
            bar_arrive(&ct.full[slot]);
          } else {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&ct.full[slot])) : "memory");
          }
          if (++slot == p.nslot) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      ++seq;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 12) {
    // ---------------- issue of the products
    if (lane == 0) {
      constexpr uint32_t id_s = instruction<DT>(KT, false), id_o = instruction<DT>(D, true);
      const uint32_t kv0 = smem_u32(sm_kv), q0 = smem_u32(sm_q);
      int k_slot = 0, v_slot = 1;       // slots of the next key and value tile
      uint32_t k_ph = 0, v_ph = 0;
      uint32_t p_par = 0;
      uint32_t q_ph = 0;
      bool ok = true;
      const auto take = [&](int& s, uint32_t& ph) {  // key and value tiles take turns in the ring
        s += 2;
        if (s >= p.nslot) {
          s -= p.nslot;
          ph ^= 1;
        }
      };
      const auto scores = [&](int s, int qt, int slot) {  // S_s = Q_qt K^T
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t qa = operand(q0 + qt * Sh::kQ + (k >> 2) * (128 * 128) + (k & 3) * 32, 0);
          const uint64_t kb = operand(kv0 + slot * Sh::kSlot + (k >> 2) * kBlk + (k & 3) * 32, 0);
          mma_ss(tmem + Sh::s_col(s), qa, kb, id_s, k > 0);
        }
        mma_commit(&ct.s_full[s]);
      };
      const auto values = [&](int s, int slot, bool first) {  // O += P_s V
        const int o = NS == 2 ? s : 0;
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          const uint64_t vb = operand(kv0 + slot * Sh::kSlot + k * 2048, kBlk);
          mma_ts(tmem + Sh::o_col(o), tmem + Sh::s_col(s) + k * 8, vb, id_o, !(first && k == 0));
        }
        mma_commit(&ct.o_done[o]);
      };
      const auto wait_p = [&](int s) {
        if (!bar_wait(&ct.p_full[s], p_par >> s & 1, ct, a.dev_status)) return false;
        p_par ^= 1u << s;
        fence_after();
        return true;
      };
      const auto wait_tile = [&](int slot, uint32_t ph) {
        if (!bar_wait(&ct.full[slot], ph, ct, a.dev_status)) return false;
        fence_async();  // the copies were ordinary writes: order them before the tensor cores' reads
        return true;
      };
      for (; ok && wk.more(); wk.next(a)) {
        const int rows = min(Sh::MG, wk.q.n * G - member * Sh::MG);
        if (rows <= 0) continue;
        const bool two = NS == 2 && rows > 128;
        if (!(ok = bar_wait(&ct.q_ready, q_ph, ct, a.dev_status))) break;
        q_ph ^= 1;
        fence_after();
        const int nt = wk.t1 - wk.t0;
        if (two) {
          for (int t = 0; ok && t <= nt; ++t) {
            for (int s = 0; ok && s < 2; ++s) {
              if (t > 0) {
                ok = wait_p(s) && (s == 1 || wait_tile(v_slot, v_ph));
                if (!ok) break;
                values(s, v_slot, t == 1);
                if (s == 1) {
                  mma_commit(&ct.empty[v_slot]);
                  take(v_slot, v_ph);
                }
              }
              if (t < nt) {
                ok = s == 1 || wait_tile(k_slot, k_ph);
                if (!ok) break;
                scores(s, s, k_slot);
                if (s == 1) {
                  mma_commit(&ct.empty[k_slot]);
                  take(k_slot, k_ph);
                }
              }
            }
          }
        } else {
          for (int t = 0; ok && t <= nt; ++t) {
            if (t < nt) {
              ok = wait_tile(k_slot, k_ph);
              if (!ok) break;
              scores(t & 1, 0, k_slot);
              mma_commit(&ct.empty[k_slot]);
              take(k_slot, k_ph);
            }
            if (t > 0) {
              const int s = (t - 1) & 1;
              ok = wait_p(s) && wait_tile(v_slot, v_ph);
              if (!ok) break;
              values(s, v_slot, t <= NS);  // the stream's first
              mma_commit(&ct.empty[v_slot]);
              take(v_slot, v_ph);
            }
          }
        }
      }
      mma_commit(&ct.drain);  // nothing runs on when the block ends
      bar_wait(&ct.drain, 0, ct, a.dev_status);
    }
  } else if (warp < 8) {
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
      if (rows <= 0) continue;
      const bool two = NS == 2 && rows > 128;
      // the group's queries into the swizzle
      for (int i = tid; i < rows * CPR; i += kSoftmaxThreads) {
        const int r = i / CPR, ch = i % CPR, mi = m0 + r, n = mi / G, g = mi - n * G;
        uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (long long)(wk.q.s + n) * a.q_stride +
                                                       (long long)(wk.h * G + g) * D) + ch);
        if (p.flip) {
          x.x ^= 0x80008000u;
          x.y ^= 0x80008000u;
          x.z ^= 0x80008000u;
          x.w ^= 0x80008000u;
        }
        const uint32_t dst = q0 + (r >> 7) * Sh::kQ + (ch >> 3) * (128 * 128) + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
      }
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&ct.q_ready);

      const int mr = (two ? wg * 128 : 0) + row;       // row of the group
      const bool live = (two ? wg * 128 : 0) + (warp & 3) * 32 < rows;  // any row of this warp
      uint64_t tree = 0;  // rows of the request that this one sees
      if (mr < rows) {
        const int i = (m0 + mr) / G;
        tree = a.tree_mask ? __ldg(a.tree_mask + wk.q.s + i) : i >= 63 ? ~0ull : (2ull << i) - 1;
      }
      const int len = wk.q.ctx + wk.q.n, nt = wk.t1 - wk.t0;
      float m = -INFINITY, l = 0.f;
      const bool mine_all = two || NS == 1;
      if (NS == 2 || wg == 0) {
        for (int ti = mine_all ? 0 : wg; ti < nt; ti += mine_all ? 1 : 2) {
          const int buf = NS == 2 ? wg : ti & 1, o = NS == 2 ? wg : 0;
          ok = __all_sync(0xffffffffu, bar_wait(&ct.s_full[buf], s_par >> buf & 1, ct, a.dev_status));
          if (!ok) break;
          s_par ^= 1u << buf;
          fence_after();
          if (live) {
            const uint32_t s_at = lanes + Sh::s_col(buf);
            const int base = (wk.t0 + ti) * KT;
            // which of the tile's keys this row sees, unless it is all
            unsigned seen[KT / 32];
            bool all = base + KT <= wk.q.ctx;
            const unsigned short* hole = ct.hole[(tile_seq + ti) & 7];
            bool holes = false;
#pragma unroll
            for (int r = 0; r < RPP; r += 2) holes |= *reinterpret_cast<const volatile unsigned*>(hole + r) != 0;
            all = all && !holes;
            if (!all) {
              const int d = wk.q.ctx - base;  // context keys of the tile
#pragma unroll
              for (int w = 0; w < KT / 32; ++w) {
                const int k = d - 32 * w;  // context keys of the word
                unsigned bits = k >= 32 ? 0xffffffffu : k > 0 ? (1u << k) - 1 : 0u;
                if (k < 32) bits |= (unsigned)(k > 0 ? tree << k : k > -64 ? tree >> -k : 0ull);
                const int v = len - base - 32 * w;  // positions of the word
                seen[w] = v >= 32 ? bits : v > 0 ? bits & ((1u << v) - 1) : 0u;
              }
              if (holes) {
#pragma unroll
                for (int w = 0; w < KT / 32; ++w)
                  for (int j = 0; j < 32; ++j) {
                    const int r = 32 * w + j;
                    if (hole[r % RPP] >> (r / RPP) & 1) seen[w] &= ~(1u << j);
                  }
              }
            }
            // S lies in registers a quarter at a time: once for the maximum, once for the weights
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < KT / 32; ++w) {
              uint32_t x[32];
              tm_load(x, s_at + 32 * w);
              if (!all) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!(seen[w] >> j & 1)) x[j] = 0xff800000u;
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(x[j]));
            }
            const bool far = m == -INFINITY ? top > -INFINITY : (top - m) * c > kRescale;
            if (__any_sync(0xffffffffu, far)) {
              const float to = fmaxf(m, top), f = m == -INFINITY ? 0.f : exp2_fast((m - to) * c);
              if (ti >= (mine_all ? 1 : 2)) {
                if (NS == 1) {  // (two streams: the scores' barrier covers the product before)
                  ok = __all_sync(0xffffffffu, bar_wait(&ct.o_done[0], (o_cnt - 1) & 1, ct, a.dev_status));
                  if (!ok) break;
                  fence_after();
                }
#pragma unroll 1
                for (int w = 0; w < D / 32; ++w) {
                  uint32_t x[32];
                  tm_load(x, lanes + Sh::o_col(o) + 32 * w);
#pragma unroll
                  for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                  tm_store32(lanes + Sh::o_col(o) + 32 * w, x);
                }
                tm_wait_store();
              }
              l *= f;
              m = to;
            }
            const float shift = m == -INFINITY ? 0.f : m * c;
#pragma unroll
            for (int w = 0; w < KT / 32; ++w) {
              uint32_t x[32], y[16];
              tm_load(x, s_at + 32 * w);
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), c, -shift));
              if (!all) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!(seen[w] >> j & 1)) x[j] = 0xff800000u;
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float e0 = exp2_fast(__uint_as_float(x[2 * j])), e1 = exp2_fast(__uint_as_float(x[2 * j + 1]));
                l += e0 + e1;
                y[j] = pack2<DT>(e0, e1);
              }
              tm_store16(s_at + 16 * w, y);  // over the quarter's own and earlier columns
            }
            tm_wait_store();
          }
          if (NS == 1 && o_cnt > 0) {  // keeps this warp within a phase of the barrier
            ok = __all_sync(0xffffffffu, bar_wait(&ct.o_done[0], (o_cnt - 1) & 1, ct, a.dev_status));
            if (!ok) break;
          }
          ++o_cnt;
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&ct.p_full[buf]);
        }
      }
      tile_seq += nt;
      // every product of the unit is done when the last of each stream is
      const bool used = NS == 1 ? wg == 0 : two || nt > wg;
      if (ok && used)
        ok = __all_sync(0xffffffffu, bar_wait(&ct.o_done[NS == 2 ? wg : 0], (o_cnt - 1) & 1, ct, a.dev_status));
      fence_after();
      if (!two && ok && (NS == 2 || wg == 0)) {  // maxima and sums change hands where the scores were
        tm_store2(lanes + Sh::s_col(NS == 2 ? wg : 0), m, l);
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
        const float2 x = tm_load2(lanes + Sh::s_col(0));
        const float2 y = NS == 2 ? tm_load2(lanes + Sh::s_col(1)) : make_float2(-INFINITY, 0.f);
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
        const int part = wk.w == w0 ? 0 : 1;
        const long long slot = ((long long)blockIdx.x * 2 + part) * p.part_rows + mr;
        const int mi = m0 + mr, i = mi / G, head = wk.h * G + mi - i * G;
        const long long orow = wk.q.s + i;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        for (int col = c0; col < c1; col += 32) {
          __syncwarp();
          uint32_t x[32];
          tm_load(x, lanes + Sh::o_col(two ? wg : 0) + col);
          if (!two) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f0);
            if (add) {
              uint32_t y[32];
              tm_load(y, lanes + Sh::o_col(1 % NS) + col);
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(fmaf(__uint_as_float(y[j]), f1, __uint_as_float(x[j])));
            }
          }
          if (mr >= rows) continue;
          if (bad & tree) {
            for (int nd = 0; nd < kTree; ++nd) {
              if (!((bad & tree) >> nd & 1)) continue;
              const int pos = wk.q.ctx + nd, pc = pos / a.cache.page_size;
              const int page = __ldg(a.block_table + (long long)wk.b * a.table_width + pc);
              const uint32_t* v = reinterpret_cast<const uint32_t*>(
                  static_cast<const uint16_t*>(a.cache.v) + page * a.cache.page_stride +
                  (pos - pc * a.cache.page_size) * a.cache.slot_stride + wk.h * a.cache.head_stride + col);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 e = unpack2<DT>(v[j]);
                if (!(fabsf(e.x) < INFINITY)) x[2 * j] = __float_as_uint(__uint_as_float(x[2 * j]) + e.x);
                if (!(fabsf(e.y) < INFINITY)) x[2 * j + 1] = __float_as_uint(__uint_as_float(x[2 * j + 1]) + e.y);
              }
            }
          }
          if (whole) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * a.out_stride + (long long)head * D + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                w[q] = pack2<DT>(__uint_as_float(x[8 * j + 2 * q]) * inv, __uint_as_float(x[8 * j + 2 * q + 1]) * inv);
              o[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4* o = reinterpret_cast<float4*>(p.part + slot * D + col);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              __stcg(o + j, make_float4(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1]),
                                        __uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])));
          }
        }
        if (mr < rows && c0 == 0) {
          if (!whole) __stcg(p.part_ml + slot, make_float2(m, l));
          else if (a.lse) a.lse[orow * a.q_heads + head] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (!whole) {
        __threadfence();
        named_sync(1, kSoftmaxThreads);
        if (tid == 0) {
          const int first = gang_of(total, gangs, wk.w - wk.t0);
          __threadfence();
          atomicAdd(p.arrive + first * groups + member, 1u);
        }
      }
      ++seq;
    }
  }
  __syncthreads();
  __syncwarp();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");

  // ---------------- heads that are split over blocks: each of these joins some rows
  if (works && !ct.abort) {
    // the share's first and last unit (the same one, maybe)
    Walk<D> jk;
    jk.begin(a, ct.start_b, ct.start_off, w0, w1);
    for (; jk.more(); jk.next(a)) {
      if (jk.t0 == 0 && jk.t1 == jk.q.tiles) continue;
      const int m0 = member * Sh::MG, rows = min(Sh::MG, jk.q.n * G - m0);
      if (rows <= 0) continue;
      const long long u0 = jk.w - jk.t0;
      const int first = gang_of(total, gangs, u0), last = gang_of(total, gangs, u0 + jk.q.tiles - 1);
      const int parts = last - first + 1;
      unsigned* arrive = p.arrive + first * groups + member;
      if (tid == 0) {
        const long long t0 = clock64();
        unsigned v;
        do {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrive) : "memory");
          if (clock64() - t0 > kWaitCycles) {
            atomicOr(a.dev_status, MOE_DEV_TIMEOUT);
            ct.abort = 1;
            break;
          }
        } while (v < (unsigned)parts);
      }
      __syncthreads();
      if (ct.abort) break;
      const int first_part = share(total, gangs, first) == u0 ? 0 : 1;
      for (int r = (gang - first) + parts * warp; r < rows; r += parts * (kThreads / 32)) {
        // lane j: every 32nd part's maximum and sum
        float top = -INFINITY;
        for (int k = lane; k < parts; k += 32) {
          const long long at = ((long long)((first + k) * groups + member) * 2 + (k ? 0 : first_part)) * p.part_rows + r;
          top = fmaxf(top, __ldcg(p.part_ml + at).x);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int mi = m0 + r, i = mi / G, head = jk.h * G + mi - i * G;
        const long long orow = jk.q.s + i;
        constexpr int PER = D / 32;  // columns of a lane
        float acc[PER], l = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) acc[j] = 0.f;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
          const long long at = ((long long)((first + k) * groups + member) * 2 + (k ? 0 : first_part)) * p.part_rows + r;
          const float2 ml = __ldcg(p.part_ml + at);
          const float f = ml.x == -INFINITY ? 1.f : exp2_fast((ml.x - top) * p.c);
          l = fmaf(ml.y, f, l);
          const float2* o = reinterpret_cast<const float2*>(p.part + at * D + lane * PER);
#pragma unroll
          for (int j = 0; j < PER / 2; ++j) {
            const float2 v = __ldcg(o + j);
            acc[2 * j] = fmaf(v.x, f, acc[2 * j]);
            acc[2 * j + 1] = fmaf(v.y, f, acc[2 * j + 1]);
          }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + orow * a.out_stride + (long long)head * D) +
                        lane * (PER / 2);
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) out[j] = pack2<DT>(acc[2 * j] * inv, acc[2 * j + 1] * inv);
        if (lane == 0 && a.lse) a.lse[orow * a.q_heads + head] = l == 0.f ? -INFINITY : (top * p.c + log2f(l)) * 0.6931471805599453f;
      }
      __syncthreads();
      if (tid == 0) {
        unsigned* done = p.done + first * groups + member;
        if (atomicAdd(done, 1u) == (unsigned)parts - 1) {  // all have seen the count: ready for the next call
          *arrive = 0;
          *done = 0;
          __threadfence();
        }
      }
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
  const int rc = check_cache(a.cache);
  if (rc != MOE_OK) return rc;
  if (!stride_ok(a.q_stride) || !stride_ok(a.out_stride)) return MOE_EINVAL;
  if (!ptr_ok(a.dev_status, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.ctx_len, 4) || !ptr_ok(a.block_table, 4) ||
      !opt_ok(a.lse, 4) || !opt_ok(a.tree_mask, 8))
    return MOE_EINVAL;
  if (a.n_rows > 0 && (!ptr_ok(a.q, 16) || !ptr_ok(a.out, 16))) return MOE_EINVAL;
  return MOE_OK;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int group_rows(const moe_tree_attention_args& a) {  // query rows of a group, as the workspace holds them
  const int rows = a.max_tree * (a.q_heads / a.kv_heads), most = a.head_dim == 256 ? 128 : 256;
  return rows < most ? rows : most;
}

struct Workspace {
  size_t counters, ml, part, total;
};
Workspace layout(const moe_tree_attention_args& a) {
  Workspace w{};
  const size_t rows = (size_t)kMaxBlocks * 2 * group_rows(a);
  w.counters = 0;
  w.ml = up256((size_t)2 * kMaxBlocks * 4);
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
  // n / page_size = (n * mul) >> shift for every n below 2^31
  int bits = 0;
  while ((1 << bits) < a.cache.page_size) ++bits;
  p.page_shift = 31 + bits;
  p.page_mul = (unsigned)((1ull << p.page_shift) / (unsigned)a.cache.page_size + 1);
  p.flip = a.scale < 0.f;
  p.c = std::fabs(a.scale) * 1.4426950408889634f;
  p.arrive = reinterpret_cast<unsigned*>(base);
  p.done = p.arrive + kMaxBlocks;
  p.part_ml = reinterpret_cast<float2*>(base + w.ml);
  p.part = reinterpret_cast<float*>(base + w.part);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = a.dtype == MOE_BF16;
  switch (a.head_dim) {
    case 64: return bf ? launch<MOE_BF16, 64>(a, p, sms, st) : launch<MOE_F16, 64>(a, p, sms, st);
    case 128: return bf ? launch<MOE_BF16, 128>(a, p, sms, st) : launch<MOE_F16, 128>(a, p, sms, st);
    default: return bf ? launch<MOE_BF16, 256>(a, p, sms, st) : launch<MOE_F16, 256>(a, p, sms, st);
  }
}
