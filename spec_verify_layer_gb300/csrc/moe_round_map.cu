// Page and slot map of a verify round (moe_round_map): block tables, cache slots,
// positions and tree masks from the requests' lengths, in one launch.
//
// Everything a thread block needs of the other requests is two prefix sums over the
// requests (rows before, fresh pages before).  Each block computes both itself (8 bytes a
// request from L2) instead of waiting for another block or a second launch, and then
// fills its share of the row arrays and of the fresh table entries; a row's page is read
// from the table where the request held it before the call and from the free list where
// it is fresh, so no block reads what another writes.  `pages` may be `pages_held` itself: blocks
// read that one from their first look to their last, so it is written by a second launch then,
// of one block, which only goes through the requests (each thread reads an entry before it
// writes it).
//
// What bounds it (GB300): latency.  Six requests with trees take 3.9 us in a graph (an empty
// launch 0.6): two dependent reads, a prefix sum, the tree's parents and masks.  1,500
// prompts of up to 1,000 tokens (9.6 MB) take 12 us: the prefix sums of the requests, and then
// a binary search a row for its request, in two steps of rows for 125 of the 608 blocks; the
// traffic alone would take 1.4.  In place the six requests take 9.5 us in a stream, apart 7.0.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kMapThreads = 256;
constexpr int kMapRows = 4 * kMapThreads;  // rows per block and step
constexpr int kMapPer = 2;  // requests of a thread at a time
constexpr int kMapMaxReq = 16384;
constexpr int kTree = 64;  // rows of a tree: bits of a mask

// n / page_size for n below 2^31, as a product (integer division is some 20 instructions).
struct ByPage {
  unsigned mul;
  int shift;
  __device__ __forceinline__ int operator()(int n) const {
    return (int)(((unsigned long long)(unsigned)n * mul) >> shift);
  }
  __device__ __forceinline__ int up(int n) const { return n > 0 ? (*this)(n - 1) + 1 : 0; }  // rounded up
};

// A request's lengths, made consistent.  flags: MOE_DEV_* bits found on the way.
struct Req {
  int ctx, rows, held, take;  // take: table columns to fill behind the held ones
};

__device__ __forceinline__ Req request(const moe_map_args& a, ByPage by, int b, unsigned& flags) {
  Req q;
  q.ctx = a.ctx_len[b];
  q.rows = a.new_len[b];
  if (q.ctx < 0 || q.rows < 0 || (long long)q.ctx + q.rows > 0x7fffffffLL) {
    flags |= MOE_DEV_LENGTH;
    q.ctx = max(q.ctx, 0);
    q.rows = 0;
  }
  const int W = a.table_width, first = by.up(q.ctx);
  q.held = a.pages_held ? a.pages_held[b] : first;
  if (q.held < first || q.held > W) {
    flags |= MOE_DEV_LENGTH;
    q.held = min(max(q.held, 0), W);
  }
  int need = by.up(q.ctx + q.rows);
  if (need > W) {
    flags |= MOE_DEV_PAGES;
    need = W;
  }
  q.take = max(0, need - q.held);
  return q;
}

__device__ __forceinline__ int checked_page(const moe_map_args& a, int page, unsigned& flags) {
  if (page >= 0 && page < a.n_pages) return page;
  flags |= MOE_DEV_INDEX;
  return -1;
}

// What a launch writes: the counts of pages, everything else, or (as it is unless they lie over
// what the requests held) both.
enum { kMapPages = 1, kMapRest = 2 };

__global__ void __launch_bounds__(kMapThreads)
    k_round_map(const __grid_constant__ moe_map_args a, const ByPage by, const int what) {
  extern __shared__ uint32_t sm[];
  uint32_t* start = sm;                // [n_req + 1] rows before a request, at most n_rows
  uint32_t* off = sm + a.n_req + 1;    // [n_req + 1] fresh pages before it
  __shared__ uint2 wsum[kMapThreads / 32];
  __shared__ int par[kTree - 1 + kMapRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned flags = 0;
  const bool lead = blockIdx.x == 0;

  // the first step's parents travel meanwhile (those of its rows and of the 63 before them,
  // which may be of the same tree)
  const auto fetch_parents = [&](int base) {
    const int lo = max(0, base - (kTree - 1)), hi = min(a.n_rows, base + kMapRows);
    for (int r = lo + tid; r < hi; r += kMapThreads) par[r - lo] = a.parents[r];
  };
  if (a.parents && what != kMapPages) fetch_parents(blockIdx.x * kMapRows);

  // kMapPer neighbouring requests a thread: their lengths are loaded together
  uint2 carry = make_uint2(0u, 0u);
  for (int b0 = 0; b0 < a.n_req; b0 += kMapThreads * kMapPer) {
    const int b = b0 + tid * kMapPer;
    Req q[kMapPer];
    unsigned f = 0;
    uint2 sum = make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < kMapPer; ++j) {
      q[j] = Req{0, 0, 0, 0};
      if (b + j < a.n_req) q[j] = request(a, by, b + j, f);
    }
#pragma unroll
    for (int j = 0; j < kMapPer; ++j) sum = make_uint2(add_sat(sum.x, (uint32_t)q[j].rows), add_sat(sum.y, (uint32_t)q[j].take));
    uint2 incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x = add_sat(incl.x, x);
        incl.y = add_sat(incl.y, y);
      }
    }
    if (lane == 31) wsum[warp] = incl;
    // what lies before this thread's requests: the lanes below, the warps below, the steps before
    uint2 before = make_uint2(__shfl_up_sync(0xffffffffu, incl.x, 1), __shfl_up_sync(0xffffffffu, incl.y, 1));
    if (lane == 0) before = make_uint2(0u, 0u);
    __syncthreads();
    before = make_uint2(add_sat(before.x, carry.x), add_sat(before.y, carry.y));
#pragma unroll
    for (int w = 0; w < kMapThreads / 32; ++w) {
      const uint2 s = wsum[w];
      if (w < warp) before = make_uint2(add_sat(before.x, s.x), add_sat(before.y, s.y));
      carry = make_uint2(add_sat(carry.x, s.x), add_sat(carry.y, s.y));
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMapPer; ++j) {
      if (b + j >= a.n_req) break;
      const uint32_t fresh = before.y;
      before = make_uint2(add_sat(before.x, (uint32_t)q[j].rows), add_sat(before.y, (uint32_t)q[j].take));
      const uint32_t end = min(before.x, (uint32_t)a.n_rows);
      start[b + j + 1] = end;
      off[b + j + 1] = before.y;
      if (lead) {
        const long long got = min((long long)q[j].take, max(0LL, (long long)a.n_free - fresh));
        if (got < q[j].take) flags |= MOE_DEV_PAGES;
        if (what & kMapRest) a.row_start[b + j + 1] = (int)end;
        if (what & kMapPages) a.pages[b + j] = q[j].held + (int)got;
      }
    }
    if (lead) flags |= f;
  }
  if (what == kMapPages) return;  // (what is wrong with the lengths the other launch reports)
  if (tid == 0) {
    start[0] = 0;
    off[0] = 0;
    if (lead) {
      a.row_start[0] = 0;
      a.n_taken[0] = (int)min(carry.y, (uint32_t)a.n_free);
      if (carry.x > (uint32_t)a.n_rows) flags |= MOE_DEV_LENGTH;
    }
  }
  __syncthreads();

  // fresh table entries
  unsigned quiet = 0;
  const uint32_t fresh = carry.y;
  for (uint32_t t = blockIdx.x * kMapThreads + tid; t < fresh; t += gridDim.x * kMapThreads) {
    const int b = last_not_above(off, a.n_req, t);
    const int held = request(a, by, b, quiet).held;
    a.block_table[(size_t)b * a.table_width + held + (t - off[b])] =
        t < (uint32_t)a.n_free ? checked_page(a, a.free_pages[t], flags) : -1;
  }

  // rows: a rolled loop, since a small call is as long as its instructions take to arrive
  const int live = (int)start[a.n_req];
  for (int base = blockIdx.x * kMapRows; base < a.n_rows; base += gridDim.x * kMapRows) {
    if (a.parents && base != (int)blockIdx.x * kMapRows) {
      __syncthreads();
      fetch_parents(base);
      __syncthreads();
    }
    const int par0 = max(0, base - (kTree - 1)), stop = min(a.n_rows, base + kMapRows);
    int b = base + tid < live ? last_not_above(start, a.n_req, (uint32_t)(base + tid)) : 0, known = -1;
    Req q{0, 0, 0, 0};  // of request `known`
#pragma unroll 1
    for (int r = base + tid; r < stop; r += kMapThreads) {
      int req = -1, pos = 0, slot = -1;
      uint64_t mask = 0;
      if (r < live) {
        while (r >= (int)start[b + 1]) ++b;
        if (b != known) {
          q = request(a, by, b, quiet);
          known = b;
        }
        req = b;
        const int s = (int)start[req], i = r - s, p = q.ctx + i, col = by(p);
        int page = -1;
        if (col < q.held) {
          page = checked_page(a, a.block_table[(size_t)req * a.table_width + col], flags);
        } else if (col - q.held < q.take) {
          const uint32_t t = off[req] + (uint32_t)(col - q.held);
          if (t < (uint32_t)a.n_free) page = checked_page(a, a.free_pages[t], flags);
        }
        int depth = i;
        if (a.parents) {
          if (i < kTree) {
            depth = -1;
            for (int n = i; n >= 0;) {  // n falls with every step
              mask |= 1ull << n;
              ++depth;
              const int up = par[s + n - par0];
              if (up < -1 || up >= n) {
                flags |= MOE_DEV_INDEX;
                break;
              }
              n = up;
            }
          } else {
            flags |= MOE_DEV_LENGTH;
          }
        } else if (a.tree_mask) {
          if (i < kTree) mask = i == kTree - 1 ? ~0ull : (2ull << i) - 1;
          else flags |= MOE_DEV_LENGTH;
        }
        pos = (int)min((long long)q.ctx + depth, 0x7fffffffLL);
        slot = page < 0 ? -1 : page * a.page_size + (p - col * a.page_size);
      }
      a.row_req[r] = req;
      a.row_pos[r] = pos;
      a.row_slot[r] = slot;
      if (a.tree_mask) a.tree_mask[r] = mask;
    }
  }
  if (flags) atomicOr(a.dev_status, flags);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_round_map(const moe_map_args* p, void* stream) {
  if (!p) return MOE_EINVAL;
  const moe_map_args& a = *p;
  if (a.n_req < 1 || a.n_rows < 0 || a.n_free < 0 || a.page_size < 1 || a.n_pages < 1 || a.table_width < 1)
    return MOE_EINVAL;
  if (!ptr_ok(a.ctx_len, 4) || !ptr_ok(a.new_len, 4) || !opt_ok(a.pages_held, 4) || !opt_ok(a.parents, 4) ||
      !ptr_ok(a.block_table, 4) || !ptr_ok(a.row_start, 4) || !ptr_ok(a.pages, 4) || !ptr_ok(a.n_taken, 4) ||
      !ptr_ok(a.dev_status, 4))
    return MOE_EINVAL;
  if (a.n_free > 0 && !ptr_ok(a.free_pages, 4)) return MOE_EINVAL;
  // pages_held in place, or apart from it
  const uintptr_t held = reinterpret_cast<uintptr_t>(a.pages_held), pages = reinterpret_cast<uintptr_t>(a.pages);
  if (held && held != pages && (held < pages ? pages - held : held - pages) < (uintptr_t)a.n_req * 4) return MOE_EINVAL;
  if (a.n_rows > 0 && (!ptr_ok(a.row_req, 16) || !ptr_ok(a.row_pos, 16) || !ptr_ok(a.row_slot, 16) ||
                       !opt_ok(a.tree_mask, 16)))
    return MOE_EINVAL;
  if (a.n_req > kMapMaxReq || a.page_size > 65536 || (int64_t)a.n_pages * a.page_size >= ((int64_t)1 << 31) ||
      (int64_t)a.n_req * a.table_width >= ((int64_t)1 << 31) || a.n_rows > (1 << 30))
    return MOE_EUNSUPPORTED;
  const int sms = current_sms();
  if (sms < 1) return MOE_ECUDA;
  const size_t smem = (size_t)(a.n_req + 1) * 8;
  if (smem > 40 * 1024) {
    // the most that any call takes: the limit is the kernel's, not the call's, and calls of other
    // threads may lie between this and the launch
    const cudaError_t e = cudaFuncSetAttribute(k_round_map, cudaFuncAttributeMaxDynamicSharedMemorySize, (kMapMaxReq + 1) * 8);
    if (e != cudaSuccess) return launch_status(e);
  }
  ByPage by;
  int bits = 0;
  while ((1 << bits) < a.page_size) ++bits;
  by.shift = 31 + bits;
  by.mul = (unsigned)((1ull << by.shift) / (unsigned)a.page_size + 1);
  // one step's rows to a block, up to four blocks an SM: what each repeats of the sums is a
  // latency that the others share
  const int steps = (a.n_rows + kMapRows - 1) / kMapRows;
  const int grid = steps < 1 ? 1 : steps > 4 * sms ? 4 * sms : steps;
  const bool in_place = held == pages;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_kernel(k_round_map, grid, kMapThreads, smem, st, a, by, (int)(in_place ? kMapRest : kMapRest | kMapPages));
  if (e != cudaSuccess || !in_place) return launch_status(e);
  return launch_status(launch_kernel(k_round_map, 1, kMapThreads, smem, st, a, by, (int)kMapPages));
}
