// Page and slot map of a verify round (moe_round_map): block tables, cache slots,
// positions and tree masks from the requests' lengths, in one launch.
//
// Everything a thread block needs of the other requests is two prefix sums over the
// requests (rows before, fresh pages before).  Each block computes both itself (8 bytes a
// request from L2) instead of waiting for another block or a second launch, and then
// fills its share of the row arrays and of the fresh table entries; a row's page is read
// from the table where the request held it before the call and from the free list where
// it is fresh, so no block reads what another writes.
#include "moe_round_ops.cuh"

namespace moe {
namespace {

constexpr int kMapThreads = 256;
constexpr int kMapRows = 4 * kMapThreads;  // rows per block and step: four a thread, 16-byte stores
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

__global__ void __launch_bounds__(kMapThreads) k_round_map(const __grid_constant__ moe_map_args a, const ByPage by) {
  extern __shared__ uint32_t sm[];
  uint32_t* start = sm;                // [n_req + 1] rows before a request, at most n_rows
  uint32_t* off = sm + a.n_req + 1;    // [n_req + 1] fresh pages before it
  __shared__ uint2 wsum[kMapThreads / 32];
  __shared__ int par[kTree - 1 + kMapRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned flags = 0;
  const bool lead = blockIdx.x == 0;

  uint2 carry = make_uint2(0u, 0u);
  for (int b0 = 0; b0 < a.n_req; b0 += kMapThreads) {
    const int b = b0 + tid;
    Req q{0, 0, 0, 0};
    unsigned f = 0;
    if (b < a.n_req) q = request(a, by, b, f);
    uint2 v = make_uint2((uint32_t)q.rows, (uint32_t)q.take), incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) {
        incl.x = add_sat(incl.x, x);
        incl.y = add_sat(incl.y, y);
      }
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    uint2 before = carry;
    for (int w = 0; w < kMapThreads / 32; ++w) {
      const uint2 s = wsum[w];
      if (w < warp) before = make_uint2(add_sat(before.x, s.x), add_sat(before.y, s.y));
      carry = make_uint2(add_sat(carry.x, s.x), add_sat(carry.y, s.y));
    }
    __syncthreads();
    incl = make_uint2(add_sat(incl.x, before.x), add_sat(incl.y, before.y));
    if (b < a.n_req) {
      const uint32_t end = min(incl.x, (uint32_t)a.n_rows);
      start[b + 1] = end;
      off[b + 1] = incl.y;
      if (lead) {
        flags |= f;
        const long long got = min((long long)q.take, max(0LL, (long long)a.n_free - (incl.y - v.y)));
        if (got < q.take) flags |= MOE_DEV_PAGES;
        a.row_start[b + 1] = (int)end;
        a.pages[b] = q.held + (int)got;
      }
    }
  }
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

  // rows, four in a row to a thread
  const int live = (int)start[a.n_req];
  for (int base = blockIdx.x * kMapRows; base < a.n_rows; base += gridDim.x * kMapRows) {
    if (a.parents) {  // this step's rows and the 63 before them, which may be of the same tree
      __syncthreads();
      const int lo = max(0, base - (kTree - 1)), hi = min(live, base + kMapRows);
      for (int r = lo + tid; r < hi; r += kMapThreads) par[r - lo] = a.parents[r];
      __syncthreads();
    }
    const int par0 = max(0, base - (kTree - 1));
    const int r0 = base + 4 * tid;
    if (r0 >= a.n_rows) continue;
    int req[4], pos[4], slot[4];
    uint64_t mask[4];
    int b = r0 < live ? last_not_above(start, a.n_req, (uint32_t)r0) : 0;
    Req q{0, 0, 0, 0};
    int off_in = 0, col = 0, page = -1;  // place in the page, table column, page of the row
    bool have = false;                   // (of request b, up to date for the row before)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + j;
      req[j] = -1;
      pos[j] = 0;
      slot[j] = -1;
      mask[j] = 0;
      if (r >= live) continue;
      while (r >= (int)start[b + 1]) {
        ++b;
        have = false;
      }
      const int s = (int)start[b], i = r - s;
      bool turn = true;  // another page
      if (!have) {
        q = request(a, by, b, quiet);
        have = true;
        col = by(q.ctx + i);
        off_in = q.ctx + i - col * a.page_size;
      } else if (++off_in == a.page_size) {
        off_in = 0;
        ++col;
      } else {
        turn = false;
      }
      if (turn) {
        page = -1;
        if (col < q.held) {
          page = checked_page(a, a.block_table[(size_t)b * a.table_width + col], flags);
        } else if (col - q.held < q.take) {
          const uint32_t t = off[b] + (uint32_t)(col - q.held);
          if (t < (uint32_t)a.n_free) page = checked_page(a, a.free_pages[t], flags);
        }
      }
      int depth = i;
      if (a.parents) {
        if (i < kTree) {
          uint64_t m = 0;
          depth = -1;
          for (int n = i; n >= 0;) {  // n falls with every step
            m |= 1ull << n;
            ++depth;
            const int up = par[s + n - par0];
            if (up < -1 || up >= n) {
              flags |= MOE_DEV_INDEX;
              break;
            }
            n = up;
          }
          mask[j] = m;
        } else {
          flags |= MOE_DEV_LENGTH;
        }
      } else if (a.tree_mask) {
        if (i < kTree) mask[j] = i == kTree - 1 ? ~0ull : (2ull << i) - 1;
        else flags |= MOE_DEV_LENGTH;
      }
      req[j] = b;
      pos[j] = (int)min((long long)q.ctx + depth, 0x7fffffffLL);
      slot[j] = page < 0 ? -1 : page * a.page_size + off_in;
    }
    if (r0 + 4 <= a.n_rows) {
      *reinterpret_cast<int4*>(a.row_req + r0) = make_int4(req[0], req[1], req[2], req[3]);
      *reinterpret_cast<int4*>(a.row_pos + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.row_slot + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.tree_mask) {
        *reinterpret_cast<ulonglong2*>(a.tree_mask + r0) = make_ulonglong2(mask[0], mask[1]);
        *reinterpret_cast<ulonglong2*>(a.tree_mask + r0 + 2) = make_ulonglong2(mask[2], mask[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        if (r0 + j >= a.n_rows) break;
        a.row_req[r0 + j] = req[j];
        a.row_pos[r0 + j] = pos[j];
        a.row_slot[r0 + j] = slot[j];
        if (a.tree_mask) a.tree_mask[r0 + j] = mask[j];
      }
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
    const cudaError_t e = cudaFuncSetAttribute(k_round_map, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return launch_status(e);
  }
  ByPage by;
  int bits = 0;
  while ((1 << bits) < a.page_size) ++bits;
  by.shift = 31 + bits;
  by.mul = (unsigned)((1ull << by.shift) / (unsigned)a.page_size + 1);
  // one step's rows to a block, up to two blocks an SM: more blocks only repeat the sums
  const int steps = (a.n_rows + kMapRows - 1) / kMapRows;
  const int grid = steps < 1 ? 1 : steps > 2 * sms ? 2 * sms : steps;
  k_round_map<<<grid, kMapThreads, smem, static_cast<cudaStream_t>(stream)>>>(a, by);
  return launch_status(cudaGetLastError());
}
