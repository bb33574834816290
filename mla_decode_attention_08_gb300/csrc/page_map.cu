// mla_page_map: tables and maps of one step from the rows' lengths.
//
// Bound by latency: two trips to L2 for the lengths and a table entry, and the
// launch; 256 rows of 8192 tokens are 8.4 MB of indices (1.3 us of traffic) in
// 6.4 us, four short rows 3.4 us.
//
// The three prefix sums over rows (cached tokens after the step, new tokens,
// new pages) are small: every block computes all of them into its shared
// memory, so no block waits for another and one launch does the whole step.
// The outputs are then flat: each thread takes entries of the concatenated
// arrays, finds their row by binary search in the prefix and computes the
// entry.  A page the step itself hands out is read from free_pages at its
// prefix, not from the table, so that no entry depends on another block's
// table writes.
#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kSaturated = 0x7FFFFFFFu;

// t / page_size: pages are mostly a power of two long.
__device__ __forceinline__ uint32_t page_of(const PageMapParams& p, uint32_t t) {
  return p.page_shift >= 0 ? t >> p.page_shift : t / static_cast<uint32_t>(p.page_size);
}
__device__ __forceinline__ uint32_t pages_for(const PageMapParams& p, uint32_t tokens) {
  const uint32_t n = page_of(p, tokens);
  return n + (tokens != n * static_cast<uint32_t>(p.page_size));
}

// Saturating sums of values <= kSaturated: associative, so a prefix either is
// exact or reads kSaturated, which no accepted total reaches.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  return min(a + b, kSaturated);
}

struct Sums {
  uint32_t kv, fresh, pages;
};

struct RowShape {
  uint32_t before, total, pages_before, pages_new;
  bool bad;
};

__device__ __forceinline__ RowShape row_shape(const PageMapParams& p, int32_t b) {
  const int32_t len = __ldg(p.kv_lens + b), add = __ldg(p.new_lens + b);
  const uint32_t page = static_cast<uint32_t>(p.page_size);
  RowShape r;
  const uint64_t cap = static_cast<uint64_t>(p.max_pages) * page;
  r.bad = len < 0 || add < 0 ||
          static_cast<uint64_t>(static_cast<uint32_t>(len)) + static_cast<uint32_t>(add) > min(cap, static_cast<uint64_t>(kSaturated));
  r.before = r.bad ? 0u : static_cast<uint32_t>(len);
  r.total = r.bad ? 0u : static_cast<uint32_t>(len) + static_cast<uint32_t>(add);
  r.pages_before = pages_for(p, r.before);
  r.pages_new = pages_for(p, r.total) - r.pages_before;
  return r;
}

// The last row whose prefix is <= at (empty rows before it are passed over).
__device__ __forceinline__ int32_t row_of(const uint32_t* prefix, int32_t lo, int32_t hi, uint32_t at) {
  // prefix[lo] <= at < prefix[hi]
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (prefix[mid] <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One row as the expansions need it.
struct RowView {
  uint32_t kv0, kv1, before, pages_before, need0;
  const int32_t* table;
};

__device__ __forceinline__ RowView view_row(const PageMapParams& p, const uint32_t* kv,
                                            const uint32_t* fresh, const uint32_t* pages, int32_t b) {
  RowView r;
  r.kv0 = kv[b];
  r.kv1 = kv[b + 1];
  r.before = r.kv1 - r.kv0 - (fresh[b + 1] - fresh[b]);
  r.pages_before = pages_for(p, r.before);
  r.need0 = pages[b];
  r.table = p.block_table + static_cast<int64_t>(b) * p.table_stride;
  return r;
}

// Page pg of the row; -1 (with the error bit) when its id is not a page of the pool.
__device__ __forceinline__ int32_t page_id(const PageMapParams& p, const RowView& r, uint32_t pg) {
  if (!MLA_DCHECK(pg < r.pages_before ? pg < static_cast<uint32_t>(p.max_pages)
                                      : r.need0 + (pg - r.pages_before) < static_cast<uint32_t>(p.num_free), p.err))
    return -1;
  const int32_t id = pg < r.pages_before ? r.table[pg] : __ldg(p.free_pages + r.need0 + (pg - r.pages_before));
  if (id < 0 || id >= p.num_pages) {
    atomicOr(p.err, MLA_DERR_KV_INDEX);
    return -1;
  }
  return id;
}

__global__ void __launch_bounds__(kThreads) page_map_kernel(const PageMapParams p) {
  extern __shared__ uint32_t sm[];
  const int32_t n = p.batch;
  uint32_t* kv = sm;                  // [n + 1]
  uint32_t* fresh = kv + n + 1;       // [n + 1]
  uint32_t* pages = fresh + n + 1;    // [n + 1]
  __shared__ Sums warp_sums[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_primary();
  pdl_launch_dependents();

  // Prefix sums: each thread a run of consecutive rows.
  const int32_t run = (n + kThreads - 1) / kThreads;
  const int32_t b0 = min(n, tid * run), b1 = min(n, b0 + run);
  Sums mine = {0, 0, 0};
  bool bad = false;
  for (int32_t b = b0; b < b1; ++b) {
    const RowShape r = row_shape(p, b);
    bad |= r.bad;
    mine.kv = sat_add(mine.kv, r.total);
    mine.fresh = sat_add(mine.fresh, r.total - r.before);
    mine.pages = sat_add(mine.pages, r.pages_new);
  }
  Sums scan = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, scan.kv, d);
    const uint32_t f = __shfl_up_sync(0xffffffffu, scan.fresh, d);
    const uint32_t g = __shfl_up_sync(0xffffffffu, scan.pages, d);
    if (lane >= d) {
      scan.kv = sat_add(scan.kv, a);
      scan.fresh = sat_add(scan.fresh, f);
      scan.pages = sat_add(scan.pages, g);
    }
  }
  if (lane == 31) warp_sums[warp] = scan;
  bad = __syncthreads_or(bad);
  Sums base = {0, 0, 0}, total = {0, 0, 0};
  for (int w = 0; w < kWarps; ++w) {
    const Sums s = warp_sums[w];
    if (w < warp) {
      base.kv = sat_add(base.kv, s.kv);
      base.fresh = sat_add(base.fresh, s.fresh);
      base.pages = sat_add(base.pages, s.pages);
    }
    total.kv = sat_add(total.kv, s.kv);
    total.fresh = sat_add(total.fresh, s.fresh);
    total.pages = sat_add(total.pages, s.pages);
  }
  const bool short_out = total.kv > static_cast<uint32_t>(p.kv_indices_len) ||
                         total.fresh > static_cast<uint32_t>(p.slots_len);
  const bool short_free = total.pages > static_cast<uint32_t>(p.num_free);
  const uint32_t gtid = blockIdx.x * kThreads + tid, gthreads = gridDim.x * kThreads;
  if (bad || short_out || short_free) {  // the same in every block: an empty step
    if (gtid == 0) {
      atomicOr(p.err, (bad ? MLA_DERR_SEQ_LEN : 0) | (short_out ? MLA_DERR_CAPACITY : 0) |
                          (short_free ? MLA_DERR_FREE_PAGES : 0));
      p.pages_used[0] = 0;
    }
    for (uint32_t i = gtid; i <= static_cast<uint32_t>(n); i += gthreads) p.qo_indptr[i] = p.kv_indptr[i] = 0;
    for (uint32_t i = gtid; i < static_cast<uint32_t>(p.slots_len); i += gthreads) {
      p.slots[i] = -1;
      p.positions[i] = 0;
    }
    return;
  }
  // Exclusive prefix of this thread's run (no total is saturated, so the
  // subtraction undoes the inclusive scan exactly).
  Sums at = {base.kv + scan.kv - mine.kv, base.fresh + scan.fresh - mine.fresh,
             base.pages + scan.pages - mine.pages};
  for (int32_t b = b0; b < b1; ++b) {
    kv[b] = at.kv;
    fresh[b] = at.fresh;
    pages[b] = at.pages;
    const RowShape r = row_shape(p, b);
    at.kv += r.total;
    at.fresh += r.total - r.before;
    at.pages += r.pages_new;
  }
  if (tid == 0) {
    kv[n] = total.kv;
    fresh[n] = total.fresh;
    pages[n] = total.pages;
  }
  __syncthreads();

  for (uint32_t i = gtid; i <= static_cast<uint32_t>(n); i += gthreads) {
    p.kv_indptr[i] = static_cast<int32_t>(kv[i]);
    p.qo_indptr[i] = static_cast<int32_t>(fresh[i]);
  }
  if (gtid == 0) p.pages_used[0] = static_cast<int32_t>(total.pages);

  const uint32_t page = static_cast<uint32_t>(p.page_size);
  // New tokens, then the padding behind them.
  for (uint32_t i = gtid; i < static_cast<uint32_t>(p.slots_len); i += gthreads) {
    int32_t slot = -1, pos = 0;
    if (i < total.fresh) {
      const int32_t b = row_of(fresh, 0, n, i);
      const RowView r = view_row(p, kv, fresh, pages, b);
      const uint32_t t = r.before + (i - fresh[b]);
      const uint32_t pg = page_of(p, t);
      const int32_t id = page_id(p, r, pg);
      pos = static_cast<int32_t>(t);
      if (id >= 0) slot = id * p.page_size + static_cast<int32_t>(t - pg * page);
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
  // New pages into the table.
  for (uint32_t i = gtid; i < total.pages; i += gthreads) {
    const int32_t b = row_of(pages, 0, n, i);
    const RowView r = view_row(p, kv, fresh, pages, b);
    const uint32_t column = r.pages_before + (i - r.need0);
    if (MLA_DCHECK(b < n && column < static_cast<uint32_t>(p.max_pages) && i < static_cast<uint32_t>(p.num_free), p.err))
      p.block_table[static_cast<int64_t>(b) * p.table_stride + column] = __ldg(p.free_pages + i);
  }
  // The index of every cached token, four at a time: each block a contiguous
  // share, whose rows are found first, so that a thread searches among those.
  const uint32_t units = total.kv / 4 + (total.kv % 4 != 0);
  const uint32_t share = (units + gridDim.x - 1) / gridDim.x;
  const uint32_t u0 = min(units, blockIdx.x * share), u1 = min(units, u0 + share);
  __shared__ int32_t ends[2];
  int32_t first_row = 0, last_row = n - 1;
  if (gridDim.x > 1) {
    if (u0 < u1 && tid < 2) ends[tid] = row_of(kv, 0, n, tid == 0 ? 4 * u0 : min(total.kv, 4 * u1) - 1);
    __syncthreads();
    first_row = ends[0];
    last_row = ends[1];
  }
  for (uint32_t u = u0 + tid; u < u1; u += kThreads) {
    uint32_t t = 4 * u;
    int32_t b = row_of(kv, first_row, last_row + 1, t);
    RowView r = view_row(p, kv, fresh, pages, b);
    uint32_t j = t - r.kv0, pg = page_of(p, j), off = j - pg * page;
    int32_t id = page_id(p, r, pg);
    int32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = id < 0 ? -1 : id * p.page_size + static_cast<int32_t>(off);
      if (++t >= total.kv) continue;  // past the end: the entries after it are not stored
      ++off;
      if (t >= r.kv1) {
        do ++b;
        while (kv[b + 1] <= t);  // over empty rows; t < total.kv = kv[n] ends it
        r = view_row(p, kv, fresh, pages, b);
        pg = off = 0;
        if (k < 3) id = page_id(p, r, pg);
      } else if (off == page) {
        off = 0;
        ++pg;
        if (k < 3) id = page_id(p, r, pg);
      }
    }
    if (!MLA_DCHECK(min(4 * u + 4, total.kv) <= static_cast<uint32_t>(p.kv_indices_len) && b <= n, p.err)) continue;
    if (4 * u + 4 <= total.kv) {
      *reinterpret_cast<int4*>(p.kv_indices + 4 * u) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (4 * u + k < total.kv) p.kv_indices[4 * u + k] = v[k];
    }
  }
}

size_t smem_of(int32_t batch) { return 3 * (static_cast<size_t>(batch) + 1) * sizeof(uint32_t); }

}  // namespace

cudaError_t page_map_prepare() {
  return cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_of(MLA_MAX_MAP_ROWS)));
}

cudaError_t launch_page_map(PageMapParams p, int32_t num_sms, cudaStream_t stream) {
  p.page_shift = -1;
  for (int32_t k = 0; k < 31; ++k)
    if (p.page_size == 1 << k) p.page_shift = k;
  // One block for every 1024 indices and 256 slots that the outputs have room for,
  // at most two an SM: each repeats the prefix sums, so more blocks only add
  // those (256 rows of 8192 tokens: 6.4 us with two blocks an SM, 7.4 with four;
  // blocks of 512 threads 7.7, and 3.9 against 3.3 us for four short rows).
  const int64_t room = static_cast<int64_t>(p.kv_indices_len) / 4 + p.slots_len;
  int64_t blocks = (room + kThreads - 1) / kThreads;
  if (blocks > 2 * num_sms) blocks = 2 * num_sms;
  if (blocks < 1) blocks = 1;
  return launch_dependent(page_map_kernel, static_cast<unsigned>(blocks), kThreads, smem_of(p.batch),
                          stream, p);
}

}  // namespace mla
