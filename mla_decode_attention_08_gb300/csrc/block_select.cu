// mla_block_select: the pages that each row attends, as the decode step's page table.
//
// Of a row's pages the first `sink` and the last `recent` are always taken, and of the
// rest those with the highest scores, the lower page where two are alike.  The last page
// is always among them, so the number of chosen tokens follows from the lengths alone:
// every block forms the prefix sums over all rows for itself, and one launch does the
// step.  A block holds its row's scores in registers, consecutive pages a thread, or of more
// than 8192 pages reads them anew from L2 whenever they are needed.  It finds the ones that are
// taken by their place in 256 equal steps between the lowest and the highest: the steps above the
// one in which the last page falls are taken whole, and in that one the pages are ranked
// against each other, or, where it holds too many for that (scores far apart, or alike), divided
// into steps again, of the scores' bits now, until few are left or all are the same.  Bound by the
// steps' latency, so scores and table entries are on their way before the row's length is known
// (4 rows of up to 128 pages 4.0 us, 6.8 when they were loaded behind it; 64 rows of up to 2048 pages
// 6.3, with the last score found bit by bit 10.8; 64 of 8192 14.1; 8 of 16384 22.3, bit by bit 198).
// Longer rows are one block's all the same, an SM that reads its row four times or more: 8 of 100000
// take 121.
#include <cfloat>

#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 256;   // of equal width between the lowest and the highest score
constexpr int kListed = 256;  // pages that are ranked against each other, at most

// Scores as integers in the same order; both zeros are alike, and a NaN counts as the
// highest, so that it is not passed over.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr uint32_t kMinusInf = 0x007FFFFFu, kPlusInf = 0xFF800000u;  // ordered(-inf), ordered(+inf)
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

struct RowCount {
  int32_t pages, taken, tokens;
  bool bad;
};
__device__ __forceinline__ RowCount count_row(const BlockSelectParams& p, int32_t b) {
  const int32_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
  const int64_t len = static_cast<int64_t>(ke) - ks;
  RowCount r;
  const uint32_t pages = pages_of(len, p.page_size);
  r.bad = ks < 0 || len < 0 || pages > static_cast<uint32_t>(p.max_pages);
  r.pages = r.bad ? 0 : static_cast<int32_t>(pages);
  r.taken = min(r.pages, p.blocks);
  // all pages but the last are full
  r.tokens = r.bad ? 0 : static_cast<int32_t>(len) - (r.pages - r.taken) * p.page_size;
  return r;
}

// The sum over the block's threads before this one, and over all (in *all).  (`sums`: read by
// the calls before, which a barrier has ended.)
__device__ __forceinline__ int32_t sum_before(int32_t v, int32_t* sums, int32_t* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t u = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int32_t before = incl - v;
  *all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    *all += sums[w];
  }
  return before;
}

// kHeld: scores that a thread holds; with 0 they are read anew whenever they are needed.
template <int kHeld>
__global__ void __launch_bounds__(kThreads, kHeld > 4 ? 1 : 2) block_select_kernel(const BlockSelectParams p) {
  extern __shared__ int32_t rows[];  // [blocks]: first cache row of each chosen page, or -1
  __shared__ int64_t sums[kWarps], totals[kWarps];
  __shared__ int32_t scan[2][kWarps];
  __shared__ int32_t counts[kSteps], listed;
  __shared__ uint2 list[kListed];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t b = blockIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
  const float* scores = p.scores + static_cast<int64_t>(b) * p.scores_stride;
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.table_stride;
  float score[kHeld > 0 ? kHeld : 1];
  int32_t entry[kHeld > 0 ? kHeld : 1];
  if constexpr (kHeld > 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int32_t j = tid * kHeld + i;
      score[i] = j < p.max_pages ? scores[j] : 0.0f;
      entry[i] = j < p.max_pages ? table[j] : -1;
    }
  }

  // Tokens of the rows before this one, and of all rows.
  int64_t before = 0, total = 0;
  bool bad = false;
  for (int32_t r = tid; r < p.batch; r += kThreads) {
    const RowCount c = count_row(p, r);
    total += c.tokens;
    if (r < b) before += c.tokens;
    bad = bad || c.bad;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    total += __shfl_xor_sync(0xffffffffu, total, d);
  }
  if (lane == 0) {
    sums[warp] = before;
    totals[warp] = total;
  }
  bad = __syncthreads_or(bad);
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += sums[w];
    total += totals[w];
  }
  const bool full = total > p.indices_len;
  const RowCount row = count_row(p, b);
  int32_t* chosen = p.chosen == nullptr ? nullptr : p.chosen + static_cast<int64_t>(b) * p.blocks;
  if (bad || full) {  // the whole step is emptied
    if (b == 0 && tid == 0) atomicOr(p.err, bad ? MLA_DERR_KV_INDPTR : MLA_DERR_CAPACITY);
    if (tid == 0) p.sel_indptr[b] = 0;
    if (tid == 0 && b == p.batch - 1) p.sel_indptr[p.batch] = 0;
    if (chosen != nullptr)
      for (int32_t i = tid; i < p.blocks; i += kThreads) chosen[i] = -1;
    return;
  }
  if (tid == 0) p.sel_indptr[b] = static_cast<int32_t>(before);
  if (tid == 0 && b == p.batch - 1) p.sel_indptr[p.batch] = static_cast<int32_t>(total);
  // Of the middle pages, [lo, hi), as many are taken as `want` says.
  const int32_t lo = p.sink, hi = row.pages - p.recent, want = p.blocks - p.sink - p.recent;
  const bool choose = row.pages > p.blocks;
  if (!MLA_DCHECK(row.pages <= p.max_pages && hi <= row.pages, p.err)) return;
  const int32_t first = tid * kHeld;  // of the pages in registers
  uint32_t held[kHeld > 0 ? kHeld : 1];
  if constexpr (kHeld > 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int32_t j = first + i;
      held[i] = choose && j >= lo && j < hi ? ordered(score[i]) : 0u;  // (0: no score's)
    }
  }
  // Calls `f(page, key)` for this thread's middle pages, in no order.
  auto each_key = [&](auto f) {
    if constexpr (kHeld > 0) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (held[i] != 0) f(first + i, held[i]);
    } else {
      constexpr int kAtOnce = 16;
      for (int32_t j0 = lo + tid; j0 < hi; j0 += kAtOnce * kThreads) {
        float x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) x[i] = j0 + i * kThreads < hi ? scores[j0 + i * kThreads] : 0.0f;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (j0 + i * kThreads < hi) f(j0 + i * kThreads, ordered(x[i]));
      }
    }
  };
  // Middle pages with a key above `threshold` are taken, and the first `ties` of those at it.
  uint32_t threshold = 0xFFFFFFFFu;
  int32_t ties = 0;
  if (choose && want > 0) {
    // Between the lowest and the highest finite score; what is not finite falls on the ends.
    uint32_t low = 0xFFFFFFFFu, high = 0;
    each_key([&](int32_t, uint32_t key) {
      if (key > kMinusInf && key < kPlusInf) {
        low = min(low, key);
        high = max(high, key);
      }
    });
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
      scan[0][warp] = static_cast<int32_t>(low);
      scan[1][warp] = static_cast<int32_t>(high);
    }
    if (tid < kSteps) counts[tid] = 0;
    if (tid == 0) listed = 0;
    __syncthreads();
    low = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(scan[0][lane % kWarps]));
    high = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(scan[1][lane % kWarps]));
    const float least = score_of(low), width = score_of(high) - least;
    // Where the width or the steps a unit pass float32's range (or there is no width), 0: all finite
    // scores share the lowest step.
    const float steps = (kSteps - 1) / width;
    const float by = width > 0.0f && width <= FLT_MAX && steps <= FLT_MAX ? steps : 0.0f;
    // (Never falls as the score rises.  With a finite width no difference overflows.)
    auto step_of = [&](uint32_t key) {
      if (key >= kPlusInf) return kSteps - 1;
      if (key <= kMinusInf || by == 0.0f) return 0;
      return static_cast<int>(fminf((score_of(key) - least) * by, kSteps - 1.0f));
    };
    each_key([&](int32_t, uint32_t key) {
      const int step = step_of(key);
      if (MLA_DCHECK(step >= 0 && step < kSteps, p.err)) atomicAdd(&counts[step], 1);
    });
    __syncthreads();
    // The highest step with which there are enough (every warp for itself): lane l has the
    // steps 8 l .. 8 l + 7.
    int32_t above = 0, inside = 0;  // pages above the step, and in it
    auto find_step = [&] {
      const int32_t need = want - above;
      int32_t c[8], own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += c[i] = counts[8 * lane + i];
      int32_t from = own;  // in this lane's steps and above
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t v = __shfl_down_sync(0xffffffffu, from, d);
        if (lane + d < 32) from += v;
      }
      int32_t over = from - own, step = -1, in = 0;
      if (over < need && from >= need) {
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          if (step >= 0) continue;
          if (over + c[i] >= need) {
            step = 8 * lane + i;
            in = c[i];
          } else {
            over += c[i];
          }
        }
      }
      const int who = __ffs(__ballot_sync(0xffffffffu, step >= 0)) - 1;
      above += __shfl_sync(0xffffffffu, over, who);
      inside = __shfl_sync(0xffffffffu, in, who);
      return __shfl_sync(0xffffffffu, step, who);
    };
    const int step = find_step();
    bool by_value = true;  // the open pages are the step's, else those with a key in [low, high]
    if (inside > kListed) {
      by_value = false;
      low = 0xFFFFFFFFu, high = 0;
      each_key([&](int32_t, uint32_t key) {
        if (step_of(key) != step) return;
        low = min(low, key);
        high = max(high, key);
      });
      low = __reduce_min_sync(0xffffffffu, low);
      high = __reduce_max_sync(0xffffffffu, high);
      if (lane == 0) {
        scan[0][warp] = static_cast<int32_t>(low);
        scan[1][warp] = static_cast<int32_t>(high);
      }
      __syncthreads();  // (counts are read, too)
      low = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(scan[0][lane % kWarps]));
      high = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(scan[1][lane % kWarps]));
      while (inside > kListed && low < high) {  // (each time a range 2^7 times smaller, or more)
        if (tid < kSteps) counts[tid] = 0;
        __syncthreads();
        const int shift = max(0, 24 - __clz(high - low));
        each_key([&](int32_t, uint32_t key) {
          const uint32_t step = (key - low) >> shift;
          if (key >= low && key <= high && MLA_DCHECK(step < kSteps, p.err)) atomicAdd(&counts[step], 1);
        });
        __syncthreads();
        low += static_cast<uint32_t>(find_step()) << shift;
        high = low + min(high - low, (1u << shift) - 1);
        __syncthreads();  // (counts are read)
      }
    }
    if (inside > kListed) {  // all alike
      threshold = low;
      ties = want - above;
    } else {
      each_key([&](int32_t j, uint32_t key) {
        if (by_value ? step_of(key) != step : key < low || key > high) return;
        const int to = atomicAdd(&listed, 1);
        if (MLA_DCHECK(to < inside && to < kListed, p.err)) list[to] = make_uint2(key, static_cast<uint32_t>(j));
      });
      __syncthreads();
      // The last page that is taken gives the threshold.
      if (tid < inside) {
        const uint2 mine = list[tid];
        int32_t over = above, alike = 0, before_it = 0;
        for (int i = 0; i < inside; ++i) {
          const uint2 other = list[i];
          over += other.x > mine.x;
          alike += other.x == mine.x;
          before_it += other.x == mine.x && other.y < mine.y;
        }
        if (over + before_it == want - 1) {  // (with all that are like it: the ones above the next lower key)
          const bool whole = before_it + 1 == alike;
          scan[0][0] = static_cast<int32_t>(mine.x - whole);
          scan[1][0] = whole ? 0 : before_it + 1;
        }
      }
      __syncthreads();
      threshold = static_cast<uint32_t>(scan[0][0]);
      ties = scan[1][0];
    }
  }
  __syncthreads();  // (scan is read)

  // The pages in order: a page's place among the chosen is the number before it.
  auto is_middle = [&](int32_t j) { return choose && j >= lo && j < hi; };
  auto put = [&](int32_t place, int32_t j, int32_t id) {
    if (place >= p.blocks || !MLA_DCHECK(place >= 0 && j >= 0 && j < row.pages, p.err)) return;
    const bool ok = id >= 0 && id < p.num_pages;
    if (!ok) atomicOr(p.err, MLA_DERR_KV_INDEX);
    rows[place] = ok ? id * p.page_size : -1;
    if (chosen != nullptr) chosen[place] = j;
  };
  int32_t all = 0;
  if constexpr (kHeld > 0) {
    int32_t alike = 0;
    if (ties > 0) each_key([&](int32_t, uint32_t key) { alike += key == threshold; });
    const int32_t rank = ties > 0 ? sum_before(alike, scan[0], &all) : 0;
    // (a tie is taken while its rank among them is below `ties`)
    int32_t taken = 0, tie = rank;
    auto takes = [&](int32_t j, uint32_t key) {
      if (!is_middle(j)) return true;
      return key > threshold || (key == threshold && tie++ < ties);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (first + i < row.pages && takes(first + i, held[i])) ++taken;
    int32_t place = sum_before(taken, scan[1], &all);
    tie = rank;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (first + i < row.pages && takes(first + i, held[i])) put(place++, first + i, entry[i]);
  } else {
    // Some consecutive pages a thread at a time; the table is read where one is taken.
    constexpr int kEach = 16;
    int32_t done = 0, tied = 0;  // pages and ties taken before
    for (int32_t base = 0; base < row.pages; base += kEach * kThreads) {
      const int32_t j0 = base + kEach * tid;
      uint32_t take = 0, equal = 0;
      float x[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) x[i] = j0 + i < row.pages ? scores[j0 + i] : 0.0f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int32_t j = j0 + i;
        if (j >= row.pages) continue;
        const uint32_t key = ordered(x[i]);
        if (!is_middle(j) || key > threshold) take |= 1u << i;
        else if (key == threshold) equal |= 1u << i;
      }
      if (ties > 0) {  // (the same for the whole block)
        const int32_t rank = tied + sum_before(__popc(equal), scan[0], &all);
        tied += all;
        // as many of this thread's, the first of them, as there is room for
        for (int32_t room = ties - rank; room > 0 && equal != 0; --room) {
          take |= equal & -equal;
          equal &= equal - 1;
        }
      }
      int32_t place = done + sum_before(__popc(take), scan[1], &all);
      done += all;
      for (; take != 0; take &= take - 1) {
        const int32_t j = j0 + __ffs(take) - 1;
        put(place++, j, table[j]);
      }
      if (ties == 0) __syncthreads();  // (scan[1] is read)
    }
  }
  if (chosen != nullptr)
    for (int32_t i = row.taken + tid; i < p.blocks; i += kThreads) chosen[i] = -1;
  __syncthreads();
  int32_t* out = p.sel_indices + before;
  const bool shifts = (p.page_size & (p.page_size - 1)) == 0;
  const int shift = __ffs(p.page_size) - 1;
  // (unsigned: a row may have close to 2^31 tokens)
  for (uint32_t t = tid; t < static_cast<uint32_t>(row.tokens); t += kThreads) {
    const uint32_t at = shifts ? t >> shift : t / static_cast<uint32_t>(p.page_size);
    if (!MLA_DCHECK(at < static_cast<uint32_t>(row.taken) && before + t < p.indices_len, p.err)) return;
    const int32_t start = rows[at];
    out[t] = start < 0 ? -1 : start + static_cast<int32_t>(t - at * p.page_size);
  }
}

}  // namespace

cudaError_t block_select_prepare() {
  for (auto kernel : {block_select_kernel<1>, block_select_kernel<4>, block_select_kernel<8>, block_select_kernel<16>, block_select_kernel<0>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MLA_SELECT_MAX_BLOCKS * 4);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Scores in registers where a row's pages fit them, as few a thread as do (64 rows of 4096 pages: 8.3
// us with eight, 12.2 with sixteen; of 16384 from L2 22.6).
cudaError_t launch_block_select(const BlockSelectParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.batch);
  const size_t smem = static_cast<size_t>(p.blocks) * 4;
  if (p.max_pages <= kThreads) return launch_dependent(block_select_kernel<1>, grid, kThreads, smem, stream, p);
  if (p.max_pages <= 4 * kThreads) return launch_dependent(block_select_kernel<4>, grid, kThreads, smem, stream, p);
  if (p.max_pages <= 8 * kThreads) return launch_dependent(block_select_kernel<8>, grid, kThreads, smem, stream, p);
  if (p.max_pages <= 16 * kThreads) return launch_dependent(block_select_kernel<16>, grid, kThreads, smem, stream, p);
  return launch_dependent(block_select_kernel<0>, grid, kThreads, smem, stream, p);
}

}  // namespace mla
