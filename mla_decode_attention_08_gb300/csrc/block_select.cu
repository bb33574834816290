// mla_block_select: the pages that each row attends, as the decode step's page table.
//
// Of a row's pages the first `sink` and the last `recent` are always taken, and of the
// rest those with the highest scores, the lower page where two are alike.  The last page
// is always among them, so the number of chosen tokens follows from the lengths alone:
// every block forms the prefix sums over all rows for itself, and one launch does the
// step.  A block then finds its row's threshold, the score of the last page that is
// taken, by radix selection (four digits of 8 bits of the scores as ordered integers,
// counted in shared memory), walks the pages in order and writes them out.
#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Scores as integers in the same order; both zeros are alike, and a NaN counts as the
// highest, so that it is not passed over.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct RowCount {
  int32_t pages, taken, tokens;
  bool bad;
};
__device__ __forceinline__ RowCount count_row(const BlockSelectParams& p, int32_t b) {
  const int32_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
  const int64_t len = static_cast<int64_t>(ke) - ks;
  RowCount r;
  const int64_t pages = (len + p.page_size - 1) / p.page_size;
  r.bad = ks < 0 || len < 0 || pages > p.max_pages;
  r.pages = r.bad ? 0 : static_cast<int32_t>(pages);
  r.taken = min(r.pages, p.blocks);
  // all pages but the last are full
  r.tokens = r.bad ? 0 : static_cast<int32_t>(len) - (r.pages - r.taken) * p.page_size;
  return r;
}

__global__ void __launch_bounds__(kThreads) block_select_kernel(const BlockSelectParams p) {
  extern __shared__ int32_t rows[];  // [blocks]: first cache row of each chosen page, or -1
  __shared__ uint32_t counts[256];
  __shared__ int64_t sums[kWarps], totals[kWarps];
  __shared__ int32_t warp_ties[kWarps], warp_taken[kWarps];
  __shared__ uint32_t digit, above;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t b = blockIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();

  // Tokens of the rows before this one, and of all rows.
  int64_t before = 0, all = 0;
  bool bad = false;
  for (int32_t r = tid; r < p.batch; r += kThreads) {
    const RowCount c = count_row(p, r);
    all += c.tokens;
    if (r < b) before += c.tokens;
    bad = bad || c.bad;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
  if (lane == 0) {
    sums[warp] = before;
    totals[warp] = all;
  }
  bad = __syncthreads_or(bad);
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += sums[w];
    all += totals[w];
  }
  const bool full = all > p.indices_len;
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
  if (tid == 0 && b == p.batch - 1) p.sel_indptr[p.batch] = static_cast<int32_t>(all);
  const float* scores = p.scores + static_cast<int64_t>(b) * p.scores_stride;
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.table_stride;

  // The threshold: of the middle pages those above it are taken, and `ties` of those at it.
  const int32_t lo = p.sink, hi = row.pages - p.recent;
  uint32_t threshold = 0;
  int32_t ties = 0;
  const bool choose = row.pages > p.blocks;
  if (choose) {
    uint32_t want = static_cast<uint32_t>(p.blocks - p.sink - p.recent);  // still to be found
    if (want == 0) threshold = 0xFFFFFFFFu;
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) counts[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int32_t j = lo + tid; j < hi; j += kThreads) {
        const uint32_t key = ordered(scores[j]);
        if ((key & mask) == threshold) atomicAdd(&counts[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      // The highest digit d for which the pages with a digit of d or more are enough.
      if (warp == 0) {
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += counts[8 * lane + i];
        uint32_t higher = mine;  // of lanes above, inclusive
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t v = __shfl_down_sync(0xffffffffu, higher, d);
          if (lane + d < 32) higher += v;
        }
        uint32_t past = higher - mine;
        if (past < want && higher >= want) {
          for (int i = 7; i >= 0; --i) {
            const uint32_t c = counts[8 * lane + i];
            if (past + c >= want) {
              digit = 8 * lane + i;
              above = past;
              break;
            }
            past += c;
          }
        }
      }
      __syncthreads();
      threshold |= digit << shift;
      want -= above;
    }
    ties = static_cast<int32_t>(want);
  }

  // The pages in order: a page's place among the chosen is the number before it.
  int32_t done_ties = 0, done = 0;
  for (int32_t j0 = 0; j0 < row.pages; j0 += kThreads) {
    const int32_t j = j0 + tid;
    const bool in = j < row.pages;
    bool take = in, tie = false;
    if (choose && in && j >= lo && j < hi) {
      const uint32_t key = ordered(scores[j]);
      tie = ties > 0 && key == threshold;
      take = key > threshold;
    }
    const uint32_t tie_mask = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_ties[warp] = __popc(tie_mask);
    __syncthreads();
    int32_t rank = done_ties + __popc(tie_mask & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) rank += warp_ties[w];
      done_ties += warp_ties[w];
    }
    if (tie && rank < ties) take = true;
    const uint32_t mask = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_taken[warp] = __popc(mask);
    __syncthreads();
    int32_t place = done + __popc(mask & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) place += warp_taken[w];
      done += warp_taken[w];
    }
    if (take && place < p.blocks) {
      const int32_t id = table[j];
      const bool ok = id >= 0 && id < p.num_pages;
      if (!ok) atomicOr(p.err, MLA_DERR_KV_INDEX);
      rows[place] = ok ? id * p.page_size : -1;
      if (chosen != nullptr) chosen[place] = j;
    }
  }
  if (chosen != nullptr)
    for (int32_t i = row.taken + tid; i < p.blocks; i += kThreads) chosen[i] = -1;
  __syncthreads();
  int32_t* out = p.sel_indices + before;
  for (int32_t t = tid; t < row.tokens; t += kThreads) {
    const int32_t at = t / p.page_size, first = rows[at];
    out[t] = first < 0 ? -1 : first + (t - at * p.page_size);
  }
}

}  // namespace

cudaError_t block_select_prepare() {
  return cudaFuncSetAttribute(block_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MLA_SELECT_MAX_BLOCKS * 4);
}

cudaError_t launch_block_select(const BlockSelectParams& p, cudaStream_t stream) {
  return launch_dependent(block_select_kernel, static_cast<unsigned>(p.batch), kThreads, static_cast<size_t>(p.blocks) * 4, stream, p);
}

}  // namespace mla
