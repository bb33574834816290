// mla_block_means: the mean cache row of every page that a step has written to.
//
// Of the new tokens' slots, in order, one ends its page when the next slot is not the
// row behind it or lies on another page; the page then holds the rows from its first
// one up to that slot.  A block has an equal share of the tokens, one behind the other, so that
// shares have about as many ends each; it finds them and sums their pages' rows, which lie one
// behind the other, from shared memory, where bulk copies bring them 36 KB at a time: a part of
// a page or several small ones.  A thread sums two dims of all rows in float32, so no threads
// join (16 bytes a thread and every eighth row cost pages of 16 a quarter more, pages of 64 4 %
// less).  Five blocks an SM: while one waits for memory the others sum (nine ragged prompts
// of up to 8000 new tokens: four 8.9 us, five 7.0, six 7.8; loads into registers instead of copies
// took 38 us for their bf16 cache, where these take 12).  Bound by the trips to memory, slots and
// then rows, and by the block that has the most pages (10.7 us where tokens were dealt out one by
// one, which left some blocks four): 27 MB of rows in 7.0 us, 3.9 TB/s.
#include <cuda_fp16.h>

#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kThreads = 288;
constexpr int kRingBytes = 64 * kQkDim;  // of rows under way: 64 of e4m3 codes, 32 of bf16
constexpr int kMaxSlots = 8;             // copies that they are, at most
constexpr int kBlocksPerSm = 5;

template <bool kE4m3>
constexpr int kRowBytes = kE4m3 ? kQkDim : 2 * kQkDim;
template <bool kE4m3>
constexpr int kRingRows = kRingBytes / kRowBytes<kE4m3>;
static_assert(2 * kThreads == kQkDim, "a thread two dims");

// A thread's two dims of a row, added to `x` and `y`.
template <bool kE4m3>
__device__ __forceinline__ void add_row(const uint8_t* row, float& x, float& y) {
  if constexpr (kE4m3) {
    const uint32_t h = cvt_e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(row));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x += v.x;
    y += v.y;
  } else {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(row);
    x += __uint_as_float(v << 16);
    y += __uint_as_float(v & 0xFFFF0000u);
  }
}

// The rows of the pages that end at `ends`, a chunk of up to `most` at a time.
struct Chunks {
  const int32_t* ends;
  int32_t count, page_size, most;
  int32_t e = 0, row = 0;     // page of the list, first row of the chunk
  int32_t page = 0, rows = 0; // the page's number and rows
  __device__ __forceinline__ Chunks(const int32_t* list, int32_t n, int32_t size, int32_t rows)
      : ends(list), count(n), page_size(size), most(rows) {
    open();
  }
  __device__ __forceinline__ void open() {
    if (e >= count) return;
    page = ends[e] / page_size;
    rows = ends[e] - page * page_size + 1;
  }
  __device__ __forceinline__ bool live() const { return e < count; }
  __device__ __forceinline__ int32_t here() const { return min(most, rows - row); }
  __device__ __forceinline__ bool ends_page() const { return row + most >= rows; }
  __device__ __forceinline__ void step() {
    row += most;
    if (row < rows) return;
    row = 0;
    ++e;
    open();
  }
};

// Bounded wait on a copy; false when it ran out (reported).
__device__ __forceinline__ bool landed(uint32_t bar, uint32_t parity, int32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - start > kWaitLimitCycles) {
      atomicOr(err, MLA_DERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) block_means_kernel(const BlockMeansParams p) {
  extern __shared__ __align__(128) uint8_t ring[];  // [slots][most rows]
  __shared__ uint64_t full[kMaxSlots];
  __shared__ int32_t ends[kThreads];
  __shared__ int32_t num_ends;
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int s = 0; s < kMaxSlots; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_mbar_init();
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  // A slot holds a page, or as much of it as the ring; the number of slots is a power of two.
  const int32_t most = min(p.page_size, kRingRows<kE4m3>);
  const uint32_t log_slots = 31 - __clz(min(kMaxSlots, kRingRows<kE4m3> / most)), slots = 1u << log_slots;
  const float scale = kE4m3 ? __ldg(p.kv_scale) : 1.0f;
  const int64_t share = (p.num_tokens + gridDim.x - 1) / gridDim.x, end = min(p.num_tokens, (blockIdx.x + 1) * share);
  uint32_t filled = 0, used = 0;  // chunks copied (thread 0) and summed, of all rounds
  bool ok = true;
  for (int64_t base = blockIdx.x * share; base < end && ok; base += kThreads) {
    __syncthreads();  // (the list is read)
    if (tid == 0) num_ends = 0;
    __syncthreads();
    const int64_t t = base + tid;
    if (t < end) {
      const int32_t slot = __ldg(p.slots + t);
      const int32_t after = t + 1 < p.num_tokens ? __ldg(p.slots + t + 1) : -1;
      if (slot >= p.limit) {
        atomicOr(p.err, MLA_DERR_KV_INDEX);
      } else if (slot >= 0 && (after != slot + 1 || (slot + 1) % p.page_size == 0)) {
        const int32_t at = atomicAdd(&num_ends, 1);
        if (MLA_DCHECK(at < kThreads, p.err)) ends[at] = slot;
      }
    }
    __syncthreads();
    const int32_t n = num_ends;
    Chunks ahead(ends, n, p.page_size, most), now(ends, n, p.page_size, most);
    // (thread 0) the next chunk into its slot, whose last one is summed
    auto fill = [&] {
      const int32_t rows = ahead.here(), bytes = rows * kRowBytes<kE4m3>;
      const int64_t first = static_cast<int64_t>(ahead.page) * p.page_size + ahead.row;
      const uint32_t s = filled & (slots - 1), bar = smem_u32(&full[s]);
      mbar_arrive_expect_tx(bar, bytes);
      if (MLA_DCHECK(first >= 0 && first + rows <= p.kv_rows && rows > 0, p.err))
        bulk_load(smem_u32(ring) + s * most * kRowBytes<kE4m3>, p.cache + first * kRowBytes<kE4m3>, bytes, bar);
      ++filled;
      ahead.step();
    };
    if (tid == 0)
      for (uint32_t s = 0; s < slots && ahead.live(); ++s) fill();
    float x = 0.0f, y = 0.0f;
    for (; now.live(); now.step(), ++used) {
      const uint32_t s = used & (slots - 1);
      ok = landed(smem_u32(&full[s]), used >> log_slots & 1, p.err);
      const uint8_t* rows = ring + s * most * kRowBytes<kE4m3> + tid * (kRowBytes<kE4m3> / kThreads);
      const int32_t here = now.here();
#pragma unroll 8
      for (int32_t r = 0; r < here; ++r) add_row<kE4m3>(rows + r * kRowBytes<kE4m3>, x, y);
      ok = __syncthreads_and(ok);
      if (!ok) break;
      if (tid == 0 && ahead.live()) fill();
      if (now.ends_page()) {
        const float count = static_cast<float>(now.rows);
        uint32_t packed;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed) : "f"(y / count * scale), "f"(x / count * scale));
        if (MLA_DCHECK(now.page >= 0 && static_cast<int64_t>(now.page) * p.page_size < p.limit, p.err))
          reinterpret_cast<uint32_t*>(p.means + static_cast<int64_t>(now.page) * kQkDim)[tid] = packed;
        x = y = 0.0f;
      }
    }
  }
  // Given up: the copies in flight land before the block's memory is given up.
  if (!ok && tid == 0)
    for (uint32_t f = filled > slots ? filled - slots : 0; f < filled; ++f)
      landed(smem_u32(&full[f & (slots - 1)]), f >> log_slots & 1, p.err);
}

}  // namespace

cudaError_t block_means_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(block_means_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(block_means_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
}

cudaError_t launch_block_means(const BlockMeansParams& p, bool e4m3, int32_t num_sms, cudaStream_t stream) {
  const int64_t blocks = kBlocksPerSm * static_cast<int64_t>(num_sms);
  const int64_t grid = p.num_tokens < blocks ? p.num_tokens : blocks;
  return e4m3 ? launch_dependent(block_means_kernel<true>, static_cast<unsigned>(grid), kThreads, kRingBytes, stream, p)
              : launch_dependent(block_means_kernel<false>, static_cast<unsigned>(grid), kThreads, kRingBytes, stream, p);
}

}  // namespace mla
