// mla_block_means: the mean cache row of every page that a step has written to.
//
// Of the new tokens' slots, in order, one ends its page when the next slot is not the
// row behind it or lies on another page; the page then holds the rows from its first
// one up to that slot.  A block walks every gridDim-th token, finds the ends among them
// and sums their pages' rows, which lie one behind the other, from shared memory, where
// bulk copies bring them 36 KB at a time.  A thread sums 16 bytes of every eighth row (bf16:
// fourth) in float32, then the sums of a dim go through shared memory.  Four blocks an SM, a
// copy each: while one waits for memory the others sum.  (One block with five copies ahead:
// 36000 new tokens in pages of 64 8.6 us, two with two 6.3, four with one 5.6; loads into
// registers instead of copies take 38 us where these take 15, nine prompts' chunks in a bf16
// cache.)  Bound by the trips to memory, slots and then rows, and by the block that has the
// most pages: nine ragged prompts of up to 8000 new tokens take 10.7 us, 27 MB of rows.
#include <cuda_fp16.h>

#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kThreads = 288;
constexpr int kSlots = 1;          // chunks that a block has copied ahead
constexpr int kSlotBytes = 64 * kQkDim;  // 64 rows of e4m3 codes, 32 of bf16
constexpr int kBlocksPerSm = 4;

template <bool kE4m3>
constexpr int kRowBytes = kE4m3 ? kQkDim : 2 * kQkDim;
template <bool kE4m3>
constexpr int kGroups = kThreads * 16 / kRowBytes<kE4m3>;  // rows that the threads read at a time
static_assert(kGroups<true> * kRowBytes<true> == kThreads * 16 && kGroups<false> * kRowBytes<false> == kThreads * 16,
              "a thread a piece");
template <bool kE4m3>
constexpr int kSmemBytes = kSlots * kSlotBytes + kGroups<kE4m3> * kQkDim * 4;

// 16 bytes of a cache row, added to `sum`.
template <bool kE4m3>
__device__ __forceinline__ void add_piece(const uint4& v, float* sum) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kE4m3) {
      const uint32_t a = cvt_e4m3x2_to_f16x2(static_cast<uint16_t>(w[i])), b = cvt_e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16));
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
      sum[4 * i] += x.x;
      sum[4 * i + 1] += x.y;
      sum[4 * i + 2] += y.x;
      sum[4 * i + 3] += y.y;
    } else {
      sum[2 * i] += __uint_as_float(w[i] << 16);
      sum[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// The rows of the pages that end at `ends`, a chunk of up to a slot's rows at a time.
template <bool kE4m3>
struct Chunks {
  static constexpr int kRows = kSlotBytes / kRowBytes<kE4m3>;
  const int32_t* ends;
  int32_t count, page_size;
  int32_t e = 0, row = 0;     // page of the list, first row of the chunk
  int32_t page = 0, rows = 0; // the page's number and rows
  __device__ __forceinline__ Chunks(const int32_t* list, int32_t n, int32_t size) : ends(list), count(n), page_size(size) { open(); }
  __device__ __forceinline__ void open() {
    if (e >= count) return;
    page = ends[e] / page_size;
    rows = ends[e] - page * page_size + 1;
  }
  __device__ __forceinline__ bool live() const { return e < count; }
  __device__ __forceinline__ int32_t here() const { return min(kRows, rows - row); }
  __device__ __forceinline__ bool ends_page() const { return row + kRows >= rows; }
  __device__ __forceinline__ void step() {
    row += kRows;
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
  constexpr int kPieces = kRowBytes<kE4m3> / 16, kDims = kE4m3 ? 16 : 8;
  extern __shared__ __align__(128) uint8_t ring[];  // [kSlots][kSlotBytes], then the groups' sums
  float* part = reinterpret_cast<float*>(ring + kSlots * kSlotBytes);  // [kGroups][576]
  __shared__ uint64_t full[kSlots];
  __shared__ int32_t ends[kThreads];
  __shared__ int32_t num_ends;
  const int tid = threadIdx.x, piece = tid % kPieces, group = tid / kPieces;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_mbar_init();
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  const float scale = kE4m3 ? __ldg(p.kv_scale) : 1.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  uint32_t filled = 0, used = 0;  // chunks copied (thread 0) and summed, of all rounds
  bool ok = true;
  for (int64_t base = blockIdx.x; base < p.num_tokens && ok; base += step) {
    __syncthreads();  // (the list is read)
    if (tid == 0) num_ends = 0;
    __syncthreads();
    const int64_t t = base + static_cast<int64_t>(tid) * gridDim.x;
    if (t < p.num_tokens) {
      const int32_t slot = __ldg(p.slots + t);
      const int32_t after = t + 1 < p.num_tokens ? __ldg(p.slots + t + 1) : -1;
      if (slot >= p.limit) {
        atomicOr(p.err, MLA_DERR_KV_INDEX);
      } else if (slot >= 0 && (after != slot + 1 || (slot + 1) % p.page_size == 0)) {
        ends[atomicAdd(&num_ends, 1)] = slot;
      }
    }
    __syncthreads();
    const int32_t n = num_ends;
    Chunks<kE4m3> ahead(ends, n, p.page_size), now(ends, n, p.page_size);
    // (thread 0) the next chunk into its slot, whose last one is summed
    auto fill = [&] {
      const int32_t rows = ahead.here(), bytes = rows * kRowBytes<kE4m3>;
      const int64_t first = static_cast<int64_t>(ahead.page) * p.page_size + ahead.row;
      const uint32_t s = filled % kSlots, bar = smem_u32(&full[s]);
      mbar_arrive_expect_tx(bar, bytes);
      if (MLA_DCHECK(first >= 0 && first + rows <= p.kv_rows && rows > 0, p.err))
        bulk_load(smem_u32(ring) + s * kSlotBytes, p.cache + first * kRowBytes<kE4m3>, bytes, bar);
      ++filled;
      ahead.step();
    };
    if (tid == 0)
      for (int s = 0; s < kSlots && ahead.live(); ++s) fill();
    float sum[kDims] = {};
    for (; now.live(); now.step(), ++used) {
      const uint32_t s = used % kSlots;
      ok = landed(smem_u32(&full[s]), used / kSlots & 1, p.err);
      const uint4* rows = reinterpret_cast<const uint4*>(ring + s * kSlotBytes);
      const int32_t here = now.here();
#pragma unroll 4
      for (int32_t r = group; r < here; r += kGroups<kE4m3>) add_piece<kE4m3>(rows[r * kPieces + piece], sum);
      if (now.ends_page()) {
#pragma unroll
        for (int i = 0; i < kDims; i += 4) {
          *reinterpret_cast<float4*>(&part[group * kQkDim + piece * kDims + i]) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
          sum[i] = sum[i + 1] = sum[i + 2] = sum[i + 3] = 0.0f;
        }
      }
      ok = __syncthreads_and(ok);
      if (!ok) break;
      if (tid == 0 && ahead.live()) fill();
      if (now.ends_page()) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int g = 0; g < kGroups<kE4m3>; ++g) {
          const float2 w = *reinterpret_cast<const float2*>(&part[g * kQkDim + 2 * tid]);
          x += w.x;
          y += w.y;
        }
        const float count = static_cast<float>(now.rows);
        uint32_t packed;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed) : "f"(y / count * scale), "f"(x / count * scale));
        reinterpret_cast<uint32_t*>(p.means + static_cast<int64_t>(now.page) * kQkDim)[tid] = packed;
        __syncthreads();  // (part is written again)
      }
    }
  }
  // Given up: the copies in flight land before the block's memory is given up.
  if (!ok && tid == 0)
    for (uint32_t f = filled > kSlots ? filled - kSlots : 0; f < filled; ++f) landed(smem_u32(&full[f % kSlots]), f / kSlots & 1, p.err);
}

}  // namespace

cudaError_t block_means_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(block_means_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<true>);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(block_means_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<false>);
}

cudaError_t launch_block_means(const BlockMeansParams& p, bool e4m3, int32_t num_sms, cudaStream_t stream) {
  // Pages end at every page_size-th token, so the blocks' stride shares no small factor
  // with page sizes: the ends then fall on all blocks alike.
  const int64_t blocks = kBlocksPerSm * static_cast<int64_t>(num_sms);
  int64_t grid = blocks;
  while (grid > 1 && (grid % 2 == 0 || grid % 3 == 0 || grid % 5 == 0 || grid % 7 == 0)) --grid;
  if (p.num_tokens <= blocks) grid = p.num_tokens;
  return e4m3 ? launch_dependent(block_means_kernel<true>, static_cast<unsigned>(grid), kThreads, kSmemBytes<true>, stream, p)
              : launch_dependent(block_means_kernel<false>, static_cast<unsigned>(grid), kThreads, kSmemBytes<false>, stream, p);
}

}  // namespace mla
