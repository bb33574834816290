// mla_block_means: the mean cache row of every page that a step has written to.
//
// Of the new tokens' slots, in order, one ends its page when the next slot is not the
// row behind it or lies on another page; the page then holds the rows from its first
// one up to that slot.  A block walks every gridDim-th token, finds the ends among them
// and averages their pages in float32, one with all of its threads (16 bytes of every
// eighth row each, bf16 every fourth; then the sums of a dim through shared memory), or
// two or four side by side where it has more.  Bound by the trips to memory, slots and
// then rows, and by the blocks that have the most pages.
#include <cuda_fp16.h>

#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kThreads = 288;
constexpr int kBatch = 8;  // rows of a thread loaded together

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

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) block_means_kernel(const BlockMeansParams p) {
  constexpr int kRowBytes = kE4m3 ? kQkDim : 2 * kQkDim;
  constexpr int kPieces = kRowBytes / 16, kGroups = kThreads / kPieces, kDims = kE4m3 ? 16 : 8;
  static_assert(kPieces * kGroups == kThreads && kPieces * kDims == kQkDim, "a thread a piece");
  __shared__ float part[kGroups][kQkDim];
  __shared__ int32_t ends[kThreads];
  __shared__ int32_t num_ends;
  const int tid = threadIdx.x, piece = tid % kPieces, group = tid / kPieces;
  pdl_wait_primary();
  pdl_launch_dependents();
  const float scale = kE4m3 ? __ldg(p.kv_scale) : 1.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t base = blockIdx.x; base < p.num_tokens; base += step) {
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
    // Teams of threads, a page each.
    const int teams = n >= 3 ? 4 : n < 1 ? 1 : n, apart = kGroups / teams;  // (rows of a thread lie `apart`)
    const int team = group / apart;
    for (int32_t e0 = 0; e0 < n; e0 += teams) {
      float sum[kDims] = {};
      if (e0 + team < n) {
        const int32_t slot = ends[e0 + team], page = slot / p.page_size;
        const int32_t rows = slot - page * p.page_size + 1;
        const int64_t first = static_cast<int64_t>(page) * p.page_size;
        const uint8_t* src = p.cache + first * kRowBytes + piece * 16;
        for (int32_t r0 = group % apart; r0 < rows; r0 += kBatch * apart) {
          uint4 v[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int32_t r = r0 + i * apart;
            v[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && MLA_DCHECK(first + r < p.kv_rows, p.err))
              v[i] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r) * kRowBytes));
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) add_piece<kE4m3>(v[i], sum);
        }
      }
#pragma unroll
      for (int i = 0; i < kDims; i += 4)
        *reinterpret_cast<float4*>(&part[group][piece * kDims + i]) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
      __syncthreads();
      for (int u = 0; u < teams && e0 + u < n; ++u) {
        float x = 0.0f, y = 0.0f;
        for (int i = u * apart; i < (u + 1) * apart; ++i) {
          const float2 w = *reinterpret_cast<const float2*>(&part[i][2 * tid]);
          x += w.x;
          y += w.y;
        }
        const int32_t slot = ends[e0 + u], page = slot / p.page_size;
        const float count = static_cast<float>(slot - page * p.page_size + 1);
        uint32_t packed;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed) : "f"(y / count * scale), "f"(x / count * scale));
        reinterpret_cast<uint32_t*>(p.means + static_cast<int64_t>(page) * kQkDim)[tid] = packed;
      }
      __syncthreads();  // (part is written again)
    }
  }
}

}  // namespace

cudaError_t launch_block_means(const BlockMeansParams& p, bool e4m3, int32_t num_sms, cudaStream_t stream) {
  // Pages end at every page_size-th token, so the blocks' stride shares no small factor
  // with page sizes: the ends then fall on all blocks alike.
  int64_t grid = 4 * static_cast<int64_t>(num_sms) + 1;
  while (grid > 1 && (grid % 2 == 0 || grid % 3 == 0 || grid % 5 == 0 || grid % 7 == 0)) --grid;
  if (grid > p.num_tokens) grid = p.num_tokens;
  return e4m3 ? launch_dependent(block_means_kernel<true>, static_cast<unsigned>(grid), kThreads, 0, stream, p)
              : launch_dependent(block_means_kernel<false>, static_cast<unsigned>(grid), kThreads, 0, stream, p);
}

}  // namespace mla
