// mla_block_scores: what a row's queries score against its pages' mean rows.
//
//   score[b][j] = max over the row's query tokens t and heads h of q[t][h] . mean[page j] / 24
//
// The means are read once, 1152 bytes a page, for 16 heads of up to four query tokens:
// bound by those bytes.  A warp takes 16 pages as the 8 columns of two bf16 products
// (m16n8k16, the heads the rows) and reads them straight into the products' operand
// registers: a lane's 16 bytes of a page are 8 neighbouring dims, which stand for the
// dims that two products expect there; the queries, in shared memory, are read in the
// same order, so the sums are over the same pairs.  At 16 rows a product this is no work
// for tcgen05, whose tiles have 128.
#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpPages = 16;                       // two columns' worth of 8
constexpr int kBlockPages = kWarps * kWarpPages;
constexpr int kChunks = kQkDim / 32;                 // of 32 dims: two products
constexpr int kAhead = 6;                            // chunks loaded together
static_assert(kChunks % kAhead == 0, "whole groups of chunks");
constexpr int kQStride = kQkDim * 2 + 64;            // bytes of a query row in shared memory: no bank twice
constexpr int kQTokenBytes = kNumHeads * kQStride;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The larger of both; a NaN stays, so that bad data is not passed over.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// kTokens: query tokens that are scored together; rows of more take the means again.
template <int kTokens>
__global__ void __launch_bounds__(kThreads) block_scores_kernel(const BlockScoresParams p) {
  extern __shared__ __align__(16) uint8_t sq[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3, col = lane >> 2;
  const int32_t b = blockIdx.y;
  const int32_t first = static_cast<int32_t>(blockIdx.x) * kBlockPages + warp * kWarpPages;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int32_t qs = __ldg(p.qo_indptr + b), qe = __ldg(p.qo_indptr + b + 1);
  const int32_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
  const int64_t len = static_cast<int64_t>(ke) - ks;
  const int64_t pages = (len + p.page_size - 1) / p.page_size;
  const bool bad_q = qs < 0 || qe < qs || qe > p.total_q, bad_k = ks < 0 || len < 0 || pages > p.max_pages;
  if ((bad_q || bad_k) && tid == 0 && blockIdx.x == 0)
    atomicOr(p.err, (bad_q ? MLA_DERR_QO_INDPTR : 0) | (bad_k ? MLA_DERR_KV_INDPTR : 0));
  const int32_t n = bad_q || bad_k ? 0 : static_cast<int32_t>(pages);
  const int32_t tokens = bad_q ? 0 : qe - qs;
  float* out = p.scores + static_cast<int64_t>(b) * p.scores_stride;
  if (static_cast<int32_t>(blockIdx.x) * kBlockPages >= n || tokens == 0) {  // (the same for the whole block)
    const int32_t j = first + lane;
    if (lane < kWarpPages && j < p.max_pages) out[j] = -INFINITY;
    return;
  }

  // The pages of this lane's column in either half, and their rows' pieces.
  const uint8_t* src[2];
  bool here[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t j = first + 8 * i + col;
    int32_t id = j < n ? __ldg(p.block_table + static_cast<int64_t>(b) * p.table_stride + j) : 0;
    here[i] = j < n;
    if (id < 0 || id >= p.num_pages) {
      atomicOr(p.err, MLA_DERR_KV_INDEX);
      here[i] = false;
      id = 0;
    }
    src[i] = reinterpret_cast<const uint8_t*>(p.means) + static_cast<int64_t>(id) * (2 * kQkDim) + 16 * quad;
  }
  float best[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) best[i][0] = best[i][1] = -INFINITY;

  for (int32_t t0 = 0; t0 < tokens; t0 += kTokens) {
    const int32_t here_tokens = min(kTokens, tokens - t0);
    if (t0 > 0) __syncthreads();
    constexpr int kRowPieces = kQkDim * 2 / 16;
    for (int i = tid; i < here_tokens * kNumHeads * kRowPieces; i += kThreads) {
      const int row = i / kRowPieces, at = i % kRowPieces;
      const uint4* q = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(qs + t0) * kNumHeads + row) * kQkDim);
      cp_async_16(smem_u32(sq + row * kQStride + 16 * at), q + at);
    }
    float acc[kTokens][2][4] = {};
    uint4 v[2][kAhead];
#pragma unroll
    for (int c = 0; c < kAhead; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) v[i][c] = here[i] ? __ldg(reinterpret_cast<const uint4*>(src[i] + 64 * c)) : make_uint4(0, 0, 0, 0);
    cp_async_wait_all();
    __syncthreads();
#pragma unroll 1
    for (int c0 = 0; c0 < kChunks; c0 += kAhead) {
#pragma unroll
      for (int c = 0; c < kAhead; ++c) {
        const uint4 v0 = v[0][c], v1 = v[1][c];
        if (c0 + kAhead < kChunks) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            v[i][c] = here[i] ? __ldg(reinterpret_cast<const uint4*>(src[i] + 64 * (c0 + kAhead + c))) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
          if (t >= here_tokens) break;
          const uint8_t* q = sq + t * kQTokenBytes + col * kQStride + 64 * (c0 + c) + 16 * quad;
          const uint4 lo = *reinterpret_cast<const uint4*>(q), hi = *reinterpret_cast<const uint4*>(q + 8 * kQStride);
          mma_16816(acc[t][0], lo.x, hi.x, lo.y, hi.y, v0.x, v0.y);
          mma_16816(acc[t][1], lo.x, hi.x, lo.y, hi.y, v1.x, v1.y);
          mma_16816(acc[t][0], lo.z, hi.z, lo.w, hi.w, v0.z, v0.w);
          mma_16816(acc[t][1], lo.z, hi.z, lo.w, hi.w, v1.z, v1.w);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (t >= here_tokens) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        best[i][0] = max_nan(best[i][0], max_nan(acc[t][i][0], acc[t][i][2]));
        best[i][1] = max_nan(best[i][1], max_nan(acc[t][i][1], acc[t][i][3]));
      }
    }
  }
  // Over the heads: lanes with the same quad hold the same two pages.
#pragma unroll
  for (int d = 4; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) best[i][e] = max_nan(best[i][e], __shfl_xor_sync(0xffffffffu, best[i][e], d));
  // Column 2 quad + e is the page of the lanes whose col is that; their `here` says whether it counts.
  uint32_t valid[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) valid[i] = __ballot_sync(0xffffffffu, here[i]);
  if (col < 2) {  // lanes 0-3 the first half, 4-7 the second
    const int i = col;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = 2 * quad + e;
      const int32_t j = first + 8 * i + c;
      const bool counts = ((i ? valid[1] : valid[0]) >> (4 * c)) & 1;
      const float best_e = i ? best[1][e] : best[0][e];
      if (j < p.max_pages) out[j] = counts ? best_e * (1.0f / 24.0f) : -INFINITY;
    }
  }
}

template <int kTokens>
cudaError_t launch_tokens(const BlockScoresParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.max_pages + kBlockPages - 1) / kBlockPages), static_cast<unsigned>(p.batch));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kTokens * kQTokenBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_scores_kernel<kTokens>, p);
}

}  // namespace

cudaError_t block_scores_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(block_scores_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kQTokenBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(block_scores_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kQTokenBytes);
}

// The rows' tokens are on the GPU; a row has total_q / batch of them as a rule, and any
// number is computed.
cudaError_t launch_block_scores(const BlockScoresParams& p, cudaStream_t stream) {
  if (p.total_q <= p.batch) return launch_tokens<1>(p, stream);
  if (p.total_q <= 2 * static_cast<int64_t>(p.batch)) return launch_tokens<2>(p, stream);
  return launch_tokens<4>(p, stream);
}

}  // namespace mla
