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
// for tcgen05, whose tiles have 128.  Several products' operands are under way at a time, across
// the groups of 16 pages that a warp works through.  64 rows of up to 131072 tokens in pages of
// 64 take 21.7 us, 115 MB at 5.3 TB/s (one group a warp at all sizes 26.8; 32 bytes a lane 29.8); 4 rows of up to
// 8192 4.8 us, launch and three trips to memory.  Two query tokens take 23.7; three and four, 30.7 and
// 31.9, have half as many bytes under way, since their sums need the registers, and read 4 KB of
// queries from shared memory for each KB of means.
#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kWarpPages = 16;                       // two columns' worth of 8
constexpr int kMaxGroups = 4;                        // of 16 pages, of a warp
constexpr int kChunks = kQkDim / 32;                 // of 32 dims: two products
// Warps of a block, which share the queries in shared memory, and chunks of the means that a warp
// has under way.  Four tokens' queries and sums leave room for two blocks of four warps an SM, so
// where there is work for more warps, blocks are wide (four tokens, 64 rows of up to 131072: 41
// us, wide 32; of up to 32768: 17.8, 13.5); with less, the queries come faster to more blocks (4
// rows of up to 8192: 6.9, wide 8.4).
template <bool kWide>
constexpr int kWarpsOf = kWide ? 8 : 4;
template <bool kWide>
constexpr int kAheadOf = kWide ? 3 : 6;
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

// 16 bytes that are not read again: past L1 (22.9 us with it, 22.3 without, 64 rows of up to 131072).
__device__ __forceinline__ uint4 load_once(const uint8_t* src) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src));
  return v;
}

// kTokens: query tokens that are scored together; rows of more take the means again.
template <int kTokens, bool kWide>
__global__ void __launch_bounds__(32 * kWarpsOf<kWide>, kWide ? 2 : 0) block_scores_kernel(const BlockScoresParams p, int32_t groups) {
  constexpr int kWarps = kWarpsOf<kWide>, kThreads = 32 * kWarps, kAhead = kAheadOf<kWide>;
  static_assert(kChunks % kAhead == 0, "whole groups of chunks");
  extern __shared__ __align__(16) uint8_t sq[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3, col = lane >> 2;
  const int32_t b = blockIdx.y;
  const int32_t block0 = static_cast<int32_t>(blockIdx.x) * kWarps * kWarpPages * groups;  // the block's first page
  const int32_t first = block0 + warp * kWarpPages * groups;                               // and the warp's
  pdl_wait_primary();
  pdl_launch_dependents();
  const int32_t qs = __ldg(p.qo_indptr + b), qe = __ldg(p.qo_indptr + b + 1);
  const int32_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
  const int64_t len = static_cast<int64_t>(ke) - ks;
  const uint32_t pages = pages_of(len, p.page_size);
  const bool bad_q = qs < 0 || qe < qs || qe > p.total_q, bad_k = ks < 0 || len < 0 || pages > static_cast<uint32_t>(p.max_pages);
  if ((bad_q || bad_k) && tid == 0 && blockIdx.x == 0)
    atomicOr(p.err, (bad_q ? MLA_DERR_QO_INDPTR : 0) | (bad_k ? MLA_DERR_KV_INDPTR : 0));
  const int32_t n = bad_q || bad_k ? 0 : static_cast<int32_t>(pages);
  const int32_t tokens = bad_q ? 0 : qe - qs;
  float* out = p.scores + static_cast<int64_t>(b) * p.scores_stride;
  if (block0 >= n || tokens == 0) {  // (the same for the whole block)
    for (int32_t j = block0 + tid; j < min(p.max_pages, block0 + kWarps * kWarpPages * groups); j += kThreads) out[j] = -INFINITY;
    return;
  }

  // The pages of this lane's column, in either half of each group; -1 where there is none.
  int32_t page[kMaxGroups][2];
#pragma unroll
  for (int u = 0; u < kMaxGroups; ++u)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t j = first + kWarpPages * u + 8 * i + col;
      const bool here = u < groups && j < n && MLA_DCHECK(j < p.max_pages, p.err);
      page[u][i] = here ? __ldg(p.block_table + static_cast<int64_t>(b) * p.table_stride + j) : -1;
      if (here && (page[u][i] < 0 || page[u][i] >= p.num_pages)) {
        atomicOr(p.err, MLA_DERR_KV_INDEX);
        page[u][i] = -1;
      }
    }
  const uint8_t* means = reinterpret_cast<const uint8_t*>(p.means) + 16 * quad;
  auto load = [&](int32_t id, int c) {
    return id >= 0 && MLA_DCHECK(id < p.num_pages, p.err) ? load_once(means + static_cast<int64_t>(id) * (2 * kQkDim) + 64 * c)
                   : make_uint4(0, 0, 0, 0);
  };
  // (a warp behind the row's pages only brings its share of the queries)
  const int32_t live = min(groups, max(0, (n - first + kWarpPages - 1) / kWarpPages));

  for (int32_t t0 = 0; t0 < tokens; t0 += kTokens) {
    const int32_t here_tokens = min(kTokens, tokens - t0);
    if (t0 > 0) __syncthreads();
    constexpr int kRowPieces = kQkDim * 2 / 16;
    for (int i = tid; i < here_tokens * kNumHeads * kRowPieces; i += kThreads) {
      const int row = i / kRowPieces, at = i % kRowPieces;
      const uint4* q = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(qs + t0) * kNumHeads + row) * kQkDim);
      if (MLA_DCHECK(qs >= 0 && qs + t0 + row / kNumHeads < p.total_q && row < kTokens * kNumHeads, p.err))
        cp_async_16(smem_u32(sq + row * kQStride + 16 * at), q + at);
    }
    uint4 v[2][kAhead];
#pragma unroll
    for (int c = 0; c < kAhead; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) v[i][c] = load(page[0][i], c);
    cp_async_wait_all();
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMaxGroups; ++u) {
      if (u >= live) break;
      float acc[kTokens][2][4] = {};
#pragma unroll 1
      for (int c0 = 0; c0 < kChunks; c0 += kAhead) {
        // the chunks that follow: this group's, or the next one's first
        const bool last = c0 + kAhead == kChunks;
        const int32_t after = last ? 0 : c0 + kAhead;
        int32_t from[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) from[i] = !last ? page[u][i] : u + 1 < kMaxGroups && u + 1 < live ? page[u + 1 < kMaxGroups ? u + 1 : u][i] : -1;
#pragma unroll
        for (int c = 0; c < kAhead; ++c) {
          const uint4 v0 = v[0][c], v1 = v[1][c];
#pragma unroll
          for (int i = 0; i < 2; ++i) v[i][c] = load(from[i], after + c);
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
      // Over the tokens, the lane's two heads of each page, and the heads: lanes with the same
      // quad hold the same two pages.
      float best[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int t = 0; t < kTokens; ++t)
            if (t < here_tokens) x = max_nan(x, max_nan(acc[t][i][e], acc[t][i][2 + e]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, d));
          best[i][e] = x;
        }
      // Column 2 quad + e is the page of the lanes whose col is that; they know whether it counts.
      uint32_t valid[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) valid[i] = __ballot_sync(0xffffffffu, page[u][i] >= 0);
      if (col < 2) {  // lanes 0-3 the first half, 4-7 the second
        const int i = col;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 2 * quad + e;
          const int32_t j = first + kWarpPages * u + 8 * i + c;
          const bool counts = ((i ? valid[1] : valid[0]) >> (4 * c)) & 1;
          float x = counts ? (i ? best[1][e] : best[0][e]) * (1.0f / 24.0f) : -INFINITY;
          if (j < p.max_pages && MLA_DCHECK(j >= 0 && j < p.max_pages, p.err)) out[j] = t0 > 0 ? max_nan(x, out[j]) : x;  // (the lane's own, of the tokens before)
        }
      }
    }
  }
  // behind the row's pages
  for (int32_t j = first + kWarpPages * live + lane; j < min(p.max_pages, first + kWarpPages * groups); j += 32) out[j] = -INFINITY;
}

// A warp's groups of 16 pages: one where the warps then fit the GPU at once (16 an SM), up to
// four where they would follow one another, since a warp's start is two trips to memory.
int64_t warps_of(const BlockScoresParams& p) { return static_cast<int64_t>(p.batch) * ((p.max_pages + kWarpPages - 1) / kWarpPages); }
int32_t warp_groups(const BlockScoresParams& p, int32_t num_sms) {
  const int64_t groups = warps_of(p) / (16 * static_cast<int64_t>(num_sms));
  return static_cast<int32_t>(groups < 1 ? 1 : groups > kMaxGroups ? kMaxGroups : groups);
}

template <int kTokens, bool kWide>
cudaError_t launch_tokens(const BlockScoresParams& p, int32_t groups, cudaStream_t stream) {
  const int64_t pages = static_cast<int64_t>(kWarpsOf<kWide>) * kWarpPages * groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.max_pages + pages - 1) / pages), static_cast<unsigned>(p.batch));
  cfg.blockDim = dim3(32 * kWarpsOf<kWide>);
  cfg.dynamicSmemBytes = kTokens * kQTokenBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_scores_kernel<kTokens, kWide>, p, groups);
}

}  // namespace

cudaError_t block_scores_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(block_scores_kernel<2, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kQTokenBytes);
  if (e != cudaSuccess) return e;
  for (auto kernel : {block_scores_kernel<4, false>, block_scores_kernel<4, true>}) {
    const cudaError_t f = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kQTokenBytes);
    if (f != cudaSuccess) return f;
  }
  return cudaSuccess;
}

// The rows' tokens are on the GPU; a row has total_q / batch of them as a rule, and any
// number is computed.
cudaError_t launch_block_scores(const BlockScoresParams& p, int32_t num_sms, cudaStream_t stream) {
  const int32_t groups = warp_groups(p, num_sms);
  if (p.total_q <= p.batch) return launch_tokens<1, false>(p, groups, stream);
  if (p.total_q <= 2 * static_cast<int64_t>(p.batch)) return launch_tokens<2, false>(p, groups, stream);
  return warps_of(p) <= 8 * static_cast<int64_t>(num_sms) ? launch_tokens<4, false>(p, groups, stream) : launch_tokens<4, true>(p, groups, stream);
}

}  // namespace mla
