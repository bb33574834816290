// mla_attn_merge: joins attention over disjoint keys by the pieces'
// log-sum-exps.
//
// With m = max_s lse_s (0 if every piece is empty) and w_s = exp(lse_s - m):
// out = sum_s w_s part_s / sum_s w_s and lse = m + log sum_s w_s.  A thread owns
// eight values of a row: it reads the row's few lses (the row's threads read
// the same ones) and each piece once.  Bound by the bytes of the pieces.
#include "ops.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 4;  // pieces whose loads are in flight together

template <bool kF32>
struct Piece;
template <>
struct Piece<false> {
  uint4 v = {};
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    v = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : (i < 4 ? v.y : (i < 6 ? v.z : v.w));
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};
template <>
struct Piece<true> {
  float4 a = {}, b = {};
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    a = __ldcs(p);
    b = __ldcs(p + 1);
  }
  __device__ __forceinline__ float get(int i) const {
    const float4& q = i < 4 ? a : b;
    return (i & 3) == 0 ? q.x : ((i & 3) == 1 ? q.y : ((i & 3) == 2 ? q.z : q.w));
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Whether `token` is one that mla_prefill_fwd has computed: it belongs to a row,
// and the row's tokens and keys lie in their tensors.  (A batch whose keys are
// split has few rows.)
__device__ __forceinline__ bool in_a_row(const MergeParams& p, int64_t token) {
  for (int32_t b = 0; b < p.batch; ++b) {
    const int32_t qs = __ldg(p.qo_indptr + b), qe = __ldg(p.qo_indptr + b + 1);
    if (token < qs || token >= qe) continue;
    const int32_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
    if (qs >= 0 && qe <= p.total_q && ks >= 0 && ke >= ks && ke <= p.total_kv &&
        ke - ks <= MLA_PREFILL_MAX_ROW_KEYS)
      return true;
  }
  return false;
}

// The first pieces' values are loaded beside the log-sum-exps, before it is known
// which of them count: one trip to memory instead of two.  Four pieces of 16384 x
// 16 rows of 128: 67 -> 55 us, 6.1 TB/s of a measured 6.7.
template <bool kF32>
__global__ void __launch_bounds__(kThreads) attn_merge_kernel(const MergeParams p, int32_t chunk_shift) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t chunks = static_cast<uint32_t>(p.dim) >> 3;
  const int64_t row = chunk_shift >= 0 ? i >> chunk_shift : i / chunks;
  const int dim0 = 8 * static_cast<int>(i - row * chunks);
  pdl_wait_primary();
  pdl_launch_dependents();
  if (row >= p.rows) return;
  if (p.qo_indptr != nullptr && !in_a_row(p, row / p.heads)) return;
  const float* lses = p.lses + row;
  Piece<kF32> x[kGroup];
#pragma unroll
  for (int k = 0; k < kGroup; ++k)
    if (k < p.pieces) x[k].load(p.parts, (k * p.rows + row) * p.dim + dim0);
  float top = -INFINITY;
  for (int s = 0; s < p.pieces; ++s) top = fmaxf(top, lses[s * p.rows]);
  if (top == -INFINITY) top = 0.0f;
  float acc[8] = {}, sum = 0.0f;
  for (int s0 = 0; s0 < p.pieces; s0 += kGroup) {
    if (s0 > 0) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
        if (s0 + k < p.pieces) x[k].load(p.parts, ((s0 + k) * p.rows + row) * p.dim + dim0);
    }
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      if (s0 + k >= p.pieces) break;
      const float w = expf(lses[(s0 + k) * p.rows] - top);
      sum += w;
      // a piece of weight zero may hold anything; a NaN weight reaches the result
      if (w == 0.0f) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, x[k].get(e), acc[e]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<uint4*>(p.out + row * p.dim + dim0) =
      make_uint4(bf16x2(acc[0] * inv, acc[1] * inv), bf16x2(acc[2] * inv, acc[3] * inv),
                 bf16x2(acc[4] * inv, acc[5] * inv), bf16x2(acc[6] * inv, acc[7] * inv));
  if (dim0 == 0 && p.lse_out != nullptr) p.lse_out[row] = top + logf(sum);
}

}  // namespace

cudaError_t launch_attn_merge(const MergeParams& p, bool f32_parts, cudaStream_t stream) {
  const int64_t items = p.rows * (p.dim / 8);
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(blocks);
  int32_t shift = -1;  // of dim / 8, where that is a power of two
  for (int32_t k = 0; k < 8; ++k)
    if (p.dim == 8 << k) shift = k;
  return f32_parts ? launch_dependent(attn_merge_kernel<true>, g, kThreads, 0, stream, p, shift)
                   : launch_dependent(attn_merge_kernel<false>, g, kThreads, 0, stream, p, shift);
}

}  // namespace mla
