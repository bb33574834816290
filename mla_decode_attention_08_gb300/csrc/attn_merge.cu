// mla_attn_merge: joins attention over disjoint keys by the pieces'
// log-sum-exps.
//
// With m = max_s lse_s (0 if every piece is empty) and w_s = exp(lse_s - m):
// out = sum_s w_s part_s / sum_s w_s and lse = m + log sum_s w_s.  A thread owns
// four to 16 values of a row: it reads the row's few lses (the row's threads read
// the same ones) and each piece once.  Bound by the bytes of the pieces.
#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// kVec consecutive values of a piece, as loaded; pair(i) are values 2 i, 2 i + 1.
template <bool kF32, int kVec>
struct Piece {
  static constexpr int kWords = kF32 ? kVec : kVec / 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at * (kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = __ldcs(p + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (kF32) return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
};

// Whether `token` is one that mla_prefill_fwd has computed: it belongs to a row,
// and the row's tokens and keys lie in their tensors.  (A batch whose keys are
// split has at most 1024 rows; the plan does not cut more.)
__device__ __forceinline__ bool in_a_row(const MergeParams& p, int64_t token) {
  for (int32_t b = 0; b < p.batch; ++b) {
    const int32_t qs = __ldcg(p.qo_indptr + b), qe = __ldcg(p.qo_indptr + b + 1);
    if (token < qs || token >= qe) continue;
    const int32_t ks = __ldcg(p.kv_indptr + b), ke = __ldcg(p.kv_indptr + b + 1);
    if (qs >= 0 && qe <= p.total_q && ks >= 0 && ke >= ks && ke <= p.total_kv &&
        ke - ks <= MLA_PREFILL_MAX_ROW_KEYS)
      return true;
  }
  return false;
}

// The first pieces' values are loaded beside the log-sum-exps, before it is known
// which of them count: one trip to memory instead of two.  Where a row is a
// multiple of 16 long a thread takes 16 of its values, which halves what the
// weights cost (the kernel issues on 8 of 10 cycles with eight).  Four pieces of
// 16384 x 16 rows of 128: 67 us with eight values and the weights first, 55 with the
// values beside them, 49.5 us with 16 (6.9 TB/s; a copy reaches 6.7).
// kGroup pieces' loads are in flight together: 16, with four values a thread, where
// a prompt's few rows have all their threads on the GPU at once and the trips to L2
// are what costs (64 queries x 16 heads of nine float32 parts: 19.3 us with the
// attention before it, 20.7 with eight, 22.6 with eight values and four in flight);
// four where the SMs' registers turn over (1000 x 16 of two parts: 23.9 us, the
// other way 34.1).
template <bool kF32, int kVec, int kGroup>
__global__ void __launch_bounds__(kThreads) attn_merge_kernel(const MergeParams p, int32_t chunk_shift) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const uint32_t chunks = static_cast<uint32_t>(p.dim) / kVec;
  const int64_t row = chunk_shift >= 0 ? i >> chunk_shift : i / chunks;
  const int dim0 = kVec * static_cast<int>(i - row * chunks);
  bool wanted = row < p.rows;
  // (The rows are an input of the attention before as well, which waited for whoever
  // wrote them.)
  if constexpr (kF32) wanted = wanted && in_a_row(p, row / p.heads);
  pdl_wait_primary();
  pdl_launch_dependents();
  if (!wanted) return;
  // (beside the pieces' loads, looked at before the stores)
  uint32_t missing = 0;
  if constexpr (kF32) {
    missing = __ldcg(p.missing);
    if (!MLA_DCHECK(dim0 + kVec <= p.dim && p.dim == 128 && p.rows == static_cast<int64_t>(p.total_q) * p.heads &&
                        p.pieces * p.rows <= p.part_rows, p.err))
      return;
  }
  const float* lses = p.lses + row;
  Piece<kF32, kVec> x[kGroup];
#pragma unroll
  for (int k = 0; k < kGroup; ++k)
    if (k < p.pieces) x[k].load(p.parts, (k * p.rows + row) * p.dim + dim0);
  float top = -INFINITY;
  for (int s = 0; s < p.pieces; ++s) top = fmaxf(top, lses[s * p.rows]);
  if (top == -INFINITY) top = 0.0f;
  uint64_t acc[kVec / 2] = {};
  float sum = 0.0f;
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
      const uint64_t w2 = pack2(w, w);
#pragma unroll
      for (int e = 0; e < kVec / 2; ++e) acc[e] = fma2(w2, x[k].pair(e), acc[e]);
    }
  }
  if (kF32 && missing != 0) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint32_t out[kVec / 2];
#pragma unroll
  for (int e = 0; e < kVec / 2; ++e) {
    float lo, hi;
    unpack2(acc[e], lo, hi);
    out[e] = bf16x2(lo * inv, hi * inv);
  }
  uint16_t* dst = p.out + row * p.dim + dim0;
  if constexpr (kVec == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  } else {
#pragma unroll
    for (int e = 0; e < kVec / 8; ++e)
      reinterpret_cast<uint4*>(dst)[e] = make_uint4(out[4 * e], out[4 * e + 1], out[4 * e + 2], out[4 * e + 3]);
  }
  if (dim0 == 0 && p.lse_out != nullptr) p.lse_out[row] = top + logf(sum);
}

template <bool kF32, int kVec, int kGroup>
cudaError_t launch_vec(const MergeParams& p, cudaStream_t stream) {
  const int32_t chunks = p.dim / kVec;
  const int64_t blocks = (p.rows * chunks + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  int32_t shift = -1;  // of `chunks`, where that is a power of two
  for (int32_t k = 0; k < 8; ++k)
    if (chunks == 1 << k) shift = k;
  return launch_dependent(attn_merge_kernel<kF32, kVec, kGroup>, static_cast<unsigned>(blocks), kThreads, 0, stream, p, shift);
}

}  // namespace

cudaError_t launch_attn_merge(const MergeParams& p, bool f32_parts, cudaStream_t stream) {
  // (The parts are rows of 128.)
  if (f32_parts) return merges_at_once(p.rows, p.num_sms) ? launch_vec<true, 4, 16>(p, stream) : launch_vec<true, 8, 4>(p, stream);
  return p.dim % 16 == 0 ? launch_vec<false, 16, 4>(p, stream) : launch_vec<false, 8, 4>(p, stream);
}

}  // namespace mla
