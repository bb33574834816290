// mla_kv_append: norm of the latent, rotation of the position parts,
// quantisation and scatter of new tokens.
//
// A token is handled by 1 + ceil(heads / 8) independent warps: one normalises
// the 512 latent values (16 a lane, sum of squares by shuffles), rotates the
// key and writes the cache row, the others rotate eight heads of the query
// each (four lanes a head).  Every value is read once and written once; nothing
// goes through shared memory.  Bound by the way to memory: a warp loads once and is
// done, so few bytes are in flight.  8192 tokens with 16 heads into a bf16 cache with the
// dense copy, 64 MB: 9 us where the inputs are in L2, 14.7 us out of DRAM (a quarter of
// its rate, warps waiting for loads); into an e4m3 cache 13.3 and 19.0 us, as the codes'
// float32 divisions add to the chain.  256 tokens, a launch and one trip: 2.7 us.
#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kRopeDim = kQkDim - kVDim;  // 64
constexpr int kPairs = kRopeDim / 2;
constexpr int kHeadsPerWarp = 8;

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// Eight e4m3 codes of x / scale (saturating, nearest even), as the per-tensor
// quantiser forms them.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = cvt_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
    const uint32_t hi = cvt_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

template <bool kE4m3>
__device__ __forceinline__ void store_cache8(const KvAppendParams& p, int32_t slot, int dim,
                                             const float (&x)[8], float scale) {
  const int64_t at = static_cast<int64_t>(slot) * kQkDim + dim;
  if (!MLA_DCHECK(at >= 0 && dim + 8 <= kQkDim && at + 8 <= p.kv_rows * kQkDim, p.err)) return;
  if constexpr (kE4m3)
    *reinterpret_cast<uint2*>(p.cache + at) = codes8(x, scale);
  else
    *reinterpret_cast<uint4*>(p.cache + 2 * at) = pack8(x);
}

// The 16 values of one lane of a 64-dim vector as the 8 pairs 8 part .. 8 part + 7
// (part 0 .. 3): two 16-byte pieces, adjacent when pairs are interleaved, 32
// dims apart when they are halves.
template <bool kInterleaved>
__device__ __forceinline__ int second_piece() { return kInterleaved ? 8 : kPairs; }
template <bool kInterleaved>
__device__ __forceinline__ int first_piece(int part) { return (kInterleaved ? 16 : 8) * part; }

template <bool kInterleaved>
__device__ __forceinline__ void rotate(float (&u)[8], float (&v)[8], const float (&c)[8],
                                       const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = kInterleaved ? (i < 4 ? u[2 * i] : v[2 * i - 8]) : u[i];
    float& b = kInterleaved ? (i < 4 ? u[2 * i + 1] : v[2 * i - 7]) : v[i];
    const float ra = a * c[i] - b * s[i], rb = b * c[i] + a * s[i];
    a = ra;
    b = rb;
  }
}

__device__ __forceinline__ void load_turn(const float* row, int part, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(row + 8 * part) + i);
    const float4 y = __ldg(reinterpret_cast<const float4*>(row + kPairs + 8 * part) + i);
    c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
    s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
  }
}

template <bool kE4m3, bool kInterleaved>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(const KvAppendParams p, uint32_t warps_per_token) {
  const int lane = threadIdx.x & 31;
  const uint64_t job = static_cast<uint64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const uint64_t token = job / warps_per_token;
  pdl_wait_primary();
  pdl_launch_dependents();
  if (token >= static_cast<uint64_t>(p.num_tokens)) return;
  const int64_t t = static_cast<int64_t>(token);
  const uint32_t part = static_cast<uint32_t>(job - token * warps_per_token);
  const int32_t slot = __ldg(p.slots + t), pos = __ldg(p.positions + t);

  if (part == 0) {
    const uint16_t* src = p.kv + t * p.kv_stride;
    const uint4 raw0 = load16(src + 8 * lane), raw1 = load16(src + kVDim / 2 + 8 * lane);
    const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(p.weight + 8 * lane));
    const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(p.weight + kVDim / 2 + 8 * lane));
    const bool turns = lane < kPairs / 8;
    const int first = kVDim + first_piece<kInterleaved>(lane), second = first + second_piece<kInterleaved>();
    uint4 k0 = {}, k1 = {};
    if (turns) {
      k0 = load16(src + first);
      k1 = load16(src + second);
    }
    if (slot < 0) return;  // padding
    if (slot >= p.kv_rows || pos < 0 || pos >= p.max_positions) {
      if (lane == 0)
        atomicOr(p.err, (slot >= p.kv_rows ? MLA_DERR_KV_INDEX : 0) |
                            (pos < 0 || pos >= p.max_positions ? MLA_DERR_POSITION : 0));
      return;
    }
    const float scale = kE4m3 ? __ldg(p.kv_scale) : 1.0f;
    float c[8], s[8];
    if (turns) load_turn(p.rope_table + static_cast<int64_t>(pos) * kRopeDim, lane, c, s);
    float a[8], b[8], wa[8], wb[8];
    unpack8(raw0, a);
    unpack8(raw1, b);
    unpack8(w0, wa);
    unpack8(w1, wb);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    float r = rsqrtf(sum * (1.0f / kVDim) + p.eps);
    // Squares below 2^-126 lose their bits.  Where they may count (no term above
    // 2^-100, and no eps beside which they vanish: one of 2^-80 is 2^29 times their
    // mean) the row is scaled by 2^100 first, and eps by its square.
    if (sum < 0x1p-100f && p.eps < 0x1p-80f) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= 0x1p100f;
        b[i] *= 0x1p100f;
        sum += a[i] * a[i] + b[i] * b[i];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      r = rsqrtf(sum * (1.0f / kVDim) + p.eps * 0x1p100f * 0x1p100f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = a[i] * r * wa[i];
      b[i] = b[i] * r * wb[i];
    }
    store_cache8<kE4m3>(p, slot, 8 * lane, a, scale);
    store_cache8<kE4m3>(p, slot, kVDim / 2 + 8 * lane, b, scale);
    uint16_t* dense = p.latent_out == nullptr ? nullptr : p.latent_out + t * kQkDim;
    if (!MLA_DCHECK(!turns || (first >= kVDim && second + 8 <= kQkDim), p.err)) return;
    if (dense != nullptr) {
      *reinterpret_cast<uint4*>(dense + 8 * lane) = pack8(a);
      *reinterpret_cast<uint4*>(dense + kVDim / 2 + 8 * lane) = pack8(b);
    }
    if (turns) {
      unpack8(k0, a);
      unpack8(k1, b);
      rotate<kInterleaved>(a, b, c, s);
      store_cache8<kE4m3>(p, slot, first, a, scale);
      store_cache8<kE4m3>(p, slot, second, b, scale);
      if (dense != nullptr) {
        *reinterpret_cast<uint4*>(dense + first) = pack8(a);
        *reinterpret_cast<uint4*>(dense + second) = pack8(b);
      }
    }
    return;
  }

  const int32_t h = static_cast<int32_t>(part - 1) * kHeadsPerWarp + (lane >> 2);
  if (h >= p.num_heads) return;
  const int first = first_piece<kInterleaved>(lane & 3), second = first + second_piece<kInterleaved>();
  const uint16_t* src = p.q_pe + t * p.q_token_stride + h * p.q_head_stride;
  uint16_t* dst = p.q_out + t * p.qo_token_stride + h * p.qo_head_stride;
  if (!MLA_DCHECK(t < p.num_tokens && h >= 0 && max(first, second) + 8 <= kRopeDim, p.err)) return;
  const uint4 r0 = load16(src + first), r1 = load16(src + second);
  if (slot < 0 || slot >= p.kv_rows || pos < 0 || pos >= p.max_positions) return;  // reported by the token's first warp
  float c[8], s[8], u[8], v[8];
  load_turn(p.rope_table + static_cast<int64_t>(pos) * kRopeDim, lane & 3, c, s);
  unpack8(r0, u);
  unpack8(r1, v);
  rotate<kInterleaved>(u, v, c, s);
  *reinterpret_cast<uint4*>(dst + first) = pack8(u);
  *reinterpret_cast<uint4*>(dst + second) = pack8(v);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, bool e4m3, bool interleaved,
                             cudaStream_t stream) {
  const uint32_t per_token = 1 + static_cast<uint32_t>((p.num_heads + kHeadsPerWarp - 1) / kHeadsPerWarp);
  const uint64_t jobs = static_cast<uint64_t>(p.num_tokens) * per_token;
  const uint64_t blocks = (jobs + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(blocks), t = 32 * kWarps;
  if (e4m3)
    return interleaved ? launch_dependent(kv_append_kernel<true, true>, g, t, 0, stream, p, per_token)
                       : launch_dependent(kv_append_kernel<true, false>, g, t, 0, stream, p, per_token);
  return interleaved ? launch_dependent(kv_append_kernel<false, true>, g, t, 0, stream, p, per_token)
                     : launch_dependent(kv_append_kernel<false, false>, g, t, 0, stream, p, per_token);
}

}  // namespace mla
