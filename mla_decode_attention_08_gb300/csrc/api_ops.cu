// Host side of the operators around the decode step: argument checks, plan,
// TMA descriptors, launches.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "kernels.h"
#include "ops.h"
#include "schedule.h"

namespace {

constexpr uint64_t kAlign = 256;
constexpr uint64_t kSchedOffset = 64;  // in a workspace's first 256 bytes, behind the error word
uint64_t round_up(uint64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A stride of bf16 elements that keeps 16-byte pieces aligned and TMA-addressable.
constexpr int64_t kMaxStride = INT64_C(1) << 36;
bool good_stride(int64_t s) { return s >= 0 && s < kMaxStride && s % 8 == 0; }
// Rows `dim` wide that lie apart (a single row's stride is not used).
bool apart(int64_t count, int64_t s, int64_t dim) { return count <= 1 || (good_stride(s) && s >= dim); }

mla_status_t check_step_workspace(const void* ws, size_t bytes) {
  if (ws == nullptr || !aligned(ws, kAlign)) return MLA_ERR_INVALID_ARG;
  return bytes < MLA_STEP_WORKSPACE_BYTES ? MLA_ERR_WORKSPACE_TOO_SMALL : MLA_OK;
}

mla_status_t launched(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

mla_status_t run_append(mla::KvAppendParams p, const void* workspace, size_t workspace_bytes,
                        bool e4m3, int32_t interleaved, cudaStream_t stream) {
  if (p.num_tokens < 0 || p.num_heads < 0 || p.num_heads > (1 << 16)) return MLA_ERR_INVALID_ARG;
  mla_status_t st = check_step_workspace(workspace, workspace_bytes);
  if (st != MLA_OK) return st;
  if (p.num_tokens == 0) return MLA_OK;
  if (p.kv == nullptr || p.weight == nullptr || p.rope_table == nullptr || p.positions == nullptr ||
      p.slots == nullptr || p.cache == nullptr || (e4m3 && p.kv_scale == nullptr))
    return MLA_ERR_INVALID_ARG;
  if (!aligned(p.kv, 16) || !aligned(p.weight, 16) || !aligned(p.rope_table, 16) ||
      !aligned(p.positions, 4) || !aligned(p.slots, 4) || !aligned(p.cache, 16) ||
      !aligned(p.kv_scale, 4) || !aligned(p.latent_out, 16))
    return MLA_ERR_INVALID_ARG;
  if (!(p.eps >= 0.0f) || !std::isfinite(p.eps) || p.max_positions < 1 || p.kv_rows < 1 ||
      p.kv_rows > INT32_MAX || !apart(p.num_tokens, p.kv_stride, mla::kQkDim))
    return MLA_ERR_INVALID_ARG;
  // In place means row by row: the dense copy lies exactly over its source.
  if (p.latent_out == p.kv && p.num_tokens > 1 && p.kv_stride != mla::kQkDim)
    return MLA_ERR_INVALID_ARG;
  if (p.num_heads > 0) {
    if (p.q_pe == nullptr || p.q_out == nullptr || !aligned(p.q_pe, 16) || !aligned(p.q_out, 16) ||
        (p.num_tokens > 1 && !good_stride(p.q_token_stride)) ||
        (p.num_heads > 1 && !good_stride(p.q_head_stride)))
      return MLA_ERR_INVALID_ARG;
    const int64_t rope = mla::kQkDim - mla::kVDim;
    if (!apart(p.num_tokens, p.qo_token_stride, rope) || !apart(p.num_heads, p.qo_head_stride, rope))
      return MLA_ERR_INVALID_ARG;
    if (p.q_pe == p.q_out && ((p.num_tokens > 1 && p.q_token_stride != p.qo_token_stride) ||
                              (p.num_heads > 1 && p.q_head_stride != p.qo_head_stride)))
      return MLA_ERR_INVALID_ARG;
  }
  int device = 0;
  st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  return launched(mla::launch_kv_append(p, e4m3, interleaved != 0, stream));
}

mla::KvAppendParams append_params(const void* kv, int64_t kv_stride, const void* weight, float eps,
                                  const float* rope_table, int32_t max_positions,
                                  const int32_t* positions, const int32_t* slots,
                                  int32_t num_tokens, void* cache, const float* kv_scale,
                                  int64_t kv_rows, void* latent_out, const void* q_pe,
                                  int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                                  int64_t qo_token_stride, int64_t qo_head_stride,
                                  int32_t num_heads, void* workspace) {
  mla::KvAppendParams p;
  p.kv = static_cast<const uint16_t*>(kv);
  p.weight = static_cast<const uint16_t*>(weight);
  p.rope_table = rope_table;
  p.positions = positions;
  p.slots = slots;
  p.cache = static_cast<uint8_t*>(cache);
  p.kv_scale = kv_scale;
  p.latent_out = static_cast<uint16_t*>(latent_out);
  p.q_pe = static_cast<const uint16_t*>(q_pe);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.err = static_cast<int32_t*>(workspace);
  p.kv_stride = kv_stride;
  p.kv_rows = kv_rows;
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.qo_token_stride = qo_token_stride;
  p.qo_head_stride = qo_head_stride;
  p.eps = eps;
  p.max_positions = max_positions;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  return p;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// bf16 [tokens][heads][dim] in boxes of 64 dims x 1 head x `rows` tokens, each
// a 128-byte-swizzled panel.
bool encode_heads(CUtensorMap* map, const void* base, int64_t tokens, int32_t heads, int32_t dim,
                  int64_t token_stride, int64_t head_stride, uint32_t rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t gdim[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t gstride[2] = {2 * static_cast<cuuint64_t>(heads > 1 ? head_stride : dim),
                                 2 * static_cast<cuuint64_t>(tokens > 1 ? token_stride : dim)};
  const cuuint32_t box[3] = {64, 1, rows}, estride[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_shared(CUtensorMap* map, const void* base, int64_t tokens, int64_t token_stride) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t gdim[2] = {mla::kPrefillRope, static_cast<cuuint64_t>(tokens)};
  const cuuint64_t gstride[1] = {2 * static_cast<cuuint64_t>(tokens > 1 ? token_stride : mla::kPrefillRope)};
  const cuuint32_t box[2] = {64, 128}, estride[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of 128 queries of any cut of `total_q` into rows, at most: as many rows as
// there may be end one query into a block.
int64_t most_blocks(int64_t total_q, int64_t batch) {
  const int64_t rows = batch < total_q ? batch : total_q;
  return rows == 0 ? 0 : (total_q - rows) / 128 + rows;
}

// Parts that a row's keys are cut into, when the (at most) `blocks` of 128 queries
// leave SMs idle, now or in a second round.  By the time that it should take, in
// twentieths of a microsecond: a job takes 2 us and 0.95 a key tile; the jobs of one
// row come in rounds, those of a batch balance over the SMs, its rows' keys on average
// at 0.7 of the longest; then the second kernel takes 2 us and its float32 parts'
// bytes, written and read at 6 TB/s while all rows' threads fit the GPU, else at 5.
// (Fitted to 50 ragged batches of 16 and five heads, each with one to twelve parts:
// what it takes is 2 % slower than the best of them on average, 14 % at worst.  Of 26
// batches of equal rows, which a plan cannot tell from them, 8 % and 29 %.)
int32_t key_splits(int64_t blocks, int64_t batch, int64_t key_tiles, int64_t sms, int64_t rows) {
  // (The second kernel looks for its tokens' rows, so thousands of empty ones are not cut.)
  if (blocks == 0 || 10 * blocks >= 13 * sms || batch > 1024) return 1;
  const bool few = mla::merges_at_once(rows, static_cast<int32_t>(sms));
  auto time = [&](int64_t s) {
    const int64_t jobs = blocks * s, longest = 40 + 19 * ((key_tiles + s - 1) / s);
    const int64_t mean = 40 + 19 * ((7 * key_tiles + 10 * s - 1) / (10 * s));
    const int64_t join = s == 1 ? 0 : 40 + s * rows * 1024 / (few ? 300000 : 250000);
    if (batch == 1 || jobs <= sms) return (jobs + sms - 1) / sms * longest + join;
    return (longest > jobs * mean / sms ? longest : jobs * mean / sms) + join;
  };
  int64_t best = 1, least = time(1);
  for (int64_t s = 2; s <= key_tiles && s * blocks <= 8 * sms; ++s)
    if (time(s) < least) least = time(best = s);
  return static_cast<int32_t>(best);
}

// Whether one row of n queries over `keys` keys takes less time in jobs of one query
// tile than in jobs of two: the longest job, or an SM's share of all, or, as far as
// they are alike, rounds of them.  (Microseconds of an SM for a job's key tile and for
// a job: 0.95 and 3.0, of two query tiles 1.75 and 3.2.  16 heads, 2560 queries over
// 8560 keys, 160 jobs of two tiles for 152 SMs: 156 us, that way 168.)
bool faster_in_pairs(int64_t n, int64_t keys, bool causal, int64_t heads, int64_t sms) {
  auto time = [&](int64_t size, double tile, double job) {
    const int64_t blocks = (n + size - 1) / size;
    auto tiles = [&](int64_t queries) {  // that the last of a row's first `queries` sees
      const int64_t seen = causal ? keys - n + queries : keys;
      return seen > 0 ? (seen + 127) / 128 : 0;
    };
    const double last = tile * tiles(n) + job, first = tile * tiles(size < n ? size : n) + job;
    const double jobs = static_cast<double>(blocks * heads), share = jobs * 0.5 * (first + last) / sms;
    const double rounds = std::ceil(jobs / sms) * last;
    double alike = 2.0 * (first + last) / last - 3.0;
    alike = alike < 0.0 ? 0.0 : alike > 1.0 ? 1.0 : alike;
    const double all = rounds > share ? share + (rounds - share) * alike : share;
    return all > last ? all : last;
  };
  return time(128, 0.95, 3.0) < time(256, 1.75, 3.2);
}

// The plan's fields for a number of parts; false if it cannot be run.
bool plan_fields(int32_t batch, int32_t total_q, int32_t max_kv_len, int32_t num_heads, int32_t num_sms,
                 int32_t splits, mla_prefill_plan_t* out) {
  mla_prefill_plan_t p;
  std::memset(&p, 0, sizeof(p));
  p.batch = batch;
  p.total_q = total_q;
  p.max_kv_len = max_kv_len;
  p.num_heads = num_heads;
  p.num_sms = num_sms;
  p.abi_version = MLA_ABI_VERSION;
  // A row of n queries has ceil(n / 256) <= n / 256 + 1 blocks, and none if it is empty.
  p.tiles = total_q / mla::kPrefillRows + (batch < total_q ? batch : total_q);
  p.splits = splits;
  if (splits < 1 || most_blocks(total_q, batch) * num_heads > INT32_MAX / splits) return false;
  uint64_t off = kAlign;  // error word
  p.ws_lse_offset = p.ws_partial_offset = off;
  if (p.splits > 1) {
    const uint64_t rows = static_cast<uint64_t>(p.splits) * total_q * num_heads;
    off += round_up(rows * sizeof(float));
    p.ws_partial_offset = off;
    off += round_up(rows * mla::kPrefillV * sizeof(float));
  }
  p.ws_bytes = off;
  *out = p;
  return true;
}

mla_status_t run_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                         const void* k_nope, int64_t kn_token_stride, int64_t kn_head_stride,
                         const void* k_rope, int64_t kr_token_stride, const void* v,
                         int64_t v_token_stride, int64_t v_head_stride, int64_t total_kv,
                         const int32_t* qo_indptr, const int32_t* kv_indptr, float scale,
                         int32_t causal, void* out, float* lse, cudaStream_t stream,
                         const mla_prefill_plan_t* plan, void* workspace, size_t workspace_bytes,
                         bool stall_stream) {
  mla_prefill_plan_t want;
  if (plan == nullptr || plan->abi_version != MLA_ABI_VERSION || plan->batch < 1 ||
      plan->batch > MLA_PREFILL_MAX_ROWS || plan->total_q < 0 || plan->max_kv_len < 0 || plan->num_heads < 1 ||
      plan->num_heads > 1024 || plan->num_sms < 1 ||
      !plan_fields(plan->batch, plan->total_q, plan->max_kv_len, plan->num_heads, plan->num_sms, plan->splits,
                   &want) ||
      std::memcmp(&want, plan, sizeof(want)) != 0)
    return MLA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, kAlign)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->ws_bytes) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (total_kv < 0 || total_kv > INT32_MAX || !(scale > 0.0f) || !std::isfinite(scale))
    return MLA_ERR_INVALID_ARG;
  if (plan->total_q == 0) return MLA_OK;
  if (q == nullptr || qo_indptr == nullptr || kv_indptr == nullptr || out == nullptr ||
      !aligned(q, 16) || !aligned(qo_indptr, 4) || !aligned(kv_indptr, 4) || !aligned(out, 16) ||
      !aligned(lse, 4) || !apart(plan->total_q, q_token_stride, mla::kPrefillQk) ||
      !apart(plan->num_heads, q_head_stride, mla::kPrefillQk))
    return MLA_ERR_INVALID_ARG;
  if (total_kv > 0 &&
      (k_nope == nullptr || k_rope == nullptr || v == nullptr || !aligned(k_nope, 16) ||
       !aligned(k_rope, 16) || !aligned(v, 16) ||
       !apart(total_kv, kn_token_stride, mla::kPrefillNope) ||
       !apart(plan->num_heads, kn_head_stride, mla::kPrefillNope) ||
       !apart(total_kv, kr_token_stride, mla::kPrefillRope) ||
       !apart(total_kv, v_token_stride, mla::kPrefillV) ||
       !apart(plan->num_heads, v_head_stride, mla::kPrefillV)))
    return MLA_ERR_INVALID_ARG;
  int device = 0;
  mla_status_t st = mla::device_ready(&device);
  if (st != MLA_OK) return st;

  mla::PrefillMaps m;
  const int32_t heads = plan->num_heads;
  if (!encode_heads(&m.q, q, plan->total_q, heads, mla::kPrefillQk, q_token_stride, q_head_stride, 128))
    return MLA_ERR_CUDA;
  if (total_kv == 0) {
    m.k_nope = m.k_rope = m.v = m.q;  // no row has keys, so no key is loaded
  } else if (!encode_heads(&m.k_nope, k_nope, total_kv, heads, mla::kPrefillNope, kn_token_stride,
                           kn_head_stride, 128) ||
             !encode_heads(&m.v, v, total_kv, heads, mla::kPrefillV, v_token_stride, v_head_stride, 64) ||
             !encode_shared(&m.k_rope, k_rope, total_kv, kr_token_stride)) {
    return MLA_ERR_CUDA;
  }
  auto* ws = static_cast<uint8_t*>(workspace);
  mla::PrefillParams p;
  p.qo_indptr = qo_indptr;
  p.kv_indptr = kv_indptr;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part = reinterpret_cast<float*>(ws + plan->ws_partial_offset);
  p.part_lse = reinterpret_cast<float*>(ws + plan->ws_lse_offset);
  p.err = reinterpret_cast<int32_t*>(ws);
  p.sched = reinterpret_cast<uint32_t*>(ws + kSchedOffset);
  p.scale = scale;
  p.batch = plan->batch;
  p.heads = heads;
  p.total_q = plan->total_q;
  p.blocks = static_cast<int32_t>(most_blocks(plan->total_q, plan->batch));
  p.walk = mla::kWalkByRows;
  if (plan->splits > 1)
    p.walk = mla::kWalkPairs;
  else if (plan->batch == 1)  // the row that was planned for
    p.walk = faster_in_pairs(plan->total_q, plan->max_kv_len, causal != 0, heads, plan->num_sms) ? mla::kWalkPairs
                                                                                               : mla::kWalkTwoTiles;
  p.num_sms = plan->num_sms;
  p.splits = plan->splits;
  p.causal = causal != 0;
  p.total_kv = total_kv;
  p.part_rows = static_cast<int64_t>((workspace_bytes - plan->ws_partial_offset) / (mla::kPrefillV * sizeof(float)));
  p.wide_out = aligned(out, 32) ? 1 : 0;
  p.stall_stream = stall_stream ? 1 : 0;
  st = launched(mla::launch_prefill(p, m, stream));
  if (st != MLA_OK || plan->splits == 1) return st;
  mla::MergeParams g;
  g.parts = p.part;
  g.lses = p.part_lse;
  g.out = p.out;
  g.lse_out = lse;
  g.rows = static_cast<int64_t>(plan->total_q) * heads;
  g.pieces = plan->splits;
  g.dim = mla::kPrefillV;
  g.missing = p.sched + 2;
  g.qo_indptr = qo_indptr;
  g.kv_indptr = kv_indptr;
  g.total_kv = total_kv;
  g.batch = plan->batch;
  g.heads = heads;
  g.total_q = plan->total_q;
  g.num_sms = plan->num_sms;
  g.part_rows = p.part_rows;
  g.err = p.err;
  return launched(mla::launch_attn_merge(g, true, stream));
}

}  // namespace

extern "C" {

mla_status_t mla_page_map(const int32_t* kv_lens, const int32_t* new_lens, int32_t batch,
                          int32_t* block_table, int64_t table_stride, int32_t max_pages,
                          int32_t page_size, int32_t num_pages, const int32_t* free_pages,
                          int32_t num_free, int32_t* qo_indptr, int32_t* kv_indptr,
                          int32_t* kv_indices, int64_t kv_indices_len, int32_t* slots,
                          int32_t* positions, int64_t slots_len, int32_t* pages_used,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (batch < 1 || batch > MLA_MAX_MAP_ROWS || max_pages < 1 || page_size < 1 || num_pages < 1 ||
      static_cast<int64_t>(page_size) * num_pages > INT32_MAX || table_stride < max_pages ||
      table_stride >= kMaxStride || num_free < 0 || kv_indices_len < 0 || kv_indices_len >= INT32_MAX ||
      slots_len < 0 || slots_len >= INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  if (kv_lens == nullptr || new_lens == nullptr || block_table == nullptr || qo_indptr == nullptr ||
      kv_indptr == nullptr || pages_used == nullptr || (kv_indices == nullptr && kv_indices_len > 0) ||
      ((slots == nullptr || positions == nullptr) && slots_len > 0) ||
      (free_pages == nullptr && num_free > 0))
    return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) ||
      !aligned(qo_indptr, 4) || !aligned(kv_indptr, 4) || !aligned(pages_used, 4) ||
      !aligned(kv_indices, 16) || !aligned(slots, 4) || !aligned(positions, 4) ||
      !aligned(free_pages, 4))
    return MLA_ERR_INVALID_ARG;
  mla_status_t st = check_step_workspace(workspace, workspace_bytes);
  if (st != MLA_OK) return st;
  int device = 0, sms = 0;
  st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return MLA_ERR_CUDA;
  mla::PageMapParams p;
  p.kv_lens = kv_lens;
  p.new_lens = new_lens;
  p.block_table = block_table;
  p.free_pages = free_pages;
  p.qo_indptr = qo_indptr;
  p.kv_indptr = kv_indptr;
  p.kv_indices = kv_indices;
  p.slots = slots;
  p.positions = positions;
  p.pages_used = pages_used;
  p.err = static_cast<int32_t*>(workspace);
  p.table_stride = table_stride;
  p.kv_indices_len = static_cast<int32_t>(kv_indices_len);
  p.slots_len = static_cast<int32_t>(slots_len);
  p.batch = batch;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.num_free = num_free;
  return launched(mla::launch_page_map(p, sms, stream));
}

mla_status_t mla_kv_append(const void* kv_bf16, int64_t kv_stride, const void* norm_weight,
                           float eps, const float* rope_table, int32_t max_positions,
                           int32_t interleaved, const int32_t* positions, const int32_t* slots,
                           int32_t num_tokens, void* cache_fp8, const float* kv_scale,
                           int64_t kv_rows, void* latent_out, const void* q_pe,
                           int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                           int64_t qo_token_stride, int64_t qo_head_stride, int32_t num_heads,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_append(append_params(kv_bf16, kv_stride, norm_weight, eps, rope_table, max_positions,
                                  positions, slots, num_tokens, cache_fp8, kv_scale, kv_rows,
                                  latent_out, q_pe, q_token_stride, q_head_stride, q_out,
                                  qo_token_stride, qo_head_stride, num_heads, workspace),
                    workspace, workspace_bytes, true, interleaved, stream);
}

mla_status_t mla_kv_append_bf16kv(const void* kv_bf16, int64_t kv_stride, const void* norm_weight,
                                  float eps, const float* rope_table, int32_t max_positions,
                                  int32_t interleaved, const int32_t* positions,
                                  const int32_t* slots, int32_t num_tokens, void* cache_bf16,
                                  int64_t kv_rows, void* latent_out, const void* q_pe,
                                  int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                                  int64_t qo_token_stride, int64_t qo_head_stride,
                                  int32_t num_heads, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
  return run_append(append_params(kv_bf16, kv_stride, norm_weight, eps, rope_table, max_positions,
                                  positions, slots, num_tokens, cache_bf16, nullptr, kv_rows,
                                  latent_out, q_pe, q_token_stride, q_head_stride, q_out,
                                  qo_token_stride, qo_head_stride, num_heads, workspace),
                    workspace, workspace_bytes, false, interleaved, stream);
}

mla_status_t mla_prefill_plan(int32_t batch, int32_t total_q, int32_t max_kv_len,
                              int32_t num_heads, int32_t num_sms, mla_prefill_plan_t* plan) {
  if (plan == nullptr || batch < 1 || batch > MLA_PREFILL_MAX_ROWS || total_q < 0 || max_kv_len < 0 ||
      num_heads < 1 || num_heads > 1024)
    return MLA_ERR_INVALID_ARG;
  if (num_sms <= 0) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  const int32_t splits = key_splits(most_blocks(total_q, batch) * num_heads, batch, mla::tiles_of_length(max_kv_len),
                                    num_sms, static_cast<int64_t>(total_q) * num_heads);
  return plan_fields(batch, total_q, max_kv_len, num_heads, num_sms, splits, plan) ? MLA_OK : MLA_ERR_INVALID_ARG;
}

mla_status_t mla_prefill_fwd(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             const void* k_nope, int64_t kn_token_stride, int64_t kn_head_stride,
                             const void* k_rope, int64_t kr_token_stride, const void* v,
                             int64_t v_token_stride, int64_t v_head_stride, int64_t total_kv,
                             const int32_t* qo_indptr, const int32_t* kv_indptr, float scale,
                             int32_t causal, void* out, float* lse, cudaStream_t stream,
                             const mla_prefill_plan_t* plan, void* workspace,
                             size_t workspace_bytes) {
  return run_prefill(q, q_token_stride, q_head_stride, k_nope, kn_token_stride, kn_head_stride, k_rope,
                     kr_token_stride, v, v_token_stride, v_head_stride, total_kv, qo_indptr, kv_indptr,
                     scale, causal, out, lse, stream, plan, workspace, workspace_bytes, false);
}

mla_status_t mla_prefill_fwd_stall_stream(const void* q, int64_t q_token_stride,
                                          int64_t q_head_stride, const void* k_nope,
                                          int64_t kn_token_stride, int64_t kn_head_stride,
                                          const void* k_rope, int64_t kr_token_stride,
                                          const void* v, int64_t v_token_stride,
                                          int64_t v_head_stride, int64_t total_kv,
                                          const int32_t* qo_indptr, const int32_t* kv_indptr,
                                          float scale, int32_t causal, void* out, float* lse,
                                          cudaStream_t stream, const mla_prefill_plan_t* plan,
                                          void* workspace, size_t workspace_bytes) {
  return run_prefill(q, q_token_stride, q_head_stride, k_nope, kn_token_stride, kn_head_stride, k_rope,
                     kr_token_stride, v, v_token_stride, v_head_stride, total_kv, qo_indptr, kv_indptr,
                     scale, causal, out, lse, stream, plan, workspace, workspace_bytes, true);
}

mla_status_t mla_attn_merge(const void* parts_bf16, const float* lses, int32_t num_parts,
                            int64_t rows, int32_t dim, void* out_bf16, float* lse_out,
                            cudaStream_t stream) {
  if (num_parts < 1 || num_parts > 64 || rows < 0 || rows > INT32_MAX || dim < 8 || dim > 1024 ||
      dim % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  if (rows == 0) return MLA_OK;
  if (parts_bf16 == nullptr || lses == nullptr || out_bf16 == nullptr || !aligned(parts_bf16, 16) ||
      !aligned(lses, 4) || !aligned(out_bf16, 16) || !aligned(lse_out, 4))
    return MLA_ERR_INVALID_ARG;
  int device = 0;
  mla_status_t st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  mla::MergeParams p;
  p.parts = parts_bf16;
  p.lses = lses;
  p.out = static_cast<uint16_t*>(out_bf16);
  p.lse_out = lse_out;
  p.rows = rows;
  p.pieces = num_parts;
  p.dim = dim;
  p.missing = nullptr;
  p.qo_indptr = p.kv_indptr = nullptr;
  p.total_kv = 0;
  p.batch = p.heads = p.total_q = p.num_sms = 0;
  p.part_rows = 0;
  p.err = nullptr;
  return launched(mla::launch_attn_merge(p, false, stream));
}

}  // extern "C"
