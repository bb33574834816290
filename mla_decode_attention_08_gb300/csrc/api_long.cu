// Host side of the operators for decode steps over long contexts: argument checks, plan,
// launches.
#include <cstring>

#include "kernels.h"
#include "ops.h"
#include "schedule.h"

namespace {

constexpr uint64_t kAlign = 256;
constexpr uint64_t kMissingOffset = 64;  // in a workspace's first 256 bytes, behind the error word
uint64_t round_up(uint64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
constexpr int64_t kMaxStride = INT64_C(1) << 36;

mla_status_t check_step_workspace(const void* ws, size_t bytes) {
  if (ws == nullptr || !aligned(ws, kAlign)) return MLA_ERR_INVALID_ARG;
  return bytes < MLA_STEP_WORKSPACE_BYTES ? MLA_ERR_WORKSPACE_TOO_SMALL : MLA_OK;
}
mla_status_t launched(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// Blocks of four queries of any cut of `total_q` into groups, at most: as many groups as
// there may be end one query into a block.
int64_t most_blocks(int64_t total_q, int64_t batch) {
  const int64_t groups = batch < total_q ? batch : total_q;
  return groups == 0 ? 0 : (total_q - groups) / mla::kSharedTokens + groups;
}

// Workers, whether blocks are shared between them, and the units that a block's start counts
// for.  A block is one worker's, or the keys of one group's blocks are cut into k equal parts,
// or all blocks' keys, one behind the other, into equal shares for all SMs, where a worker whose
// share has the end of one block and the start of another does two jobs.  By the time that it
// should take, in eightieths of a microsecond: a key tile 140, a block's start and end 400, the
// rest of a call 400, or 680 for that and a first part and its join, where each part costs 1 and
// each part of the same block 12; groups' keys on average at 0.7 of the longest.  (Of 90 batches
// run with 8 to 20 cuts each, the one taken is 2 % slower than the best on average, 14 % at
// most: 4 short groups.  Blocks that are one worker's take up to 5 times the best's time where
// they are few and long, equal shares 1.4 times where they are many and short.)
// More groups than the second kernel looks through are not cut, whatever their blocks' time, so
// their whole blocks are dealt out by those shares, each to the worker that its start falls to: 256
// queries over 32768 keys among 1100 groups of one over up to 200 take 571 us, by count 3147; 2000
// groups of up to eight over up to 3000 651, by count 743.  By count where blocks can differ by
// no tile (16384 groups of one over 30 keys: 1080, by shares 1097), and of fewer groups, where
// whole blocks are only taken if as many of the longest are fast enough (300 of one over up to 1000:
// 42, by shares 45).
struct Cut {
  int32_t workers, split, start;
};
constexpr int32_t kStartUnits = 4;
constexpr int64_t kMostCutGroups = 1024;
Cut cut_of(int64_t blocks, int64_t batch, int64_t key_tiles, int64_t sms) {
  Cut best = {static_cast<int32_t>(blocks < sms ? (blocks > 0 ? blocks : 1) : sms), 0, 0};
  if (blocks == 0) return best;
  if (batch > kMostCutGroups) {  // (the second kernel looks for its tokens' groups)
    if (blocks > sms && key_tiles > 1) best.start = kStartUnits;
    return best;
  }
  int64_t least = (blocks + sms - 1) / sms * (400 + 140 * key_tiles) + 400;
  auto take = [&](int64_t share, int64_t of_block, int64_t parts, int64_t workers, int32_t start) {
    const int64_t time = 680 + 140 * share + 12 * of_block + parts;
    if (time >= least) return;
    least = time;
    best = Cut{static_cast<int32_t>(workers), 1, start};
  };
  if (batch == 1)
    for (int64_t k = 2; k <= key_tiles && k * blocks <= sms; ++k) take((key_tiles + k - 1) / k, k, k * blocks, k * blocks, 0);
  const int64_t units = (batch == 1 ? blocks * key_tiles : 7 * blocks * key_tiles / 10) + kStartUnits * blocks;
  const int64_t share = (units + sms - 1) / sms;
  if (key_tiles > 0) take(share, key_tiles / share, (sms < units ? sms : units) + blocks, sms, kStartUnits);
  return best;
}

// The plan's fields for a number of workers; false if it cannot be run.
bool plan_fields(int32_t batch, int32_t total_q, int32_t max_kv_len, int32_t num_sms, Cut cut,
                 mla_shared_plan_t* out) {
  mla_shared_plan_t p;
  std::memset(&p, 0, sizeof(p));
  p.batch = batch;
  p.total_q = total_q;
  p.max_kv_len = max_kv_len;
  p.num_sms = num_sms;
  p.workers = cut.workers;
  p.split = cut.split;
  p.start = cut.start;
  p.abi_version = MLA_ABI_VERSION;
  if (cut.workers < 1 || cut.workers > MLA_SHARED_MAX_WORKERS || (cut.split != 0 && cut.split != 1) ||
      cut.start < 0 || cut.start > 64 || (cut.split == 1 && batch > kMostCutGroups))
    return false;
  uint64_t off = kAlign;  // error word
  p.ws_lse_offset = p.ws_partial_offset = off;
  if (cut.split == 1) {
    const uint64_t rows = 2ull * cut.workers * mla::kSharedTokens * mla::kNumHeads;
    off += round_up(rows * sizeof(float));
    p.ws_partial_offset = off;
    off += round_up(rows * mla::kVDim * sizeof(uint16_t));
  }
  p.ws_bytes = off;
  *out = p;
  return true;
}

mla_status_t run_shared(const void* q, const void* kv, const float* kv_scale, const int32_t* qo_indptr,
                        const int32_t* kv_indptr, void* out, float* lse, cudaStream_t stream,
                        const mla_shared_plan_t* plan, const int32_t* kv_indices, int64_t kv_indices_len,
                        int64_t kv_rows, void* workspace, size_t workspace_bytes, bool stall_stream) {
  mla_shared_plan_t want;
  if (plan == nullptr || plan->abi_version != MLA_ABI_VERSION || plan->batch < 1 ||
      plan->batch > MLA_SHARED_MAX_GROUPS || plan->total_q < 0 || plan->max_kv_len < 0 || plan->num_sms < 1 ||
      !plan_fields(plan->batch, plan->total_q, plan->max_kv_len, plan->num_sms, Cut{plan->workers, plan->split, plan->start},
                   &want) ||
      std::memcmp(&want, plan, sizeof(want)) != 0)
    return MLA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, kAlign)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->ws_bytes) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (kv_rows < 1 || kv_rows > INT32_MAX ||
      (kv_indices != nullptr && (kv_indices_len < 0 || kv_indices_len > INT32_MAX)))
    return MLA_ERR_INVALID_ARG;
  if (plan->total_q == 0) return MLA_OK;
  if (q == nullptr || kv == nullptr || kv_scale == nullptr || qo_indptr == nullptr || kv_indptr == nullptr ||
      out == nullptr || !aligned(q, 16) || !aligned(kv, 16) || !aligned(kv_scale, 4) || !aligned(qo_indptr, 4) ||
      !aligned(kv_indptr, 4) || !aligned(kv_indices, 4) || !aligned(out, 16) || !aligned(lse, 4))
    return MLA_ERR_INVALID_ARG;
  int device = 0;
  mla_status_t st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  mla::SharedMaps m = {};
  if (kv_indices == nullptr && !mla::cache_maps(kv, kv_rows, device, &m.latent, &m.rope)) return MLA_ERR_CUDA;
  auto* ws = static_cast<uint8_t*>(workspace);
  mla::SharedParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.kv_scale = kv_scale;
  p.qo_indptr = qo_indptr;
  p.kv_indptr = kv_indptr;
  p.kv_indices = kv_indices;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part = reinterpret_cast<uint16_t*>(ws + plan->ws_partial_offset);
  p.part_lse = reinterpret_cast<float*>(ws + plan->ws_lse_offset);
  p.err = reinterpret_cast<int32_t*>(ws);
  p.missing = reinterpret_cast<uint32_t*>(ws + kMissingOffset);
  p.kv_rows = kv_rows;
  p.kv_limit = kv_indices != nullptr ? kv_indices_len : kv_rows;
  p.batch = plan->batch;
  p.total_q = plan->total_q;
  p.workers = plan->workers;
  p.split = plan->split;
  p.start = plan->start;
  p.stall_stream = stall_stream ? 1 : 0;
  st = launched(mla::launch_shared(p, m, stream));
  return st != MLA_OK || plan->split == 0 ? st : launched(mla::launch_shared_join(p, plan->num_sms, stream));
}

mla_status_t run_means(const void* cache, const float* kv_scale, bool e4m3, int64_t kv_rows,
                       const int32_t* slots, int64_t num_tokens, void* means, int32_t num_pages,
                       int32_t page_size, const void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || page_size < 1 || num_pages < 1 || kv_rows < 1 ||
      kv_rows > INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  mla_status_t st = check_step_workspace(workspace, workspace_bytes);
  if (st != MLA_OK) return st;
  if (num_tokens == 0) return MLA_OK;
  if (cache == nullptr || (e4m3 && kv_scale == nullptr) || slots == nullptr || means == nullptr ||
      !aligned(cache, 16) || !aligned(kv_scale, 4) || !aligned(slots, 4) || !aligned(means, 16))
    return MLA_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return MLA_ERR_CUDA;
  mla::BlockMeansParams p;
  p.cache = static_cast<const uint8_t*>(cache);
  p.kv_scale = kv_scale;
  p.slots = slots;
  p.means = static_cast<uint16_t*>(means);
  p.err = static_cast<int32_t*>(const_cast<void*>(workspace));
  p.kv_rows = kv_rows;
  const int64_t covered = static_cast<int64_t>(num_pages) * page_size;
  p.limit = covered < kv_rows ? covered : kv_rows;
  p.num_tokens = num_tokens;
  p.page_size = page_size;
  return launched(mla::launch_block_means(p, e4m3, sms, stream));
}

}  // namespace

extern "C" {

mla_status_t mla_shared_plan(int32_t batch, int32_t total_q, int32_t max_kv_len, int32_t num_sms,
                             mla_shared_plan_t* plan) {
  if (plan == nullptr || batch < 1 || batch > MLA_SHARED_MAX_GROUPS || total_q < 0 || max_kv_len < 0)
    return MLA_ERR_INVALID_ARG;
  if (num_sms <= 0) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  // (no more workers than the workspace is laid out for: a GPU has fewer SMs)
  const int32_t sms = num_sms < MLA_SHARED_MAX_WORKERS ? num_sms : MLA_SHARED_MAX_WORKERS;
  const Cut cut = cut_of(most_blocks(total_q, batch), batch, mla::tiles_of_length(max_kv_len), sms);
  return plan_fields(batch, total_q, max_kv_len, num_sms, cut, plan) ? MLA_OK : MLA_ERR_INVALID_ARG;
}

mla_status_t mla_shared_fwd(const void* q_bf16, const void* kv_fp8, const float* kv_scale,
                            const int32_t* qo_indptr, const int32_t* kv_indptr, void* out_bf16, float* lse,
                            cudaStream_t stream, const mla_shared_plan_t* plan, const int32_t* kv_indices,
                            int64_t kv_indices_len, int64_t kv_rows, void* workspace, size_t workspace_bytes) {
  return run_shared(q_bf16, kv_fp8, kv_scale, qo_indptr, kv_indptr, out_bf16, lse, stream, plan, kv_indices,
                    kv_indices_len, kv_rows, workspace, workspace_bytes, false);
}

mla_status_t mla_shared_fwd_stall_stream(const void* q_bf16, const void* kv_fp8, const float* kv_scale,
                                         const int32_t* qo_indptr, const int32_t* kv_indptr, void* out_bf16,
                                         float* lse, cudaStream_t stream, const mla_shared_plan_t* plan,
                                         const int32_t* kv_indices, int64_t kv_indices_len, int64_t kv_rows,
                                         void* workspace, size_t workspace_bytes) {
  return run_shared(q_bf16, kv_fp8, kv_scale, qo_indptr, kv_indptr, out_bf16, lse, stream, plan, kv_indices,
                    kv_indices_len, kv_rows, workspace, workspace_bytes, true);
}

mla_status_t mla_block_means(const void* kv_fp8, const float* kv_scale, int64_t kv_rows, const int32_t* slots,
                             int64_t num_tokens, void* means, int32_t num_pages, int32_t page_size,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_means(kv_fp8, kv_scale, true, kv_rows, slots, num_tokens, means, num_pages, page_size, workspace,
                   workspace_bytes, stream);
}

mla_status_t mla_block_means_bf16kv(const void* kv_bf16, int64_t kv_rows, const int32_t* slots,
                                    int64_t num_tokens, void* means, int32_t num_pages, int32_t page_size,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_means(kv_bf16, nullptr, false, kv_rows, slots, num_tokens, means, num_pages, page_size, workspace,
                   workspace_bytes, stream);
}

mla_status_t mla_block_scores(const void* q_bf16, int32_t total_q, const void* means, int32_t num_pages,
                              const int32_t* block_table, int64_t table_stride, int32_t max_pages,
                              const int32_t* qo_indptr, const int32_t* kv_indptr, int32_t batch,
                              int32_t page_size, float* scores, int64_t scores_stride, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  if (batch < 1 || batch > MLA_MAX_MAP_ROWS || total_q < 0 || max_pages < 1 || max_pages > MLA_MAX_ROW_PAGES || num_pages < 1 || page_size < 1 ||
      table_stride < max_pages || table_stride >= kMaxStride || scores_stride < max_pages ||
      scores_stride >= kMaxStride)
    return MLA_ERR_INVALID_ARG;
  if ((q_bf16 == nullptr && total_q > 0) || means == nullptr || block_table == nullptr || qo_indptr == nullptr ||
      kv_indptr == nullptr || scores == nullptr || !aligned(q_bf16, 16) || !aligned(means, 16) ||
      !aligned(block_table, 4) || !aligned(qo_indptr, 4) || !aligned(kv_indptr, 4) || !aligned(scores, 4))
    return MLA_ERR_INVALID_ARG;
  mla_status_t st = check_step_workspace(workspace, workspace_bytes);
  if (st != MLA_OK) return st;
  int device = 0, sms = 0;
  st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return MLA_ERR_CUDA;
  mla::BlockScoresParams p;
  p.q = static_cast<const uint16_t*>(q_bf16);
  p.means = static_cast<const uint16_t*>(means);
  p.block_table = block_table;
  p.qo_indptr = qo_indptr;
  p.kv_indptr = kv_indptr;
  p.scores = scores;
  p.err = static_cast<int32_t*>(workspace);
  p.table_stride = table_stride;
  p.scores_stride = scores_stride;
  p.batch = batch;
  p.total_q = total_q;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_size = page_size;
  return launched(mla::launch_block_scores(p, sms, stream));
}

mla_status_t mla_block_select(const float* scores, int64_t scores_stride, const int32_t* block_table,
                              int64_t table_stride, int32_t max_pages, const int32_t* kv_indptr, int32_t batch,
                              int32_t page_size, int32_t num_pages, int32_t blocks, int32_t sink, int32_t recent,
                              int32_t* sel_indptr, int32_t* sel_indices, int64_t sel_indices_len,
                              int32_t* chosen, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (batch < 1 || batch > MLA_MAX_MAP_ROWS || max_pages < 1 || max_pages > MLA_MAX_ROW_PAGES || page_size < 1 || num_pages < 1 ||
      static_cast<int64_t>(page_size) * num_pages > INT32_MAX || table_stride < max_pages ||
      table_stride >= kMaxStride || scores_stride < max_pages || scores_stride >= kMaxStride || blocks < 1 ||
      blocks > MLA_SELECT_MAX_BLOCKS || sink < 0 || recent < 1 || sink > blocks - recent || sel_indices_len < 0 ||
      sel_indices_len > INT32_MAX)
    return MLA_ERR_INVALID_ARG;
  if (scores == nullptr || block_table == nullptr || kv_indptr == nullptr || sel_indptr == nullptr ||
      (sel_indices == nullptr && sel_indices_len > 0) || !aligned(scores, 4) || !aligned(block_table, 4) ||
      !aligned(kv_indptr, 4) || !aligned(sel_indptr, 4) || !aligned(sel_indices, 4) || !aligned(chosen, 4))
    return MLA_ERR_INVALID_ARG;
  mla_status_t st = check_step_workspace(workspace, workspace_bytes);
  if (st != MLA_OK) return st;
  int device = 0;
  st = mla::device_ready(&device);
  if (st != MLA_OK) return st;
  mla::BlockSelectParams p;
  p.scores = scores;
  p.block_table = block_table;
  p.kv_indptr = kv_indptr;
  p.sel_indptr = sel_indptr;
  p.sel_indices = sel_indices;
  p.chosen = chosen;
  p.err = static_cast<int32_t*>(workspace);
  p.table_stride = table_stride;
  p.scores_stride = scores_stride;
  p.indices_len = sel_indices_len;
  p.batch = batch;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.blocks = blocks;
  p.sink = sink;
  p.recent = recent;
  return launched(mla::launch_block_select(p, stream));
}

}  // extern "C"
