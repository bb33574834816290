// Parameter blocks and launchers of the operators around the decode step and over long
// contexts (internal to libmla_decode).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "../../include/mla_decode.h"

namespace mla {

// api.cu: MLA_OK when the current device is an sm_103 part whose kernels are set up.
mla_status_t device_ready(int* device);
// api.cu: the descriptors of an e4m3 cache's latent and rope boxes (tiles of 128 rows).
bool cache_maps(const void* kv_fp8, int64_t rows, int device, CUtensorMap* latent, CUtensorMap* rope);

// A launch as a programmatic dependent of the previous kernel of the stream:
// the kernel may be scheduled while that one finishes and waits for it
// (griddepcontrol.wait) before it touches global memory.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

struct PageMapParams {
  const int32_t* kv_lens;
  const int32_t* new_lens;
  int32_t* block_table;
  const int32_t* free_pages;
  int32_t* qo_indptr;
  int32_t* kv_indptr;
  int32_t* kv_indices;
  int32_t* slots;
  int32_t* positions;
  int32_t* pages_used;
  int32_t* err;
  int64_t table_stride;
  int32_t kv_indices_len, slots_len;
  int32_t batch, max_pages, page_size, num_pages, num_free;
  int32_t page_shift;      // set by the launch: log2 of page_size, or -1
};

struct KvAppendParams {
  const uint16_t* kv;
  const uint16_t* weight;
  const float* rope_table;
  const int32_t* positions;
  const int32_t* slots;
  uint8_t* cache;          // e4m3 codes or bf16 rows
  const float* kv_scale;   // e4m3 only
  uint16_t* latent_out;    // or null
  const uint16_t* q_pe;
  uint16_t* q_out;
  int32_t* err;
  int64_t kv_stride, kv_rows;
  int64_t q_token_stride, q_head_stride, qo_token_stride, qo_head_stride;
  float eps;
  int32_t max_positions, num_tokens, num_heads;
};

cudaError_t page_map_prepare();
cudaError_t launch_page_map(PageMapParams p, int32_t num_sms, cudaStream_t stream);
cudaError_t launch_kv_append(const KvAppendParams& p, bool e4m3, bool interleaved,
                             cudaStream_t stream);

// Joins `pieces` outputs [pieces][rows][dim] by their log-sum-exps
// [pieces][rows].  bf16 pieces (the public operator) or float ones (the split
// of mla_prefill_fwd, a row for each token and head; tokens that it has not
// computed are left alone).
struct MergeParams {
  const void* parts;
  const float* lses;
  uint16_t* out;
  float* lse_out;          // or null
  int64_t rows;
  int32_t pieces, dim;
  const uint32_t* missing;   // of float pieces: nonzero if not all were computed, and nothing is to be joined
  const int32_t* qo_indptr;  // of float pieces
  const int32_t* kv_indptr;
  int64_t total_kv;
  int32_t batch, heads, total_q, num_sms;
  // of float pieces, for the debug build's checks: rows that the workspace has room for, and the error word
  int64_t part_rows;
  int32_t* err;
};
// Whether float parts of `rows` rows of 128 are joined by threads that are all on the
// GPU at once: four values each, two blocks of 256 an SM.
inline bool merges_at_once(int64_t rows, int32_t sms) { return rows * (128 / 4) <= static_cast<int64_t>(sms) * 2 * 256; }
cudaError_t launch_attn_merge(const MergeParams& p, bool f32_parts, cudaStream_t stream);

// mla_prefill_fwd: a persistent block an SM; a job is up to 256 queries of a row
// and head over one split of its keys.
struct PrefillParams {
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  uint16_t* out;           // bf16 [total_q][heads][128]
  float* lse;              // [total_q][heads] or null
  float* part;             // splits > 1: [splits][total_q][heads][128]
  float* part_lse;         // splits > 1: [splits][total_q][heads]
  int32_t* err;
  uint32_t* sched;         // jobs handed out, blocks done: both zero between calls; then
                           // whether parts of this call are missing (see MergeParams)
  float scale;
  int32_t batch, heads, total_q, splits, causal, num_sms;
  int32_t blocks;          // of 128 queries, at most
  int32_t walk;            // kWalk...
  int64_t total_kv;
  int64_t part_rows;       // rows of parts that the workspace has room for (for the debug build's checks)
  int32_t wide_out;        // out is 32-byte aligned
  int32_t stall_stream;    // test hook: no copies are issued, so the waits run out
};
struct PrefillMaps {
  CUtensorMap q, k_nope, k_rope, v;
};
constexpr int kPrefillQk = MLA_PREFILL_QK_DIM, kPrefillNope = MLA_PREFILL_NOPE_DIM;
constexpr int kPrefillRope = kPrefillQk - kPrefillNope, kPrefillV = MLA_PREFILL_V_DIM;
// Jobs of two query tiles, of one whose key tiles alternate, or as the rows say.
constexpr int32_t kWalkByRows = 0, kWalkTwoTiles = 1, kWalkPairs = 2;
constexpr int kPrefillRows = 256;  // query rows of a job: two tiles of 128
size_t prefill_smem_bytes();
cudaError_t prefill_prepare();
cudaError_t launch_prefill(const PrefillParams& p, const PrefillMaps& maps, cudaStream_t stream);

// mla_shared_fwd: a persistent block an SM, a worker; a job is up to four query tokens of a
// group over its keys, or the part of them that falls to the worker.
struct SharedParams {
  const uint16_t* q;         // bf16 [total_q][16][576]
  const uint8_t* kv;         // e4m3 codes [kv_rows][576]
  const float* kv_scale;
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  const int32_t* kv_indices; // or null: keys are rows of the cache
  uint16_t* out;             // bf16 [total_q][16][512]
  float* lse;                // [total_q][16] or null
  uint16_t* part;            // if split: half [2 * workers][4 chunks][4 tokens][128 dims][16]
  float* part_lse;           // if split: [2 * workers][64]
  int32_t* err;
  uint32_t* missing;         // nonzero if not all parts of this call were computed
  int64_t kv_rows;
  int64_t kv_limit;          // keys that kv_indptr may count: kv_indices' entries, or kv_rows
  int32_t batch, total_q, workers;
  int32_t split;             // whether a block's keys may be shared by workers
  int32_t start;             // units of work that a block's start counts for
  int32_t stall_stream;      // test hook: no copies are issued, so the waits run out
};
struct SharedMaps {
  CUtensorMap latent, rope;  // (zeros with kv_indices: those keys are copied without descriptors)
};
constexpr int kSharedTokens = 4;  // query tokens of a job
size_t shared_smem_bytes();
cudaError_t shared_prepare();
cudaError_t launch_shared(const SharedParams& p, const SharedMaps& maps, cudaStream_t stream);
cudaError_t launch_shared_join(const SharedParams& p, int32_t num_sms, cudaStream_t stream);

struct BlockMeansParams {
  const uint8_t* cache;      // e4m3 codes or bf16 rows
  const float* kv_scale;     // e4m3 only
  const int32_t* slots;
  uint16_t* means;           // bf16 [num_pages][576]
  int32_t* err;
  int64_t kv_rows;
  int64_t limit;             // slots below it lie in the cache and on a page with a mean
  int64_t num_tokens;
  int32_t page_size;
};
cudaError_t block_means_prepare();
cudaError_t launch_block_means(const BlockMeansParams& p, bool e4m3, int32_t num_sms, cudaStream_t stream);

struct BlockScoresParams {
  const uint16_t* q;         // bf16 [total_q][16][576]
  const uint16_t* means;     // bf16 [num_pages][576]
  const int32_t* block_table;
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  float* scores;
  int32_t* err;
  int64_t table_stride, scores_stride;
  int32_t batch, total_q, max_pages, num_pages, page_size;
};
cudaError_t block_scores_prepare();
cudaError_t launch_block_scores(const BlockScoresParams& p, int32_t num_sms, cudaStream_t stream);

struct BlockSelectParams {
  const float* scores;
  const int32_t* block_table;
  const int32_t* kv_indptr;
  int32_t* sel_indptr;
  int32_t* sel_indices;
  int32_t* chosen;           // [batch][blocks] or null
  int32_t* err;
  int64_t table_stride, scores_stride, indices_len;
  int32_t batch, max_pages, num_pages, page_size;
  int32_t blocks, sink, recent;
};
cudaError_t block_select_prepare();
cudaError_t launch_block_select(const BlockSelectParams& p, cudaStream_t stream);

}  // namespace mla
