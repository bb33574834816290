// mla_prefill_fwd: attention of prompts with keys and values expanded for each
// head (192-dim queries, keys = 128 dims of the head | 64 rotated dims shared by
// the heads, 128-dim values).
//
// Persistent blocks, one an SM, take jobs from a counter.  A job is up to 256
// queries of one row and head as two tiles of 128 (t = 0, 1), over the row's keys
// (or a split of them) in tiles of 128 (j):
//   * warp 3 takes the jobs, long ones first, and finds their row,
//   * warp 2 streams K(j) (three 64-dim panels of 128 keys) and V(j) (two panels
//     of 64 keys x 128 dims) by TMA into a ring of eight 16 KB slots,
//   * warps 0 and 1 issue S_t = Q_t . K(j)^T and O_t += P_t . V(j) of a tile each
//     (tcgen05, float32 accumulators in TMEM, P_t read from TMEM),
//   * warps 4-7 and 8-11 run the online softmax of tile t, a thread a row: S out
//     of TMEM, running maximum and sum in registers, P back over S as bf16.
// TMEM is full: S_0 | S_1 | O_0 | O_1, 128 columns each, P_t in S_t's first 64.
// The two tiles alternate: while the tensor cores work on one tile's products
// the other tile's softmax runs.  K and V are read from shared memory for both
// tiles, so a block moves 80 KB for 2 x 128 x 128 x 320 multiply-adds.
//
// That takes 2 x 128 queries a job, and a row's last job is its longest.  Where such
// jobs would leave SMs idle (few of them, or few long ones), a job is one query tile
// and its key tiles alternate ("pairs" below): tile T goes to issuer and softmax T & 1,
// each with its own S and O over the same queries, and the second accumulator is
// joined to the first at the job's end, out of TMEM.  K and V are then read from
// shared memory for one query tile only, a key tile takes 0.95 us and not 1.75 / 2,
// but jobs are half as long, and a row's jobs follow each other without a pause.
// (16 heads, both ways: one prompt of 1000 tokens 14.4 us and 19.2, of 2000 23 and
// 32, of 4000 62 and 59; 64 queries over 8256 keys 22.6 and 25.6; 8 rows of up to 64
// queries over up to 4000 keys 42 and 52; 12 prompts of up to 2047 tokens 106 and 98;
// 16384 tokens in one 10 % longer.)
//
// Bound by the chain of one tile (scores 768 cycles of the tensor pipe, softmax
// ~1250, values 512, and the looks at barriers between them) against the other
// tile's: ~3300 cycles for a key tile of both where the pipe alone needs 2560,
// and ~6700 more a job.  One prompt of 16384 tokens, 16 heads, causal: 753-770 us,
// 1.8 PFLOP/s, in a burst of five (a plain bf16 product reaches 1.97 in one); over
// thousands of calls 858 us, 1.6 PFLOP/s, with the SM clock at 1.65 GHz under the power
// limit (a plain product sustains 1.77).  12 prompts of up to 2047 tokens: 96-98 us.
//
// P is rounded to bf16 because the second product's operands have one type and V is
// bf16; its sum is taken before the rounding, whose errors have independent signs.  Both
// roundings together leave the output 0.0018 to 0.0022 off in the 2-norm, where rounding
// the output alone leaves 0.0016.  The exponential's approximation (2^-22) is far below.
#include <cstddef>

#include "ops.h"
#include "ptx.cuh"
#include "kernels.h"

namespace mla {
namespace {

constexpr int kTile = 128;
constexpr int kPanelBytes = 16384;
constexpr int kQPanels = kPrefillQk / 64;              // per query tile
constexpr int kKPanels = kPrefillQk / 64;              // per key tile: 2 of the head, 1 shared
constexpr int kVPanels = 2;                            // 64 keys x 128 dims each
constexpr int kFillsPerTile = kKPanels + kVPanels;
constexpr int kSlots = 8;
constexpr int kOffQ = 0;
constexpr int kOffRing = kOffQ + 2 * kQPanels * kPanelBytes;
constexpr int kOffMisc = kOffRing + kSlots * kPanelBytes;
// Pairs: one query tile, two buffers of K and of V, and the running maximum and
// sum of the softmax that is joined to the other.
constexpr int kOffPairK = kOffQ + kQPanels * kPanelBytes;
constexpr int kOffPairV = kOffPairK + 2 * kKPanels * kPanelBytes;
constexpr int kOffStats = kOffPairV + 2 * kVPanels * kPanelBytes;
static_assert(kOffStats + 2 * kTile * static_cast<int>(sizeof(float2)) <= kOffMisc, "room of the pairs' layout");
// Three warpgroups: two of softmax, one with the MMA issuers, the producer and
// the scheduler, whose registers go to the softmax (a row of 128 scores stays in
// registers; 200 and 104 take the same time).
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 192, kOtherRegs = 120;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168,
              "register split exceeds the launch allocation");
constexpr int kMmaWarp = 0, kProducerWarp = 2, kSchedulerWarp = 3, kFirstSoftmaxWarp = 4;  // issuers 0 and 1
constexpr uint32_t kLayoutSw128 = 2;
constexpr uint32_t kColS = 0, kColO = 256;             // + 128 t
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescQK = idesc_bf16(kTile, kTile, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(kTile, kPrefillV, false, true);
// The running reference of the exponent follows the maximum only when it is
// passed by more than this many powers of two: P then stays below 2^8, which
// costs bf16 nothing, and most tiles rescale nothing.
constexpr float kRescaleThreshold = 8.0f;

// One job: up to 256 queries (pairs: 128) of a row and head over a part of the row's keys.
struct Job {
  int32_t q0, nq;       // first query token (of the batch) and number of queries
  int32_t k0, len;      // the row's first key and number of keys
  int32_t see;          // keys that the first query sees, when causal
  int32_t head, split;
  int32_t j0, nt0, nt1; // first key tile, and key tiles of query tiles 0 and 1
  int32_t live;         // 0: no more jobs
  __device__ __forceinline__ int32_t tiles() const { return max(nt0, nt1); }
  // The tile (counted from j0) that the row's end cuts, or -1.
  __device__ __forceinline__ int32_t partial() const {
    const int32_t j = len / kTile - j0;
    return len % kTile != 0 && j >= 0 && j < tiles() ? j : -1;
  }
};

// The block works through jobs; key tiles are numbered through all of them (T),
// and so are each query tile's tiles and jobs: the numbers give the phases.
struct Misc {
  uint64_t job_full[2], job_empty[2];
  uint64_t claim;       // the copies of a job's last tiles are due: take the next job
  uint64_t q_full[2], q_empty[2];
  // Of key tile T's K and V, T & 1: landed, and released by both issuers.
  uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2];
  uint64_t s_full[2];   // S_t complete, and with it every product before it
  uint64_t p_head[2];   // the first three quarters of P_t written (and O_t rescaled)
  uint64_t p_full[2];   // all of it
  uint64_t o_full[2];   // the job's last product of tile t complete
  uint64_t o_free[2];   // the job's O_t read out
  uint64_t turn[2];     // the other tile's products are issued
  // Key tile T's V, T & 1, is zeroed behind the row's end.  One a buffer: issuer 0 can
  // be a tile ahead of issuer 1, which may not yet have looked at V(T) when V(T + 1) is
  // zeroed.  Of one buffer it cannot: V(T + 2) is zeroed after K(T + 2) was copied, hence
  // after both issuers released V(T), which issuer 1 does behind its wait.
  uint64_t v_clean[2];
  // Pairs: of buffer b, K and V released; the query tile released by both issuers;
  // softmax b's maximum and sum written and O_b complete.
  uint64_t pair_k_empty[2], pair_v_empty[2], pair_q_empty, joined[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int32_t pairs;        // jobs are of one query tile, and their key tiles alternate
  volatile int32_t abort_flag;
  Job job[2];
};
__device__ __forceinline__ uint8_t* block_memory(Misc* ms, int at) {
  return reinterpret_cast<uint8_t*>(ms) - kOffMisc + at;
}
// What reads a job: two issuers, the producer and eight softmax warps.
constexpr uint32_t kJobReaders = 11;
constexpr int kSmemBytes = kOffMisc + static_cast<int>(sizeof(Misc)) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of one block");
static_assert(kPrefillV == 128 && kPrefillNope == 128 && kPrefillRope == 64, "tile layout");

// Bounded wait on an mbarrier phase; false when the call is being abandoned.
// (Inlined: code whose register count setmaxnreg raised admits no calls.)
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Misc* ms, int32_t* err) {
  const long long start = clock64();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 15) == 0) {
      if (ms->abort_flag) return false;
      if (clock64() - start > kWaitLimitCycles) {
        ms->abort_flag = 1;
        atomicOr(err, MLA_DERR_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_on(const uint64_t* bar, uint32_t parity, Misc* ms, int32_t* err) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  return wait_slow(b, parity, ms, err);
}
// The same by a whole warp, which polls and gives up together: no lane runs ahead,
// so nothing has to be brought together again (16384-token prompt: 766 us; the
// lanes each on their own, then a vote, 781; one lane for the warp 961).
__device__ __forceinline__ bool warp_wait_on(const uint64_t* bar, uint32_t parity, Misc* ms, int32_t* err) {
  const uint32_t b = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
  const long long start = clock64();
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    if ((n & 15) == 0) {
      const bool late = clock64() - start > kWaitLimitCycles;
      if (__any_sync(0xffffffffu, late || ms->abort_flag)) {
        if (late && !ms->abort_flag) atomicOr(err, MLA_DERR_TIMEOUT);
        ms->abort_flag = 1;
        return false;
      }
    }
  }
}
// Bounded wait while draining at the end of a call.
__device__ __forceinline__ void drain(const uint64_t* bar, uint32_t parity) {
  const long long start = clock64();
  for (uint32_t n = 0;; ++n) {
    if (mbar_try_wait(smem_u32(bar), parity)) return;
    if ((n & 15) == 15 && clock64() - start > kWaitLimitCycles) return;
  }
}

__device__ __forceinline__ int32_t parts_of(int32_t n, int32_t size) { return n / size + (n % size != 0); }

// A row of the batch.
struct Row {
  int32_t qs, n, ks, len;
  // Key tiles that block i's last query reaches.
  __device__ __forceinline__ int32_t tiles(bool causal, int32_t last) const {
    const int32_t keys = causal ? max(0, min(len, len - n + 1 + last)) : len;
    return parts_of(keys, kTile);
  }
  // The same of block i of `size` queries.
  __device__ __forceinline__ int32_t block_tiles(bool causal, int32_t i, int32_t size) const {
    return tiles(causal, min(n, (i + 1) * size) - 1);
  }
};
// (`back`: set when the row ends before it begins; a bad row is reported by one block.)
__device__ __forceinline__ Row load_row(const PrefillParams& p, int32_t b, bool report, bool& back) {
  Row r = {0, 0, 0, 0};
  if (b >= p.batch) return r;
  const int32_t qs = __ldg(p.qo_indptr + b), qe = __ldg(p.qo_indptr + b + 1);
  const int32_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
  const bool bad_q = qs < 0 || qe < qs || qe > p.total_q;
  const bool bad_k = ks < 0 || ke < ks || ke > p.total_kv || ke - ks > MLA_PREFILL_MAX_ROW_KEYS;
  back = back || qe < qs;
  if (report && (bad_q || bad_k))
    atomicOr(p.err, (bad_q ? MLA_DERR_QO_INDPTR : 0) | (bad_k ? MLA_DERR_KV_INDPTR : 0));
  if (!bad_q && !bad_k) r = Row{qs, qe - qs, ks, ke - ks};
  return r;
}

// The batch as the scheduler warp holds it.  Up to 32 rows: a row a lane, handed
// out from the row with the most key tiles to the one with the fewest, each row's
// blocks of queries from its last, which sees the most keys: the blocks at work at
// one time share few rows' keys, which stay in L2, and the last jobs to start are
// short.  (12 prompts of up to 2047 tokens: 99 us; blocks by falling length over
// all rows 102 us, with 331 MB read from DRAM for 184 MB of inputs.)  More rows: a
// run of consecutive rows a lane, and the batch's blocks from the last one on; that
// many rows even out.
//
// Pairs, when no row has more than a tile of queries, when the host says so, or, if
// it leaves that open, when the longest job of two tiles takes longer than nine
// tenths of an SM's share of all jobs.  (Of 40 batches the slower way is taken for
// three, by 5, 6 and 14 %; with eight tenths or 0.95 for more.  All that the host
// weighs for one row, weighed here, would right them, but at 0.3 to 0.9 us a call.)
constexpr float kTileCost = 1.75f, kJobCost = 3.2f;  // microseconds of two query tiles: a key tile, a job
constexpr float kFull = 0.9f;
// Rows that overlap, which decreasing offsets make (and which are reported), could
// have any number of blocks.  No more are worked on than rows in order can have, so
// some rows may be left out: the joining kernel is told, which would otherwise join
// what an earlier call left in the workspace for them.  Sums stay below this, which
// is more.
constexpr int32_t kManyBlocks = 1 << 25;
struct Batch {
  Row row;
  int32_t b0, b1, first, count, total;
  int32_t size;         // queries of a block: 256, or 128 in pairs
  // More than 32 rows: the row before which the lane's search stands, and the
  // blocks of its run before that row.  A block's jobs come in falling order, so
  // the search only moves back.
  int32_t at, before;
};
__device__ __forceinline__ Batch count_rows(const PrefillParams& p) {
  const int lane = threadIdx.x & 31;
  const int32_t run = (p.batch + 31) / 32;
  Batch r;
  r.b0 = min(p.batch, lane * run);
  r.b1 = min(p.batch, r.b0 + run);
  const bool causal = p.causal != 0;
  r.row = Row{0, 0, 0, 0};
  bool one = true, back = false;
  int32_t blocks = 0, halves = 0, longest = 0;
  float work = 0.0f;
  for (int32_t b = r.b0; b < r.b1; ++b) {
    r.row = load_row(p, b, blockIdx.x == 0, back);
    const int32_t n = parts_of(r.row.n, kPrefillRows);
    if (n == 0) continue;
    const int32_t least = r.row.block_tiles(causal, 0, kPrefillRows), most = r.row.block_tiles(causal, n - 1, kPrefillRows);
    blocks = min(blocks + n, kManyBlocks);
    halves = min(halves + parts_of(r.row.n, kTile), kManyBlocks);
    one = one && r.row.n <= kTile;
    longest = max(longest, most);
    work += n * (kTileCost * 0.5f * (least + most) + kJobCost);
  }
  if (blockIdx.x == 0) {
    back = __any_sync(0xffffffffu, back);
    if (lane == 0) p.sched[2] = back;  // (of every call anew)
  }
  bool pairs = p.walk == kWalkPairs || __all_sync(0xffffffffu, one);
  if (p.walk == kWalkByRows && !pairs) {
    longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) work += __shfl_xor_sync(0xffffffffu, work, d);
    pairs = work * p.heads < kFull * p.num_sms * (kTileCost * longest + kJobCost);
  }
  r.size = pairs ? kTile : kPrefillRows;
  r.count = pairs ? halves : blocks;
  if (p.batch <= 32) {
    r.total = __reduce_add_sync(0xffffffffu, r.count);
    r.first = 0;
    const int32_t size = r.count > 0 ? r.row.block_tiles(causal, r.count - 1, r.size) : 0;
    for (int l = 0; l < p.batch; ++l) {
      const int32_t other = __shfl_sync(0xffffffffu, size, l), blocks = __shfl_sync(0xffffffffu, r.count, l);
      if (other > size || (other == size && l < lane)) r.first += blocks;
    }
  } else {
    int32_t incl = r.count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    r.first = incl - r.count;
    r.total = __shfl_sync(0xffffffffu, incl, 31);
  }
  r.total = min(r.total, p.blocks);
  r.at = r.b1;
  r.before = r.count;
  return r;
}

// Job `index` into `job` (one warp).  Heads run fastest, so that the blocks at
// work read the same keys' neighbourhood for all heads and it stays in L2.
__device__ __forceinline__ void find_job(const PrefillParams& p, Batch& r, uint32_t index, Job* job) {
  const int lane = threadIdx.x & 31;
  const uint32_t rest = index / p.heads, order = rest / p.splits;
  const bool causal = p.causal != 0;
  if (order >= static_cast<uint32_t>(r.total)) {
    if (lane == 0) job->live = job->nq = job->nt0 = job->nt1 = 0;
    __syncwarp();
    return;
  }
  const int32_t rank = static_cast<int32_t>(order);
  Row row = r.row;
  int32_t block = -1;  // of `row`, in the lane that has it
  if (p.batch <= 32) {
    const int32_t k = rank - r.first;
    if (k >= 0 && k < r.count) block = r.count - 1 - k;
  } else {
    const int32_t i = r.total - 1 - rank - r.first;
    if (i >= 0 && i < r.count) {
      bool back = false;
      while (i < r.before) {
        r.row = load_row(p, --r.at, false, back);
        r.before -= parts_of(r.row.n, r.size);
      }
      row = r.row;
      block = i - r.before;
    }
  }
  if (block >= 0) {
    const int32_t i0 = block * r.size, nq = min(r.size, row.n - i0);
    const int32_t split = static_cast<int32_t>(rest % p.splits);
    const int32_t all = row.block_tiles(causal, block, r.size), share = (all + p.splits - 1) / p.splits;
    const int32_t j0 = min(all, split * share), j1 = min(all, j0 + share);
    job->q0 = row.qs + i0;
    job->nq = nq;
    job->k0 = row.ks;
    job->len = row.len;
    job->see = row.len - row.n + i0 + 1;
    job->head = static_cast<int32_t>(index % p.heads);
    job->split = split;
    job->j0 = j0;
    job->nt0 = max(0, min(j1, row.tiles(causal, i0 + min(nq, kTile) - 1)) - j0);
    job->nt1 = nq > kTile ? j1 - j0 : 0;
    job->live = 1;
  }
  __syncwarp();
}

// Whether the block works in pairs; known with its first job.  (Abandoned: either.)
__device__ __forceinline__ bool in_pairs(const PrefillParams& p, Misc* ms) {
  return warp_wait_on(&ms->job_full[0], 0, ms, p.err) && ms->pairs != 0;
}

// Job number `k` of this block, for one of its readers (a whole warp).
__device__ __forceinline__ bool next_job(const PrefillParams& p, Misc* ms, uint32_t k, Job& job) {
  if (!warp_wait_on(&ms->job_full[k & 1], (k >> 1) & 1, ms, p.err)) return false;
  job = ms->job[k & 1];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ms->job_empty[k & 1]));
  return job.live != 0;
}

// ------------------------------------------------------------ producer (one warp, lane 0 copies)
// K(T) is the ring's fills 5 T .. 5 T + 2 and V(T) 5 T + 3 and 5 T + 4, fill f in
// slot f % 8: K(T) takes the slots of K(T - 2)'s last panel and V(T - 2), V(T)
// those of K(T - 1)'s first two.
__device__ __forceinline__ uint32_t ring_slot(uint32_t f) { return f % kSlots; }

struct Loads {
  uint32_t k = 0, v = 0, q0 = 0, q1 = 0;  // copies issued: key tiles, and query tiles 0 and 1
};

// The next job is taken when this many key tiles of the present one are still to
// be copied: late enough that no block sits on a job that another could start and
// that the heads of a block of queries stay abreast, early enough to hide the
// counter and the search, since the copies run two tiles ahead.  (76 rows of up to
// 256 tokens: 52.3 us, with two tiles 54.1; 12 prompts of up to 2047 tokens: 99 us,
// and 105 with the next job taken as a job starts.)
constexpr int32_t kClaimTiles = 1;

// Whether a copy that starts at this token does so inside its tensor (debug build; a
// failed check ends the call through the abort flag).
__device__ __forceinline__ bool copy_ok(const PrefillParams& p, Misc* ms, const Job& job, int32_t token, int64_t tokens) {
  if (MLA_DCHECK(token >= 0 && token < tokens && job.head >= 0 && job.head < p.heads, p.err)) return true;
  ms->abort_flag = 1;
  return false;
}

// The copies of one job (lane 0).
__device__ __forceinline__ bool load_job(const PrefillParams& p, const PrefillMaps& m, Misc* ms, uint32_t sbase,
                                         const Job& job, Loads& l, uint64_t keep, uint64_t once) {
  const uint32_t ring = sbase + kOffRing;
  const int32_t n = job.tiles(), claim = max(0, n - kClaimTiles);
  if (n == 0) mbar_arrive(smem_u32(&ms->claim));
  auto load_q = [&](int t, uint32_t& count) {
    if (!wait_on(&ms->q_empty[t], (count + 1) & 1, ms, p.err)) return false;  // (the first passes)
    if (!copy_ok(p, ms, job, job.q0 + t * kTile, p.total_q)) return false;
    ++count;
    const uint32_t bar = smem_u32(&ms->q_full[t]);
    mbar_arrive_expect_tx(bar, kQPanels * kPanelBytes);
    for (int c = 0; c < kQPanels; ++c)
      tma_load_3d(sbase + kOffQ + (t * kQPanels + c) * kPanelBytes, &m.q, 64 * c, job.head, job.q0 + t * kTile,
                  bar, once);
    return true;
  };
  for (int32_t j = 0; j < n; ++j) {
    const uint32_t T = l.k, f = T * kFillsPerTile;
    const int32_t key = job.k0 + (job.j0 + j) * kTile;
    if (j == claim) mbar_arrive(smem_u32(&ms->claim));
    if (T > 1 && !wait_on(&ms->v_empty[T & 1], ((T >> 1) + 1) & 1, ms, p.err)) return false;
    if (!copy_ok(p, ms, job, key, p.total_kv)) return false;
    uint32_t bar = smem_u32(&ms->k_full[T & 1]);
    mbar_arrive_expect_tx(bar, kKPanels * kPanelBytes);
    tma_load_3d(ring + ring_slot(f) * kPanelBytes, &m.k_nope, 0, job.head, key, bar, keep);
    tma_load_3d(ring + ring_slot(f + 1) * kPanelBytes, &m.k_nope, 64, job.head, key, bar, keep);
    tma_load_2d(ring + ring_slot(f + 2) * kPanelBytes, &m.k_rope, 0, key, bar, keep);
    ++l.k;
    if (j == 0 && job.nt0 > 0 && !load_q(0, l.q0)) return false;
    if (j == 0 && job.nt1 > 0 && !load_q(1, l.q1)) return false;
    if (T > 0 && !wait_on(&ms->k_empty[(T - 1) & 1], ((T - 1) >> 1) & 1, ms, p.err)) return false;
    bar = smem_u32(&ms->v_full[T & 1]);
    mbar_arrive_expect_tx(bar, kVPanels * kPanelBytes);
#pragma unroll
    for (int h = 0; h < kVPanels; ++h) {
      const uint32_t dst = ring + ring_slot(f + kKPanels + h) * kPanelBytes;
      tma_load_3d(dst, &m.v, 0, job.head, key + 64 * h, bar, keep);
      tma_load_3d(dst + kPanelBytes / 2, &m.v, 64, job.head, key + 64 * h, bar, keep);
    }
    ++l.v;
  }
  return true;
}

// The same for pairs: key tile T's K and V in buffer T & 1.
__device__ __forceinline__ bool load_pair_job(const PrefillParams& p, const PrefillMaps& m, Misc* ms, uint32_t sbase,
                                              const Job& job, Loads& l, uint64_t keep, uint64_t once) {
  const int32_t n = job.tiles(), claim = max(0, n - kClaimTiles);
  if (n == 0) mbar_arrive(smem_u32(&ms->claim));
  for (int32_t j = 0; j < n; ++j) {
    const uint32_t b = l.k & 1, before = ((l.k >> 1) + 1) & 1;  // (the first of each pass)
    const int32_t key = job.k0 + (job.j0 + j) * kTile;
    if (j == claim) mbar_arrive(smem_u32(&ms->claim));
    if (!wait_on(&ms->pair_k_empty[b], before, ms, p.err)) return false;
    if (!copy_ok(p, ms, job, key, p.total_kv)) return false;
    uint32_t bar = smem_u32(&ms->k_full[b]), dst = sbase + kOffPairK + b * kKPanels * kPanelBytes;
    mbar_arrive_expect_tx(bar, kKPanels * kPanelBytes);
    tma_load_3d(dst, &m.k_nope, 0, job.head, key, bar, keep);
    tma_load_3d(dst + kPanelBytes, &m.k_nope, 64, job.head, key, bar, keep);
    tma_load_2d(dst + 2 * kPanelBytes, &m.k_rope, 0, key, bar, keep);
    ++l.k;
    if (j == 0) {
      if (!wait_on(&ms->pair_q_empty, (l.q0 + 1) & 1, ms, p.err)) return false;
      if (!copy_ok(p, ms, job, job.q0, p.total_q)) return false;
      ++l.q0;
      bar = smem_u32(&ms->q_full[0]);
      mbar_arrive_expect_tx(bar, kQPanels * kPanelBytes);
      for (int c = 0; c < kQPanels; ++c)
        tma_load_3d(sbase + kOffQ + c * kPanelBytes, &m.q, 64 * c, job.head, job.q0, bar, once);
    }
    if (!wait_on(&ms->pair_v_empty[b], before, ms, p.err)) return false;
    bar = smem_u32(&ms->v_full[b]);
    dst = sbase + kOffPairV + b * kVPanels * kPanelBytes;
    mbar_arrive_expect_tx(bar, kVPanels * kPanelBytes);
    for (int h = 0; h < kVPanels; ++h) {
      tma_load_3d(dst + h * kPanelBytes, &m.v, 0, job.head, key + 64 * h, bar, keep);
      tma_load_3d(dst + h * kPanelBytes + kPanelBytes / 2, &m.v, 64, job.head, key + 64 * h, bar, keep);
    }
    ++l.v;
  }
  return true;
}

__device__ __forceinline__ void run_producer(const PrefillParams& p, const PrefillMaps& m, Misc* ms, uint32_t sbase) {
  const int lane = threadIdx.x & 31;
  const uint64_t keep = l2_policy_evict_normal(), once = l2_policy_evict_first();
  Loads l;
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    if (lane == 0) {
      if (p.stall_stream)
        mbar_arrive(smem_u32(&ms->claim));
      else
        ok = ms->pairs ? load_pair_job(p, m, ms, sbase, job, l, keep, once)
                       : load_job(p, m, ms, sbase, job, l, keep, once);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  }
  if (!ms->abort_flag) return;  // the issuers wait for every copy
  // Abandoned: the copies in flight land before the block's memory is given up.
  if (lane == 0) {
    if (l.q0 > 0) drain(&ms->q_full[0], (l.q0 - 1) & 1);
    if (l.q1 > 0) drain(&ms->q_full[1], (l.q1 - 1) & 1);
    for (uint32_t T = l.k > 2 ? l.k - 2 : 0; T < l.k; ++T) drain(&ms->k_full[T & 1], (T >> 1) & 1);
    for (uint32_t T = l.v > 2 ? l.v - 2 : 0; T < l.v; ++T) drain(&ms->v_full[T & 1], (T >> 1) & 1);
  }
  __syncwarp();
}

// ------------------------------------------------------------ scheduler (one warp)
// The first job is the block's own, the others are taken from a counter.
__device__ __forceinline__ void run_scheduler(const PrefillParams& p, Misc* ms) {
  const int lane = threadIdx.x & 31;
  Batch rows = count_rows(p);
  if (lane == 0) ms->pairs = rows.size == kTile;
  uint32_t index = blockIdx.x;
  for (uint32_t k = 0;; ++k) {
    Job* job = &ms->job[k & 1];
    if (!warp_wait_on(&ms->job_empty[k & 1], ((k >> 1) + 1) & 1, ms, p.err)) return;  // (the first two pass)
    find_job(p, rows, index, job);
    const int32_t live = job->live;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ms->job_full[k & 1]));
    if (live == 0 || !warp_wait_on(&ms->claim, k & 1, ms, p.err)) return;
    if (lane == 0) index = gridDim.x + atomicAdd(p.sched, 1u);
    index = __shfl_sync(0xffffffffu, index, 0);
  }
}

// ------------------------------------------------------------ V behind the row's end
// The row's last key tile may end inside the tile.  The rows of V behind it are
// another row's, or never written: their probabilities are zero, but zero times
// NaN is NaN, so issuer 0 zeroes them in shared memory (while the tile's softmax
// runs) before either product reads them; of pairs, the issuer whose tile it is.
__device__ __forceinline__ void clean_v(uint8_t* v0, uint8_t* v1, int32_t keys) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int32_t i = keys * 16 + lane; i < kTile * 16; i += 32) {
    const int32_t key = i >> 4, piece = i & 15;
    *reinterpret_cast<uint4*>((key < 64 ? v0 : v1) + (piece >> 3) * (kPanelBytes / 2) + (key & 63) * 128 + (piece & 7) * 16) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// ------------------------------------------------------------ MMA issuers (a warp a tile, an elected lane issues)
// The tensor pipe takes hardly more than one of these products ahead (measured:
// 48 of 128 x 128 x 16 issued back to back block the issuer until ~100 cycles
// before they end, 64 cycles each), and a look at a barrier takes 100 to 150
// cycles beside the products' own reads of shared memory.  So each tile has its
// own issuer, which waits for what its next products need while the other
// tile's run, and they take turns: P_t(j) . V(j) and Q_t . K(j + 1)^T are issued
// together, the turn handed over one product before their end.  (A 16384-token
// prompt: one issuer for both tiles 913 us, two without turns 1252 us, as both
// tiles' softmax then fall together, two in turn 776 us at that time.  A single S
// for both tiles with one issuer for the scores and one for the values: 829 us.)
__device__ __forceinline__ void run_mma(const PrefillParams& p, Misc* ms, uint32_t sbase, uint32_t tmem, int t) {
  const uint64_t q_desc = smem_desc(sbase + kOffQ + t * kQPanels * kPanelBytes, 1024, 1024, kLayoutSw128);
  const uint64_t k_desc = smem_desc(sbase + kOffRing, 1024, 1024, kLayoutSw128);
  const uint64_t v_desc = smem_desc(sbase + kOffRing, kPanelBytes / 2, 1024, kLayoutSw128);
  constexpr uint32_t kPanel = kPanelBytes >> 4;  // a panel, in descriptor address units
  const uint32_t other_turn = smem_u32(&ms->turn[t ^ 1]);
  const uint32_t d_s = tmem + kColS + 128 * t, d_o = tmem + kColO + 128 * t;
  constexpr int kHandover = 1;   // products issued after the turn is handed over
  constexpr int kHeadSteps = 6;  // k-steps of 16 keys in p_head
  // A wait of this warp; tile 0 starts, so its first turn is the phase before the first.
  auto on = [&](const uint64_t* bar, uint32_t parity) { return warp_wait_on(bar, parity & 1, ms, p.err); };
  // (bit b of clean_phase: the phase of v_clean[b] to wait for next)
  uint32_t turns = t, T = 0, mine = 0, jobs = 0, clean_phase = 0;
  bool duo = false;  // both tiles have keys: they take turns
  // S_t = Q_t . K(T)^T (one lane)
  auto qk = [&](uint32_t tile, bool last, bool hand_over) {
    const uint32_t f = tile * kFillsPerTile;
#pragma unroll
    for (int c = 0; c < kKPanels; ++c) {
      const uint64_t a = q_desc + c * kPanel, b = k_desc + ring_slot(f + c) * kPanel;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (4 * c + kk == 4 * kKPanels - kHandover && hand_over) mbar_arrive(other_turn);
        umma_f16(d_s, a + 2 * kk, b + 2 * kk, kIdescQK, c != 0 || kk != 0);
      }
    }
    umma_commit(smem_u32(&ms->s_full[t]));
    umma_commit(smem_u32(&ms->k_empty[tile & 1]));
    if (last) umma_commit(smem_u32(&ms->q_empty[t]));
  };
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    const int32_t nt = t ? job.nt1 : job.nt0, n = job.tiles(), clean = job.partial();
    if (n == 0) continue;
    duo = job.nt0 > 0 && job.nt1 > 0;
    ok = (nt == 0 || on(&ms->q_full[t], jobs)) && on(&ms->k_full[T & 1], T >> 1);
    if (!ok) break;
    tc_fence_after();
    if (elect_one()) {
      if (nt > 0) {
        qk(T, nt == 1, false);  // beside the other tile's last products of the job before
      } else {  // the other tile alone reads this K
        mbar_arrive(smem_u32(&ms->k_empty[T & 1]));
      }
    }
    __syncwarp();
    for (int32_t j = 0; j < n && ok; ++j, ++T) {
      const bool here = j < nt, next = j + 1 < nt;
      ok = on(&ms->v_full[T & 1], T >> 1);
      if (ok && j == clean) {
        if (t == 0) {
          const uint32_t f = T * kFillsPerTile + kKPanels;
          clean_v(block_memory(ms, kOffRing + ring_slot(f) * kPanelBytes),
                  block_memory(ms, kOffRing + ring_slot(f + 1) * kPanelBytes), job.len % kTile);
          if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ms->v_clean[T & 1]));
          __syncwarp();
        } else {
          ok = on(&ms->v_clean[T & 1], clean_phase >> (T & 1));
          clean_phase ^= 1u << (T & 1);
        }
      }
      // K(T + 1) has mostly landed too; looked at here, it costs no pause between
      // the products.
      const bool k_ready = ok && j + 1 < n &&
                           __all_sync(0xffffffffu, mbar_test_wait(smem_u32(&ms->k_full[(T + 1) & 1]), ((T + 1) >> 1) & 1));
      ok = ok && (j != 0 || nt == 0 || on(&ms->o_free[t], jobs + 1)) && (!duo || on(&ms->turn[t], ++turns)) &&
           (!here || on(&ms->p_head[t], mine));
      if (!ok) break;
      tc_fence_after();
      const uint32_t f = T * kFillsPerTile + kKPanels;
      const uint64_t v0 = v_desc + ring_slot(f) * kPanel, v1 = v_desc + ring_slot(f + 1) * kPanel;
      if (here) {
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kHeadSteps; ++kk)
            umma_f16_ts(d_o, d_s + 8 * kk, (kk < 4 ? v0 : v1) + (kk & 3) * 128, kIdescPV, j != 0 || kk != 0);
        }
        __syncwarp();
        ok = on(&ms->p_full[t], mine++);
        if (!ok) break;
        tc_fence_after();
      }
      if (elect_one()) {
        if (here) {
#pragma unroll
          for (int kk = kHeadSteps; kk < 8; ++kk) umma_f16_ts(d_o, d_s + 8 * kk, v1 + (kk & 3) * 128, kIdescPV, 1);
          if (!next) umma_commit(smem_u32(&ms->o_full[t]));
          umma_commit(smem_u32(&ms->v_empty[T & 1]));
        } else {
          mbar_arrive(smem_u32(&ms->v_empty[T & 1]));
        }
        if (!next && duo) mbar_arrive(other_turn);
      }
      __syncwarp();
      if (j + 1 == n) continue;
      ok = k_ready || on(&ms->k_full[(T + 1) & 1], (T + 1) >> 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        if (next)
          qk(T + 1, j + 2 == nt, duo);
        else
          mbar_arrive(smem_u32(&ms->k_empty[(T + 1) & 1]));
      }
      __syncwarp();
    }
    jobs += nt > 0;
  }
  if (elect_one()) umma_commit(smem_u32(&ms->mma_done));
  __syncwarp();
}

// Pairs: issuer t has the key tiles T with T & 1 == t, in buffer t, and its products
// depend on nothing of the other issuer's: the chain of a tile (load, scores,
// softmax, values) runs beside the other's.
__device__ __forceinline__ void run_pair_mma(const PrefillParams& p, Misc* ms, uint32_t sbase, uint32_t tmem, int t) {
  const int k_at = kOffPairK + t * kKPanels * kPanelBytes, v_at = kOffPairV + t * kVPanels * kPanelBytes;
  const uint64_t q_desc = smem_desc(sbase + kOffQ, 1024, 1024, kLayoutSw128);
  const uint64_t k_desc = smem_desc(sbase + k_at, 1024, 1024, kLayoutSw128);
  const uint64_t v_desc = smem_desc(sbase + v_at, kPanelBytes / 2, 1024, kLayoutSw128);
  constexpr uint32_t kPanel = kPanelBytes >> 4;
  const uint32_t d_s = tmem + kColS + 128 * t, d_o = tmem + kColO + 128 * t;
  constexpr int kHeadSteps = 6;
  auto on = [&](const uint64_t* bar, uint32_t parity) { return warp_wait_on(bar, parity & 1, ms, p.err); };
  uint32_t T = 0, mine = 0, jobs = 0, own_jobs = 0;
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    const int32_t n = job.tiles(), clean = job.partial(), first = (T ^ t) & 1;
    if (n == 0) continue;
    T += n;
    ok = on(&ms->q_full[0], jobs++);
    if (!ok) break;
    if (first >= n) {  // the job's one tile is the other issuer's
      if (elect_one()) mbar_arrive(smem_u32(&ms->pair_q_empty));
      __syncwarp();
      continue;
    }
    for (int32_t j = first; j < n; j += 2, ++mine) {
      const bool last = j + 2 >= n;
      ok = on(&ms->k_full[t], mine);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < kKPanels; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16(d_s, q_desc + c * kPanel + 2 * kk, k_desc + c * kPanel + 2 * kk, kIdescQK, c != 0 || kk != 0);
        umma_commit(smem_u32(&ms->s_full[t]));
        umma_commit(smem_u32(&ms->pair_k_empty[t]));
        if (last) umma_commit(smem_u32(&ms->pair_q_empty));
      }
      __syncwarp();
      ok = on(&ms->v_full[t], mine);
      if (!ok) break;
      if (j == clean) clean_v(block_memory(ms, v_at), block_memory(ms, v_at + kPanelBytes), job.len % kTile);
      ok = (j != first || on(&ms->o_free[t], own_jobs + 1)) && on(&ms->p_head[t], mine);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kHeadSteps; ++kk)
          umma_f16_ts(d_o, d_s + 8 * kk, v_desc + (kk >> 2) * kPanel + (kk & 3) * 128, kIdescPV, j != first || kk != 0);
      }
      __syncwarp();
      ok = on(&ms->p_full[t], mine);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = kHeadSteps; kk < 8; ++kk)
          umma_f16_ts(d_o, d_s + 8 * kk, v_desc + (kk >> 2) * kPanel + (kk & 3) * 128, kIdescPV, 1);
        if (last) umma_commit(smem_u32(&ms->o_full[t]));
        umma_commit(smem_u32(&ms->pair_v_empty[t]));
      }
      __syncwarp();
    }
    ++own_jobs;
  }
  if (elect_one()) umma_commit(smem_u32(&ms->mma_done));
  __syncwarp();
}

// ------------------------------------------------------------ softmax
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 bytes of a row.  A warp's lanes write 32 different rows, one cache line each,
// which holds up the other warps' barriers while it lasts: whole 32-byte sectors
// take half the instructions of 16-byte pieces (which an output that is only
// 16-byte aligned gets).
__device__ __forceinline__ void store_row32(void* dst, const uint32_t* w, int32_t wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// One job of softmax t (a warpgroup): its query tile, or of pairs its key tiles.
// `tiles`, `jobs` and `joins` count what was done before: this warpgroup's tiles,
// its jobs with tiles, and of pairs the joinings.
template <bool kPairs>
__device__ __forceinline__ bool softmax_job(const PrefillParams& p, Misc* ms, uint32_t tmem, const Job& job, int t,
                                            int32_t first, uint32_t& tiles, uint32_t& jobs, uint32_t& joins) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int row0 = (kPairs ? 0 : t * kTile) + quad * 32, qi = row0 + lane;  // this thread's query of the job
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t s_addr = tmem + lanes + kColS + 128 * t, o_addr = tmem + lanes + kColO + 128 * t;
  constexpr int32_t kStep = kPairs ? 2 : 1;
  const int32_t n = kPairs ? job.nt0 : t ? job.nt1 : job.nt0;
  const float sl = p.scale * 1.4426950408889634f;    // scores to powers of two
  // keys that this row, and the warp's first row, see
  const int32_t sees = p.causal ? min(job.len, job.see + qi) : job.len;
  const int32_t warp_sees = p.causal ? min(job.len, job.see + row0) : job.len;
  float ref = -INFINITY, sum = 0.0f;
  for (int32_t j = first; j < n; j += kStep, ++tiles) {
    if (!warp_wait_on(&ms->s_full[t], tiles & 1, ms, p.err)) return false;
    tc_fence_after();
    uint32_t raw[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, raw[c]);
    tmem_wait_ld();
    const int32_t key0 = (job.j0 + j) * kTile;
    if (warp_sees - key0 < kTile) {
      const int32_t lim = sees - key0, warp_lim = warp_sees - key0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (warp_lim >= 32 * c + 32) continue;  // all of the warp's rows see these keys
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (32 * c + i >= lim) raw[c][i] = 0xFF800000u;  // -inf
      }
    }
    float top[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      top[c] = __uint_as_float(raw[c][0]);
#pragma unroll
      for (int i = 1; i < 32; ++i) top[c] = fmaxf(top[c], __uint_as_float(raw[c][i]));
    }
    const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    // (a first finite maximum is infinitely far above -inf; two -inf are not apart)
    const bool moves = high > ref && (high - ref) * sl > kRescaleThreshold;
    if (__any_sync(0xffffffffu, moves)) {
      const float alpha = moves ? ex2((ref - high) * sl) : 1.0f;
      if (moves) ref = high;
      sum *= alpha;
      if (j > first) {  // O_t's last product is complete: S_t(j) was issued after it
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(o_addr + 16 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(o_addr + 16 * c, o);
        }
      }
    }
    const float off = ref == -INFINITY ? 0.0f : -ref * sl;
    const uint64_t sl2 = pack2(sl, sl), off2 = pack2(off, off);
    uint64_t part[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = 2 * i;
        float x, y;
        unpack2(fma2(pack2(__uint_as_float(raw[c][e]), __uint_as_float(raw[c][e + 1])), sl2, off2), x, y);
        x = ex2(x);
        y = ex2(y);
        part[i & 1] = add2(part[i & 1], pack2(x, y));
        pk[i] = bf16x2(x, y);
      }
      tmem_st16(s_addr + 16 * c, pk);
      if (c == 2) {  // the products of the first 96 keys may start
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms->p_head[t]));
      }
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&ms->p_full[t]));
    float s0, s1, s2, s3;
    unpack2(part[0], s0, s1);
    unpack2(part[1], s2, s3);
    sum += (s0 + s1) + (s2 + s3);
  }

  // Epilogue.  A row that saw no key has sum 0; a NaN score makes it NaN, which reaches
  // the output and the log-sum-exp (and through them the joined parts).
  if (n > first) {
    if (!warp_wait_on(&ms->o_full[t], jobs & 1, ms, p.err)) return false;
    ++jobs;
    tc_fence_after();
  }
  // Pairs: the softmax without the job's first tile hands over its maximum and sum
  // (written after its O is complete, so after the last ones were read), the other
  // weights both accumulators by them.
  const bool join = kPairs && n > 1;
  float weight = 1.0f, other_weight = 0.0f;
  if (join) {
    float2* stats = reinterpret_cast<float2*>(block_memory(ms, kOffStats)) + quad * 32 + lane;
    if (first != 0) {
      stats[t * kTile] = make_float2(ref, sum);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->joined[t]));
      return true;
    }
    if (!warp_wait_on(&ms->joined[t ^ 1], joins & 1, ms, p.err)) return false;
    ++joins;
    tc_fence_after();
    const float2 other = stats[(t ^ 1) * kTile];
    const float high = fmaxf(ref, other.x);
    weight = ref == high ? 1.0f : ex2((ref - high) * sl);  // (-inf is not apart from -inf)
    other_weight = other.x == high ? 1.0f : ex2((other.x - high) * sl);
    sum = weight * sum + other_weight * other.y;
    ref = high;
  }
  bool live = qi < job.nq;
  if (live)
    live = MLA_DCHECK(job.q0 >= 0 && job.q0 + qi < p.total_q && job.head >= 0 && job.head < p.heads && job.split >= 0 &&
                          job.split < p.splits &&
                          (p.splits == 1 || static_cast<int64_t>(p.splits) * p.total_q * p.heads <= p.part_rows), p.err);
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  const int64_t at = static_cast<int64_t>(job.q0 + qi) * p.heads + job.head;
  const int64_t part_at = static_cast<int64_t>(job.split) * p.total_q * p.heads + at;
  // (one copy of a chunk's code: it runs once a job, and unrolled it is fetched
  // from far away every time)
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    if (n > 0) {
      tmem_ld32(o_addr + 32 * c, o);
      if (join) {
        uint32_t x[32];
        tmem_ld32(tmem + lanes + kColO + 128 * (t ^ 1) + 32 * c, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          o[i] = __float_as_uint(__uint_as_float(o[i]) * weight + __uint_as_float(x[i]) * other_weight);
      } else {
        tmem_wait_ld();
      }
      if (c == 3) {  // the next job's products may overwrite O_t
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ms->o_free[t]));
          if (join) mbar_arrive(smem_u32(&ms->o_free[t ^ 1]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0;
    }
    if (live && p.splits == 1) {
      uint16_t* dst = p.out + at * kPrefillV + 32 * c;
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
      store_row32(dst, w, p.wide_out);
      store_row32(dst + 16, w + 8, p.wide_out);
    } else if (live) {
      float* dst = p.part + part_at * kPrefillV + 32 * c;
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) store_row32(dst + 8 * i, o + 8 * i, 1);
    }
    __syncwarp();
  }
  if (live) {
    const float lse = sum != 0.0f ? ref * p.scale + logf(sum) : -INFINITY;
    if (p.splits > 1)
      p.part_lse[part_at] = lse;
    else if (p.lse != nullptr)
      p.lse[at] = lse;
  }
  __syncwarp();
  return true;
}

template <bool kPairs>
__device__ __forceinline__ void run_softmax(const PrefillParams& p, Misc* ms, uint32_t tmem, int t) {
  uint32_t tiles = 0, jobs = 0, joins = 0;
  int32_t first = kPairs ? t : 0;  // of pairs, this warpgroup's first key tile of the job
  Job job;
  for (uint32_t k = 0; next_job(p, ms, k, job); ++k) {
    const bool mine = kPairs ? first == 0 || job.nt0 > 1 : job.nq > t * kTile;
    if (mine && !softmax_job<kPairs>(p, ms, tmem, job, t, first, tiles, jobs, joins)) return;
    if (kPairs) first ^= job.nt0 & 1;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ PrefillMaps maps, const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Misc* ms = reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&ms->tmem_base), kTmemCols);
  if (tid == kProducerWarp * 32) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ms->k_full[t]), 1);
      mbar_init(smem_u32(&ms->v_full[t]), 1);
      mbar_init(smem_u32(&ms->k_empty[t]), 2);
      mbar_init(smem_u32(&ms->v_empty[t]), 2);
      mbar_init(smem_u32(&ms->q_full[t]), 1);
      mbar_init(smem_u32(&ms->s_full[t]), 1);
      mbar_init(smem_u32(&ms->p_head[t]), 4);
      mbar_init(smem_u32(&ms->p_full[t]), 4);
      mbar_init(smem_u32(&ms->o_full[t]), 1);
      mbar_init(smem_u32(&ms->o_free[t]), 4);
      mbar_init(smem_u32(&ms->q_empty[t]), 1);
      mbar_init(smem_u32(&ms->job_full[t]), 1);
      mbar_init(smem_u32(&ms->job_empty[t]), kJobReaders);
      mbar_init(smem_u32(&ms->turn[t]), 1);
      mbar_init(smem_u32(&ms->v_clean[t]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ms->pair_k_empty[b]), 1);
      mbar_init(smem_u32(&ms->pair_v_empty[b]), 1);
      mbar_init(smem_u32(&ms->joined[b]), 4);
    }
    mbar_init(smem_u32(&ms->pair_q_empty), 2);
    mbar_init(smem_u32(&ms->claim), 1);
    mbar_init(smem_u32(&ms->mma_done), 2);
    ms->abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k_nope);
    prefetch_tensormap(&maps.k_rope);
    prefetch_tensormap(&maps.v);
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem_base;
  if (warp >= kFirstSoftmaxWarp) {
    setmaxnreg_inc<kSoftmaxRegs>();
    const int t = (warp - kFirstSoftmaxWarp) >> 2;
    if (in_pairs(p, ms))
      run_softmax<true>(p, ms, tmem, t);
    else
      run_softmax<false>(p, ms, tmem, t);
  } else {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kProducerWarp)
      run_producer(p, maps, ms, sbase);
    else if (warp == kSchedulerWarp)
      run_scheduler(p, ms);
    else if (in_pairs(p, ms))
      run_pair_mma(p, ms, sbase, tmem, warp - kMmaWarp);
    else
      run_mma(p, ms, sbase, tmem, warp - kMmaWarp);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // (What is known above is read anew here.  Kept over the roles it made the issuers
  // spill a word: 3 % of the ragged batch, and 0.35 us of a launch for its local memory.)
  if (threadIdx.x >> 5 == kMmaWarp) {
    const bool one = (threadIdx.x & 31) == 0;
    if (one) drain(&ms->mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(ms->tmem_base, kTmemCols);
    // (Abandoned: the parts are not whole.  Block 0 has written the word long before a wait runs out.)
    if (one && ms->abort_flag) p.sched[2] = 1;
    // The last block leaves the counters zero for the workspace's next call.
    if (one && atomicAdd(p.sched + 1, 1u) == gridDim.x - 1) {
      p.sched[0] = 0;
      p.sched[1] = 0;
    }
  }
}

}  // namespace

size_t prefill_smem_bytes() { return kSmemBytes; }

cudaError_t prefill_prepare() {
  return cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

cudaError_t launch_prefill(const PrefillParams& p, const PrefillMaps& maps, cudaStream_t stream) {
  const int64_t jobs = static_cast<int64_t>(p.blocks) * p.heads * p.splits;
  if (jobs > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const int64_t grid = jobs < p.num_sms ? jobs : p.num_sms;
  return launch_dependent(prefill_kernel, static_cast<unsigned>(grid), kThreads, kSmemBytes, stream,
                          maps, p);
}

}  // namespace mla
