// mla_shared_fwd: decode queries of many rows over keys that all of them see (a prefix
// that the rows of a group share), e4m3 cache, with the log-sum-exp that joins the
// result to each row's own keys.
//
// The decode step reads a row's keys once for its 16 heads, and is bound by those
// bytes.  Here a block takes four query tokens, 64 rows of 16 heads each, over the same
// keys, so that the tensor cores bound it.  For a tile of 128 keys (T):
//   S^T[key][row]  = K(T) . Q^T      128 x 128 x 576: 64 rows of high terms, 64 of low
//   O^T[dim][row] += V(T)^T . P^T    4 x 128 x 64 x 128, once for P's high terms and
//                                    once for its low ones
// K(T) and V(T) are the same e4m3 codes in shared memory (V the first 512 dims), read
// by key for the first product and by dim for the second, so nothing is converted.  A
// bf16 query is two e4m3 terms, q 2^k = hi + lo / 8, exact down to 2^-13 of the row's
// largest magnitude; a probability p in [0, 2^8] is hi + lo, to 2^-8 of itself and 2^-10,
// which is 2^-14 of the row's reference (2^4).  TMEM is full: two S of 128 columns, O in
// four chunks of 64.
//
// Persistent blocks, one an SM, are workers.  Every four query tokens of a group, with their
// keys, are a block of units, a unit a key tile and some for its start; all blocks' units
// one behind the other are cut into equal ranges, a worker each.  A job is what a range has
// of one block, or, of blocks that are not cut, the whole of each that begins in the range:
//   * warp 3 finds the jobs,
//   * the keys come as four panels of 128 dims a tile into two buffers, and the 64 rotated
//     dims into one: by warp 2 through TMA in boxes of 128 rows, or, by a page table, by
//     warps 20-27 in 16-byte copies (TMA's gathers of four rows take 74 cycles each to
//     issue from one warp, 160 a tile, and 20 from four; alone, the copies of four warps
//     bring a panel in 500 cycles and of eight in 330),
//   * warps 0 and 1 issue the products S and O, each as soon as it can,
//   * four warpgroups, warps 4-19, run the softmax of a query token each, a thread a key: the
//     maximum over keys is over lanes, so it is only looked for when a score passes the
//     running reference by four powers of two, which few tiles' do.
// A job without all of its block's keys leaves a part of half precision, in units of the
// cache's codes (at most 448; 11 bits, 2^-4 of the output's rounding: blocks store at 30 bytes
// a cycle, and float32 parts took 4300 cycles a job), and a second kernel joins them.
//
// A tile's products are 18 of 64 cycles and 32 of 48, 2690 in all; it takes 2950.  The second
// product reads 6 KB of operands for 32 cycles' work and waits for shared memory.  256
// queries over 32768 keys take 204 us (1.43 PFLOP/s), by a page table 235, where a buffer's way
// back is longer than TMA's; 64 over 8192 26.8 and 28.9, 8 over 1000 12.3 and 13.4, of which a
// job's start (finding it, the query's two terms) is 4.5 and the second kernel 3.
#include <cstddef>

#include <cuda_fp16.h>

#include "kernels.h"
#include "ops.h"
#include "ptx.cuh"
#include "schedule.h"

namespace mla {
namespace {

constexpr int kTokens = kSharedTokens;             // query tokens of a block
constexpr int kRows = kTokens * kNumHeads;         // 64
constexpr int kPanelBytes = kTileTokens * 128;     // 128 keys (or operand rows) x 128 dims
constexpr int kPanels = kVDim / 128;               // latent panels of a tile
constexpr int kRopeBytes = kTileTokens * 64;
constexpr int kPBytes = kTileTokens * kRows;       // one term of P: a key's 64 rows are contiguous
constexpr int kOffKeys = 0;                        // [2][kPanels]
constexpr int kOffRope = kOffKeys + 2 * kPanels * kPanelBytes;
constexpr int kOffQ = kOffRope + kRopeBytes;       // [kPanels], 64 rows of high terms, then 64 of low
constexpr int kOffQRope = kOffQ + kPanels * kPanelBytes;
constexpr int kOffP = kOffQRope + kRopeBytes;      // high terms, low terms
constexpr int kOffMisc = kOffP + 2 * kPBytes;

constexpr int kScoreWarp = 0, kValueWarp = 1, kProducerWarp = 2, kSchedulerWarp = 3, kFirstSoftmaxWarp = 4;
constexpr uint32_t kSoftmaxWarps = 4 * kTokens, kCopyWarps = 8;
constexpr int kFirstCopyWarp = kFirstSoftmaxWarp + static_cast<int>(kSoftmaxWarps);
// Threads of a block, and registers: launched with 96 a thread (72 with a page table),
// of which the softmax warpgroups take the others' share.
template <bool kPaged>
__host__ __device__ constexpr int threads() { return 32 * (kFirstCopyWarp + (kPaged ? static_cast<int>(kCopyWarps) : 0)); }
template <bool kPaged>
__host__ __device__ constexpr int softmax_regs() { return kPaged ? 88 : 104; }
template <bool kPaged>
__host__ __device__ constexpr int other_regs() { return kPaged ? 48 : 64; }
static_assert(kTokens * 128 * softmax_regs<false>() + (threads<false>() - kTokens * 128) * other_regs<false>() <= threads<false>() * 96 &&
                  kTokens * 128 * softmax_regs<true>() + (threads<true>() - kTokens * 128) * other_regs<true>() <= threads<true>() * 72,
              "register split exceeds the launch allocation");
// What reads a job: two issuers, the softmax, and the producer or the copying warps.
template <bool kPaged>
__host__ __device__ constexpr uint32_t job_readers() { return 2 + kSoftmaxWarps + (kPaged ? kCopyWarps : 1); }
constexpr uint32_t kBarSoftmax = 1;                // + g: named barrier of a softmax warpgroup
constexpr uint32_t kLayoutSw128 = 2, kLayoutSw64 = 4;
constexpr uint32_t kColS = 0, kColO = 256;         // S of tile T at 128 (T & 1); chunk c of O at + 64 c
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescQK = idesc_e4m3(128, 128, false, false);
constexpr uint32_t kIdescPV = idesc_e4m3(128, kRows, true, true);
constexpr float kSmScaleLog2 = 1.4426950408889634f / 24.0f;  // dot products to powers of two
// A probability is 2^(s - reference + 4), computed 2^8 smaller (split_p): the reference
// stands at kTop.  It follows a maximum that passes it by four powers of two, so none is
// above 2^8, which e4m3 holds.  The farther apart the two, the rarer the maximum is looked
// for (normal scores of two powers of two: in half of 64 tiles with a distance of two, in
// three with four; 308 and 252 us for 256 queries over 32768 keys) and the coarser the small
// probabilities: with these one of 2^-13 of the reference's is still a step of the low term.
constexpr float kTop = -4.0f;

struct Job {
  int32_t q0, nq;    // first query token, number of them (up to four)
  int32_t k0, keys;  // first key of the part (of all groups' keys), and keys
  int32_t slot;      // of the part in the workspace; -1: these are all of the block's keys
  int32_t live;      // 0: no more jobs
  int64_t end;       // unit behind the block's last
  __device__ __forceinline__ int32_t tiles() const { return (keys + kTileTokens - 1) / kTileTokens; }
};

// Key tiles are numbered through all of a block's jobs (T), and so are the jobs that
// have any; the numbers give the barriers' phases.  The waits of each barrier come in
// order, and none can be two phases behind: what completes a phase needs, through the
// other roles, that its waiters have passed the one before (said at each).
struct Misc {
  uint64_t job_full[2], job_empty[2];
  uint64_t key_full[2 * kPanels], key_empty[2 * kPanels];  // panel c of tile T: kPanels (T & 1) + c
  uint64_t rope_full, rope_empty;
  uint64_t q_full;       // a job's query operand written ...
  uint64_t q_empty;      // ... and read by its last scores
  uint64_t s_full[2];    // S(T) complete, T & 1 ...
  uint64_t s_free[2];    // ... and read; S(T + 2) is issued behind that
  uint64_t p_full[4];    // 32 keys' P(T) written (those of warp w of the warpgroups), O rescaled ...
  // ... and read by the last chunk, T & 1; P(T + 1) is written behind that.  With the last 32 keys
  // O(T) is complete: who waits for that has not waited for O(T - 1) and O(T - 2), of which the
  // latter is, since warp 3 waits for each before it writes the next P.
  uint64_t p_free[2][4];
  uint64_t o_free;       // a job's O read out
  uint64_t mma_done;     // both issuers' last products
  uint32_t tmem_base;
  volatile int32_t abort_flag;
  Job job[2];
  // Of a warpgroup's rows, its token's heads:
  alignas(16) float red[kTokens][4][kNumHeads];  // [warpgroup][warp][row]: maxima, sums
  alignas(16) float scale[kTokens][kNumHeads];   // products to powers of two
  alignas(16) float off[kTokens][kNumHeads];     // kTop less the reference
  alignas(16) float factor[kTokens][kNumHeads];  // of O: rescaling, at the end the division
};
constexpr int kSmemBytes = kOffMisc + static_cast<int>(sizeof(Misc));
static_assert(kSmemBytes <= 232448, "shared memory of one block");

// Bounded waits on an mbarrier phase by a whole warp, which polls and gives up
// together; false when the call is being abandoned.
__device__ __forceinline__ bool warp_wait_on(const uint64_t* bar, uint32_t parity, Misc* ms, int32_t* err) {
  const uint32_t b = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(b, parity & 1))) return true;
  const long long start = clock64();
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity & 1))) return true;
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
    if (mbar_try_wait(smem_u32(bar), parity & 1)) return;
    if ((n & 15) == 15 && clock64() - start > kWaitLimitCycles) return;
  }
}

// ------------------------------------------------------------ who does what
struct Group {
  int32_t qs, n, ks, len;
};
// A group from its offsets.  (`back`: set when the group ends before it begins; a bad group has no
// tokens.)
__device__ __forceinline__ Group group_of(const SharedParams& p, int32_t qs, int32_t qe, int32_t ks, int32_t ke, bool report,
                                          bool& back) {
  const bool bad_q = qs < 0 || qe < qs || qe > p.total_q;
  const bool bad_k = ks < 0 || ke < ks || ke > p.kv_limit || ke - ks > MLA_SHARED_MAX_KEYS;
  back = back || qe < qs;
  if (report && (bad_q || bad_k))
    atomicOr(p.err, (bad_q ? MLA_DERR_QO_INDPTR : 0) | (bad_k ? MLA_DERR_KV_INDPTR : 0));
  return bad_q || bad_k ? Group{0, 0, 0, 0} : Group{qs, qe - qs, ks, ke - ks};
}
__device__ __forceinline__ Group load_group(const SharedParams& p, int32_t g, bool report, bool& back) {
  return group_of(p, __ldg(p.qo_indptr + g), __ldg(p.qo_indptr + g + 1), __ldg(p.kv_indptr + g), __ldg(p.kv_indptr + g + 1), report,
                  back);
}
__device__ __forceinline__ int64_t blocks_of(const Group& g) { return (g.n + kTokens - 1) / kTokens; }

// A block's units: its key tiles (one if it has none) behind `start` ones, or one where blocks are
// dealt out by their number.
__device__ __forceinline__ int64_t units_of(const SharedParams& p, const Group& g) {
  return p.split || p.start > 0 ? p.start + max(1, tiles_of_length(g.len)) : 1;
}
// A bound on units that keeps the shares' products within 64 bits.
constexpr int64_t kManyUnits = INT64_C(1) << 48;

// The groups as a warp holds them: a run of consecutive groups a lane, or every lane the only one.
struct Batch {
  int64_t first, count;  // units before the lane's run, and in it
  int32_t at;            // the group of the run that the last job was found in (or before it) ...
  int64_t at_unit;       // ... and units before it
  Shares shares;
  Group only;
};
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ Batch count_groups(const SharedParams& p) {
  const int lane = threadIdx.x & 31;
  const int32_t run = (p.batch + 31) / 32;
  Batch r;
  r.only = Group{};
  bool back = false;
  if (p.batch == 1) {
    r.at = 0;
    r.only = load_group(p, 0, blockIdx.x == 0 && lane == 0, back);
    r.first = 0;
    r.shares.all = r.count = min(blocks_of(r.only) * units_of(p, r.only), kManyUnits / 32);
  } else {
    r.at = min(p.batch, lane * run);
    const int32_t g1 = min(p.batch, r.at + run);
    r.count = 0;
    constexpr int kAtOnce = 4;  // offsets loaded together: one by one, each is a trip to L2
    for (int32_t i0 = r.at; i0 < g1; i0 += kAtOnce) {
      int32_t q[kAtOnce + 1], k[kAtOnce + 1];
#pragma unroll
      for (int i = 0; i <= kAtOnce; ++i) {
        q[i] = __ldg(p.qo_indptr + min(i0 + i, g1));
        k[i] = __ldg(p.kv_indptr + min(i0 + i, g1));
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i0 + i >= g1) break;
        const Group g = group_of(p, q[i], q[i + 1], k[i], k[i + 1], blockIdx.x == 0, back);
        r.count = min(r.count + blocks_of(g) * units_of(p, g), kManyUnits / 32);
      }
    }
    int64_t incl = r.count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    r.first = r.at_unit = incl - r.count;
    r.shares.all = __shfl_sync(0xffffffffu, incl, 31);
  }
  back = __any_sync(0xffffffffu, back);
  if (blockIdx.x == 0 && lane == 0) *p.missing = back;  // (of every call anew)
  // Groups overlap where offsets of queries decrease (which is reported) and could come to
  // any amount of work, so nothing is done then, and nothing joined.
  if (back) r.shares.all = 0;
  r.shares.workers = min(static_cast<int64_t>(p.workers), r.shares.all);
  return r;
}

// The job at unit `u` of this worker's share, which ends at `stop`: at unit `at` of group g.
__device__ __forceinline__ void make_job(const SharedParams& p, const Group& g, int64_t u, int64_t at, int64_t stop, Job* job) {
  const int64_t size = units_of(p, g), block = quotient(at, size), begin = u - (at - block * size);
  const int32_t tiles = tiles_of_length(g.len);
  const SharedPiece piece = p.split ? shared_piece(begin, tiles, p.start, u, stop) : uncut_piece(begin, tiles, u);
  job->q0 = g.qs + static_cast<int32_t>(block) * kTokens;
  // (a share that ends among a block's start units, or begins inside a block that is not cut, has none
  // of it: a job without query tokens, which all roles pass over)
  job->nq = piece.whole || piece.j1 > piece.j0 ? min(kTokens, g.n - static_cast<int32_t>(block) * kTokens) : 0;
  job->k0 = g.ks + piece.j0 * kTileTokens;
  job->keys = piece.j1 > piece.j0 ? min(g.len, piece.j1 * kTileTokens) - piece.j0 * kTileTokens : 0;
  job->slot = piece.whole ? -1 : static_cast<int32_t>(shared_slot(blockIdx.x, piece.j0 == 0));
  job->live = 1;
  job->end = begin + size;
}

// The job at unit `u` of this worker's share into `job` (a warp); none behind the share's end.
// Units only rise, so a lane looks on from the group where it found the last one.
__device__ __forceinline__ void find_job(const SharedParams& p, Batch& r, int64_t u, Job* job) {
  const int64_t c = blockIdx.x;
  int64_t stop = 0;
  if (c < r.shares.workers) stop = r.shares.begin(c + 1);
  if (u >= stop) {
    if ((threadIdx.x & 31) == 0) job->live = job->nq = job->keys = 0;
  } else if (p.batch == 1) {
    if ((threadIdx.x & 31) == 0) make_job(p, r.only, u, u, stop, job);
  } else if (u >= r.first && u < r.first + r.count) {
    bool back = false;
    Group g = load_group(p, r.at, false, back);
    while (u - r.at_unit >= blocks_of(g) * units_of(p, g)) {  // (ends within the lane's run)
      if (!MLA_DCHECK(r.at + 1 < p.batch, p.err)) break;
      r.at_unit += blocks_of(g) * units_of(p, g);
      g = load_group(p, ++r.at, false, back);
    }
    make_job(p, g, u, u - r.at_unit, stop, job);
  }
  __syncwarp();
}

// ------------------------------------------------------------ scheduler (one warp)
// The first job is found before the roles start, and known to them when they do.
__device__ __forceinline__ void run_scheduler(const SharedParams& p, Batch& groups, Misc* ms) {
  const int lane = threadIdx.x & 31;
  int64_t u = 0;
  for (uint32_t k = 0;; ++k) {
    Job* job = &ms->job[k & 1];
    if (k > 0) {
      if (k > 1 && !warp_wait_on(&ms->job_empty[k & 1], (k >> 1) - 1, ms, p.err)) return;
      find_job(p, groups, u, job);
    }
    const int32_t live = job->live;
    u = job->end;
    __syncwarp();
    if (lane == 0 && k > 0) mbar_arrive(smem_u32(&ms->job_full[k & 1]));
    if (live == 0) return;
  }
}

// Job number `k` of this block, for one of its readers (a whole warp).
__device__ __forceinline__ bool next_job(const SharedParams& p, Misc* ms, uint32_t k, Job& job) {
  if (k > 0 && !warp_wait_on(&ms->job_full[k & 1], (k - 1) >> 1, ms, p.err)) return false;
  job = ms->job[k & 1];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ms->job_empty[k & 1]));
  return job.live != 0;
}

// ------------------------------------------------------------ keys by TMA (one warp)
__device__ __forceinline__ void run_producer(const SharedParams& p, const SharedMaps& m, Misc* ms, uint32_t sbase) {
  const int lane = threadIdx.x & 31;
  // (several blocks read a key at about the same time)
  const uint64_t keep = l2_policy_evict_normal();
  uint32_t T = 0, ropes = 0, panels = 0;  // tiles done; copies of rope panels and of latent ones
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    const int32_t n = p.stall_stream ? 0 : job.tiles();
    for (int32_t j = 0; j < n && ok; ++j, ++T) {
      const int32_t key = job.k0 + j * kTileTokens;
      if (!MLA_DCHECK(key >= 0 && key < p.kv_rows, p.err)) {
        ms->abort_flag = 1;
        ok = false;
        break;
      }
      if (T > 0) ok = warp_wait_on(&ms->rope_empty, T - 1, ms, p.err);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&ms->rope_full), kRopeBytes);
        tma_load_2d(sbase + kOffRope, &m.rope, kVDim, key, smem_u32(&ms->rope_full), keep);
      }
      ++ropes;
#pragma unroll 1
      for (int c = 0; c < kPanels; ++c) {
        const uint32_t at = kPanels * (T & 1) + c;
        if (T > 1) ok = warp_wait_on(&ms->key_empty[at], (T >> 1) - 1, ms, p.err);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(smem_u32(&ms->key_full[at]), kPanelBytes);
          tma_load_2d(sbase + kOffKeys + at * kPanelBytes, &m.latent, 128 * c, key, smem_u32(&ms->key_full[at]), keep);
        }
        ++panels;
      }
      __syncwarp();
    }
  }
  if (!ms->abort_flag) return;  // the issuers wait for every copy
  // Abandoned: the copies in flight land before the block's memory is given up.
  if (lane == 0) {
    if (ropes > 0) drain(&ms->rope_full, ropes - 1);
    for (uint32_t f = panels > 2 * kPanels ? panels - 2 * kPanels : 0; f < panels; ++f)
      drain(&ms->key_full[f % (2 * kPanels)], f / (2 * kPanels));
  }
  __syncwarp();
}

// ------------------------------------------------------------ keys by a page table (eight warps)
constexpr int kCopyThreads = 32 * kCopyWarps;

// A thread's rows of a tile: it copies piece t & 7 of latent row 16 i + t / 8 and piece t & 3 of
// the rotated dims of row 32 i + t / 4.
constexpr int kLatentRows = kTileTokens * 8 / kCopyThreads, kRopeRows = kTileTokens * 4 / kCopyThreads;
static_assert(kLatentRows * kCopyThreads == kTileTokens * 8 && kCopyThreads % 8 == 0, "whole panels");
struct CopyRows {
  int32_t latent[kLatentRows], rope[kRopeRows];
  // (keys behind the part's end repeat its last one)
  __device__ __forceinline__ void load(const SharedParams& p, const Job& job, int32_t j) {
    const int t = threadIdx.x - 32 * kFirstCopyWarp;
    const int32_t* at = p.kv_indices + job.k0;
    const int32_t last = job.keys - 1, key = j * kTileTokens;
    if (!MLA_DCHECK(job.k0 >= 0 && job.keys > 0 && static_cast<int64_t>(job.k0) + job.keys <= p.kv_limit, p.err)) {
#pragma unroll
      for (int i = 0; i < kLatentRows; ++i) latent[i] = 0;
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i) rope[i] = 0;
      return;
    }
#pragma unroll
    for (int i = 0; i < kLatentRows; ++i) latent[i] = __ldg(at + min(last, key + (t >> 3) + i * (kCopyThreads / 8)));
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) rope[i] = __ldg(at + min(last, key + (t >> 2) + i * (kCopyThreads / 4)));
  }
  __device__ __forceinline__ void check(const SharedParams& p) {
    bool bad = false;
    auto one = [&](int32_t& row) {
      const bool out = row < 0 || row >= p.kv_rows;
      bad = bad || out;
      row = out ? 0 : row;
    };
#pragma unroll
    for (int i = 0; i < kLatentRows; ++i) one(latent[i]);
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) one(rope[i]);
    if (bad) atomicOr(p.err, MLA_DERR_KV_INDEX);
  }
};

__device__ __forceinline__ void run_copies(const SharedParams& p, Misc* ms, uint32_t sbase) {
  const int t = threadIdx.x - 32 * kFirstCopyWarp;
  const int piece = t & 7, row0 = t >> 3, rope_piece = t & 3, rope_row0 = t >> 2;
  const uint8_t* latent = p.kv + 16 * piece;
  const uint8_t* rope = p.kv + kVDim + 16 * rope_piece;
  auto at_row = [&](const uint8_t* first, int32_t row) {
    return first + static_cast<int64_t>(MLA_DCHECK(row >= 0 && row < p.kv_rows, p.err) ? row : 0) * kQkDim;
  };
  // (of the rows that a thread copies all have the same place in a swizzle's pattern)
  const uint32_t latent_at = sbase + kOffKeys + row0 * 128 + ((piece ^ (row0 & 7)) << 4);
  const uint32_t rope_at = sbase + kOffRope + rope_row0 * 64 + ((rope_piece ^ ((rope_row0 >> 1) & 3)) << 4);
  CopyRows rows, next;
  uint32_t T = 0;
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    const int32_t n = p.stall_stream ? 0 : job.tiles();
    if (n > 0) next.load(p, job, 0);
    for (int32_t j = 0; j < n && ok; ++j, ++T) {
      rows = next;
      rows.check(p);
      if (j + 1 < n) next.load(p, job, j + 1);
      if (T > 0) ok = warp_wait_on(&ms->rope_empty, T - 1, ms, p.err);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i)
        cp_async_16(rope_at + i * (kCopyThreads / 4) * 64, at_row(rope, rows.rope[i]));
      cp_async_arrive(smem_u32(&ms->rope_full));
#pragma unroll 1
      for (int c = 0; c < kPanels; ++c) {
        const uint32_t at = kPanels * (T & 1) + c;
        if (T > 1) ok = warp_wait_on(&ms->key_empty[at], (T >> 1) - 1, ms, p.err);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kLatentRows; ++i)
          cp_async_16(latent_at + at * kPanelBytes + i * (kCopyThreads / 8) * 128,
                      at_row(latent, rows.latent[i]) + 128 * c);
        cp_async_arrive(smem_u32(&ms->key_full[at]));
      }
    }
  }
  cp_async_wait_all();  // (nothing lands behind the block's end)
}

// ------------------------------------------------------------ MMA issuers (a warp each, an elected lane issues)
// Keys behind the part's end lie in the tile's boxes too (another row's, or never
// written): their probabilities are zero, but zero times NaN is NaN, so they are zeroed
// in shared memory before either product reads them.
__device__ __forceinline__ void clean_keys(uint8_t* panels, int32_t keys) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < kPanels; ++c)
#pragma unroll 1
    for (int32_t i = keys * 8 + lane; i < kTileTokens * 8; i += 32)
      *reinterpret_cast<uint4*>(panels + c * kPanelBytes + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// S(T) = K(T) . Q^T, panel by panel as they land.
template <bool kPaged>
__device__ __forceinline__ void run_scores(const SharedParams& p, Misc* ms, uint8_t* smem, uint32_t sbase, uint32_t tmem) {
  constexpr uint32_t kPanel = kPanelBytes >> 4;  // in descriptor address units
  const uint64_t key_k = smem_desc(sbase + kOffKeys, 1024, 1024, kLayoutSw128);
  const uint64_t rope_k = smem_desc(sbase + kOffRope, 512, 512, kLayoutSw64);
  const uint64_t q_k = smem_desc(sbase + kOffQ, 1024, 1024, kLayoutSw128);
  const uint64_t q_rope = smem_desc(sbase + kOffQRope, 512, 512, kLayoutSw64);
  auto on = [&](const uint64_t* bar, uint32_t parity) { return warp_wait_on(bar, parity, ms, p.err); };
  uint32_t T = 0, jobs = 0;
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    const int32_t n = job.tiles();
    if (n == 0) continue;
    for (int32_t j = 0; j < n && ok; ++j, ++T) {
      const uint32_t d = tmem + kColS + 128 * (T & 1), first = kPanels * (T & 1);
      const int32_t keys = job.keys - j * kTileTokens;
      const bool clean = !kPaged && keys < kTileTokens;
      // A job's first keys land before its query, and a look at a barrier costs 100 cycles.
      const bool landed = j == 0 || clean;
      if (landed) {
        for (int c = 0; c < kPanels && ok; ++c) ok = on(&ms->key_full[first + c], T >> 1);
        if (!ok) break;
        if (clean) clean_keys(smem + kOffKeys + first * kPanelBytes, keys);
      }
      ok = (T < 2 || on(&ms->s_free[T & 1], (T >> 1) - 1)) && on(&ms->rope_full, T) && (j > 0 || on(&ms->q_full, jobs));
      if (!ok) break;
      if (kPaged) fence_proxy_async_smem();  // the copies' writes, observed above, before the products' reads
      tc_fence_after();
      if (elect_one()) {
        umma_f8(d, rope_k, q_rope, kIdescQK, 0);
        umma_f8(d, rope_k + 2, q_rope + 2, kIdescQK, 1);
        umma_commit(smem_u32(&ms->rope_empty));
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < kPanels; ++c) {
        ok = ok && (landed || on(&ms->key_full[first + c], T >> 1));
        if (!ok) break;
        if (kPaged && !landed) fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = key_k + (first + c) * kPanel, b = q_k + c * kPanel;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma_f8(d, a + 2 * kk, b + 2 * kk, kIdescQK, 1);
          if (c == kPanels - 1) {
            umma_commit(smem_u32(&ms->s_full[T & 1]));
            if (j == n - 1) umma_commit(smem_u32(&ms->q_empty));
          }
        }
        __syncwarp();
      }
    }
    ++jobs;
  }
  if (elect_one()) umma_commit(smem_u32(&ms->mma_done));
  __syncwarp();
}

// O(T) += V(T)^T . P(T)^T.  (The panels have landed: S(T), which P(T) comes from, read them.)
__device__ __forceinline__ void run_values(const SharedParams& p, Misc* ms, uint32_t sbase, uint32_t tmem) {
  constexpr uint32_t kPanel = kPanelBytes >> 4;
  const uint64_t key_mn = smem_desc(sbase + kOffKeys, 1024, 1024, kLayoutSw128);
  const uint64_t p_mn = smem_desc(sbase + kOffP, 512, 512, kLayoutSw64);
  auto on = [&](const uint64_t* bar, uint32_t parity) { return warp_wait_on(bar, parity, ms, p.err); };
  uint32_t T = 0, jobs = 0;
  Job job;
  bool ok = true;
  for (uint32_t k = 0; ok && next_job(p, ms, k, job); ++k) {
    const int32_t n = job.tiles();
    if (n == 0) continue;
    ok = jobs == 0 || on(&ms->o_free, jobs - 1);
    ++jobs;
    for (int32_t j = 0; j < n && ok; ++j, ++T) {
      const uint64_t a = key_mn + kPanels * (T & 1) * kPanel;
      // 32 keys of a chunk: 4 KB of a panel, 2 KB of a term of P
      auto products = [&](int c, int kk) {
        const uint32_t d = tmem + kColO + kRows * c;
        umma_f8(d, a + c * kPanel + 256 * kk, p_mn + 128 * kk, kIdescPV, j != 0 || kk != 0);
        umma_f8(d, a + c * kPanel + 256 * kk, p_mn + (kPBytes >> 4) + 128 * kk, kIdescPV, 1);
      };
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // the first chunk, as the keys' P are written
        ok = ok && on(&ms->p_full[kk], T);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) products(0, kk);
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) {
        umma_commit(smem_u32(&ms->key_empty[kPanels * (T & 1)]));
#pragma unroll
        for (int c = 1; c < kPanels; ++c) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            products(c, kk);
            if (c == kPanels - 1) umma_commit(smem_u32(&ms->p_free[T & 1][kk]));
          }
          umma_commit(smem_u32(&ms->key_empty[kPanels * (T & 1) + c]));
        }
      }
      __syncwarp();
    }
  }
  if (elect_one()) umma_commit(smem_u32(&ms->mma_done));
  __syncwarp();
}

// ------------------------------------------------------------ softmax (a warpgroup a token)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// Sum of v[h] over the warp's lanes, for h = (lane >> 1) & 15: four exchanges that move
// half of what is left to the partner.
__device__ __forceinline__ float transposed_sum16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 8, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float send = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}
// Whether any thread of warpgroup g says so (and a barrier of its threads).
__device__ __forceinline__ bool any_of_group(bool v, int g) {
  uint32_t r;
  asm volatile("{ .reg .pred a, b; setp.ne.u32 a, %1, 0; bar.red.or.pred b, %2, 128, a; selp.u32 %0, 1, 0, b; }"
               : "=r"(r) : "r"(static_cast<uint32_t>(v)), "r"(kBarSoftmax + g) : "memory");
  return r != 0;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 32 bytes, aligned so.
__device__ __forceinline__ void store_sector(uint16_t* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}
// Two e4m3 terms without the conversion instructions, whose rate is a fraction of the
// others'.  A half precision value below 2 in magnitude has a fifth exponent bit of zero, so
// its bits 13 .. 7 are the e4m3 code of the value times 2^8, cut to its four leading bits:
// denormals included, since both formats' exponents end 2^8 apart.  The high term is that
// cut value, the low term the rest, which half precision holds exactly, rounded.
constexpr uint32_t kCut = 0xFF80FF80u, kRound = 0x00800080u, kSigns = 0x80008000u;
// The codes of two pairs, at bits 15 .. 8 of each half, packed.
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }

// 16 probabilities p 2^-8, 0 <= p <= 2^8, given as pairs: p = hi + lo.  The low term is below a
// step of the high one, 2^-3 p, so that half of its own step is 2^-8 p at most.
__device__ __forceinline__ void split_p(const uint32_t (&h)[8], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = h[2 * k], b = h[2 * k + 1];
    hi[k] = pack_codes(a << 1, b << 1);
    lo[k] = pack_codes((half2_sub(a, a & kCut) << 1) + kRound, (half2_sub(b, b & kCut) << 1) + kRound);
  }
}
// bf16 arithmetic on pairs (exact or rounded to nearest; denormals are kept).
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The bf16 bits of 2^e, twice.
__device__ __forceinline__ uint32_t bf16x2_power(int e) { return static_cast<uint32_t>(e + 127) * 0x00800080u; }
// The same for a query's bf16 values, scaled so that the largest is below 2^-111: their exponent's
// upper four bits are zero then, and bits 10 .. 4 are the e4m3 code of the value times 2^120.
constexpr int kQueryPower = -120;
constexpr uint32_t kQueryCut = 0xFFF0FFF0u;
__device__ __forceinline__ uint32_t signed_codes(uint32_t v, uint32_t round) {
  return ((v * 16 + round) & ~kSigns) | (v & kSigns);
}
// 16 query values, scaled by `up` to at most 448 2^-120, as hi + lo / 8 in units of 2^-120.
// They have eight leading bits, so the rest has four and both terms are exact (but for
// denormals, which are rounded).
__device__ __forceinline__ void split_q(const uint4& a, const uint4& b, uint32_t up, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t x[8], y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t v = bf16x2_mul(w[k], up);
    x[k] = signed_codes(v, 0);
    y[k] = signed_codes(bf16x2_mul(bf16x2_sub(v, v & kQueryCut), bf16x2_power(3)), kRound);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    hi[k] = pack_codes(x[2 * k], x[2 * k + 1]);
    lo[k] = pack_codes(y[2 * k], y[2 * k + 1]);
  }
}
// The query operand's rows of warpgroup g's token, each row scaled by a power of two so
// that its largest magnitude lies in (224, 448], and what turns its products into powers of
// two (NaN for a row that is not finite, whose output becomes NaN).  A warp has four of
// the 16 rows: a lane 16 latent dims of each and 16 of the rotated dims of one (half of the
// lanes write what the others do).  Rows are written as they arrive.  Of a token that is not
// there nothing is written, nor read: its columns of both products mean nothing.
__device__ __forceinline__ void write_q(const SharedParams& p, Misc* ms, uint32_t sbase, const Job& job, int g, float kv_scale) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  constexpr int kWarpRows = kNumHeads / 4;
  static_assert(kVDim / 16 == 32 && 2 * kWarpRows * ((kQkDim - kVDim) / 16) == 32, "a lane a piece");
  if (g >= job.nq || !MLA_DCHECK(job.q0 >= 0 && job.q0 + g < p.total_q, p.err)) {
    if (lane == 0) mbar_arrive(smem_u32(&ms->q_full));
    return;
  }
  const int row0 = kWarpRows * warp;
  const int rope_row = row0 + (lane >> 2) % kWarpRows, rope_ch = kVDim / 16 + (lane & 3);
  const uint16_t* src = p.q + (static_cast<int64_t>(job.q0 + g) * kNumHeads) * kQkDim;
  uint4 raw[kWarpRows + 1][2];  // the rotated dims last
#pragma unroll
  for (int i = 0; i <= kWarpRows; ++i) {
    const int r = (i + kWarpRows) % (kWarpRows + 1);  // they come first
    const uint4* at = reinterpret_cast<const uint4*>(src + (r < kWarpRows ? (row0 + r) * kQkDim + 16 * lane
                                                                          : rope_row * kQkDim + 16 * rope_ch));
    raw[r][0] = __ldg(at);
    raw[r][1] = __ldg(at + 1);
  }
  auto largest = [&](const uint4 (&v)[2]) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
  };
  // Scaled by 2^by, in two steps where that is no bf16 (rows of 2^15 and more).
  auto store = [&](uint4 (&v)[2], int by, uint32_t at, uint32_t low_at) {
    uint32_t hi[4], lo[4];
    if (__any_sync(0xffffffffu, by < -126)) {
      const uint32_t first = bf16x2_power(by < -126 ? -120 : 0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(bf16x2_mul(v[i].x, first), bf16x2_mul(v[i].y, first), bf16x2_mul(v[i].z, first), bf16x2_mul(v[i].w, first));
      by = by < -126 ? by + 120 : by;
    }
    split_q(v[0], v[1], bf16x2_power(by), hi, lo);
    st_shared_v4(at, hi);
    st_shared_v4(low_at, lo);
  };
  uint32_t rope_top = largest(raw[kWarpRows]);
  rope_top = max(rope_top, __shfl_xor_sync(0xffffffffu, rope_top, 1));
  rope_top = max(rope_top, __shfl_xor_sync(0xffffffffu, rope_top, 2));
  // (all rows' maxima first: the rows' conversions then overlap)
  uint32_t top[kWarpRows];
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) top[r] = __reduce_max_sync(0xffffffffu, largest(raw[r]));
  int rope_by = 0;
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) {
    top[r] = max(top[r], __shfl_sync(0xffffffffu, rope_top, 4 * r));
    // The exponent e of the largest magnitude m 2^e, 1 <= m < 2, of bf16 bits: scaled by 2^k to
    // 2^8 m where m <= 1.75, else to 2^7 m.  (Zeros and denormals: clamped.)
    const int e = static_cast<int>(top[r] >> 7) - 127;
    int k = (top[r] & 0x7Fu) <= 0x60u ? 8 - e : 7 - e;
    k = top[r] == 0 ? 0 : min(k, 126);
    if ((lane >> 2) % kWarpRows == r) rope_by = k + kQueryPower;
    const int row = kNumHeads * g + row0 + r;
    if (lane == r)
      ms->scale[g][row0 + r] = top[r] >= 0x7F80u ? __int_as_float(0x7FC00000)
                                                 : __int_as_float((127 - k) << 23) * kv_scale * kSmScaleLog2;
    const uint32_t at = sbase + kOffQ + (lane >> 3) * kPanelBytes + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
    store(raw[r], k + kQueryPower, at, at + kRows * 128);
  }
  const int row = kNumHeads * g + rope_row;
  const uint32_t at = sbase + kOffQRope + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4);
  store(raw[kWarpRows], rope_by, at, at + kRows * 64);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&ms->q_full));
}

// A warpgroup's warps meet at named barriers, so none may leave alone: a wait that ran
// out is passed over (the others then return at once, and what is computed is not
// written), and a job is taken by all four warps or by none.
__device__ __forceinline__ bool next_job_of_group(const SharedParams& p, Misc* ms, uint32_t k, Job& job, int g) {
  const bool live = next_job(p, ms, k, job);
  return k == 0 ? live : !any_of_group(!live, g);
}

__device__ __forceinline__ void run_softmax(const SharedParams& p, Misc* ms, uint32_t sbase, uint32_t tmem, int g) {
  const int t = threadIdx.x & 127, warp = t >> 5, lane = t & 31, row = lane & 15;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t bar = kBarSoftmax + g;
  const float kv_scale = __ldg(p.kv_scale);
  const uint32_t s_hi = tmem + lanes + kColS + kNumHeads * g, s_lo = s_hi + kRows;
  const uint32_t o_addr = tmem + lanes + kColO + kNumHeads * g;
  // this thread's key of a tile: its row of either term of P, 16 bytes a warpgroup
  const uint32_t p_at = sbase + kOffP + t * kRows + ((g ^ ((t >> 1) & 3)) << 4);
  uint32_t T = 0, jobs = 0;
  Job job, next;
  bool live = next_job_of_group(p, ms, 0, job, g);
  if (live && job.tiles() > 0) write_q(p, ms, sbase, job, g, kv_scale);
  const ulonglong2* scales = reinterpret_cast<const ulonglong2*>(ms->scale[g]);  // four rows each
  const ulonglong2* offs = reinterpret_cast<const ulonglong2*>(ms->off[g]);
  const ulonglong2* factors = reinterpret_cast<const ulonglong2*>(ms->factor[g]);
  for (uint32_t k = 0; live; ++k) {
    const int32_t n = job.tiles();
    const bool here = g < job.nq;
    float off = 0.0f;     // of row `lane % 16` of the warpgroup, alike in its four warps
    uint64_t sum[8];      // of pairs of rows: this thread's keys'
#pragma unroll
    for (int h = 0; h < 8; ++h) sum[h] = 0;
    for (int32_t j = 0; j < n; ++j, ++T) {
      warp_wait_on(&ms->s_full[T & 1], T >> 1, ms, p.err);
      tc_fence_after();
      if (!here) {  // nothing to read; P of a token that is not there means nothing
        if (lane == 0) mbar_arrive(smem_u32(&ms->s_free[T & 1]));
        if (T > 0) warp_wait_on(&ms->p_free[(T - 1) & 1][warp], (T - 1) >> 1, ms, p.err);
        if (lane == 0) mbar_arrive(smem_u32(&ms->p_full[warp]));
        continue;
      }
      const bool partial = (j + 1) * kTileTokens > job.keys;  // (the same for the whole block)
      const bool seen = j * kTileTokens + t < job.keys;
      const uint32_t s_at = 128 * (T & 1);
      const uint64_t eighth = pack2(0.125f, 0.125f);
      // Scores as powers of two over the reference, kTop up.
      uint64_t x[8];
      auto exponents = [&] {
        uint32_t hi[16], lo[16];
        tmem_ld16(s_hi + s_at, hi);
        tmem_ld16(s_lo + s_at, lo);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const ulonglong2 a = scales[h], o = offs[h];
          const int r = 4 * h;
          x[2 * h] = fma2(fma2(pack2(lo[r], lo[r + 1]), eighth, pack2(hi[r], hi[r + 1])), a.x, o.x);
          x[2 * h + 1] = fma2(fma2(pack2(lo[r + 2], lo[r + 3]), eighth, pack2(hi[r + 2], hi[r + 3])), a.y, o.y);
        }
      };
      bool look = j == 0;
      if (!look) {
        exponents();
        float high = -INFINITY;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          float u, v;
          unpack2(x[h], u, v);
          high = fmaxf(high, fmaxf(u, v));
        }
        look = any_of_group(seen && high > 0.0f, g);
      }
      const bool moved = look && j > 0;
      if (look) {
        float mine = 0.0f;  // the maximum of row `lane % 16`
        {
          uint32_t hi[16], lo[16];
          tmem_ld16(s_hi + s_at, hi);
          tmem_ld16(s_lo + s_at, lo);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            const float s = fmaf(__uint_as_float(lo[h]), 0.125f, __uint_as_float(hi[h])) * ms->scale[g][h];
            const float m = warp_max(seen ? s : -INFINITY);
            mine = row == h ? m : mine;
          }
        }
        ms->red[g][warp][row] = mine;
        named_bar_sync(bar, 128);
        mine = fmaxf(fmaxf(ms->red[g][0][row], ms->red[g][1][row]), fmaxf(ms->red[g][2][row], ms->red[g][3][row]));
        float factor = 1.0f;
        if (j == 0 || mine + off > 0.0f) {
          const float to = kTop - mine;
          factor = ex2(to - off);  // (of a job's first tile nothing is scaled)
          off = to;
        }
        // (the four warps write the same)
        ms->off[g][row] = off;
        ms->factor[g][row] = factor;
        __syncwarp();
        if (moved) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const ulonglong2 f = factors[h];
            sum[2 * h] = mul2(sum[2 * h], f.x);
            sum[2 * h + 1] = mul2(sum[2 * h + 1], f.y);
          }
        }
        exponents();  // (anew, so that a row that stands has the bits it has beside any other rows)
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->s_free[T & 1]));
      uint32_t hi[4], lo[4], halves[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        float u, v;
        unpack2(x[h], u, v);
        u = ex2(u);
        v = ex2(v);
        if (partial) {
          u = seen ? u : 0.0f;
          v = seen ? v : 0.0f;
        }
        sum[h] = add2(sum[h], pack2(u, v));
        halves[h] = half2_bits(u, v);
      }
      split_p(halves, hi, lo);
      if (T > 0) warp_wait_on(&ms->p_free[(T - 1) & 1][warp], (T - 1) >> 1, ms, p.err);  // this warp's keys' P(T - 1) are read
      // (and the other warpgroups' rows of the job before have left through P's memory)
      if (j == 0 && jobs > 0) warp_wait_on(&ms->o_free, jobs - 1, ms, p.err);
      st_shared_v4(p_at, hi);
      st_shared_v4(p_at + kPBytes, lo);
      fence_proxy_async_smem();
      if (moved) {
        warp_wait_on(&ms->p_free[(T - 1) & 1][3], (T - 1) >> 1, ms, p.err);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kPanels; ++c) {
          uint32_t o[16];
          tmem_ld16(o_addr + kRows * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ms->factor[g][i]);
          tmem_st16(o_addr + kRows * c, o);
        }
        tmem_wait_st();
        tc_fence_before();
        named_bar_sync(bar, 128);  // (each key's products add to all four warps' dims)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->p_full[warp]));
    }

    // ------------------------------------------------ sums over the keys
    float lse = -INFINITY;  // of row `lane % 16`, in the warpgroup's first warp
    if (here) {
      named_bar_sync(bar, 128);  // (red and factor are read)
      float v[16];
#pragma unroll
      for (int h = 0; h < 8; ++h) unpack2(sum[h], v[2 * h], v[2 * h + 1]);
      const float s16 = transposed_sum16(v);
      if ((lane & 1) == 0) ms->red[g][warp][lane >> 1] = s16;
      named_bar_sync(bar, 128);
      if (warp == 0) {
        const float s = (ms->red[g][0][row] + ms->red[g][1][row]) + (ms->red[g][2][row] + ms->red[g][3][row]);
        // (P is 2^8 times what was summed; a part is left in units of codes)
        ms->factor[g][row] = s != 0.0f ? (job.slot >= 0 ? 1.0f : kv_scale) * 0x1p-8f / s : 0.0f;
        if (n > 0) lse = kLn2 * (log2f(s) - off);
      }
      named_bar_sync(bar, 128);
    }

    // ------------------------------------------------ the next job's query, while the last products run
    const bool more = next_job_of_group(p, ms, k + 1, next, g);
    if (more && next.tiles() > 0) {
      if (jobs > 0 || n > 0) warp_wait_on(&ms->q_empty, jobs + (n > 0) - 1, ms, p.err);
      write_q(p, ms, sbase, next, g, kv_scale);
    }
    if (n > 0) {
      warp_wait_on(&ms->p_free[(T - 1) & 1][3], (T - 1) >> 1, ms, p.err);
      tc_fence_after();
    }

    // ------------------------------------------------ output
    // A thread has one dim of a chunk.  Parts keep that order, [chunk][token][dim][head]: 16
    // heads are a sector.  Rows of the output go through shared memory (P's, which is
    // free: a quarter for a warpgroup) to leave in 16-byte pieces.
    const bool parts = job.slot >= 0;
    const bool fits = !ms->abort_flag && MLA_DCHECK(!here || (parts ? job.slot < 2 * p.workers && p.split
                                                                    : job.q0 >= 0 && job.q0 + g < p.total_q), p.err);
    uint8_t* stage = reinterpret_cast<uint8_t*>(ms) - kOffMisc + kOffP + g * (2 * kPBytes / kTokens);
#pragma unroll 1
    for (int c = 0; c < (here ? kPanels : 0); ++c) {  // the token's 16 rows of a chunk
      uint16_t* dst = p.out + (static_cast<int64_t>(job.q0 + g) * kNumHeads) * kVDim + 128 * c;
      if (n == 0) {  // no keys: zeros (P's memory may be at work; of a part the log-sum-exp says so)
        if (fits && !parts)
          for (int i = t >> 4; i < 16; i += 8)
            *reinterpret_cast<uint4*>(dst + i * kVDim + 8 * (t & 15)) = make_uint4(0, 0, 0, 0);
        continue;
      }
      uint32_t o[16];
      tmem_ld16(o_addr + kRows * c, o);
      tmem_wait_ld();
      const float4* by = reinterpret_cast<const float4*>(ms->factor[g]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 f = by[q];
        o[4 * q] = __float_as_uint(__uint_as_float(o[4 * q]) * f.x);
        o[4 * q + 1] = __float_as_uint(__uint_as_float(o[4 * q + 1]) * f.y);
        o[4 * q + 2] = __float_as_uint(__uint_as_float(o[4 * q + 2]) * f.z);
        o[4 * q + 3] = __float_as_uint(__uint_as_float(o[4 * q + 3]) * f.w);
      }
      if (parts) {
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) w[h] = half2_bits(__uint_as_float(o[2 * h]), __uint_as_float(o[2 * h + 1]));
        if (fits)
          store_sector(p.part + ((static_cast<int64_t>(job.slot) * kPanels + c) * kTokens + g) * (128 * kNumHeads) + t * kNumHeads, w);
        continue;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(__uint_as_float(o[i])));
        reinterpret_cast<uint16_t*>(stage)[i * 128 + t] = b;
      }
      named_bar_sync(bar, 128);
      if (fits) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = 8 * q + (t >> 4), piece = t & 15;  // 256 bytes a row
          *reinterpret_cast<uint4*>(dst + i * kVDim + 8 * piece) = reinterpret_cast<const uint4*>(stage)[i * 16 + piece];
        }
      }
      named_bar_sync(bar, 128);
    }
    if (t < 16 && here && fits) {
      if (parts)
        p.part_lse[static_cast<int64_t>(job.slot) * kRows + g * kNumHeads + t] = lse;
      else if (p.lse != nullptr)
        p.lse[(static_cast<int64_t>(job.q0) + g) * kNumHeads + t] = lse;
    }
    __syncwarp();
    if (n > 0) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->o_free));
      ++jobs;
    }
    named_bar_sync(bar, 128);  // (factor is read)
    job = next;
    live = more;
  }
}

template <bool kPaged>
__global__ void __launch_bounds__(threads<kPaged>(), 1)
    shared_kernel(const __grid_constant__ SharedMaps maps, const SharedParams p) {
  // (aligned as the panels' swizzle needs it: there is no room to align it here)
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc* ms = reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == kScoreWarp) tmem_alloc(smem_u32(&ms->tmem_base), kTmemCols);
  if (tid == kProducerWarp * 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms->job_full[i]), 1);
      mbar_init(smem_u32(&ms->job_empty[i]), job_readers<kPaged>());
      mbar_init(smem_u32(&ms->s_full[i]), 1);
      mbar_init(smem_u32(&ms->s_free[i]), kSoftmaxWarps);
    }
    for (int i = 0; i < 2 * kPanels; ++i) {
      mbar_init(smem_u32(&ms->key_full[i]), kPaged ? kCopyThreads : 1);
      mbar_init(smem_u32(&ms->key_empty[i]), 1);
    }
    mbar_init(smem_u32(&ms->rope_full), kPaged ? kCopyThreads : 1);
    mbar_init(smem_u32(&ms->rope_empty), 1);
    mbar_init(smem_u32(&ms->q_full), kSoftmaxWarps);
    mbar_init(smem_u32(&ms->q_empty), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&ms->p_full[i]), kTokens);
      mbar_init(smem_u32(&ms->p_free[0][i]), 1);
      mbar_init(smem_u32(&ms->p_free[1][i]), 1);
    }
    mbar_init(smem_u32(&ms->o_free), kSoftmaxWarps);
    mbar_init(smem_u32(&ms->mma_done), 2);
    ms->abort_flag = 0;
    fence_mbar_init();
    if (!kPaged) {
      prefetch_tensormap(&maps.latent);
      prefetch_tensormap(&maps.rope);
    }
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  Batch groups = {};
  if (warp == kSchedulerWarp) {
    groups = count_groups(p);
    find_job(p, groups, blockIdx.x < groups.shares.workers ? groups.shares.begin(blockIdx.x) : 0, &ms->job[0]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem_base;
  if (warp >= kFirstSoftmaxWarp && warp < kFirstCopyWarp) {
    setmaxnreg_inc<softmax_regs<kPaged>()>();
    run_softmax(p, ms, sbase, tmem, (warp - kFirstSoftmaxWarp) >> 2);
  } else {
    setmaxnreg_dec<other_regs<kPaged>()>();
    if (warp == kScoreWarp)
      run_scores<kPaged>(p, ms, smem, sbase, tmem);
    else if (warp == kValueWarp)
      run_values(p, ms, sbase, tmem);
    else if (warp == kSchedulerWarp)
      run_scheduler(p, groups, ms);
    else if (kPaged && warp >= kFirstCopyWarp)
      run_copies(p, ms, sbase);
    else if (!kPaged && warp == kProducerWarp)
      run_producer(p, maps, ms, sbase);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreWarp) {
    const bool one = (threadIdx.x & 31) == 0;
    if (one) drain(&ms->mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
    // (Abandoned: the parts are not whole.  Block 0 has written the word long before a wait runs out.)
    if (one && ms->abort_flag) *p.missing = 1;
  }
}

// ------------------------------------------------------------ joining
// A block a token, chunk of 128 dims and half of the heads: out = sum_w 2^(..) part_w over the
// workers that share the token's block of queries.  A thread has eight heads of a dim, eight
// parts in flight, the first ones' values beside the log-sum-exps; the weights are formed once
// a block (by every thread they took longer than the bytes), and the rows are turned through
// shared memory.  Rows whose keys one worker had are written already.
constexpr int kJoinThreads = 128, kJoinAhead = 8, kJoinHeads = 8;
constexpr int kJoinStep = kJoinThreads / kJoinHeads;  // parts whose weights are formed together
constexpr int kJoinPerSm = 8;                         // blocks, at most
constexpr int kJoinOwnBytes = 3 << 10;                  // of shared memory (its arrays)
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm) shared_join_kernel(const SharedParams p) {
  __shared__ __align__(16) uint16_t rows[kJoinHeads][kJoinThreads];
  __shared__ __align__(16) float weight[kJoinStep][kJoinHeads];
  __shared__ float red[2][kJoinThreads / 32][kJoinHeads];
  __shared__ int64_t sums[2][kJoinThreads / 32];
  __shared__ int32_t mine;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t token = static_cast<int32_t>(blockIdx.x) / (2 * kPanels), c = static_cast<int32_t>(blockIdx.x) % (2 * kPanels) >> 1;
  const int32_t head0 = kJoinHeads * (static_cast<int32_t>(blockIdx.x) & 1);
  if (tid == 0) mine = -1;
  __syncthreads();
  bool back = false;
  int64_t all = 0, before = 0;
  for (int32_t g = tid; g < p.batch; g += kJoinThreads) {
    const Group x = load_group(p, g, false, back);
    const int64_t n = blocks_of(x) * units_of(p, x);
    all = min(all + n, kManyUnits / 32);
    if (x.qs + x.n <= token) before = min(before + n, kManyUnits / 32);
    if (token >= x.qs && token < x.qs + x.n) mine = g;  // (of groups that overlap any: nothing is joined then)
  }
  all = warp_sum(all);
  before = warp_sum(before);
  if (lane == 0) {
    sums[0][warp] = all;
    sums[1][warp] = before;
  }
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    all += sums[0][w];
    before += sums[1][w];
  }
  const int32_t own = mine;
  int32_t w0 = 0, w1 = 0, place = 0;
  if (own >= 0) {
    const Group x = load_group(p, own, false, back);
    const int32_t n = tiles_of_length(x.len), block = (token - x.qs) / kTokens;
    const Shares shares = {all, min(static_cast<int64_t>(p.workers), all)};
    const int64_t tile0 = before + block * units_of(p, x) + p.start;
    w0 = static_cast<int32_t>(shares.owner(tile0));
    w1 = n > 0 ? static_cast<int32_t>(shares.owner(tile0 + n - 1)) : w0;
    place = token - x.qs - block * kTokens;
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  if (w0 == w1) return;
  const uint32_t missing = __ldcg(p.missing);  // (looked at behind the parts, which are read all the same)
  if (!MLA_DCHECK(token < p.total_q && w0 >= 0 && w1 < p.workers && place >= 0 && place < kTokens, p.err)) return;
  // The first worker's part is its last job's, the others' their first.
  auto slot = [&](int32_t w) { return shared_slot(w, w == w0); };
  const uint16_t* part = p.part + (static_cast<int64_t>(c) * kTokens + place) * (128 * kNumHeads) + tid * kNumHeads + head0;
  constexpr int64_t kSlot = static_cast<int64_t>(kRows) * kVDim;
  uint4 v[kJoinAhead];
  auto load = [&](int32_t at) {
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i)
      if (at + i <= w1) v[i] = __ldcs(reinterpret_cast<const uint4*>(part + slot(at + i) * kSlot));
  };
  load(w0);
  // Thread (i, h): head h of the parts i, i + 16, ...
  const int h = tid % kJoinHeads, first = w0 + tid / kJoinHeads;
  const float* lses = p.part_lse + place * kNumHeads + head0 + h;
  const float lse0 = first <= w1 ? __ldcg(lses + slot(first) * kRows) : -INFINITY;
  float top = lse0;
  for (int32_t w = first + kJoinStep; w <= w1; w += kJoinStep) top = fmaxf(top, __ldcg(lses + slot(w) * kRows));
  auto over_parts = [&](float x, int which, auto join) {  // over the threads of a head
    x = join(x, __shfl_xor_sync(0xffffffffu, x, 8));
    x = join(x, __shfl_xor_sync(0xffffffffu, x, 16));
    if (lane < kJoinHeads) red[which][warp][lane] = x;
    __syncthreads();
    return join(join(red[which][0][h], red[which][1][h]), join(red[which][2][h], red[which][3][h]));
  };
  top = over_parts(top, 0, [](float a, float b) { return fmaxf(a, b); });
  float sum = 0.0f, acc[kJoinHeads] = {};
  for (int32_t at = w0; at <= w1; at += kJoinStep) {
    const int32_t w = at + tid / kJoinHeads;
    float f = 0.0f;
    // (every part has keys; a NaN reaches the result)
    if (w <= w1) f = expf((at == w0 ? lse0 : __ldcg(lses + slot(w) * kRows)) - top);
    sum += f;
    if (at > w0) __syncthreads();  // (the weights before are read)
    weight[tid / kJoinHeads][h] = f;
    __syncthreads();
#pragma unroll
    for (int half = 0; half < kJoinStep; half += kJoinAhead) {
      if (at + half > w1) break;
      if (at + half > w0) load(at + half);
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) {
        if (at + half + i > w1) break;
        const uint32_t halves[kJoinHeads / 2] = {v[i].x, v[i].y, v[i].z, v[i].w};
        const float4 f0 = *reinterpret_cast<const float4*>(&weight[half + i][0]), f1 = *reinterpret_cast<const float4*>(&weight[half + i][4]);
        const float fs[kJoinHeads] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int e = 0; e < kJoinHeads / 2; ++e) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&halves[e]));
          acc[2 * e] = fmaf(fs[2 * e], x.x, acc[2 * e]);
          acc[2 * e + 1] = fmaf(fs[2 * e + 1], x.y, acc[2 * e + 1]);
        }
      }
    }
  }
  sum = over_parts(sum, 1, [](float a, float b) { return a + b; });
  if (missing != 0) return;  // (the same for the whole block)
  if (tid < kJoinHeads) {
    weight[0][tid] = __ldg(p.kv_scale) / sum;
    if (c == 0 && p.lse != nullptr) p.lse[static_cast<int64_t>(token) * kNumHeads + head0 + tid] = top + logf(sum);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kJoinHeads; ++e) {
    uint16_t b;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(acc[e] * weight[0][e]));
    rows[e][tid] = b;
  }
  __syncthreads();
  uint16_t* out = p.out + (static_cast<int64_t>(token) * kNumHeads + head0) * kVDim + 128 * c;
  *reinterpret_cast<uint4*>(out + (tid >> 4) * kVDim + 8 * (tid & 15)) = *reinterpret_cast<const uint4*>(&rows[tid >> 4][8 * (tid & 15)]);
}

}  // namespace

// Shared memory that a block of the second kernel asks for beside its own, so that no more than
// `blocks` of them share an SM (of its 228 KB each also costs 1 KB).
static int32_t join_room(int32_t blocks) { return 228 * 1024 / blocks - 1024 - kJoinOwnBytes; }

size_t shared_smem_bytes() { return kSmemBytes; }

cudaError_t shared_prepare() {
  cudaError_t e = cudaFuncSetAttribute(shared_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(shared_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, join_room(1));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(shared_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

cudaError_t launch_shared(const SharedParams& p, const SharedMaps& maps, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.workers);
  return p.kv_indices != nullptr
             ? launch_dependent(shared_kernel<true>, grid, threads<true>(), kSmemBytes, stream, maps, p)
             : launch_dependent(shared_kernel<false>, grid, threads<false>(), kSmemBytes, stream, maps, p);
}

cudaError_t launch_shared_join(const SharedParams& p, int32_t num_sms, cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(p.total_q) * 2 * kPanels;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  // Few blocks are spread over the SMs: left alone, the first SMs that are done take eight each, and
  // what an SM can load bounds the call (13 queries over 9000 keys 36 us, spread 24; 64 over 8192
  // 34.4, spread 31.7).
  const int64_t each = blocks / num_sms + 1;
  const size_t room = each < kJoinPerSm ? join_room(static_cast<int32_t>(each)) : 0;
  return launch_dependent(shared_join_kernel, static_cast<unsigned>(blocks), kJoinThreads, room, stream, p);
}

}  // namespace mla
