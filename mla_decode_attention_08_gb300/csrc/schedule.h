// Integer formulas of the token-balanced split-KV schedule, shared by the host
// planner and the kernels so both compute the same ranges.
//
// Rows are cut into tiles of kTileTokens tokens; all rows' tiles, row after
// row (each row with tiles preceded by row_start_units units for its start),
// form one sequence of T units; worker c of a grid of G takes the units
// [floor(c*T/G), floor((c+1)*T/G)).  This is the persistent form of the
// flash-decoding split (kernelbot-amd-mixed-mla submission 722089,
// `_mla_multihead_stage1` splits each row into contiguous ranges; submissions
// 663509 and 738050 hand a persistent kernel precomputed work maps).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MLA_HD __host__ __device__ __forceinline__
#else
#define MLA_HD inline
#endif

namespace mla {

constexpr int kNumHeads = 16;
constexpr int kQkDim = 576;
constexpr int kVDim = 512;
constexpr int kTileTokens = 128;

MLA_HD int32_t tiles_of_length(int64_t len) {
  return len > 0 ? static_cast<int32_t>((len + kTileTokens - 1) / kTileTokens) : 0;
}

// Workers for a batch: the fewest that still give no worker more than
// k = ceil(U / min(num_sms, U)) tiles, U = B * ceil(max_kv_len / 128), i.e.
// ceil(U / k).  Fewer workers than SMs when that does not lengthen the longest
// range: the ranges then hold k tiles each and, for rows of a multiple of k
// tiles, start at row starts (bs 32 x 1024: 128 workers of two tiles instead
// of 152 of one or two, some of which straddle two rows).
MLA_HD int32_t plan_grid(int32_t batch, int32_t max_kv_len, int32_t num_sms) {
  const int64_t upper = static_cast<int64_t>(batch) * tiles_of_length(max_kv_len);
  const int64_t g0 = upper < num_sms ? upper : num_sms;
  if (g0 < 1) return 1;
  const int64_t k = (upper + g0 - 1) / g0;
  return static_cast<int32_t>((upper + k - 1) / k);
}

// Clusters of s CTAs (one 227 KB CTA per SM) that a GPU of num_sms SMs runs at
// once, estimated from the GB300 GPC layout (measured: 15 clusters of 8, 36 of
// 4 and 76 of 2 on 152 SMs): num_sms / 10, 7 num_sms / 32 and num_sms / 2.
MLA_HD int32_t cluster_capacity(int32_t s, int32_t num_sms) {
  return s == 8 ? num_sms / 10 : (s == 4 ? num_sms * 7 / 32 : num_sms / 2);
}

// Cluster split for small batches of one query token per row: every row gets
// a cluster of s CTAs that share its tiles (rank r takes the row's tiles
// [r k, min((r + 1) k, nt)), k = ceil(nt / s)) and combine their partial
// results after one cluster barrier, with no second kernel.  s is the
// largest of 8, 4, 2 with s <= ceil(max_kv_len / 128) whose clusters for the
// whole batch fit the GPU at once; it is used (else 0: the persistent split)
// when its longest share, ceil(nt / s) tiles, is at most two tiles longer than
// the persistent schedule's longest range.
MLA_HD int32_t plan_cluster(int32_t batch, int32_t qo_len, int32_t max_kv_len, int32_t num_sms) {
  const int32_t nt = tiles_of_length(max_kv_len);
  if (qo_len != 1 || batch < 1 || num_sms < 1 || nt < 2) return 0;
  int32_t s = 8;
  while (s >= 2 && (s > nt || batch > cluster_capacity(s, num_sms))) s >>= 1;
  if (s < 2) return 0;
  const int64_t upper = static_cast<int64_t>(batch) * nt;
  const int64_t g0 = upper < num_sms ? upper : num_sms;
  const int64_t longest = (upper + g0 - 1) / g0;
  return (nt + s - 1) / s <= longest + 2 ? s : 0;
}

// Row starts.  A worker whose range takes on a new row pays for that row's
// start (its query's preparation and the previous segment's epilogue, about
// three tiles' streaming time) on top of its tiles, and such workers finished
// last.  So when the ranges are long, every row with tiles is preceded in the
// global sequence by kRowStartUnits units that stand for its start: a range
// that takes on a row start gets that many fewer tiles.  With short ranges
// (fewer than kRowStartMinRange tiles each) the units would cost more than
// they balance (ranges of 2 tiles become 2 or 3), and rows start with their
// tiles.  The rule depends only on the batch's tile count T and the grid:
// units per row start = kRowStartUnits when ceil(T / grid) >= kRowStartMinRange,
// else 0 (e4m3 and MXFP4 caches; a bf16 cache's rows start with their tiles).
constexpr int32_t kRowStartUnits = 3;
constexpr int32_t kRowStartMinRange = 8;
MLA_HD int32_t row_start_units(int32_t total_tiles, int32_t grid) {
  if (grid < 1 || total_tiles < 1) return 0;
  const int64_t k = (static_cast<int64_t>(total_tiles) + grid - 1) / grid;
  return k >= kRowStartMinRange ? kRowStartUnits : 0;
}

// floor(c * total / grid) for 0 <= c <= grid and total >= 0, without a 64-bit
// division (a slow call on the GPU): with total = q * grid + r it is
// c * q + floor(c * r / grid), and c * r < grid^2 fits 32 bits whenever
// grid < 65536.
MLA_HD int32_t worker_begin(int32_t c, int32_t total, int32_t grid) {
  const uint32_t g = static_cast<uint32_t>(grid);
  const uint32_t q = static_cast<uint32_t>(total) / g, r = static_cast<uint32_t>(total) % g;
  const uint64_t cr = static_cast<uint64_t>(c) * r;
  const uint32_t extra = cr <= 0xFFFFFFFFull ? static_cast<uint32_t>(cr) / g
                                             : static_cast<uint32_t>(cr / g);
  return static_cast<int32_t>(static_cast<uint32_t>(c) * q + extra);
}

// Worker holding global tile t (0 <= t < total): the largest c with
// worker_begin(c) <= t, i.e. floor(((t + 1) * grid - 1) / total).  A float
// estimate is stepped to the exact answer with worker_begin.
MLA_HD int32_t worker_of_tile(int32_t t, int32_t total, int32_t grid) {
  int32_t c = static_cast<int32_t>(static_cast<float>(t) * static_cast<float>(grid) /
                                   static_cast<float>(total));
  c = c < 0 ? 0 : (c > grid - 1 ? grid - 1 : c);
  while (c > 0 && worker_begin(c, total, grid) > t) --c;
  while (c + 1 < grid && worker_begin(c + 1, total, grid) <= t) ++c;
  return c;
}

// Workspace slot of worker c's partial for a split row whose tiles start at
// prefix_b: slot 2c when c's range begins inside that row, else 2c + 1.
MLA_HD int32_t partial_slot(int32_t c, int32_t worker_t0, int32_t prefix_b) {
  return worker_t0 >= prefix_b ? 2 * c : 2 * c + 1;
}

// Equal shares of `all` units of work for `workers` workers (at most `all` of them, so that
// none is empty): worker c has the units [begin(c), begin(c + 1)), and unit u is owner(u)'s.
// (all below 2^50 and workers below 2^13, so the products fit 64 bits.)
// (Division in 32 bits where both fit: in 64 bits it takes the GPU some hundred cycles.)
MLA_HD int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}
struct Shares {
  int64_t all, workers;
  MLA_HD int64_t begin(int64_t c) const { return quotient(c * all, workers); }
  MLA_HD int64_t owner(int64_t u) const { return quotient((u + 1) * workers - 1, all); }
};

// What a worker whose units end at `stop` has of a block of `tiles` key tiles (one unit each,
// behind `start` units for the block's start, which begin at unit `begin`), from unit u of it on:
// the key tiles [j0, j1).  A block without key tiles has one unit behind its start
// and is whole where that unit is.
struct SharedPiece {
  int32_t j0, j1;
  bool whole;
};
MLA_HD SharedPiece shared_piece(int64_t begin, int32_t tiles, int32_t start, int64_t u, int64_t stop) {
  const int64_t tile0 = begin + start;
  int64_t j0 = u - tile0, j1 = stop - tile0;
  j0 = j0 < 0 ? 0 : j0;
  j1 = j1 < 0 ? 0 : j1 > tiles ? tiles : j1;
  SharedPiece p;
  p.j0 = static_cast<int32_t>(j0 < tiles ? j0 : tiles);
  p.j1 = static_cast<int32_t>(j1);
  p.whole = p.j0 == 0 && p.j1 == tiles && stop > tile0;
  return p;
}
// The same of blocks that are not cut: a block is whole and the worker's that has its first unit, and
// nothing at its other units, where a worker's share may begin.
MLA_HD SharedPiece uncut_piece(int64_t begin, int32_t tiles, int64_t u) {
  return u == begin ? SharedPiece{0, tiles, true} : SharedPiece{0, 0, false};
}
// Where the worker leaves that piece, if it is not whole: its first piece may continue a block
// (slot 2 c), its last may begin one (slot 2 c + 1).
MLA_HD int64_t shared_slot(int64_t c, bool begins) { return 2 * c + (begins ? 1 : 0); }

// Pages of a row of `len` tokens, 0 .. 2^31 - 1 (anything for other lengths): divided in 32 bits, since in 64
// bits it takes the GPU some hundred cycles.
MLA_HD uint32_t pages_of(int64_t len, int32_t page_size) {
  return (static_cast<uint32_t>(len) + static_cast<uint32_t>(page_size) - 1u) / static_cast<uint32_t>(page_size);
}

}  // namespace mla
