// Exposes how the kernels' schedule.h cuts the blocks of shared keys to the CPU tests.
#include <cstdint>

#include "schedule.h"

extern "C" int64_t share_begin(int64_t all, int64_t workers, int64_t c) { return mla::Shares{all, workers}.begin(c); }
extern "C" int64_t share_owner(int64_t all, int64_t workers, int64_t u) { return mla::Shares{all, workers}.owner(u); }
extern "C" int64_t piece_slot(int64_t c, bool begins) { return mla::shared_slot(c, begins); }
extern "C" void piece_of(int64_t begin, int32_t tiles, int32_t start, int64_t u, int64_t stop, int32_t out[3]) {
  const mla::SharedPiece p = mla::shared_piece(begin, tiles, start, u, stop);
  out[0] = p.j0, out[1] = p.j1, out[2] = p.whole;
}
