// Exposes to the CPU tests which worker has a block of shared keys that is not cut (schedule.h).
#include <cstdint>

#include "schedule.h"

extern "C" int64_t share_begin(int64_t all, int64_t workers, int64_t c) { return mla::Shares{all, workers}.begin(c); }
extern "C" void uncut_piece_of(int64_t begin, int32_t tiles, int64_t u, int32_t out[3]) {
  const mla::SharedPiece p = mla::uncut_piece(begin, tiles, u);
  out[0] = p.j0, out[1] = p.j1, out[2] = p.whole;
}
