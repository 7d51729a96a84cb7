// The tile schedule at extents near 2^31, for tests/test_extents.py.
#include <stdint.h>

#include "schedule.h"

using namespace rd;

extern "C" long long group_tiles(int op, int32_t lo, int32_t hi, int tm, int n_tiles) {
  return tiles_of_group(op, lo, hi, tm, n_tiles, 1);
}

// tile t of one group of rows [lo, hi): m_idx, row_load, nkb, and the last K block's row
template <int OP, int TM>
static void decode(int32_t lo, int32_t hi, int32_t kc, int t, int32_t* out) {
  const int32_t bound[2] = {lo, hi};
  const int32_t tile_start[2] = {0, OP == kOpDw ? 0 : 0x7FFFFFFF};
  SchedView v = {};
  v.bound = bound;
  v.tile_start = tile_start;
  v.g_local = 1;
  v.n_tiles = 1;
  v.band_tiles = 48;
  v.dw_m_tiles = 1;
  v.kc = kc;
  const Tile tl = decode_tile_view<OP, TM>(v, t);
  out[0] = tl.m_idx;
  out[1] = tl.row_load;
  out[2] = tl.nkb;
  out[3] = OP == kOpDw ? dw_block_row(tl, tl.nkb - 1) : 0;
}

extern "C" void decode_tile_of(int dw, int tm, int32_t lo, int32_t hi, int32_t kc, int t, int32_t* out) {
  if (dw) decode<kOpDw, 128>(lo, hi, kc, t, out);
  else if (tm == 256) decode<kOpFwd, 256>(lo, hi, kc, t, out);
  else decode<kOpFwd, 128>(lo, hi, kc, t, out);
}
