// Host build of the windowed walks (csrc/window_iter.cuh) for
// test_window_iter_cpu.py, as iter_harness.cpp builds the ring's.
#include <algorithm>
namespace ra {
using std::max;
using std::min;
}  // namespace ra
#define __ldg(p) (*(p))
#include "window_iter.cuh"

namespace {

int geometry(int S, int tile, int window, int n_sink, ra::WinGeometry* g) {
  *g = ra::WinGeometry();
  if (ra::make_geometry(1, 1, 1, S, 128, 1, 1, 0.f, RA_ORDER_CONTIGUOUS, -1, tile, g) != RA_OK)
    return -1;
  g->window = window;
  g->n_sink = n_sink;
  g->sink_splits = 1;
  return 0;
}

}  // namespace

extern "C" {

// Key tiles met by the `rows` query rows from tile ti: (first position, valid,
// work) each; -2 when the length told differs.
int ra_win_walk(int S, int tile, int window, int n_sink, int ti, int rows, int* out, int cap) {
  ra::WinGeometry g;
  if (geometry(S, tile, window, n_sink, &g) != 0) return -1;
  const int q_lo = ti * g.tile, q_valid = std::min(rows, S - q_lo);
  ra::WinKvIter it;
  it.init(g, 0, q_lo, q_valid);
  const int length = it.length(g);
  ra::KvTile kv;
  int n = 0;
  while (it.next(g, kv)) {
    if (n < cap) {
      int* e = out + 3 * n;
      e[0] = kv.lo; e[1] = kv.valid; e[2] = kv.work;
    }
    ++n;
  }
  return length == n ? n : -2;
}

// Query tiles met by key tile ti among those whose first position is in
// [share_lo, share_hi): (head, first position, valid, mask) each.
int ra_win_qwalk(int S, int window, int n_sink, int ti, int heads, int share_lo, int share_hi,
                 int* out, int cap) {
  ra::WinGeometry g;
  if (geometry(S, 128, window, n_sink, &g) != 0) return -1;
  ra::WinQIterT<128> it;
  it.init(g, 0, ti * 128, ra::tile_tokens(g, 0, ti), 0, heads, share_lo, share_hi);
  ra::QTile q;
  int n = 0;
  while (it.next(g, q)) {
    if (n < cap) {
      int* e = out + 4 * n;
      e[0] = q.h; e[1] = q.lo; e[2] = q.valid; e[3] = q.mask ? 1 : 0;
    }
    ++n;
  }
  return n;
}

// First positions of the tiles that hold a first token, by ordinal.
int ra_win_sink_tiles(int S, int n_sink, int most, int* lo) {
  ra::WinGeometry g;
  if (geometry(S, 128, 1, n_sink, &g) != 0) return -1;
  int n = 0, seg, ti;
  for (int o = 0; o < most; ++o)
    if (ra::sink_tile(g, o, seg, ti)) lo[n++] = seg * g.seg_len + ti * g.tile;
  return n;
}

}  // extern "C"
