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

int geometry(int S, int P, int order, int tile, int window, int n_sink, ra::WinGeometry* g) {
  *g = ra::WinGeometry();
  if (ra::make_geometry(1, 1, 1, S, 128, P, 1, 0.f, order, -1, tile, g) != RA_OK) return -1;
  g->window = window;
  g->n_sink = n_sink;
  g->sink_splits = 1;
  return 0;
}

}  // namespace

extern "C" {

int ra_win_facts(int S, int P, int order, int tile, int* facts) {
  ra::WinGeometry g;
  if (geometry(S, P, order, tile, 1, 0, &g) != 0) return -1;
  facts[0] = g.seg_len;
  facts[1] = g.n_seg;
  facts[2] = g.nt;
  return 0;
}

// Key tiles met by the `rows` query rows from tile (seg, ti): (step, source,
// first position, valid, work) each; -2 when the counted length differs.
int ra_win_walk(int S, int P, int order, int tile, int window, int n_sink, int seg, int ti,
                int rows, int* out, int cap) {
  ra::WinGeometry g;
  if (geometry(S, P, order, tile, window, n_sink, &g) != 0) return -1;
  const int r = ra::seg_owner(g, seg);
  const int q_lo = seg * g.seg_len + ti * g.tile;
  const int q_valid = std::min(rows, ra::seg_tokens(g, seg) - ti * g.tile);
  if (q_valid <= 0) return 0;
  ra::WinKvIter it;
  it.init(g, r, q_lo, q_valid);
  ra::KvTile kv;
  int n = 0;
  while (it.next(g, kv)) {
    if (n < cap) {
      int* e = out + 5 * n;
      e[0] = kv.step; e[1] = kv.src; e[2] = kv.lo; e[3] = kv.valid; e[4] = kv.work;
    }
    ++n;
  }
  return ra::win_walk_length(g, r, q_lo, q_valid) == n ? n : -2;
}

// Query tiles met by key tile (seg, ti) among those whose first position is
// in [share_lo, share_hi): (head, first position, valid, mask) each.
int ra_win_qwalk(int S, int P, int order, int window, int n_sink, int seg, int ti, int heads,
                 int share_lo, int share_hi, int* out, int cap) {
  ra::WinGeometry g;
  if (geometry(S, P, order, 128, window, n_sink, &g) != 0) return -1;
  const int kv_lo = seg * g.seg_len + ti * g.tile;
  const int valid = ra::tile_tokens(g, seg, ti);
  ra::WinQIterT<128> it;
  it.init(g, ra::seg_owner(g, seg), kv_lo, valid, 0, heads, share_lo, share_hi);
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
int ra_win_sink_tiles(int S, int P, int order, int n_sink, int most, int* lo) {
  ra::WinGeometry g;
  if (geometry(S, P, order, 128, 1, n_sink, &g) != 0) return -1;
  int n = 0, seg, ti;
  for (int o = 0; o < most; ++o)
    if (ra::sink_tile(g, o, seg, ti)) lo[n++] = seg * g.seg_len + ti * g.tile;
  return n;
}

}  // extern "C"
