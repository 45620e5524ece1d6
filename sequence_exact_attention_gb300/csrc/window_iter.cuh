// Walks of attention with a sliding window and a few first tokens that stay
// visible: query i sees key j <= i when j > i - window or j < n_sink.
//
// A window meets the blocks before its own, few of the ring's, so these walks
// do not follow the ring: positions are counted through (one rank, one
// segment), and ranks, chunks and their order change nothing. (Walked chunk by
// chunk, 32 tokens of 8 ranks were 36 tile pairs instead of 1.)
//
// WinKvIter: the key tiles that some row of the query rows sees, in position
// order; the tiles between the first tokens and the rows' windows are jumped
// over, so a walk costs what it visits. WinQIterT the other way round: the
// query tiles that see a key tile, limited to a share of them (by their first
// position) where the work on one key tile is split.
#pragma once

#include "q_iter.cuh"
#include "ring_iter.cuh"

namespace ra {

struct WinKvIter {
  int ti, end;      // next tile, past the last
  int n_first, w0;  // tiles of first tokens that the windows left behind; the windows' first
  int q_lo, q_hi;

  __device__ __forceinline__ void init(const WinGeometry& g, int, int q_first, int q_valid) {
    q_lo = q_first;
    q_hi = q_first + q_valid - 1;
    end = q_valid > 0 ? q_hi / g.tile + 1 : 0;
    w0 = min(max(q_lo - g.window + 1, 0) / g.tile, end);
    n_first = min((g.n_sink + g.tile - 1) / g.tile, w0);
    ti = n_first > 0 ? 0 : w0;
  }
  // Key tiles in all.
  __device__ __forceinline__ int length() const { return n_first + end - w0; }

  __device__ __forceinline__ bool next(const WinGeometry& g, KvTile& kv) {
    if (ti >= end) return false;
    kv.step = kv.src = kv.seg = 0;
    kv.id = ti;
    kv.lo = ti * g.tile;
    kv.valid = min(g.tile, g.S - kv.lo);
    const int hi = kv.lo + kv.valid;
    const bool all_allowed = hi - 1 <= q_lo && (kv.lo > q_hi - g.window || hi <= g.n_sink);
    kv.work = (all_allowed && kv.valid == g.tile) ? kNoMask : kMask;
    if (++ti == n_first) ti = w0;
    return true;
  }
};

template <int kT>
struct WinQIterT {
  int h, h_end;           // query heads of the group
  int ti, first, end;     // next tile of head h; its first and past its last
  int kv_lo, kv_hi;

  // The tiles whose first position is in [share_lo, share_hi).
  __device__ __forceinline__ void init(const WinGeometry& g, int, int kv_lo_, int kv_valid,
                                       int h_begin, int h_end_, int share_lo, int share_hi) {
    h = h_begin;
    h_end = kv_valid > 0 ? h_end_ : h_begin;
    kv_lo = kv_lo_;
    kv_hi = kv_lo_ + kv_valid - 1;
    // the last query position that sees a key of the tile
    const int p_max = kv_lo < g.n_sink ? g.S - 1 : min(kv_hi + g.window - 1, g.S - 1);
    first = max(kv_lo / kT, (share_lo + kT - 1) / kT);
    end = min(p_max / kT + 1, (share_hi + kT - 1) / kT);
    ti = first;
  }
  __device__ __forceinline__ bool next(const WinGeometry& g, QTile& o) {
    if (ti >= end) {
      ti = first;
      ++h;
    }
    if (h >= h_end || first >= end) return false;
    o.h = h;
    o.seg = 0;
    o.ti = ti;
    o.lo = ti * kT;
    o.valid = min(kT, g.S - o.lo);
    o.mask = kv_hi > o.lo ||
             (o.lo + o.valid - 1 >= kv_lo + g.window && kv_hi >= g.n_sink);
    ++ti;
    return true;
  }
};

// The o-th key tile of those that hold a first token; false when there is none.
__device__ __forceinline__ bool sink_tile(const WinGeometry& g, int o, int& seg, int& ti) {
  seg = 0;
  ti = o;
  return o * g.tile < g.n_sink && o * g.tile < g.S;
}

// The geometry of packed sequence b, its window and first tokens.
__device__ __forceinline__ void varlen_window_geometry(const WinGeometry& gp, int b,
                                                       WinGeometry& gs, int& row0,
                                                       int* status = nullptr) {
  gs = gp;
  varlen_geometry(gp, b, gs, row0, status);
}

}  // namespace ra
