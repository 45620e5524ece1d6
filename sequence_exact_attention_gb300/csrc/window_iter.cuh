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
  int lo, end;               // first position of the next tile; past the last tile
  int first_end, w0;         // tiles of first tokens that the windows left behind end
                             // here; the windows' first tile
  int full_to, window_from, sink_to;   // tiles that need no mask start here

  __device__ __forceinline__ void init(const WinGeometry& g, int, int q_lo, int q_valid) {
    const int q_hi = q_lo + q_valid - 1;
    end = q_valid > 0 ? (q_hi / g.tile + 1) * g.tile : 0;
    w0 = min(max(q_lo - g.window + 1, 0) / g.tile * g.tile, end);
    first_end = min((g.n_sink + g.tile - 1) / g.tile * g.tile, w0);
    lo = first_end > 0 ? 0 : w0;
    // all keys are at or before the first query (a ragged tile never is), and in
    // the last query's window or first tokens
    full_to = q_lo - g.tile + 1;
    window_from = q_hi - g.window + 1;
    sink_to = g.n_sink - g.tile;
  }
  // Key tiles in all.
  __device__ __forceinline__ int length(const WinGeometry& g) const {
    return (first_end + end - w0) / g.tile;
  }

  __device__ __forceinline__ bool next(const WinGeometry& g, KvTile& kv) {
    if (lo >= end) return false;
    kv.step = kv.src = kv.seg = kv.id = 0;
    kv.lo = lo;
    kv.valid = min(g.tile, g.S - lo);
    kv.work = lo <= full_to && (lo >= window_from || lo <= sink_to) ? kNoMask : kMask;
    lo += g.tile;
    if (lo == first_end) lo = w0;
    return true;
  }
};

template <int kT>
struct WinQIterT {
  int h, h_end;              // query heads of the group
  int lo, first, end;        // next tile's first position; of a head's first tile, past its last
  int masked_to, masked_from;    // tiles that start before, or whose last query is from here on

  // The tiles whose first position is in [share_lo, share_hi).
  __device__ __forceinline__ void init(const WinGeometry& g, int, int kv_lo, int kv_valid,
                                       int h_begin, int h_end_, int share_lo, int share_hi) {
    const int kv_hi = kv_lo + kv_valid - 1;
    // the last query position that sees a key of the tile
    const int p_max = kv_lo < g.n_sink ? g.S - 1 : min(kv_hi + g.window - 1, g.S - 1);
    first = max(kv_lo, share_lo + kT - 1) / kT * kT;
    end = min(p_max + 1, share_hi);
    lo = first;
    h = h_begin;
    h_end = kv_valid > 0 && first < end ? h_end_ : h_begin;
    masked_to = kv_hi;
    masked_from = kv_hi >= g.n_sink ? kv_lo + g.window : 0x7fffffff;
  }
  __device__ __forceinline__ bool next(const WinGeometry& g, QTile& o) {
    if (h >= h_end) return false;
    o.h = h;
    o.seg = 0;
    o.ti = lo / kT;
    o.lo = lo;
    o.valid = min(kT, g.S - lo);
    o.mask = lo < masked_to || lo + o.valid - 1 >= masked_from;
    lo += kT;
    if (lo >= end) {
      lo = first;
      ++h;
    }
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
