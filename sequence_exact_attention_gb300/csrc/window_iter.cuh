// Walks of attention with a sliding window and a few first tokens that stay
// visible: query i sees key j <= i when j > i - window or j < n_sink.
//
// WinKvIter is KvIter over the key tiles that some row of the query rows
// sees, in the same ring order; the tiles between the first tokens and the
// rows' windows are jumped over, so a walk costs what it visits. WinQIterT is
// QIterT the other way round, over the query tiles that see a key tile,
// limited to a share of them (by their first position) where the work on one
// key tile is split.
#pragma once

#include "q_iter.cuh"
#include "ring_iter.cuh"

namespace ra {

struct WinKvIter : KvIter {
  __device__ __forceinline__ bool next(const WinGeometry& g, KvTile& kv) {
    while (t < t_end) {
      if (rem > 0 && lo <= q_hi) {
        const int valid = min(g.tile, rem);
        if (lo >= g.n_sink && lo + valid - 1 <= q_lo - g.window) {
          // hidden from the first row, and so from all: jump over the whole
          // tiles that are (a ragged one ends its segment)
          const int skip = max(1, (q_lo - g.window + 1 - lo) / g.tile);
          lo += skip * g.tile;
          rem -= skip * g.tile;
          id += skip;
          continue;
        }
        kv.step = t;
        kv.src = src;
        kv.seg = seg;
        kv.id = id;
        kv.lo = lo;
        kv.valid = valid;
        const bool all_allowed = lo + valid - 1 <= q_lo &&
                                 (lo > q_hi - g.window || lo + valid <= g.n_sink);
        kv.work = (all_allowed && valid == g.tile) ? kNoMask : kMask;
        lo += g.tile;
        rem -= g.tile;
        ++id;
        return true;
      }
      if (++which >= g.segs_per_rank) {
        which = 0;
        ++t;
        if (--src < 0) src += g.P;
      }
      start_segment(g);
    }
    return false;
  }
};

// Number of key tiles WinKvIter walks (walks are a window long: counted by
// walking).
__device__ __forceinline__ int win_walk_length(const WinGeometry& g, int r, int q_lo,
                                               int q_valid) {
  WinKvIter it;
  it.init(g, r, q_lo, q_valid);
  KvTile kv;
  int n = 0;
  while (it.next(g, kv)) ++n;
  return n;
}

template <int kT>
struct WinQIterT : QIterT<kT> {
  using Base = QIterT<kT>;
  int p_max;              // last query position that sees a key of the tile
  int share_lo, share_hi; // tiles whose first position is in [share_lo, share_hi)

  __device__ __forceinline__ void start_segment(const WinGeometry& g) {
    const int s0 = rank_seg(g, this->r, this->which) * g.seg_len;
    this->len = seg_tokens(g, rank_seg(g, this->r, this->which));
    const int tiles = (this->len + kT - 1) / kT;
    auto first_from = [&](int p) { return p <= s0 ? 0 : (p - s0 + kT - 1) / kT; };
    this->ti = max(this->kv_lo <= s0 ? 0 : (this->kv_lo - s0) / kT, first_from(share_lo));
    this->ti_end = min(min(tiles, first_from(share_hi)), p_max < s0 ? 0 : (p_max - s0) / kT + 1);
    if (s0 + this->len <= this->kv_lo) this->ti_end = 0;     // all before the key tile
  }
  __device__ __forceinline__ void init(const WinGeometry& g, int src_, int kv_lo_, int kv_valid,
                                       int h_begin, int h_end_, int share_lo_, int share_hi_) {
    this->h = h_begin;
    this->h_end = kv_valid > 0 ? h_end_ : h_begin;
    this->src = src_;
    this->t = 0;
    this->r = src_;
    this->which = 0;
    this->kv_lo = kv_lo_;
    this->kv_hi = kv_lo_ + kv_valid - 1;
    p_max = kv_lo_ < g.n_sink ? g.S - 1 : min(this->kv_hi + g.window - 1, g.S - 1);
    share_lo = share_lo_;
    share_hi = share_hi_;
    start_segment(g);
  }
  __device__ __forceinline__ bool next(const WinGeometry& g, QTile& o) {
    while (this->h < this->h_end) {
      if (this->ti < this->ti_end) {
        const int seg = rank_seg(g, this->r, this->which);
        o.h = this->h;
        o.seg = seg;
        o.ti = this->ti;
        o.lo = seg * g.seg_len + this->ti * kT;
        o.valid = min(kT, this->len - this->ti * kT);
        o.mask = this->kv_hi > o.lo ||
                 (o.lo + o.valid - 1 >= this->kv_lo + g.window && this->kv_hi >= g.n_sink);
        ++this->ti;
        return true;
      }
      if (++this->which >= g.segs_per_rank) {
        this->which = 0;
        if (++this->t >= g.P) {
          this->t = 0;
          ++this->h;
        }
        this->r = this->src + this->t;
        if (this->r >= g.P) this->r -= g.P;
      }
      if (this->h < this->h_end) start_segment(g);
    }
    return false;
  }
};

// The o-th key tile, in position order, of the tiles that hold a first token
// (key position below n_sink); false when there is no such tile.
__device__ __forceinline__ bool sink_tile(const WinGeometry& g, int o, int& seg, int& ti) {
  const int per = max(1, (g.seg_len + g.tile - 1) / g.tile);
  seg = o / per;
  ti = o - seg * per;
  return seg < g.n_seg && seg * g.seg_len + ti * g.tile < g.n_sink && tile_tokens(g, seg, ti) > 0;
}

// The geometry of packed sequence b, its window and first tokens.
__device__ __forceinline__ void varlen_window_geometry(const WinGeometry& gp, int b,
                                                       WinGeometry& gs, int& row0,
                                                       int* status = nullptr) {
  gs = gp;
  varlen_geometry(gp, b, gs, row0, status);
}

}  // namespace ra
