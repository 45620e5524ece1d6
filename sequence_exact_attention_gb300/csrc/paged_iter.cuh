// The paged kernels' walks: a sequence's rows, the tiles of slots that a block of them
// sees, and which CTA takes which chunk. Also built for the host, by a CPU test.
#pragma once

#include "paged_internal.h"

namespace ra {

// A sequence's new tokens: their first row in q and out, how many they are, and
// the slots in use with them. Offsets are brought into the tensors' range.
struct PagedSeq {
  int row0, n, len;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedAttnArgs& a, int b) {
  PagedSeq s;
  if (a.cu) {
    s.row0 = min(max(a.cu[b], 0), a.rows);
    s.n = min(min(max(a.cu[b + 1] - s.row0, 0), a.T), a.rows - s.row0);
  } else {
    s.row0 = b * a.T;
    s.n = a.T;
  }
  s.len = min(max(a.lens[b], 0), a.max_len);
  return s;
}

// Whether a sequence of a packed call is the launch's that `a` is of.
__device__ __forceinline__ bool paged_mine(const PagedAttnArgs& a, const PagedSeq& s) {
  if (a.few_rows == 0) return true;
  return (s.n * (a.H_q / a.p.H_kv) <= a.few_rows) == (a.block_rows <= 16);
}

// Whether the row at position p sees slot j.
__device__ __forceinline__ bool paged_sees(const PagedAttnArgs& a, int p, int j) {
  return j <= p && (a.window <= 0 || j > p - a.window || j < a.n_sink);
}

// The tiles of kTile slots that rows at positions pmin to pmax see: those of the
// first slots that the windows have left behind, then the windows' own.
template <int kTile>
struct PagedSpan {
  int hi;              // slots from here on are invisible to every row
  int pmin, pmax;
  int n_sink_tiles, w0;
  int n;               // tiles in all
  __device__ __forceinline__ void init(const PagedAttnArgs& a, int p0, int p1) {
    pmin = p0;
    pmax = p1;
    hi = max(p1 + 1, 0);
    const int lo = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
    w0 = lo / kTile;
    n_sink_tiles = min((min(a.n_sink, hi) + kTile - 1) / kTile, w0);
    n = n_sink_tiles + max((hi + kTile - 1) / kTile - w0, 0);
  }
  __device__ __forceinline__ int tile(int v) const {
    return v < n_sink_tiles ? v : v - n_sink_tiles + w0;
  }
  // Whether some row sees one of the n slots from j0 on, a run that starts below hi.
  __device__ __forceinline__ bool meets(const PagedAttnArgs& a, int j0, int n_slots) const {
    return a.window <= 0 || j0 + n_slots > pmin - a.window + 1 || j0 < a.n_sink;
  }
  // Whether every row sees all of the n slots from j0 on.
  __device__ __forceinline__ bool whole(const PagedAttnArgs& a, int j0, int n_slots) const {
    return j0 + n_slots - 1 <= pmin &&
           (a.window <= 0 || j0 > pmax - a.window || j0 + n_slots <= a.n_sink);
  }
};

// A CTA's block and its chunk of it, or (split -1) all of it.
struct PagedWork {
  int item, split;
};
__device__ __forceinline__ PagedWork paged_work(const PagedAttnArgs& a, int cta) {
  if (cta < a.n_whole) return {cta, -1};
  const int x = cta - a.n_whole, cut = a.n_cut * a.n_split;
  if (x < cut) return {a.n_whole + x / a.n_split, x % a.n_split};
  return {a.n_whole + a.n_cut + x - cut, -1};
}
// The row of the partial results that is row r of chunk `split` of block `item`.
__device__ __forceinline__ long long paged_part(const PagedAttnArgs& a, int item, int split, int r) {
  return ((long long)(item - a.n_whole) * a.n_split + split) * a.block_rows + r;
}

}  // namespace ra
