// Host build of the paged attention's plan (csrc/paged_plan.cpp) and walks
// (csrc/paged_iter.cuh) for test_paged_plan_cpu.py: every CTA of every launch of a call.
#include <algorithm>
namespace ra {
using std::max;
using std::min;
}  // namespace ra
#include "paged_iter.cuh"

namespace {

// The block of query rows that item `item` of a launch is: sequence (below 0: there is no
// such block), head, number among the sequence's.
struct Block {
  int b, hk, rb;
};
Block block_of(const ra::PagedAttnArgs& a, int item) {
  const int H = a.p.H_kv;
  if (a.block_rows <= 16) return {item / a.n_rb / H, item / a.n_rb % H, item % a.n_rb};
  const int tokens = 2 * (128 / (a.H_q / H));
  auto blocks = [&](int b) {
    const ra::PagedSeq s = ra::paged_seq(a, b);
    if (!a.cu) return a.n_rb;
    return ra::paged_mine(a, s) ? (s.n + tokens - 1) / tokens : 0;
  };
  if (!a.cu && a.rb_major) {
    const int bh = item % (a.B * H);
    return {bh / H, bh % H, a.n_rb - 1 - item / (a.B * H)};
  }
  for (int b = 0; b < a.B; ++b) {
    const int n = blocks(b);
    if (item < n * H) {
      if (a.rb_major) return {b, item % H, n - 1 - item / H};
      return {b, item / n, n - 1 - item % n};
    }
    item -= n * H;
  }
  return {-1, 0, 0};
}

struct Out {
  int* rows;
  int cap, n;
  void add(std::initializer_list<int> x) {
    if (n < cap) std::copy(x.begin(), x.end(), rows + 9 * n);
    ++n;
  }
};

// (launch, first sequence, head, first row, rows, slots a tile, split, first slot of a tile
// or -1 for a chunk without one, part's first row or -1) of a launch's CTAs.
template <int kTile>
void walk(const ra::PagedAttnArgs& a, int launch, int first_seq, Out* out) {
  const int grp = a.H_q / a.p.H_kv, few = a.block_rows <= 16;
  const long long ctas = few ? (long long)a.n_items * a.n_split
                             : a.n_items + (long long)a.n_cut * (a.n_split - 1);
  for (long long cta = 0; cta < ctas; ++cta) {
    ra::PagedWork w = ra::paged_work(a, (int)cta);
    if (few) w = {(int)(cta % a.n_items), a.n_split > 1 ? (int)(cta / a.n_items) : -1};
    const Block blk = block_of(a, w.item);
    if (blk.b < 0) continue;
    const ra::PagedSeq s = ra::paged_seq(a, blk.b);
    if (!ra::paged_mine(a, s)) continue;
    const int per = few ? a.block_rows : 2 * (128 / grp) * grp;
    const int r0 = blk.rb * per, R = std::min(s.n * grp - r0, per);
    if (R <= 0) continue;
    ra::PagedSpan<kTile> sp;
    const int first = s.len - s.n;
    sp.init(a, first + r0 / grp, first + (r0 + R - 1) / grp);
    const int from = std::max(w.split, 0) * a.chunk;
    const int to = w.split < 0 ? sp.n : std::min(sp.n, from + a.chunk);
    const int part = w.split < 0 ? -1 : (int)ra::paged_part(a, w.item, w.split, 0);
    if (to <= from)
      out->add({launch, first_seq + blk.b, blk.hk, r0, R, kTile, w.split, -1, part});
    for (int v = from; v < to; ++v)
      out->add({launch, first_seq + blk.b, blk.hk, r0, R, kTile, w.split, sp.tile(v) * kTile, part});
  }
}

}  // namespace

extern "C" {

// The CTAs' walks of a call, nine numbers each; their number, or below 0 where the plan
// refuses. `launches`: for each, (block_rows, rows of parts, sequences, tiles expanded a
// sequence or, below 0, by page).
int ra_paged_walks(int B, int T, int total, int H_q, int H_kv, int D, int page, int n_pages, int quant,
                   int max_len, int window, int n_sink, const int* lens, const int* cu, int* rows, int cap,
                   int* launches, int launch_cap) {
  ra::PagedAttnArgs a = {}, few = {};
  a.p.n_pages = n_pages;
  a.p.H_kv = H_kv;
  a.p.page = page;
  a.p.D = D;
  a.p.quant = quant;
  a.B = B;
  a.T = T;
  a.packed = cu != nullptr;
  a.rows = cu ? total : B * T;
  a.H_q = H_q;
  a.max_len = max_len;
  a.window = window >= max_len ? 0 : window;
  a.n_sink = a.window > 0 ? std::min(n_sink, max_len) : 0;
  a.lens = lens;
  a.cu = cu;
  a.table = lens;                    // never read
  size_t bytes = 0;
  if (ra::paged_attn_plan(&a, &few, &bytes) != RA_OK) return -1;
  Out out = {rows, cap, 0};
  int n = 0;
  auto launch = [&](const ra::PagedAttnArgs& x, int first_seq) {
    if (n < launch_cap) {
      int* l = launches + 4 * n;
      l[0] = x.block_rows;
      l[1] = x.n_cut * x.n_split * x.block_rows;
      l[2] = x.B;
      l[3] = x.by_page ? -1 : x.n_expanded;
    }
    if (x.block_rows <= 16 && ra::paged_rows_tile(x.p.D, x.p.quant != 0) == 64) walk<64>(x, n, first_seq, &out);
    else walk<128>(x, n, first_seq, &out);
    ++n;
  };
  if (few.n_items > 0) launch(few, 0);
  for (int b0 = 0; b0 < B; b0 += a.n_group) {
    ra::PagedAttnArgs g;
    if (ra::paged_attn_group(a, b0, &g) != RA_OK) return -2;
    launch(g, b0);
  }
  if (n < launch_cap) launches[4 * n] = 0;
  return out.n;
}

}  // extern "C"
