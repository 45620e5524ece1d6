// How an attention call over pages is cut up: which kernel, its blocks of query rows
// and its chunks of slots. Host only, and the same where there is no device to ask,
// as the workspace's size follows from it: the card's numbers are a GB300's.
#include <algorithm>

#include "paged_internal.h"

namespace ra {
namespace {

constexpr long long kSms = 152;

// Tiles of `tile` slots that a run of T new tokens sees at most.
long long tiles_seen(const PagedAttnArgs& a, int tile, long long T) {
  const long long all = ((long long)a.max_len + tile - 1) / tile;
  if (a.window <= 0) return all;
  const long long seen = ((long long)a.n_sink + tile - 1) / tile +
                         ((long long)a.window + T - 1 + tile - 1) / tile + 1;
  return seen < all ? seen : all;
}

// Rows of partial results.
size_t parts(const PagedAttnArgs& a) {
  return (size_t)a.n_cut * a.n_split * a.block_rows;
}

// How the visible tiles of blocks are cut: those of `count` blocks behind the first
// `whole` ones into `want` chunks, but none under `least` tiles.
ra_status cut(PagedAttnArgs* a, long long items, long long whole, long long count, long long tiles,
              long long want, long long least) {
  long long chunk = (tiles + want - 1) / want;
  if (chunk < least) chunk = least;
  const long long n_split = tiles > chunk ? (tiles + chunk - 1) / chunk : 1;
  if (n_split == 1) count = 0;
  if (items > 0x7fffffffLL || items + count * (n_split - 1) > 0x7fffffffLL) return RA_ERR_RANGE;
  a->n_items = (int)items;
  a->n_whole = (int)whole;
  a->n_cut = (int)count;
  a->chunk = (int)chunk;
  a->n_split = (int)n_split;
  return RA_OK;
}

// Few rows, R of T tokens a sequence and head: chunks that fill whole waves of resident
// CTAs best, two waves by preference (sequences of different lengths then even out), but
// none under two tiles, where joining would cost more than it spreads.
ra_status plan_few(PagedAttnArgs* a, long long R, long long T) {
  a->block_rows = R <= 8 ? 8 : 16;
  const long long n_rb = (R + a->block_rows - 1) / a->block_rows;
  a->n_rb = (int)n_rb;
  const long long items = (long long)a->B * a->p.H_kv * n_rb;
  const long long wave = 2 * kSms;
  long long best = 1, best_full = 0;
  for (int w = 2; w >= 1; --w) {
    const long long n = wave * w / items;
    const long long full = n * items * 1000 / (wave * w);
    if (full > best_full + 20) {
      best = n;
      best_full = full;
    }
  }
  const int tile = paged_rows_tile(a->p.D, a->p.quant != 0);
  return cut(a, items, 0, items, tiles_seen(*a, tile, T), best, 2);
}

// Many rows: a CTA a multiprocessor, in whole waves; the blocks left over are cut into
// as many chunks as end first, counted in tiles: a CTA takes some 4 to begin and end,
// the join's launch and its rows some 6.
ra_status plan_many(PagedAttnArgs* a) {
  a->block_rows = 256;
  const int grp = a->H_q / a->p.H_kv, tokens = 2 * (128 / grp);
  const long long n_rb = ((long long)a->T + tokens - 1) / tokens;
  a->n_rb = (int)n_rb;
  // of packed sequences: how many blocks there are at most, and, where the short ones
  // have their own launch, if the others have T tokens each
  long long blocks = a->B * n_rb, likely = blocks;
  if (a->packed) {
    const long long most = a->rows / tokens + a->B;
    if (most < blocks) blocks = most;
    likely = blocks;
    if (a->few_rows > 0) {
      const long long over = a->rows > a->B ? a->rows - a->B : 0;
      const long long n = (over + a->T - 2) / (a->T - 1);
      if (n * n_rb < likely) likely = n * n_rb;
    }
  }
  const long long items = blocks * a->p.H_kv;
  const long long tiles = tiles_seen(*a, 128, tokens < a->T ? tokens : a->T);
  const long long whole = likely * a->p.H_kv / kSms * kSms, rest = likely * a->p.H_kv - whole;
  long long best = 1, best_cost = tiles + 4;
  for (long long s = 2; rest > 0 && s * 4 <= tiles; ++s) {
    const long long cost = (rest * s + kSms - 1) / kSms * ((tiles + s - 1) / s + 4) + 6;
    if (cost < best_cost) {
      best = s;
      best_cost = cost;
    }
    if (rest * s > 8 * kSms) break;
  }
  // keys and values within half of the 126 MB L2
  a->rb_major = (long long)a->B * a->max_len * a->p.H_kv * a->p.D * 4 <= (64ll << 20);
  if (a->p.quant) {
    // (the expansion counts shares of tiles in 32 bits, also where it goes by page)
    const long long e = tiles_seen(*a, 128, a->T);
    if ((long long)a->B * e * a->p.H_kv > 0x7fffffffLL / (a->p.D / kPagedShare))
      return RA_ERR_RANGE;
    a->n_expanded = (int)e;
  }
  return cut(a, items, whole, rest, tiles, best, 4);
}

// One of the two expanded tensors' values.
size_t expanded(const PagedAttnArgs& a) {
  if (a.by_page) return (size_t)a.p.n_pages * a.p.H_kv * a.p.page * a.p.D;
  return (size_t)a.B * a.n_expanded * a.p.H_kv * 128 * a.p.D;
}
// The workspace of a launch.
size_t launch_bytes(const PagedAttnArgs& a) {
  return 4 * expanded(a) + parts(a) * (a.p.D + 2) * sizeof(float) + (size_t)a.n_cut * sizeof(int4);
}

// A launch of many rows for n of the call's sequences; its tensors are still the call's.
ra_status plan_group(const PagedAttnArgs& a, int n, PagedAttnArgs* group) {
  *group = a;
  group->B = n;
  if (!a.packed) group->rows = n * a.T;
  return plan_many(group);
}

}  // namespace

ra_status paged_attn_plan(PagedAttnArgs* a, PagedAttnArgs* few, size_t* bytes) {
  const int grp = a->H_q / a->p.H_kv;
  const long long R = (long long)a->T * grp;
  // What is more than few rows. bf16 pages of many rows are read once, by tiles; 8-bit
  // ones are expanded first, five times their bytes, so blocks of 16 rows that read the
  // pages again (from L2, mostly) are ahead for longer: 8 x 32K slots of 4 heads, D =
  // 128, 25 rows 128 instead of 245 us, 40 rows 176; of short windows they are as fast.
  const int limit = a->p.quant ? 48 : 16;
  few->n_items = 0;
  a->n_group = a->B;
  ra_status st;
  if (R <= limit) {
    st = plan_few(a, R, a->T);
  } else {
    // 8-bit pages: packed sequences of which many have to be short, single tokens beside
    // pieces of prompts, get a launch of their own, which reads one byte a value where
    // the tiles' expansion moves five and its tiles two. It costs some 13 us, what 2^25
    // values take. 63 tokens and a piece of 512 behind 8K slots, 8 heads, D = 128: 290
    // instead of 971 us; 28 tokens and 4 x 256 behind 4K 157 instead of 306; 15 and 256
    // behind 1K (2.3e7 values) 54 instead of 41. bf16 pages have less to gain: 367
    // instead of 387, 150 instead of 158, 46 instead of 23.
    const int short_rows = grp > 16 ? grp : 16;
    if (a->packed && a->p.quant && short_rows <= limit && 2ll * a->rows <= (long long)a->B * a->T &&
        a->B * tiles_seen(*a, 128, a->T) * a->p.H_kv * 128 * a->p.D >= 1ll << 25)
      a->few_rows = short_rows;
    // The expanded tiles of 64 places of 128K slots, 8 heads, D = 128, would take 34 GB,
    // few of which may be used. Where they pass kPagedExpanded, the pool's pages are expanded
    // instead, each to a page (63 tokens and a piece of 512 behind 8K slots at such a table:
    // 2.1 GB), or, of a pool too large as well, a group of sequences at a time, in equal
    // groups. (A group without a piece costs 15 us: 466 instead of 368 us for 8 of them.)
    if (a->p.quant) {
      const size_t seen = (size_t)tiles_seen(*a, 128, a->T), one = seen * a->p.H_kv * 128 * a->p.D;
      const size_t most = std::max<size_t>(kPagedExpanded / (4 * one), 1);
      if ((size_t)a->B > most) {
        a->by_page = 1;
        if (4 * expanded(*a) > kPagedExpanded) {
          a->by_page = 0;
          const int groups = (a->B - 1) / (int)most + 1;
          a->n_group = (a->B - 1) / groups + 1;
        }
      }
    }
    *bytes = 0;
    PagedAttnArgs group;
    for (int n : {a->n_group, a->B % a->n_group}) {      // the last group may be smaller
      if (n == 0) continue;
      st = plan_group(*a, n, &group);
      if (st != RA_OK) return st;
      *bytes = std::max(*bytes, launch_bytes(group));
    }
    if (a->few_rows > 0) {
      *few = *a;
      st = plan_few(few, short_rows, short_rows / grp);
      if (st == RA_OK) *bytes = std::max(*bytes, launch_bytes(*few));
    }
    return st;
  }
  if (st == RA_OK) *bytes = launch_bytes(*a);
  return st;
}

ra_status paged_attn_group(const PagedAttnArgs& a, int b0, PagedAttnArgs* group) {
  *group = a;
  if (a.block_rows != 0) return RA_OK;      // few rows: planned already, and one launch
  const ra_status st = plan_group(a, std::min(a.n_group, a.B - b0), group);
  if (st != RA_OK) return st;
  group->table += (size_t)b0 * a.width;
  group->lens += b0;
  if (a.packed) {
    group->cu += b0;
  } else {
    const size_t row = (size_t)b0 * a.T * a.H_q;
    group->q = static_cast<const __nv_bfloat16*>(a.q) + row * a.p.D;
    group->out = static_cast<__nv_bfloat16*>(a.out) + row * a.p.D;
    if (a.lse) group->lse += row;
  }
  return RA_OK;
}

void paged_attn_place(PagedAttnArgs* a, void* workspace) {
  __nv_bfloat16* e = static_cast<__nv_bfloat16*>(workspace);
  a->expanded_k = e;
  a->expanded_v = e + expanded(*a);
  a->part_o = reinterpret_cast<float*>(e + 2 * expanded(*a));
  a->part_ml = a->part_o + parts(*a) * a->p.D;
  a->part_block = reinterpret_cast<int4*>(a->part_ml + parts(*a) * 2);
}

}  // namespace ra
