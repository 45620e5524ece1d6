// How an attention call over pages is cut up: which kernel, its blocks of query rows
// and its chunks of slots. Host only, and the same where there is no device to ask,
// as the workspace's size follows from it: the card's numbers are a GB300's.
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
  return (size_t)(a.n_items - a.n_whole) * a.n_split * a.block_rows;
}

}  // namespace

ra_status paged_attn_plan(PagedAttnArgs* a, size_t* bytes) {
  const int grp = a->H_q / a->p.H_kv;
  const long long R = (long long)a->T * grp;
  long long items, whole = 0, tiles, best = 1, least;
  // What is more than few rows. bf16 pages of many rows are read once, by tiles; 8-bit
  // ones are expanded first, five times their bytes, so blocks of 16 rows that read the
  // pages again (from L2, mostly) are ahead for longer: 8 x 32K slots of 4 heads, D =
  // 128, 25 rows 128 instead of 245 us, 40 rows 173; of short windows they are as fast.
  if (R <= (a->p.quant ? 48 : 16)) {
    // Few rows: chunks that fill whole waves of resident CTAs best, two waves by
    // preference (sequences of different lengths then even out), but none under two
    // tiles, where joining would cost more than it spreads.
    a->block_rows = R <= 8 ? 8 : 16;
    const long long n_rb = (R + a->block_rows - 1) / a->block_rows;
    a->n_rb = (int)n_rb;
    items = (long long)a->B * a->p.H_kv * n_rb;
    const int tile = paged_rows_tile(a->p.D, a->p.quant != 0);
    tiles = tiles_seen(*a, tile, a->T);
    least = 2;
    const long long wave = 2 * kSms;
    long long best_full = 0;
    for (int w = 2; w >= 1; --w) {
      const long long n = wave * w / items;
      const long long full = n * items * 1000 / (wave * w);
      if (full > best_full + 20) {
        best = n;
        best_full = full;
      }
    }
  } else {
    // Many rows: a CTA a multiprocessor, in whole waves; the blocks left over are cut
    // into as many chunks as end first, counted in tiles: a CTA takes some 4 to begin
    // and end, the join's launch and its rows some 6.
    a->block_rows = 256;
    const int block_tokens = 2 * (128 / grp);
    const long long n_rb = ((long long)a->T + block_tokens - 1) / block_tokens;
    long long blocks = a->B * n_rb;
    const long long most = a->rows / block_tokens + a->B;     // of packed sequences
    if (a->packed && most < blocks) blocks = most;
    items = blocks * a->p.H_kv;
    if (items > 0x7fffffffLL) return RA_ERR_RANGE;
    a->n_rb = (int)n_rb;
    tiles = tiles_seen(*a, 128, block_tokens < a->T ? block_tokens : a->T);
    least = 4;
    whole = items / kSms * kSms;
    const long long rest = items - whole;
    long long best_cost = tiles + 4;
    for (long long s = 2; rest > 0 && s * least <= tiles; ++s) {
      const long long cost = (rest * s + kSms - 1) / kSms * ((tiles + s - 1) / s + 4) + 6;
      if (cost < best_cost) {
        best = s;
        best_cost = cost;
      }
      if (rest * s > 8 * kSms) break;
    }
    // keys and values within half of the 126 MB L2
    a->rb_major = (long long)a->B * a->max_len * a->p.H_kv * a->p.D * 4 <= (64ll << 20);
  }
  long long chunk = (tiles + best - 1) / best;
  if (chunk < least) chunk = least;
  const long long n_split = tiles > chunk ? (tiles + chunk - 1) / chunk : 1;
  if (n_split == 1) whole = items;
  if (whole + (items - whole) * n_split > 0x7fffffffLL) return RA_ERR_RANGE;
  a->n_items = (int)items;
  a->n_whole = (int)whole;
  a->chunk = (int)chunk;
  a->n_split = (int)n_split;
  size_t n = parts(*a) * (a->p.D + 2) * sizeof(float);
  if (a->block_rows == 256 && a->p.quant) {
    const long long e = tiles_seen(*a, 128, a->T);
    if ((long long)a->B * e * a->p.H_kv > 0x7fffffffLL) return RA_ERR_RANGE;
    a->n_expanded = (int)e;
    n += (size_t)a->B * e * a->p.H_kv * 128 * a->p.D * 2 * 2;
  }
  *bytes = n;
  return RA_OK;
}

void paged_attn_place(PagedAttnArgs* a, void* workspace) {
  __nv_bfloat16* e = static_cast<__nv_bfloat16*>(workspace);
  const size_t tensor = (size_t)a->B * a->n_expanded * a->p.H_kv * 128 * a->p.D;
  a->expanded_k = e;
  a->expanded_v = e + tensor;
  a->part_o = reinterpret_cast<float*>(e + 2 * tensor);
  a->part_ml = a->part_o + parts(*a) * a->p.D;
}

}  // namespace ra
