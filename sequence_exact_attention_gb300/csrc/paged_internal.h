// Internal declarations of the paged key/value cache: its format, the
// arguments of its kernels and their launchers.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ring_attn.h"

namespace ra {

// A pool of pages: rows of D values (one slot of one key/value head),
// [n_pages, H_kv, page, D] bfloat16, or e4m3 codes with one power of two a row,
// its biased exponent in ks, vs [n_pages, H_kv, page]: a code c stands for
// c 2^(byte - 127). Slot j of sequence b is row j % page of page
// table[b * width + j / page].
struct PagePool {
  uint8_t *k, *v, *ks, *vs;
  int n_pages, H_kv, page, D;
  int quant;               // 1: e4m3 codes
};
constexpr int kPageMin = 16, kPageMax = 128;

// append and read.
struct PagedRowArgs {
  PagePool p;
  const int* table;
  int width;
  void* k;                 // [B, T, H_kv, D] or, with cu, [rows, H_kv, D]
  void* v;
  const int* start;        // [B], or null for 0
  const int* n_new;        // [B] tokens that count, or null for T (append)
  const int* cu;           // [B + 1] packed rows' offsets, or null (append)
  int B, T;
  long long rows;          // B * T, or the packed rows
  int* status;
};
ra_status launch_paged_append(const PagedRowArgs& a, int dtype, cudaStream_t stream);
ra_status launch_paged_read(const PagedRowArgs& a, int dtype, cudaStream_t stream);

// Attention of each sequence's new tokens over its slots.
struct PagedAttnArgs {
  const void* q;           // [rows, H_q, D] bf16
  PagePool p;
  const int* table;
  int width;
  const int* lens;         // [B] slots in use, the new tokens' included
  const int* cu;           // [B + 1] offsets of packed rows, or null: T rows a sequence
  void* out;               // [rows, H_q, D] bf16
  float* lse;              // [B, H_q, T] or, packed, [H_q, rows]; may be null
  int B, T, rows, H_q;     // T: new tokens a sequence; packed: at most so many
  int packed;
  int max_len;             // bound on lens
  int window, n_sink;      // window 0: every slot up to the query's own
  float scale_log2;        // softmax scale * log2(e)
  // plan (paged_attn_plan): a sequence's new tokens give n * H_q / H_kv query rows
  // a key/value head, cut into blocks, few rows (block_rows 8 or 16: paged_attn.cu) or
  // many (256: paged_tiles.cu). Of the n_items blocks n_cut, behind the first n_whole,
  // have their visible tiles cut into n_split chunks of `chunk` tiles; the others go to
  // one CTA each.
  int block_rows, n_items, n_whole, n_cut, n_split, chunk;
  int n_rb;                // blocks of the longest sequence and head
  int few_rows;            // packed: sequences of up to so many rows a head are the few rows'
                           // kernel's, longer ones the other's; 0: all are this one's
  int n_group;             // many rows: sequences a launch (paged_attn_group)
  int rb_major;            // many rows: the blocks' order, see there
  int n_expanded;          // many rows over 8-bit pages: tiles a sequence's rows see at most
  int by_page;             // 1: they are expanded page by page, to a pool of bf16 pages
  float* part_o;           // [n_cut][n_split][block_rows][D]
  float* part_ml;          // [n_cut][n_split][block_rows][2]: maximum (base 2), sum
  int4* part_block;        // many rows: [n_cut] the block's first row in q, its tokens (0: there
                           // is no such block), its key/value head
  __nv_bfloat16* expanded_k;     // [B][n_expanded][H_kv][128][D] or, by page, as the pool
  __nv_bfloat16* expanded_v;
  int* status;
};

// Few rows: slots of a tile, 32 KB of keys and values at most.
constexpr int paged_rows_tile(int D, bool quant) { return !quant && D == 128 ? 64 : 128; }

// Many rows over 8-bit pages: a tile of 128 slots of one head is expanded in D / kPagedShare
// shares.
constexpr int kPagedShare = 32;

// Fills the plan fields for the sizes in `a`, and, where short sequences of a packed
// call have a launch of their own, makes `few` that launch's arguments (else its n_items
// is 0); bytes: the workspace needed. Then a->n_group sequences are a launch: all, or, where
// neither their expanded tiles nor the pool's pages fit in kPagedExpanded bytes, fewer.
ra_status paged_attn_plan(PagedAttnArgs* a, PagedAttnArgs* few, size_t* bytes);
constexpr size_t kPagedExpanded = size_t(4) << 30;
// The arguments of the launch of sequences b0 on, a->n_group at most, of a planned call.
ra_status paged_attn_group(const PagedAttnArgs& a, int b0, PagedAttnArgs* group);
// Puts a launch's parts into the workspace, which a call's launches use in turn.
void paged_attn_place(PagedAttnArgs* a, void* workspace);
// The launchers of the two kernels and of the join of their chunks.
ra_status launch_paged_rows(const PagedAttnArgs& a, cudaStream_t stream);
ra_status launch_paged_tiles(const PagedAttnArgs& a, cudaStream_t stream);
ra_status launch_paged_join(const PagedAttnArgs& a, cudaStream_t stream);

// TMA map of a pool's keys or values as [n_pages * H_kv, D / cols, page, cols], cols
// being 64 values (bfloat16) or D (codes): a box is `box_rows` rows of one page and
// `box_parts` of its parts of `cols` values, one part after the other, swizzled over
// the bytes of a part's row (128, or 64 where D is 64 and codes are held).
bool make_page_map(CUtensorMap* m, const PagePool& p, const void* ptr, int box_rows, int box_parts);
// TMA map of bf16 queries [rows, H_q, D]: a box is 64 columns of `heads` heads of
// `tokens` rows, a row of the box after the other, 128-byte swizzle.
bool make_query_map(CUtensorMap* m, const void* q, int rows, int H_q, int D, int heads, int tokens);

}  // namespace ra
