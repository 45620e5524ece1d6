// extern "C" entry points of the paged key/value cache: argument checks on the
// host, then one launcher.
#include <cstdint>

#include "host_checks.h"
#include "paged_internal.h"
#include "ra_internal.h"

using namespace ra;

namespace {

PagePool pool_of(const ra_pages& p) {
  return {static_cast<uint8_t*>(p.k), static_cast<uint8_t*>(p.v),
          static_cast<uint8_t*>(p.k_scale), static_cast<uint8_t*>(p.v_scale),
          p.n_pages, p.H_kv, p.page, p.D, p.dtype == RA_E4M3};
}

// The sizes and the type of a pool.
ra_status check_sizes(const ra_pages* p) {
  if (!p) return RA_ERR_NULL;
  if (p->dtype != RA_BF16 && p->dtype != RA_E4M3) return RA_ERR_DTYPE;
  if (p->n_pages <= 0 || p->H_kv <= 0) return RA_ERR_SHAPE;
  if (p->page < kPageMin || p->page > kPageMax || (p->page & (p->page - 1)) != 0)
    return RA_ERR_SHAPE;
  if (p->D != 64 && p->D != 128) return RA_ERR_HEADDIM;
  // pages and heads are counted in 32 bits, rows and values in 64
  if ((long long)p->n_pages * p->H_kv > kMaxElems) return RA_ERR_RANGE;
  return RA_OK;
}

ra_status check_pages(const ra_pages* p, const int* table, int width) {
  const ra_status st = check_sizes(p);
  if (st != RA_OK) return st;
  if (!p->k || !p->v || !table) return RA_ERR_NULL;
  if (p->dtype == RA_E4M3 && (!p->k_scale || !p->v_scale)) return RA_ERR_NULL;
  if (width <= 0) return RA_ERR_SHAPE;
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(table, 4)) return RA_ERR_ALIGN;
  if (p->dtype == RA_E4M3 && (!aligned(p->k_scale, 16) || !aligned(p->v_scale, 16)))
    return RA_ERR_ALIGN;
  return RA_OK;
}

size_t pool_bytes(const ra_pages& p) {
  return (size_t)p.n_pages * p.H_kv * p.page * p.D * (p.dtype == RA_E4M3 ? 1 : 2);
}
size_t scale_bytes(const ra_pages& p) {
  return p.dtype == RA_E4M3 ? (size_t)p.n_pages * p.H_kv * p.page : 0;
}
size_t table_bytes(int B, int width) { return (size_t)B * width * 4; }

// Token tensors [tokens, H, D].
ra_status check_tokens(long long tokens, int H, int D) {
  return tokens > kMaxElems || tokens * H > kMaxElems || tokens * H * D > kMaxElems ? RA_ERR_RANGE
                                                                                    : RA_OK;
}

ra_status append(const ra_pages* pages, const int* table, int width, const void* k, const void* v,
                 const int* start, const int* n_new, const int* cu, int B, int T, long long rows,
                 int dtype, int* status, void* stream) {
  if (!k || !v || !start) return RA_ERR_NULL;
  if (dtype != RA_BF16 && dtype != RA_F32) return RA_ERR_DTYPE;
  ra_status st = check_pages(pages, table, width);
  if (st != RA_OK) return st;
  if (B <= 0 || T <= 0 || rows <= 0) return RA_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16)) return RA_ERR_ALIGN;
  if (!aligned(start, 4) || !aligned(n_new, 4) || !aligned(cu, 4) || !aligned(status, 4))
    return RA_ERR_ALIGN;
  st = check_tokens(rows, pages->H_kv, pages->D);
  if (st != RA_OK) return st;
  const size_t n = (size_t)rows * pages->H_kv * pages->D * (dtype == RA_F32 ? 4 : 2);
  const Bytes ins[] = {{k, n}, {v, n}, {table, table_bytes(B, width)}, {start, (size_t)B * 4},
                       {n_new, (size_t)B * 4}, {cu, ((size_t)B + 1) * 4}};
  const Bytes outs[] = {{pages->k, pool_bytes(*pages)}, {pages->v, pool_bytes(*pages)},
                        {pages->k_scale, scale_bytes(*pages)},
                        {pages->v_scale, scale_bytes(*pages)}, {status, 4}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  PagedRowArgs a = {};
  a.p = pool_of(*pages);
  a.table = table;
  a.width = width;
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.start = start;
  a.n_new = n_new;
  a.cu = cu;
  a.B = B;
  a.T = T;
  a.rows = rows;
  a.status = status;
  return launch_paged_append(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

// Sizes of an attention call, brought to the form the plan wants.
ra_status attn_sizes(const ra_pages& p, bool varlen, int B, int T, long long rows, int H_q,
                     int max_len, int window, int n_sink, PagedAttnArgs* a) {
  if (B <= 0 || T <= 0 || rows <= 0 || H_q <= 0) return RA_ERR_SHAPE;
  if (H_q % p.H_kv != 0 || H_q / p.H_kv > 128) return RA_ERR_SHAPE;
  if (max_len <= 0 || max_len > (1 << 30) || window < 0 || n_sink < 0) return RA_ERR_RANGE;
  // a block's rows, and the launch's blocks, are counted in 32 bits
  if ((long long)T * (H_q / p.H_kv) > (1 << 30) || (long long)B * p.H_kv > kMaxElems)
    return RA_ERR_RANGE;
  const ra_status st = check_tokens(rows, H_q, p.D);
  if (st != RA_OK) return st;
  a->p = pool_of(p);
  a->B = B;
  a->T = T;
  a->rows = (int)rows;
  a->packed = varlen;
  a->H_q = H_q;
  a->max_len = max_len;
  // a window that no query leaves is none
  a->window = window >= max_len ? 0 : window;
  a->n_sink = a->window > 0 ? (n_sink < max_len ? n_sink : max_len) : 0;
  return RA_OK;
}

ra_status launch(const PagedAttnArgs& a, cudaStream_t s) {
  const ra_status st = a.block_rows <= 16 ? launch_paged_rows(a, s) : launch_paged_tiles(a, s);
  return st != RA_OK || a.n_split == 1 ? st : launch_paged_join(a, s);
}

ra_status attn(const void* q, const ra_pages* pages, const int* table, int width, const int* lens,
               const int* cu, bool varlen, void* out, float* lse, int B, int T, long long rows,
               int H_q, int max_len, int window, int n_sink, float scale, int dtype,
               void* workspace, size_t workspace_bytes, int* status, void* stream) {
  if (!q || !lens || !out || (varlen && !cu)) return RA_ERR_NULL;
  if (dtype != RA_BF16) return RA_ERR_DTYPE;
  ra_status st = check_pages(pages, table, width);
  if (st != RA_OK) return st;
  PagedAttnArgs a = {}, few = {};
  st = attn_sizes(*pages, varlen, B, T, rows, H_q, max_len, window, n_sink, &a);
  if (st != RA_OK) return st;
  if (max_len > (long long)width * pages->page) return RA_ERR_RANGE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return RA_ERR_ALIGN;
  if (!aligned(lens, 4) || !aligned(cu, 4) || !aligned(lse, 4) || !aligned(status, 4))
    return RA_ERR_ALIGN;
  a.q = q;
  a.table = table;
  a.width = width;
  a.lens = lens;
  a.cu = cu;
  a.out = out;
  a.lse = lse;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / __builtin_sqrtf((float)pages->D)) * 1.4426950408889634f;
  a.status = status;
  size_t need = 0;
  st = paged_attn_plan(&a, &few, &need);
  if (st != RA_OK) return st;
  if (need > 0 && !workspace) return RA_ERR_NULL;
  if (workspace_bytes < need) return RA_ERR_BUFFER;
  const size_t n = (size_t)rows * H_q;
  const Bytes ins[] = {{q, n * pages->D * 2}, {pages->k, pool_bytes(*pages)},
                       {pages->v, pool_bytes(*pages)}, {pages->k_scale, scale_bytes(*pages)},
                       {pages->v_scale, scale_bytes(*pages)}, {table, table_bytes(B, width)},
                       {lens, (size_t)B * 4}, {cu, ((size_t)B + 1) * 4}};
  const Bytes outs[] = {{out, n * pages->D * 2}, {lse, n * 4}, {workspace, need}, {status, 4}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (few.n_items > 0) {
    paged_attn_place(&few, workspace);
    st = launch(few, s);
    if (st != RA_OK) return st;
  }
  for (long long b0 = 0; b0 < B; b0 += a.n_group) {
    PagedAttnArgs group;
    st = paged_attn_group(a, (int)b0, &group);
    if (st != RA_OK) return st;
    paged_attn_place(&group, workspace);
    st = launch(group, s);
    if (st != RA_OK) return st;
  }
  return RA_OK;
}

}  // namespace

extern "C" {

ra_status paged_append(const ra_pages* pages, const int* table, int width, const void* k,
                       const void* v, const int* start, const int* n_new, int B, int T, int dtype,
                       int* dev_status, void* stream) {
  return append(pages, table, width, k, v, start, n_new, nullptr, B, T, (long long)B * T, dtype,
                dev_status, stream);
}

ra_status paged_append_varlen(const ra_pages* pages, const int* table, int width, const void* k,
                              const void* v, const int* start, const int* cu_seqlens, int n_seq,
                              int total, int dtype, int* dev_status, void* stream) {
  if (!cu_seqlens) return RA_ERR_NULL;
  return append(pages, table, width, k, v, start, nullptr, cu_seqlens, n_seq, 1, total, dtype,
                dev_status, stream);
}

ra_status paged_read(const ra_pages* pages, const int* table, int width, const int* start, void* k,
                     void* v, int B, int T, int dtype, int* dev_status, void* stream) {
  if (!k && !v) return RA_ERR_NULL;
  if (dtype != RA_BF16 && dtype != RA_F32) return RA_ERR_DTYPE;
  ra_status st = check_pages(pages, table, width);
  if (st != RA_OK) return st;
  if (B <= 0 || T <= 0) return RA_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16)) return RA_ERR_ALIGN;
  if (!aligned(start, 4) || !aligned(dev_status, 4)) return RA_ERR_ALIGN;
  st = check_tokens((long long)B * T, pages->H_kv, pages->D);
  if (st != RA_OK) return st;
  const size_t n = (size_t)B * T * pages->H_kv * pages->D * (dtype == RA_F32 ? 4 : 2);
  const Bytes ins[] = {{pages->k, pool_bytes(*pages)}, {pages->v, pool_bytes(*pages)},
                       {pages->k_scale, scale_bytes(*pages)},
                       {pages->v_scale, scale_bytes(*pages)}, {table, table_bytes(B, width)},
                       {start, (size_t)B * 4}};
  const Bytes outs[] = {{k, n}, {v, n}, {dev_status, 4}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  PagedRowArgs a = {};
  a.p = pool_of(*pages);
  a.table = table;
  a.width = width;
  a.k = k;
  a.v = v;
  a.start = start;
  a.B = B;
  a.T = T;
  a.rows = (long long)B * T;
  a.status = dev_status;
  return launch_paged_read(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

ra_status paged_attn_workspace(const ra_pages* pages, int B, int S_q, int total, int H_q,
                               int max_len, int window, int n_sink, int varlen, size_t* bytes) {
  if (!bytes) return RA_ERR_NULL;
  ra_status st = check_sizes(pages);
  if (st != RA_OK) return st;
  PagedAttnArgs a = {}, few = {};
  st = attn_sizes(*pages, varlen != 0, B, S_q, varlen ? total : (long long)B * S_q, H_q, max_len,
                  window, n_sink, &a);
  if (st != RA_OK) return st;
  return paged_attn_plan(&a, &few, bytes);
}

ra_status paged_attn(const void* q, const ra_pages* pages, const int* table, int width,
                     const int* lens, void* out, float* lse, int B, int S_q, int H_q, int max_len,
                     int window, int n_sink, float scale, int dtype, void* workspace,
                     size_t workspace_bytes, int* dev_status, void* stream) {
  return attn(q, pages, table, width, lens, nullptr, false, out, lse, B, S_q, (long long)B * S_q,
              H_q, max_len, window, n_sink, scale, dtype, workspace, workspace_bytes, dev_status,
              stream);
}

ra_status paged_attn_varlen(const void* q, const ra_pages* pages, const int* table, int width,
                            const int* lens, const int* cu_seqlens, void* out, float* lse,
                            int n_seq, int total, int max_seqlen, int H_q, int max_len, int window,
                            int n_sink, float scale, int dtype, void* workspace,
                            size_t workspace_bytes, int* dev_status, void* stream) {
  return attn(q, pages, table, width, lens, cu_seqlens, true, out, lse, n_seq, max_seqlen, total,
              H_q, max_len, window, n_sink, scale, dtype, workspace, workspace_bytes, dev_status,
              stream);
}

}  // extern "C"
