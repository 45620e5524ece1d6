// extern "C" entry points of the 4-bit key/value cache: argument checks on
// the host, then one launcher.
#include <cstdint>

#include "host_checks.h"
#include "kv4_internal.h"
#include "ra_internal.h"

using namespace ra;

namespace {

// Bytes of one of a call's two token tensors, code tensors, meta tensors.
size_t token_bytes(const Kv4RowArgs& a, int dtype) {
  return (size_t)a.B * a.T * a.H_kv * a.D * (dtype == RA_F32 ? 4 : 2);
}
template <class Args>
size_t code_bytes(const Args& a) {
  return (size_t)a.B * a.H_kv * a.C * (a.D / 2);
}
template <class Args>
size_t meta_bytes(const Args& a) {
  return (size_t)a.B * a.H_kv * a.C * (a.D / kKv4Group) * 4;
}

ra_status check_cache(const Kv4Cache& c, int B, int H_kv, int D, int C) {
  if (!c.kc || !c.km || !c.vc || !c.vm) return RA_ERR_NULL;
  if (B <= 0 || H_kv <= 0 || C <= 0) return RA_ERR_SHAPE;
  if (D != 64 && D != 128) return RA_ERR_HEADDIM;
  if (C % kKv4SlotAlign != 0) return RA_ERR_SHAPE;
  if (!aligned(c.kc, 16) || !aligned(c.vc, 16) || !aligned(c.km, 16) || !aligned(c.vm, 16))
    return RA_ERR_ALIGN;
  // slots and their rows are counted in 64 bits; a head's slots in 32
  if ((long long)B * H_kv > kMaxElems) return RA_ERR_RANGE;
  return RA_OK;
}

Kv4Cache cache_of(void* kc, void* km, void* vc, void* vm) {
  return {static_cast<uint8_t*>(kc), static_cast<uint32_t*>(km), static_cast<uint8_t*>(vc),
          static_cast<uint32_t*>(vm)};
}
Kv4Cache cache_of(const void* kc, const void* km, const void* vc, const void* vm) {
  return cache_of(const_cast<void*>(kc), const_cast<void*>(km), const_cast<void*>(vc),
                  const_cast<void*>(vm));
}

ra_status check_rows(const Kv4RowArgs& a, int dtype) {
  if (dtype != RA_BF16 && dtype != RA_F32) return RA_ERR_DTYPE;
  ra_status st = check_cache(a.c, a.B, a.H_kv, a.D, a.C);
  if (st != RA_OK) return st;
  if (a.T <= 0) return RA_ERR_SHAPE;
  if (!aligned(a.k, 16) || !aligned(a.v, 16)) return RA_ERR_ALIGN;
  if (!aligned(a.start, 4) || !aligned(a.n_new, 4) || !aligned(a.status, 4)) return RA_ERR_ALIGN;
  if ((long long)a.B * a.T > kMaxElems || (long long)a.B * a.T * a.H_kv > kMaxElems ||
      (long long)a.B * a.T * a.H_kv * a.D > kMaxElems)
    return RA_ERR_RANGE;
  return RA_OK;
}

// Sizes of an attention call, brought to the form the plan wants.
ra_status attn_sizes(int B, int S_q, int H_q, int H_kv, int D, int C, int max_len, int window,
                     int n_sink, Kv4AttnArgs* a) {
  if (B <= 0 || S_q <= 0 || H_q <= 0 || H_kv <= 0 || C <= 0) return RA_ERR_SHAPE;
  if (H_q % H_kv != 0 || C % kKv4SlotAlign != 0) return RA_ERR_SHAPE;
  if (D != 64 && D != 128) return RA_ERR_HEADDIM;
  if (max_len <= 0 || max_len > C || window < 0 || n_sink < 0) return RA_ERR_RANGE;
  if ((long long)B * S_q > kMaxElems || (long long)B * S_q * H_q > kMaxElems ||
      (long long)B * S_q * H_q * D > kMaxElems || C > (1 << 30))
    return RA_ERR_RANGE;
  a->B = B; a->S_q = S_q; a->H_q = H_q; a->H_kv = H_kv; a->D = D; a->C = C;
  a->max_len = max_len;
  // a window that no query leaves is none
  a->window = window >= max_len ? 0 : window;
  a->n_sink = a->window > 0 ? (n_sink < max_len ? n_sink : max_len) : 0;
  return RA_OK;
}

}  // namespace

extern "C" {

ra_status kv4_append(const void* k, const void* v, void* k_codes, void* k_meta, void* v_codes,
                     void* v_meta, const int* start, const int* n_new, int B, int T, int H_kv,
                     int D, int C, int dtype, int* dev_status, void* stream) {
  if (!k || !v || !start) return RA_ERR_NULL;
  Kv4RowArgs a = {};
  a.c = cache_of(k_codes, k_meta, v_codes, v_meta);
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.start = start;
  a.n_new = n_new;
  a.B = B; a.T = T; a.H_kv = H_kv; a.D = D; a.C = C;
  a.status = dev_status;
  ra_status st = check_rows(a, dtype);
  if (st != RA_OK) return st;
  const Bytes ins[] = {{k, token_bytes(a, dtype)}, {v, token_bytes(a, dtype)},
                       {start, (size_t)B * 4}, {n_new, (size_t)B * 4}};
  const Bytes outs[] = {{k_codes, code_bytes(a)}, {k_meta, meta_bytes(a)},
                        {v_codes, code_bytes(a)}, {v_meta, meta_bytes(a)}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  return launch_kv4_append(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

ra_status kv4_read(const void* k_codes, const void* k_meta, const void* v_codes,
                   const void* v_meta, const int* start, void* k, void* v, int B, int T,
                   int H_kv, int D, int C, int dtype, int* dev_status, void* stream) {
  if (!k && !v) return RA_ERR_NULL;
  Kv4RowArgs a = {};
  a.c = cache_of(k_codes, k_meta, v_codes, v_meta);
  a.k = k;
  a.v = v;
  a.start = start;
  a.B = B; a.T = T; a.H_kv = H_kv; a.D = D; a.C = C;
  a.status = dev_status;
  ra_status st = check_rows(a, dtype);
  if (st != RA_OK) return st;
  const Bytes ins[] = {{k_codes, code_bytes(a)}, {k_meta, meta_bytes(a)}, {v_codes, code_bytes(a)},
                       {v_meta, meta_bytes(a)}, {start, (size_t)B * 4}};
  const Bytes outs[] = {{k, token_bytes(a, dtype)}, {v, token_bytes(a, dtype)}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  return launch_kv4_read(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

ra_status kv4_attn_workspace(int B, int S_q, int H_q, int H_kv, int D, int C, int max_len,
                             int window, int n_sink, int with_score, size_t* bytes) {
  if (!bytes) return RA_ERR_NULL;
  Kv4AttnArgs a = {};
  const ra_status st = attn_sizes(B, S_q, H_q, H_kv, D, C, max_len, window, n_sink, &a);
  if (st != RA_OK) return st;
  return kv4_attn_plan(&a, with_score != 0, bytes);
}

ra_status kv4_attn(const void* q, const void* k_codes, const void* k_meta, const void* v_codes,
                   const void* v_meta, const int* lens, void* out, float* lse, float* score,
                   int B, int S_q, int H_q, int H_kv, int D, int C, int max_len, int window,
                   int n_sink, float scale, int dtype, void* workspace, size_t workspace_bytes,
                   int* dev_status, void* stream) {
  if (!q || !lens || !out) return RA_ERR_NULL;
  if (dtype != RA_BF16) return RA_ERR_DTYPE;
  Kv4AttnArgs a = {};
  ra_status st = attn_sizes(B, S_q, H_q, H_kv, D, C, max_len, window, n_sink, &a);
  if (st != RA_OK) return st;
  a.c = cache_of(k_codes, k_meta, v_codes, v_meta);
  st = check_cache(a.c, B, H_kv, D, C);
  if (st != RA_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return RA_ERR_ALIGN;
  if (!aligned(lens, 4) || !aligned(lse, 4) || !aligned(score, 4) || !aligned(dev_status, 4))
    return RA_ERR_ALIGN;
  size_t need = 0;
  st = kv4_attn_plan(&a, score != nullptr, &need);
  if (st != RA_OK) return st;
  if (need > 0 && !workspace) return RA_ERR_NULL;
  if (workspace_bytes < need) return RA_ERR_BUFFER;
  const size_t rows = (size_t)B * S_q * H_q;
  const Bytes ins[] = {{q, rows * D * 2}, {k_codes, code_bytes(a)}, {k_meta, meta_bytes(a)},
                       {v_codes, code_bytes(a)}, {v_meta, meta_bytes(a)}, {lens, (size_t)B * 4}};
  const Bytes outs[] = {{out, rows * D * 2}, {lse, rows * 4},
                        {score, (size_t)B * H_kv * C * 4}, {workspace, need}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  a.q = q;
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  a.score = score;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / __builtin_sqrtf((float)D)) * 1.4426950408889634f;
  // partial outputs, their (maximum, sum), the logits, the rows' log-sums: each a
  // multiple of 16 bytes
  float* ws = static_cast<float*>(workspace);
  const size_t parts = (size_t)B * H_kv * a.n_rb * a.n_split * a.rows;
  a.part_o = ws;
  if (a.n_split > 1) ws += parts * D;
  a.part_ml = ws;
  if (a.n_split > 1) ws += parts * 2;
  a.logits = ws;
  a.row_lse2 = ws + (size_t)B * H_kv * a.n_rb * a.slots * a.log_rows;
  a.status = dev_status;
  return launch_kv4_attn(a, reinterpret_cast<cudaStream_t>(stream));
}

ra_status kv4_evict(const void* k_codes, const void* k_meta, const void* v_codes,
                    const void* v_meta, const float* score, const int* lens, void* dst_k_codes,
                    void* dst_k_meta, void* dst_v_codes, void* dst_v_meta, float* dst_score,
                    int* dst_lens, int* kept, int B, int H_kv, int D, int C, int C_dst,
                    int budget, int n_sink, int n_recent, int* dev_status, void* stream) {
  if (!score || !lens || !dst_lens || !kept) return RA_ERR_NULL;
  Kv4EvictArgs a = {};
  a.src = cache_of(k_codes, k_meta, v_codes, v_meta);
  a.dst = cache_of(dst_k_codes, dst_k_meta, dst_v_codes, dst_v_meta);
  ra_status st = check_cache(a.src, B, H_kv, D, C);
  if (st != RA_OK) return st;
  st = check_cache(a.dst, B, H_kv, D, C_dst);
  if (st != RA_OK) return st;
  if (budget <= 0 || budget > C_dst || n_sink < 0 || n_recent < 0 ||
      (long long)n_sink + n_recent > budget || C > (1 << 30))
    return RA_ERR_RANGE;
  if (!aligned(score, 4) || !aligned(lens, 4) || !aligned(dst_score, 4) ||
      !aligned(dst_lens, 4) || !aligned(kept, 4) || !aligned(dev_status, 4))
    return RA_ERR_ALIGN;
  a.B = B; a.H_kv = H_kv; a.D = D; a.C = C; a.C_dst = C_dst;
  a.budget = budget; a.n_sink = n_sink; a.n_recent = n_recent;
  // nothing that is written may be part of what is read
  const size_t dst_rows = (size_t)B * H_kv * C_dst;
  const size_t code = dst_rows * (D / 2), meta = dst_rows * (D / kKv4Group) * 4;
  const Bytes ins[] = {{k_codes, code_bytes(a)}, {k_meta, meta_bytes(a)}, {v_codes, code_bytes(a)},
                       {v_meta, meta_bytes(a)}, {score, (size_t)B * H_kv * C * 4},
                       {lens, (size_t)B * 4}};
  const Bytes outs[] = {{dst_k_codes, code}, {dst_k_meta, meta}, {dst_v_codes, code},
                        {dst_v_meta, meta}, {dst_score, dst_rows * 4},
                        {dst_lens, (size_t)B * 4}, {kept, (size_t)B * H_kv * budget * 4}};
  if (overlap(outs, ins)) return RA_ERR_BUFFER;
  st = check_device(nullptr);
  if (st != RA_OK) return st;
  a.score = score;
  a.dst_score = dst_score;
  a.lens = lens;
  a.dst_lens = dst_lens;
  a.kept = kept;
  a.status = dev_status;
  return launch_kv4_evict(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
