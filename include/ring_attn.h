/*
 * ring_attn.h - C ABI of the GB300 (sm_103a) exact ring-attention library.
 *
 * What it computes. Glossary "sequence parallelism transformers":
 *  - §Sequence Parallelism Fundamentals ("Sequence Dimension Splitting"): the
 *    length-S sequence is cut into P chunks, one per rank. Here the ranks are
 *    virtual: all P live on the one GPU running the call.
 *  - §Ring Attention: each rank keeps its query block; at step t it attends
 *    to the key/value block that started on rank (r - t) mod P (blocks move
 *    from rank i to i+1 each step) and accumulates the outputs; after P
 *    steps the result equals full softmax attention.
 *  - §Implementation Considerations ("Numerical Stability", "Load
 *    Balancing"): partial results are combined with an exact log-sum-exp
 *    merge; the zig-zag chunk order (2P halves, rank r owns halves r and
 *    2P-1-r) balances causal work across ranks.
 * Uneven lengths follow the mvp-engine "sequence-parallel" skill (seq_len
 * divisible by the split, else pad explicitly and mask): the sequence counts
 * as padded to the next multiple of P (contiguous) or 2P (zig-zag), every
 * chunk (half) spans L = ceil(S/P) (ceil(S/2P)) positions starting at a
 * multiple of L, and the padding positions (S and beyond) hold no token:
 * they are never read, never written and never attended to. A trailing
 * chunk can therefore be short or empty. The padding is virtual; tensors
 * keep exactly S rows.
 *
 * For each batch b, query head h and query position i, with key/value head
 * hk = h / (H_q / H_kv) and allowed keys A(i) = {0..S-1} (non-causal) or
 * {0..i} (causal, global positions):
 *     lse[b,h,i] = log sum_{j in A(i)} exp(scale * <q_i, k_j>)      (natural log)
 *     out[b,i,h] = sum_{j in A(i)} exp(scale * <q_i, k_j> - lse) * v_j
 *
 * Layouts (all row-major, contiguous, "BSHD": sequence is dimension 1):
 *     q, out      [B, S, H_q,  D]
 *     k, v        [B, S, H_kv, D]
 *     lse         [B, H_q, S]            float32
 * Element types: RA_BF16 (bfloat16 in and out, float32 accumulation) or
 * RA_F32 (float32 throughout).
 *
 * Conventions shared by every entry point:
 *  - Every data pointer is a DEVICE pointer on the current CUDA device, owned
 *    by the caller. Tensor pointers (q, k, v, out, o_*) are 16-byte aligned;
 *    lse, visit logs and status words 4-byte aligned (else RA_ERR_ALIGN).
 *    The library allocates no device memory and keeps no state between calls
 *    except read-only per-device facts and the one scratch array that
 *    ring_attn_bwd_noalloc uses (module memory, held until exit).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). Calls enqueue work and return; they never synchronise.
 *  - Arguments are checked on the host before anything is enqueued; on error
 *    nothing is launched and the status says why. A failed launch returns
 *    RA_ERR_LAUNCH. A device-side bounded wait that expired is reported in
 *    `dev_status` (where the call takes one) as RA_ERR_TIMEOUT, after the
 *    stream has run the kernel.
 *  - Two builds export this same ABI: libringattn.so and the bounds-checked
 *    libringattn_debug.so. In the checked build every global-memory access
 *    a kernel computes from indices is tested against its tensor's extent.
 *    A violation skips the access and sets RA_ERR_RANGE in `dev_status`;
 *    there is no trap. In the release build the checks compile away.
 *  - `scale <= 0` means 1/sqrt(D).
 *  - Tensors stay in natural token order in every chunk order: the order only
 *    decides which virtual rank owns which tokens and the sequence of steps.
 */
#ifndef RING_ATTN_H
#define RING_ATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  RA_OK = 0,
  RA_ERR_NULL = 1,     /* a required pointer is NULL                              */
  RA_ERR_SHAPE = 2,    /* a size <= 0, H_q % H_kv != 0, merge n out of range,
                          a cache capacity that is not a multiple of 16          */
  RA_ERR_HEADDIM = 3,  /* D is not 64 or 128 (attention), not 32-256 (merge)     */
  RA_ERR_ALIGN = 4,    /* a data pointer is not 16-byte aligned                    */
  RA_ERR_DTYPE = 5,    /* unknown dtype or order value                             */
  RA_ERR_DEVICE = 6,   /* current device is not compute capability 10.3            */
  RA_ERR_LAUNCH = 7,   /* CUDA runtime error while preparing or launching          */
  RA_ERR_TIMEOUT = 8,  /* a device-side bounded wait expired (dev_status only)     */
  RA_ERR_BUFFER = 9,   /* a caller buffer is too small; caches: one that a call
                          writes overlaps another of its buffers                 */
  RA_ERR_RANGE = 10,   /* a size overflows 32-bit indexing, or step out of range;
                          in dev_status: a slot without a page (paged_*), or, in
                          the checked build only, a device index out of its
                          tensor's range                                          */
  RA_ERR_SCRATCH = 11  /* the problem needs more scratch than the library's
                          built-in array holds (ring_attn_bwd_noalloc)           */
} ra_status;

/* RA_E4M3 (8 bits) is a type of pages only. */
typedef enum { RA_BF16 = 0, RA_F32 = 1, RA_E4M3 = 2 } ra_dtype;
typedef enum { RA_ORDER_CONTIGUOUS = 0, RA_ORDER_ZIGZAG = 1 } ra_order;

/* Classes of a (query set, key set) pair under the causal rule j <= i. */
enum { RA_CLASS_SKIP = 0, RA_CLASS_FULL = 1, RA_CLASS_PARTIAL = 2 };

/* Largest n accepted by attn_lse_merge_n. */
#define RA_MERGE_MAX_N 16

/*
 * ring_attn_fwd - exact attention computed as a ring of P virtual ranks,
 * bfloat16 inputs and output, contiguous chunk order. Defined by glossary
 * "sequence parallelism transformers", §Ring Attention ("Block-Wise
 * Attention", "Ring Communication", "Computation": each rank keeps its query
 * block, attends to every key/value block as it passes, and accumulates
 * exactly the full-attention result).
 *
 * All P ring steps run inside one kernel launch: every query tile keeps its
 * running (max, sum, unnormalised output) on chip across steps, which is the
 * log-sum-exp merge of the per-step partials done in registers. Under a
 * causal mask, key tiles that lie entirely after the query tile are skipped.
 * `lse` may be NULL (not written). Errors: RA_ERR_NULL (q, k, v or out NULL),
 * RA_ERR_SHAPE, RA_ERR_HEADDIM, RA_ERR_ALIGN, RA_ERR_RANGE (B*S*H*D beyond
 * 2^31 elements per tensor), RA_ERR_DEVICE, RA_ERR_LAUNCH.
 */
ra_status ring_attn_fwd(const void* q, const void* k, const void* v,
                        void* out, float* lse,
                        int B, int H_q, int H_kv, int S, int D, int P,
                        int causal, float scale, void* stream);

/*
 * ring_attn_fwd_ex - ring_attn_fwd with every option. Defined by the same
 * glossary, §Ring Attention (the per-step partial results of `step`), and
 * §Implementation Considerations ("Load Balancing": the zig-zag `order`).
 *
 * dtype   RA_BF16 (tensor-core path) or RA_F32 (exact float32 CUDA-core path).
 * order   RA_ORDER_CONTIGUOUS (rank r owns [rS/P, (r+1)S/P)) or
 *         RA_ORDER_ZIGZAG (rank r owns halves r and 2P-1-r of length S/2P).
 * step    -1: all P steps, folded on chip (same result as ring_attn_fwd).
 *         t in [0, P): ring step t only. Every rank r attends to the chunk of
 *         rank (r - t) mod P and the call writes that step's PARTIAL result:
 *         `out` is then float32 [B, S, H_q, D] whatever `dtype` is, and `lse`
 *         (required) is the partial lse; rows with no allowed key in that
 *         chunk get out = 0 and lse = -inf. Folding the P partials with
 *         attn_lse_merge / attn_lse_merge_n gives the full result.
 * visit_log  NULL, or a device int32 buffer of ring_attn_visit_log_len(...)
 *         elements: for every (b, h, query tile) the key tiles the kernel
 *         visited, in visit order (layout at ring_attn_visit_log_len).
 * dev_status NULL, or a device int the kernel sets to RA_ERR_TIMEOUT if one of
 *         its bounded waits expired (it is never cleared by the library; the
 *         caller zeroes it).
 */
ra_status ring_attn_fwd_ex(const void* q, const void* k, const void* v,
                           void* out, float* lse,
                           int B, int H_q, int H_kv, int S, int D, int P,
                           int causal, float scale,
                           int dtype, int order, int step,
                           int* visit_log, int* dev_status, void* stream);

/*
 * ring_attn_fwd_varlen - ring attention over a batch of packed sequences of
 * different lengths.
 *
 * Sequence b occupies rows [cu_seqlens[b], cu_seqlens[b+1]) of the packed
 * tensors and is its own ring problem: its S_b tokens are cut into P chunks
 * (or 2P halves) of ceil(S_b / P) (ceil(S_b / 2P)) positions, padded like an
 * uneven S (see above), and its queries attend only to its own keys. Layouts:
 *     q, out   [total, H_q,  D]      k, v   [total, H_kv, D]
 *     lse      [H_q, total]          float32 (may be NULL)
 * cu_seqlens: DEVICE int32 array of n_seq + 1 nondecreasing offsets with
 * cu_seqlens[0] = 0 and cu_seqlens[n_seq] = total. max_seqlen >= every S_b
 * (it sizes the launch). The kernels clamp offsets into [0, total] and
 * lengths into [0, max_seqlen], so a malformed array never moves an access
 * outside the tensors (its sequences are then simply wrong). A sequence of
 * length 0 writes nothing. dtype RA_BF16 or RA_F32; all steps; no visit log.
 * Errors: RA_ERR_NULL, RA_ERR_SHAPE (n_seq, total or max_seqlen <= 0,
 * H_q % H_kv), RA_ERR_HEADDIM, RA_ERR_ALIGN (cu_seqlens 4-byte), RA_ERR_DTYPE,
 * RA_ERR_RANGE, RA_ERR_DEVICE, RA_ERR_LAUNCH.
 */
ra_status ring_attn_fwd_varlen(const void* q, const void* k, const void* v,
                               void* out, float* lse, const int* cu_seqlens,
                               int n_seq, int total, int max_seqlen,
                               int H_q, int H_kv, int D, int P, int causal,
                               float scale, int dtype, int order,
                               int* dev_status, void* stream);

/*
 * ring_attn_fwd_ulysses - exact attention in the sequence-parallel layout of
 * Ulysses-style sequence parallelism (glossary "sequence parallelism
 * transformers", §Ulysses Sequence Parallelism: an all-to-all turns the
 * sequence-parallel layout into a head-parallel one, each rank computes full
 * attention for its subset of heads, and a second all-to-all restores the
 * sequence-parallel layout).
 *
 * Virtual rank p holds the contiguous shard of C = ceil(S/P) positions
 * [p*C, min((p+1)*C, S)) of every batch and head, and the tensors are the P
 * ranks' local tensors stacked:
 *     q, out  [P, B, C, H_q,  D]      k, v  [P, B, C, H_kv, D]
 *     lse     [P, B, H_q, C]          float32 (may be NULL)
 * (rows of a last, partly filled shard past S are neither read nor written).
 * Rank r's head-parallel work is heads [r*H_q/P, (r+1)*H_q/P) (and the kv
 * heads they read) over all S positions. On one GPU both all-to-alls are an
 * index map inside the kernel's loads and stores: nothing is copied. The
 * result is full attention, as for every other entry point. H_q and H_kv
 * must be multiples of P (else RA_ERR_SHAPE). dtype RA_BF16 or RA_F32; all
 * steps; no visit log. Errors as ring_attn_fwd_ex.
 */
ra_status ring_attn_fwd_ulysses(const void* q, const void* k, const void* v,
                                void* out, float* lse,
                                int B, int H_q, int H_kv, int S, int D, int P,
                                int causal, float scale, int dtype,
                                int* dev_status, void* stream);

/*
 * ring_attn_visit_log_len - size of the visit log of ring_attn_fwd_ex.
 *
 * The kernel for `dtype` cuts every chunk (contiguous) or half (zig-zag) of
 * length L into query and key tiles of `*tile_rows` rows (the last one shorter
 * when L is not a multiple). Tiles are numbered globally: the segment's index
 * in position order times `*tiles_per_segment` plus the tile's index in it.
 * The log holds, for each (b, h, query tile id), `*stride` ints: the number
 * of visits n, then n entries of 4 ints (step, source rank, key tile id,
 * class). Total length = B * H_q * n_query_tiles * stride, returned in *len.
 * Host-only; never touches the GPU.
 */
ra_status ring_attn_visit_log_len(int B, int H_q, int S, int D, int P,
                                  int dtype, int order,
                                  int* tile_rows, int* tiles_per_segment,
                                  int* n_query_tiles, int* stride,
                                  long long* len);

/*
 * ring_attn_bwd_workspace - bytes of device workspace ring_attn_bwd needs
 * for this shape (written to *bytes). Host only; never touches the GPU.
 * The workspace holds two float32 statistics per query row of the forward
 * result, negated (-lse in base 2 and -delta_i, delta_i = <dout_i, out_i>),
 * stored per (b, h, query tile) with every tile padded to the kernels' tile
 * height; its contents are the library's own and only its phases read them.
 * Errors: RA_ERR_NULL (bytes NULL), RA_ERR_SHAPE, RA_ERR_HEADDIM,
 * RA_ERR_DTYPE (order), RA_ERR_RANGE.
 */
ra_status ring_attn_bwd_workspace(int B, int H_q, int S, int D, int P,
                                  int order, size_t* bytes);

/*
 * ring_attn_bwd - gradients of ring attention with respect to q, k and v,
 * bfloat16 (glossary "sequence parallelism transformers", §Implementation
 * Considerations: the backward pass runs over the same ring as the forward).
 *
 * For an upstream gradient dout = dL/d(out), with p_ij = exp(s_ij - lse_i)
 * on the allowed pairs of the forward definition above:
 *     dV_j = sum_i p_ij dout_i
 *     ds_ij = p_ij (<dout_i, v_j> - delta_i),   delta_i = <dout_i, out_i>
 *     dQ_i = scale * sum_j ds_ij k_j,   dK_j = scale * sum_i ds_ij q_i
 * A key/value head's dk and dv sum over the query heads of its group.
 * Ring structure: the dq of a query tile is accumulated on chip over the key
 * tiles in the forward's ring order; the dk, dv of a key tile over the query
 * tiles of ranks src, src+1, ..., src+P-1 (mod P) in step order, which is
 * the order in which the block, travelling the ring, meets them on its way
 * back to its owner. All P steps run; there is no single-step mode.
 *
 * q [B,S,H_q,D], k and v [B,S,H_kv,D], out and dout [B,S,H_q,D]: bfloat16
 *   device tensors; out and lse are the forward's results for the same
 *   arguments (lse float32 [B,H_q,S], natural log, as ring_attn_fwd_ex
 *   writes it).
 * dq [B,S,H_q,D], dk and dv [B,S,H_kv,D]: bfloat16, overwritten (not
 *   accumulated into). They must not overlap any input.
 * dtype RA_BF16 only (RA_ERR_DTYPE otherwise); order as in ring_attn_fwd_ex.
 * workspace / workspace_bytes: a device buffer of at least
 *   ring_attn_bwd_workspace(...) bytes (else RA_ERR_BUFFER), 16-byte aligned,
 *   owned by the caller; its contents on entry are ignored and on return
 *   undefined. The call allocates no memory of its own.
 * dev_status as in ring_attn_fwd_ex.
 * Errors: as ring_attn_fwd_ex, plus RA_ERR_BUFFER.
 */
ra_status ring_attn_bwd(const void* q, const void* k, const void* v,
                        const void* out, const float* lse, const void* dout,
                        void* dq, void* dk, void* dv,
                        int B, int H_q, int H_kv, int S, int D, int P,
                        int causal, float scale, int dtype, int order,
                        void* workspace, size_t workspace_bytes,
                        int* dev_status, void* stream);

/* Size of the scratch array built into the library for ring_attn_bwd_noalloc. */
#define RA_BWD_NOALLOC_MAX_BYTES (8u << 20)

/*
 * ring_attn_bwd_noalloc - ring_attn_bwd without a caller workspace; the call
 * allocates no memory at all. The pages have no counterpart to this entry
 * point: it exists for callers that cannot call cudaMalloc, such as a plugin
 * whose host framework owns the device memory through its own pool and hands
 * it no workspace, or a latency-critical path on which cudaMalloc / cudaFree
 * may synchronise the device.
 *
 * Arguments and results are those of ring_attn_bwd without `workspace` and
 * `workspace_bytes`: the caller still passes every input and output. The
 * workspace lives instead in a file-scope device array of
 * RA_BWD_NOALLOC_MAX_BYTES (8 MiB) that every GPU which loads the library
 * holds until the process exits. It fits ring_attn_bwd_workspace(...) <=
 * 8 MiB, i.e. up to 2^20 tile-padded query rows (B * H_q * S rounded up per
 * 128-row tile of each chunk or half); the S = 32768, H_q = 32 causal
 * zig-zag problem fits exactly. A larger problem returns RA_ERR_SCRATCH
 * before anything is launched.
 *  - The first call on a device looks up the array's device address (with
 *    that device current) and caches it; make that first call before any
 *    stream capture begins.
 *  - Every call shares the one array and it keeps the last call's contents.
 *    Nothing in it has to start at zero: the prep phase overwrites every
 *    entry a call reads. Calls whose work overlaps on the GPU (two streams,
 *    or two host threads on one device) race on the array: serialise them.
 *  - dev_status and every other convention as ring_attn_bwd.
 * Errors: as ring_attn_bwd, with RA_ERR_SCRATCH in place of RA_ERR_BUFFER.
 */
ra_status ring_attn_bwd_noalloc(const void* q, const void* k, const void* v,
                                const void* out, const float* lse, const void* dout,
                                void* dq, void* dk, void* dv,
                                int B, int H_q, int H_kv, int S, int D, int P,
                                int causal, float scale, int dtype, int order,
                                int* dev_status, void* stream);

/* Phases of the backward pass (bit flags) for ring_attn_bwd_ex. */
enum { RA_BWD_PREP = 1, RA_BWD_DKDV = 2, RA_BWD_DQ = 4, RA_BWD_ALL = 7 };

/*
 * ring_attn_bwd_ex - ring_attn_bwd restricted to the phases in `phases` (a
 * nonzero OR of RA_BWD_*, else RA_ERR_RANGE), enqueued in the order prep,
 * dK/dV, dQ; one kernel launch per phase. The prep phase writes the
 * workspace (-lse in base 2 and -delta per query row); the dK/dV phase
 * (writes dk, dv) and the dQ phase (writes dq) read it and are independent
 * of each other, so after the prep phase they may run on two streams at
 * once. A phase needs the prep phase of the same arguments to have run
 * before it on the device. ring_attn_bwd is phases = RA_BWD_ALL.
 */
ra_status ring_attn_bwd_ex(const void* q, const void* k, const void* v,
                           const void* out, const float* lse, const void* dout,
                           void* dq, void* dk, void* dv,
                           int B, int H_q, int H_kv, int S, int D, int P,
                           int causal, float scale, int dtype, int order,
                           void* workspace, size_t workspace_bytes, int phases,
                           int* dev_status, void* stream);

/*
 * ring_attn_bwd_varlen - ring_attn_bwd for packed sequences, with the
 * layouts and cu_seqlens / max_seqlen conventions of ring_attn_fwd_varlen
 * (dout, dq like q; dk, dv like k; lse [H_q, total]). The workspace size is
 * ring_attn_bwd_workspace(n_seq, H_q, max_seqlen, D, P, order, ...).
 * bf16 only. Errors: as ring_attn_fwd_varlen, plus RA_ERR_BUFFER.
 */
ra_status ring_attn_bwd_varlen(const void* q, const void* k, const void* v,
                               const void* out, const float* lse, const void* dout,
                               void* dq, void* dk, void* dv, const int* cu_seqlens,
                               int n_seq, int total, int max_seqlen,
                               int H_q, int H_kv, int D, int P, int causal,
                               float scale, int dtype, int order,
                               void* workspace, size_t workspace_bytes,
                               int* dev_status, void* stream);

/*
 * ring_attn_bwd_ulysses - ring_attn_bwd for tensors in the sequence-parallel
 * layout of ring_attn_fwd_ulysses (q, out, dout, dq [P, B, C, H_q, D]; k, v,
 * dk, dv [P, B, C, H_kv, D]; lse [P, B, H_q, C]; C = ceil(S/P)). The
 * all-to-alls are again index maps in the loads and stores. H_q and H_kv must
 * be multiples of P. The workspace size is ring_attn_bwd_workspace(B, H_q, S,
 * D, P, RA_ORDER_CONTIGUOUS, ...). bf16 only. Errors: as ring_attn_bwd.
 */
ra_status ring_attn_bwd_ulysses(const void* q, const void* k, const void* v,
                                const void* out, const float* lse, const void* dout,
                                void* dq, void* dk, void* dv,
                                int B, int H_q, int H_kv, int S, int D, int P,
                                int causal, float scale, int dtype,
                                void* workspace, size_t workspace_bytes,
                                int* dev_status, void* stream);

/*
 * ring_attn_fwd_window - attention with a sliding window and a few first
 * tokens that stay visible. The pages have no counterpart; definition and
 * layouts are those of ring_attn_fwd_ex (causal, all steps), with the allowed
 * keys
 *     A(i) = { j <= i : j > i - window  or  j < n_sink }
 * P and order are checked as there and change nothing, not a bit of the result:
 * a window meets the blocks before its own, wherever the ring keeps them.
 * window >= 1 (1: only the query's own token, and the first ones), n_sink >=
 * 0, else RA_ERR_RANGE; values of S and more mean all tokens. A query tile
 * meets only the key tiles that some row of it sees, so the work grows with
 * S * window. dtype RA_BF16 or RA_F32; no visit log. Errors as
 * ring_attn_fwd_ex.
 * Keys and values must be finite where a query does not see them, too: a
 * hidden key has weight 0, and 0 times an infinity is not a number (in the
 * backward so must queries, out and dout).
 * A row that sees a NaN score has NaN in out and in lse.
 * ring_attn_fwd_window_varlen - the same for packed sequences (conventions of
 * ring_attn_fwd_varlen): windows and first tokens are each sequence's own. A
 * sequence's results depend on its own rows only, whatever the others hold;
 * cu_seqlens[n_seq] may be less than `total`: rows behind the last sequence
 * are not written and may hold anything (also in the backward).
 */
ra_status ring_attn_fwd_window(const void* q, const void* k, const void* v,
                               void* out, float* lse, int B, int H_q, int H_kv,
                               int S, int D, int P, int window, int n_sink,
                               float scale, int dtype, int order,
                               int* dev_status, void* stream);
ra_status ring_attn_fwd_window_varlen(const void* q, const void* k, const void* v,
                                      void* out, float* lse, const int* cu_seqlens,
                                      int n_seq, int total, int max_seqlen,
                                      int H_q, int H_kv, int D, int P, int window,
                                      int n_sink, float scale, int dtype, int order,
                                      int* dev_status, void* stream);

/*
 * ring_attn_bwd_window - gradients of ring_attn_fwd_window (formulas and
 * conventions of ring_attn_bwd, sums over A(i)); ring_attn_bwd_window_varlen
 * those of the packed form. RA_BF16 only. The workspace size comes from
 * ring_attn_bwd_window_workspace with the call's sizes (packed: B = n_seq,
 * S = max_seqlen, varlen = 1); beside the row statistics it holds float32
 * parts of dK and dV of the key tiles whose work is shared out: those with
 * first tokens, which the whole sequence sees, and all where key/value heads
 * and tiles are few. Gradients repeat bit for bit. Errors as ring_attn_bwd, RA_ERR_RANGE for window and n_sink.
 */
ra_status ring_attn_bwd_window_workspace(int B, int H_q, int H_kv, int S, int D, int P,
                                         int window, int n_sink, int order, int varlen,
                                         size_t* bytes);
ra_status ring_attn_bwd_window(const void* q, const void* k, const void* v,
                               const void* out, const float* lse, const void* dout,
                               void* dq, void* dk, void* dv,
                               int B, int H_q, int H_kv, int S, int D, int P,
                               int window, int n_sink, float scale, int dtype,
                               int order, void* workspace, size_t workspace_bytes,
                               int* dev_status, void* stream);
ra_status ring_attn_bwd_window_varlen(const void* q, const void* k, const void* v,
                                      const void* out, const float* lse,
                                      const void* dout, void* dq, void* dk, void* dv,
                                      const int* cu_seqlens, int n_seq, int total,
                                      int max_seqlen, int H_q, int H_kv, int D, int P,
                                      int window, int n_sink, float scale, int dtype,
                                      int order, void* workspace,
                                      size_t workspace_bytes, int* dev_status,
                                      void* stream);

/*
 * attn_lse_merge - exact merge of two partial attention results over
 * disjoint key sets (glossary "sequence parallelism transformers",
 * §Ring Attention and §Implementation Considerations):
 *     lse = log(exp(lse_a) + exp(lse_b))
 *     out = exp(lse_a - lse) * o_a + exp(lse_b - lse) * o_b
 * evaluated with the larger lse factored out. A side with lse = -inf
 * contributes nothing; both -inf gives out = 0, lse = -inf.
 * o_a, o_b, out: [B, S, H, D] of `dtype`; lse_a, lse_b, lse: float32
 * [B, H, S]. `out` may alias o_a or o_b and `lse` may alias lse_a or lse_b
 * (each element is read before it is written, by the same thread).
 */
ra_status attn_lse_merge(const void* o_a, const float* lse_a,
                         const void* o_b, const float* lse_b,
                         void* out, float* lse,
                         int B, int H, int S, int D, int dtype, void* stream);

/*
 * attn_lse_merge_n - the same merge over n partials in one pass
 * (1 <= n <= RA_MERGE_MAX_N):
 *     lse = M + log sum_t exp(lse_t - M),  M = max_t lse_t
 *     out = sum_t exp(lse_t - lse) * o_t
 * `o` and `lse` are HOST arrays of n device pointers. Aliasing as for
 * attn_lse_merge. D is 32, 64, 128 or 256 here.
 */
ra_status attn_lse_merge_n(const void* const* o, const float* const* lse,
                           int n, void* out, float* out_lse,
                           int B, int H, int S, int D, int dtype, void* stream);

/*
 * ring_attn_plan - the ring schedule as an int32 table, host only. Defined
 * by glossary "sequence parallelism transformers", §Sequence Parallelism
 * Fundamentals (P chunks of S/P tokens) and §Ring Attention ("Ring
 * Communication": at step t rank r holds the block of rank (r - t) mod P).
 * One row of RA_PLAN_COLS ints per (rank, step), rank-major then step:
 *   rank, step, src = (rank - step) mod P, class of the whole (query chunk,
 *   key chunk) pair, segment length L (padded, see above), first and second
 *   query segment starts,
 *   first and second key segment starts (-1 where a rank owns one segment).
 * `table_len` is the capacity in ints (>= P*P*RA_PLAN_COLS, else
 * RA_ERR_BUFFER). Never touches the GPU.
 */
#define RA_PLAN_COLS 9
ra_status ring_attn_plan(int S, int P, int causal, int order,
                         int* table, size_t table_len);

/*
 * ring_attn_expiry_test - exercises the failure path of the tensor-core
 * kernel's bounded waits; for tests, never needed in normal use.
 * Runs the bf16 kernel on B = H_q = H_kv = 1, D = 128, P = 1, non-causal,
 * 1 <= S <= 4096 (q, k, v, out [1, S, 1, 128] bf16; lse [1, 1, S]) with the
 * load of the first value tile withheld, so the wait for it expires after
 * about two seconds. The kernel then gives up in every role, waits (bounded)
 * for the copies and tensor-core work it issued, frees its tensor memory,
 * returns, and sets *dev_status (device int, required) to RA_ERR_TIMEOUT.
 * `out` and `lse` are left partly unwritten. The CUDA context stays usable.
 * Returns RA_OK when the kernel was launched (the expiry shows in dev_status
 * after the stream has run it), else an argument or launch error.
 */
ra_status ring_attn_expiry_test(const void* q, const void* k, const void* v,
                                void* out, float* lse, int S, int* dev_status,
                                void* stream);

/*
 * The 4-bit key/value cache: what a served sequence has attended to so far,
 * kept at 4.5 bits a value for the decoding steps that follow a prompt. The
 * pages have no counterpart; it continues the forward above (the same
 * definition of attention, the same lse, so that its partial results merge
 * with attn_lse_merge).
 *
 * A cache of capacity C holds, for each sequence b and key/value head, C
 * slots; a slot is one token's key row and value row of D values, in groups
 * of 64 along D:
 *     k_codes, v_codes   [B, H_kv, C, D / 2]      bytes: dimension 2i in the
 *                        low, 2i + 1 in the high half of byte i of a row
 *     k_meta, v_meta     [B, H_kv, C, D / 64, 2]  bfloat16: scale, zero point
 * A code c stands for scale * (c - 8) + zero. C is a multiple of 16, D 64 or
 * 128; the four tensors are 16-byte aligned. How many slots a sequence uses
 * is the caller's `lens` (device int32 [B]); slots past it may hold anything,
 * including NaN. Nothing here reads lens on the host, so a step can be
 * captured into a graph and replayed while lens grows. A tensor that a call
 * writes (its workspace too) may not overlap any other of the call's
 * (RA_ERR_BUFFER).
 *
 * kv4_append - quantises T tokens a sequence, k and v [B, T, H_kv, D] of
 * `dtype` (RA_BF16 or RA_F32), into slots start[b], start[b] + 1, ...
 * (start: device int32 [B]). n_new: NULL, or device int32 [B]: only the first
 * n_new[b] tokens of sequence b count, the rest of a padded batch is not
 * written. Per group, in float32: scale = bf16(max / 15 - min / 15), zero =
 * bf16(min + 8 scale), code = clamp(rint((x - zero) / scale) + 8, 0, 15), or
 * 8 where scale is 0. A group that holds an infinity or a NaN reads back as
 * NaN. A slot outside [0, C) is not written and sets RA_ERR_RANGE in
 * `dev_status` (device int, may be NULL).
 */
ra_status kv4_append(const void* k, const void* v, void* k_codes, void* k_meta,
                     void* v_codes, void* v_meta, const int* start,
                     const int* n_new, int B, int T, int H_kv, int D, int C,
                     int dtype, int* dev_status, void* stream);

/*
 * kv4_read - the values of slots start[b] ... start[b] + T - 1 (start NULL:
 * from slot 0), as k and v [B, T, H_kv, D] of `dtype` (either may be NULL).
 * A slot outside [0, C) gives zeros and sets RA_ERR_RANGE in `dev_status`.
 */
ra_status kv4_read(const void* k_codes, const void* k_meta, const void* v_codes,
                   const void* v_meta, const int* start, void* k, void* v,
                   int B, int T, int H_kv, int D, int C, int dtype,
                   int* dev_status, void* stream);

/* Bytes of workspace kv4_attn needs for these sizes (host only; 0 for short
 * axes without scores). Errors as kv4_attn's sizes. */
ra_status kv4_attn_workspace(int B, int S_q, int H_q, int H_kv, int D, int C,
                             int max_len, int window, int n_sink,
                             int with_score, size_t* bytes);

/*
 * kv4_attn - attention of S_q new tokens a sequence (one in plain decoding)
 * over its cache, which already holds them (append first).
 * lens: device int32 [B], slots in use, the S_q new ones included (clamped to
 * [0, max_len]); max_len in [1, C] bounds them and sizes the launch. Query t
 * of sequence b is at slot p = lens[b] - S_q + t and sees the slots j <= p;
 * with window > 0 only those with j > p - window or j < n_sink (window 0: no
 * window, n_sink is ignored). Slots are counted as they lie, so after an
 * eviction a window counts kept slots. Head h reads key/value head
 * h / (H_q / H_kv). A row that sees no slot gets out = 0, lse = -inf.
 * A row's results depend on the slots that it sees alone, to the bit, whatever
 * the others hold (a later drafted token that is not finite, say); a value that
 * is not finite reaches its own group of 64 dimensions.
 *     q, out  [B, S_q, H_q, D] bfloat16    lse  [B, H_q, S_q] float32 or NULL
 * score: NULL, or float32 [B, H_kv, C]: every slot's attention weight, summed
 * over the queries and the heads of its group, is ADDED to it.
 * dtype RA_BF16; queries of up to 2^90 in magnitude and logits of up to 2^28
 * (beyond them results may not be finite). scale <= 0 means 1 / sqrt(D). The
 * workspace is the caller's, 16-byte aligned; its contents do not matter. Calls
 * that may overlap on the GPU need workspaces of their own. Results repeat bit
 * for bit.
 * Errors: RA_ERR_NULL, RA_ERR_SHAPE, RA_ERR_HEADDIM, RA_ERR_ALIGN,
 * RA_ERR_DTYPE, RA_ERR_RANGE (max_len, window, n_sink, sizes), RA_ERR_BUFFER,
 * RA_ERR_DEVICE, RA_ERR_LAUNCH.
 */
ra_status kv4_attn(const void* q, const void* k_codes, const void* k_meta,
                   const void* v_codes, const void* v_meta, const int* lens,
                   void* out, float* lse, float* score, int B, int S_q, int H_q,
                   int H_kv, int D, int C, int max_len, int window, int n_sink,
                   float scale, int dtype, void* workspace,
                   size_t workspace_bytes, int* dev_status, void* stream);

/*
 * kv4_evict - cuts every sequence down to `budget` slots a head by its
 * accumulated weights, into another cache of capacity C_dst >= budget.
 * Of n = lens[b] > budget slots a head keeps the first n_sink, the last
 * n_recent and, of those between, the budget - n_sink - n_recent with the
 * largest score (score float32 [B, H_kv, C]; among equal scores the lowest
 * slot, NaN below every number). n <= budget keeps all. Kept slots keep their
 * order. Outputs: the four dst tensors' first min(n, budget) slots, dst_score
 * [B, H_kv, C_dst] likewise (may be NULL), dst_lens [B] = min(n, budget), and
 * kept int32 [B, H_kv, budget], each kept slot's place in the source, -1 past
 * the last. Slots past the last stay as they were. n_sink + n_recent <=
 * budget (else RA_ERR_RANGE). Source and destination are two caches: evict
 * into a spare one and swap the two.
 */
ra_status kv4_evict(const void* k_codes, const void* k_meta, const void* v_codes,
                    const void* v_meta, const float* score, const int* lens,
                    void* dst_k_codes, void* dst_k_meta, void* dst_v_codes,
                    void* dst_v_meta, float* dst_score, int* dst_lens, int* kept,
                    int B, int H_kv, int D, int C, int C_dst, int budget,
                    int n_sink, int n_recent, int* dev_status, void* stream);

/*
 * The paged key/value cache: what served sequences have attended to so far, in
 * pages that the caller hands out from one pool, in bfloat16 or 8 bits. The pages
 * have no counterpart in the sources; it continues the forward above (the same
 * attention, the same lse, so that its results merge with attn_lse_merge).
 *
 * A page holds `page` slots (16, 32, 64 or 128) of every key/value head; a slot is
 * one token's key row and value row of D values (64 or 128):
 *     k, v               [n_pages, H_kv, page, D]   bfloat16 (RA_BF16), or e4m3
 *                        codes (RA_E4M3)
 *     k_scale, v_scale   [n_pages, H_kv, page]      RA_E4M3 only (else NULL): a
 *                        byte b in 1..254 a row; a code c stands for c 2^(b - 127)
 * all 16-byte aligned. Which page holds which slots is the caller's table, device
 * int32 [B, width]: slot j of sequence b is row j % page of page
 * table[b][j / page]. An entry outside [0, n_pages) is a page that is not there;
 * only entries of slots that a call touches are read. Sequences may share pages
 * that no call writes. Nothing here reads tables, lengths or offsets on the host,
 * so a step can be captured into a graph and replayed while they change. A tensor
 * that a call writes (its workspace too) may not overlap any other of the call's
 * (RA_ERR_BUFFER).
 */
typedef struct {
  void* k;
  void* v;
  void* k_scale;
  void* v_scale;
  int n_pages, H_kv, page, D;
  int dtype;                 /* RA_BF16 or RA_E4M3 */
} ra_pages;

/*
 * paged_append - writes T tokens a sequence, k and v [B, T, H_kv, D] of `dtype`
 * (RA_BF16 or RA_F32), to slots start[b], start[b] + 1, ... (start: device int32
 * [B]). n_new: NULL, or device int32 [B]: only the first n_new[b] tokens of
 * sequence b count. bfloat16 pages: each value rounded once. 8 bits: a row's
 * scale is 2^e, e the least from -117 on with max |x| / 2^e <= 448 over its finite
 * values, its codes e4m3(x / 2^e), half to even; an infinity or a NaN reads back
 * as NaN, it alone. (What rounds to 2^128, from 1.9375 2^127 on, reads back as an
 * infinity.) A slot without a page is not written and sets RA_ERR_RANGE in
 * `dev_status` (device int, may be NULL). The slots that a call writes have to be
 * different ones.
 * paged_append_varlen - the same of packed tokens: k, v [total, H_kv, D], sequence
 * b's in rows [cu_seqlens[b], cu_seqlens[b + 1]) (device int32 [n_seq + 1], not
 * decreasing); rows that no sequence has are passed over.
 * Errors: RA_ERR_NULL, RA_ERR_SHAPE, RA_ERR_HEADDIM, RA_ERR_ALIGN, RA_ERR_DTYPE,
 * RA_ERR_RANGE (sizes), RA_ERR_BUFFER, RA_ERR_DEVICE, RA_ERR_LAUNCH.
 */
ra_status paged_append(const ra_pages* pages, const int* table, int width, const void* k,
                       const void* v, const int* start, const int* n_new, int B, int T,
                       int dtype, int* dev_status, void* stream);
ra_status paged_append_varlen(const ra_pages* pages, const int* table, int width,
                              const void* k, const void* v, const int* start,
                              const int* cu_seqlens, int n_seq, int total, int dtype,
                              int* dev_status, void* stream);

/*
 * paged_read - the values of slots start[b] ... start[b] + T - 1 (start NULL: from
 * slot 0), as k and v [B, T, H_kv, D] of `dtype` (either may be NULL). What 8 bits
 * hold is a bfloat16 number. A slot without a page gives zeros and sets
 * RA_ERR_RANGE in `dev_status`.
 */
ra_status paged_read(const ra_pages* pages, const int* table, int width, const int* start,
                     void* k, void* v, int B, int T, int dtype, int* dev_status,
                     void* stream);

/* Bytes of workspace that paged_attn needs for these sizes, and (varlen = 1, B =
 * n_seq, S_q = max_seqlen) paged_attn_varlen of `total` rows; host only. Of the
 * pages their sizes, number and type count. Partial results of long contexts take some
 * hundred MB at most; 8-bit pages besides, where S_q tokens are many (more than 48
 * query rows a key/value head), 4 GB at most of bfloat16 keys and values (of what the
 * windows see of B sequences of max_len slots, or of the whole pool, or of some
 * sequences at a time), or what one sequence of max_len slots takes, if that is more: a
 * max_len near the real lengths saves memory and time. */
ra_status paged_attn_workspace(const ra_pages* pages, int B, int S_q, int total, int H_q,
                               int max_len, int window, int n_sink, int varlen,
                               size_t* bytes);

/*
 * paged_attn - attention of S_q new tokens a sequence (one in plain decoding) over
 * its slots, which already hold them (append first).
 * lens: device int32 [B], slots in use, the new ones included (clamped to
 * [0, max_len]); max_len in [1, width * page] bounds them and sizes the launch.
 * Query t of sequence b is at slot p = lens[b] - S_q + t and sees the slots j <= p;
 * with window > 0 only those with j > p - window or j < n_sink (window 0: no
 * window, n_sink is ignored). Head h reads key/value head h / (H_q / H_kv); H_q /
 * H_kv is 128 at most. A row that sees no slot gets out = 0, lse = -inf.
 *     q, out  [B, S_q, H_q, D] bfloat16    lse  [B, H_q, S_q] float32 or NULL
 * paged_attn_varlen - the same of packed tokens, a prompt's pieces of different
 * lengths and single tokens side by side: sequence b's are rows [cu_seqlens[b],
 * cu_seqlens[b + 1]) of q, out [total, H_q, D], lse [H_q, total]; max_seqlen bounds
 * their numbers. Malformed offsets are brought into range; rows that no sequence
 * has are left as they were.
 * A row's results depend on the slots that it sees alone, to the bit, whatever the
 * others hold (slots past lens[b], behind the windows, later tokens' slots): NaN and
 * infinities included. A value that is not finite makes its own dimension of the rows
 * that see it infinite with its sign, or NaN if it is NaN, if there are infinities of
 * both signs, or (possibly) where the slot's weight is below 2^-100 of the row's
 * largest. Finite values of up to 2^88 in magnitude (beyond them results may be
 * infinite). A slot whose page is not there is not seen, and sets RA_ERR_RANGE in
 * `dev_status` where a row would have seen it; pages that every window has left behind
 * may be taken out of the table.
 * dtype RA_BF16. scale <= 0 means 1 / sqrt(D). The workspace is the caller's,
 * 16-byte aligned; its contents do not matter. Calls that may overlap on the GPU
 * need workspaces of their own. Results repeat bit for bit.
 * Errors: as paged_append, RA_ERR_RANGE for max_len, window, n_sink, too.
 */
ra_status paged_attn(const void* q, const ra_pages* pages, const int* table, int width,
                     const int* lens, void* out, float* lse, int B, int S_q, int H_q,
                     int max_len, int window, int n_sink, float scale, int dtype,
                     void* workspace, size_t workspace_bytes, int* dev_status,
                     void* stream);
ra_status paged_attn_varlen(const void* q, const ra_pages* pages, const int* table,
                            int width, const int* lens, const int* cu_seqlens, void* out,
                            float* lse, int n_seq, int total, int max_seqlen, int H_q,
                            int max_len, int window, int n_sink, float scale, int dtype,
                            void* workspace, size_t workspace_bytes, int* dev_status,
                            void* stream);

/* Human-readable text of a status; never NULL. */
const char* ring_attn_strerror(int status);

/* Library ABI version (major * 100 + minor); 103 adds the backward, the
 * packed variable-length and the Ulysses-layout entry points, 104 the 4-bit
 * key/value cache and the windowed entry points, 105 the paged cache. */
int ring_attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RING_ATTN_H */
