// Internal declarations of the 4-bit key/value cache: its format, the
// arguments of its kernels and their launchers.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "ring_attn.h"

namespace ra {

// One cache: rows of D values (one slot of one key/value head) in groups of
// 64 along D. codes [B, H_kv, C, D / 2], dimension 2i in the low and 2i + 1
// in the high half of byte i; meta [B, H_kv, C, D / 64] words, the group's
// bfloat16 scale in the low and its zero point in the high half. A code c
// stands for scale * (c - 8) + zero.
struct Kv4Cache {
  uint8_t* kc;
  uint32_t* km;
  uint8_t* vc;
  uint32_t* vm;
};

// Lets a kernel use `bytes` of dynamic shared memory on the current device;
// asked for once a device (`done` has a bit for each, the first 64).
template <class Kernel>
bool allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

constexpr int kKv4Group = 64;
constexpr int kKv4SlotAlign = 16;    // capacities are multiples of it

// append and read: `T` tokens a sequence, slots from start[b] on.
struct Kv4RowArgs {
  Kv4Cache c;
  void* k;                // [B, T, H_kv, D]
  void* v;
  const int* start;       // [B], or null for 0
  const int* n_new;       // [B] tokens that count, or null for T (append)
  int B, T, H_kv, D, C;
  int* status;
};
ra_status launch_kv4_append(const Kv4RowArgs& a, int dtype, cudaStream_t stream);
ra_status launch_kv4_read(const Kv4RowArgs& a, int dtype, cudaStream_t stream);

// Attention of S_q query tokens a sequence over its cache.
struct Kv4AttnArgs {
  const void* q;          // [B, S_q, H_q, D] bf16
  Kv4Cache c;
  const int* lens;        // [B] slots in use, the S_q query tokens' included
  void* out;              // [B, S_q, H_q, D] bf16
  float* lse;             // [B, H_q, S_q], may be null
  float* score;           // [B, H_kv, C], may be null: += weight of every slot
  int B, S_q, H_q, H_kv, D, C;
  int max_len;            // bound on lens
  int window, n_sink;     // window 0: every slot up to the query's own
  float scale_log2;       // softmax scale * log2(e)
  // plan (kv4_attn_plan): a query token's group of H_q / H_kv heads gives
  // R = S_q * H_q / H_kv rows a key/value head, cut into n_rb blocks of
  // `rows`; each block's visible tiles of kKv4Tile slots are cut into
  // n_split chunks of `chunk` tiles.
  int rows, n_rb, n_split, chunk;
  int slots;              // max_len rounded up to a tile: the logits' slots
  int log_rows;           // rows a slot's logits take: those in use, in fours
  float* part_o;          // [B * H_kv * n_rb][n_split][rows][D]
  float* part_ml;         // [B * H_kv * n_rb][n_split][rows][2]
  float* logits;          // [B * H_kv * n_rb][slots][log_rows], with score
  float* row_lse2;        // [B * H_kv * n_rb][rows] log-sums, base 2, with score
  int* status;
};
constexpr int kKv4Tile = 128;        // slots a CTA works on at a time

// Fills the plan fields for the sizes in `a`; bytes: the workspace needed
// (0 when one chunk a block suffices and no score is kept).
ra_status kv4_attn_plan(Kv4AttnArgs* a, bool score, size_t* bytes);
ra_status launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream);

// Eviction: the kept slots of every sequence and head, into another cache.
struct Kv4EvictArgs {
  Kv4Cache src, dst;
  const float* score;     // [B, H_kv, C]
  float* dst_score;       // [B, H_kv, C_dst], may be null
  const int* lens;        // [B]
  int* dst_lens;          // [B]
  int* kept;              // [B, H_kv, budget] source slots, -1 past the last
  int B, H_kv, D, C, C_dst;
  int budget, n_sink, n_recent;    // n_sink + n_recent <= budget <= C_dst
  int* status;
};
ra_status launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream);

}  // namespace ra
