// Device code that the paged cache's kernels share: number formats, boxes of
// pages, blocks of query rows.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "checks.cuh"
#include "paged_internal.h"
#include "paged_iter.cuh"

namespace ra {

// Two e4m3 codes (lo in the low byte), to nearest, half to even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes, in the low 16 bits, as two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
  return r;
}
__device__ __forceinline__ float2 half2_values(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// 2^(byte - 127).
__device__ __forceinline__ float pow2_byte(int byte) { return __uint_as_float((uint32_t)byte << 23); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// The table's entry for a sequence's slots from p * page on; -1 past its end. (Whether it is
// a page is tested where it is used, not here: a test would wait for the load.)
__device__ __forceinline__ int paged_entry(const PagedAttnArgs& a, int b, int p) {
  const long long at = (long long)b * a.width + p;
  if (p >= a.width || !in_range(at, 1, (long long)a.B * a.width, a.status)) return -1;
  return a.table[at];
}
__device__ __forceinline__ bool paged_held(const PagedAttnArgs& a, int id) {
  return id >= 0 && id < a.p.n_pages;
}
// What the bounds checks know of the pool's rows and of the partial results'.
__device__ __forceinline__ long long paged_pool_rows(const PagePool& p) {
  return (long long)p.n_pages * p.H_kv * p.page;
}
__device__ __forceinline__ long long paged_part_rows(const PagedAttnArgs& a) {
  return (long long)a.n_cut * a.n_split * a.block_rows;
}

// Sums of x over a warp's lanes up to each.
__device__ __forceinline__ int warp_prefix(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The block of query rows that item `item` is; every lane of a warp calls it. Few
// rows: by sequence and head. Many: blocks of late tokens (the longest
// walks) come first, across all heads of a sequence (and the sequences, where all
// have T new tokens) when keys and values fit in L2 anyway, else within each head.
// Packed sequences are looked up among their numbers of blocks: the launch knows
// only how many there are at most (b = -1 past the last).
struct PagedBlock {
  int b, hk, rb;
};
__device__ __forceinline__ PagedBlock paged_block(const PagedAttnArgs& a, int item) {
  const int H_kv = a.p.H_kv;
  if (a.block_rows <= 16) return {item / a.n_rb / H_kv, item / a.n_rb % H_kv, item % a.n_rb};
  if (!a.cu) {
    if (a.rb_major) {
      const int bh = item % (a.B * H_kv);
      return {bh / H_kv, bh % H_kv, a.n_rb - 1 - item / (a.B * H_kv)};
    }
    const int bh = item / a.n_rb;
    return {bh / H_kv, bh % H_kv, a.n_rb - 1 - item % a.n_rb};
  }
  const int lane = threadIdx.x & 31, tokens = 2 * (128 / (a.H_q / H_kv));
  int before = 0;                                  // blocks of a head before these 32 sequences
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int nb = 0;
    if (b < a.B) {
      const PagedSeq s = paged_seq(a, b);
      if (paged_mine(a, s)) nb = (s.n + tokens - 1) / tokens;
    }
    const int sum = warp_prefix(nb, lane);
    const uint32_t past = __ballot_sync(0xffffffffu, item < (long long)(before + sum) * H_kv);
    if (past) {
      const int src = __ffs(past) - 1;
      const int n = __shfl_sync(0xffffffffu, nb, src);
      const int in = item - (before + __shfl_sync(0xffffffffu, sum, src) - n) * H_kv;
      if (a.rb_major) return {b0 + src, in % H_kv, n - 1 - in / H_kv};
      return {b0 + src, in / n, n - 1 - in % n};
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return {-1, 0, 0};
}

// The place of a row's log-sum.
__device__ __forceinline__ long long paged_lse_at(const PagedAttnArgs& a, int b, int row, int t,
                                                  int h) {
  return a.cu ? (long long)h * a.rows + row : ((long long)b * a.H_q + h) * a.T + t;
}

}  // namespace ra
