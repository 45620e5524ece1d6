// Pieces of an attention kernel on the tcgen05 tensor cores that works on 128
// query rows by 128 keys at a time: scores and weights in tensor memory, keys and
// values in shared memory as boxes of 64 bf16 columns with the 128-byte swizzle.
#pragma once

#include <cstdint>

#include "fastmath.cuh"
#include "sm100.cuh"

namespace ra {
namespace tc {

constexpr int kTile = 128;                 // rows of a query tile and of a key tile
constexpr int kBoxBytes = kTile * 64 * 2;  // one box: 128 rows x 64 bf16

// Barrier among `count` threads of the CTA (ids 1-15; 0 is __syncthreads).
__device__ __forceinline__ void named_bar_sync(uint32_t id, uint32_t count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Three phase tests issued back to back (their shared-memory round trips
// overlap); true when all three phases have completed.
__device__ __forceinline__ bool mbar_test3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1,
                                           uint32_t b2, uint32_t p2) {
  const bool t0 = sm100::mbar_test_wait(b0, p0);
  const bool t1 = sm100::mbar_test_wait(b1, p1);
  const bool t2 = sm100::mbar_test_wait(b2, p2);
  return t0 && t1 && t2;
}

// The N columns of this thread's O row at tO, times alpha.
template <int N>
__device__ __forceinline__ void scale_cols(uint32_t tO, float alpha) {
#pragma unroll
  for (int c = 0; c < N / 32; ++c) {
    uint32_t uo[32];
    sm100::tmem_ld32(tO + c * 32, uo);
    sm100::tmem_ld_wait(uo);
#pragma unroll
    for (int i = 0; i < 32; ++i) uo[i] = __float_as_uint(__uint_as_float(uo[i]) * alpha);
    sm100::tmem_st32(tO + c * 32, uo);
  }
}

// Running 3-input maxima of 32 scores into 8 chains.
__device__ __forceinline__ void max_chunk(const uint32_t (&u)[32], float (&m8)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m8[i] = fastmath::fmax3(m8[i], __uint_as_float(u[i]), __uint_as_float(u[i + 8]));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m8[i] = fastmath::fmax3(m8[i], __uint_as_float(u[16 + i]), __uint_as_float(u[24 + i]));
}

__device__ __forceinline__ float max8(const float (&m8)[8]) {
  return fastmath::fmax3(fastmath::fmax3(m8[0], m8[1], m8[2]),
                         fastmath::fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
}

// p = 2^(s * scale * log2(e) - m) for 32 scores (packed FMA, two ex2 a pair),
// added to the two partial row sums and stored as 16 TMEM columns of bf16
// pairs at taddr.
__device__ __forceinline__ void exp_chunk(const uint32_t (&u)[32], uint64_t sl2x2,
                                          uint64_t neg_m2, uint64_t& sum2a, uint64_t& sum2b,
                                          uint32_t taddr) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x2 = fastmath::ffma2(
        fastmath::pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), sl2x2, neg_m2);
    float x0, x1;
    fastmath::unpack2(x2, x0, x1);
    const float p0 = sm100::ex2_approx(x0), p1 = sm100::ex2_approx(x1);
    if (i & 1) sum2b = fastmath::fadd2(sum2b, fastmath::pack2(p0, p1));
    else sum2a = fastmath::fadd2(sum2a, fastmath::pack2(p0, p1));
    pk[i] = sm100::pack_bf16x2(p0, p1);
  }
  sm100::tmem_st16(taddr, pk);
}

// S_i = Q_i K^T: M = 128 query rows, N = 128 keys, K = D in steps of 16.
template <int D>
__device__ __forceinline__ void issue_s(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc) {
  constexpr uint32_t idesc = sm100::idesc_bf16_f32(128, kTile, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    // 4 K steps of 16 columns per 64-column box; no carry into other fields
    const uint32_t off16 = ((kk / 4) * kBoxBytes + (kk % 4) * 32) >> 4;
    sm100::umma_ss(d_tmem, q_desc + off16, k_desc + off16, idesc, kk > 0 ? 1u : 0u);
  }
}

// O_i (+)= P_i V: A = P_i (bf16, TMEM), B = V (MN-major), M = 128, N = D,
// K = 128 keys in steps of 16 (8 TMEM columns of bf16 pairs each). P_i lies
// in the first 64 columns of S_i, or (kOwnCols) in the first 32 of each
// part's 64.
template <int D, bool kOwnCols>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint64_t v_desc,
                                         bool accumulate) {
  constexpr uint32_t idesc = sm100::idesc_bf16_f32(128, D, true);
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    sm100::umma_ts(o_tmem, p_tmem + (kOwnCols ? (kk / 4) * 64 + (kk % 4) * 8 : kk * 8),
                   v_desc + (uint64_t)((kk * 2048) >> 4), idesc, (accumulate || kk > 0) ? 1u : 0u);
}

}  // namespace tc
}  // namespace ra
