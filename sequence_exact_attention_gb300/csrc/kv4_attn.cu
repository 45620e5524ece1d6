// Attention of a few query tokens a sequence over a cache held in 4 bits.
//
// For a query row (token t, head h) at slot p = len - S_q + t of its
// sequence, over the visible slots j <= p (with a window: and j > p - window
// or j < n_sink), k_j and v_j being what the codes stand for:
//   s_j = scale <q, k_j>,  lse = log sum exp(s_j),  out = sum exp(s_j - lse) v_j
// and, on request, score[j] += sum over the rows of a key/value head of
// exp(s_j - lse).
//
// With k = sk (c - 8) + zk a group of 64 dimensions, and v likewise,
//   <q, k_j> = sum_groups sk (<q, c_j> - 8 <q, 1>) + zk <q, 1>
//   out      = sum_j (p_j sv) (c_j - 8) + sum_j p_j zv
// so the matrix units see the codes themselves, and scales and zero points are
// applied in float32: nothing is lost to a dequantised copy, and none is
// written. A code becomes an operand by one mask: as the low bits of a half a
// nibble n is the subnormal n 2^-24, in bits 4-7 it is 16 n 2^-24, exact both;
// the powers of two go into the query (1/16 for the dimensions that sit in
// high nibbles) and the results. In the scores the 8 comes off as the first
// addend. For the outputs sum_j w_j 8, of the weights w as they were rounded,
// is a product with a constant operand, one for all dimensions of a group, and
// is taken off every kFlush tiles: taken off at the end it left a long axis'
// output with the rounding of sums many times its size (2.4e-3 instead of 8e-4
// at 131072 slots), and of the unrounded weights with their roundings times 8
// (1.4e-3). (Making c - 8 from each pair of codes took two operations more a
// pair: 340 instead of 285 instructions on 16 slots; a product with the
// constant for every 16 dimensions took 4 us more at the size below.)
//
// What bounds it: the cache's bytes, 144 a slot and head at D = 128, read
// once. A row has 2 * 2 * D flops a slot, some 4 to 16 rows share a slot, far
// below what the tensor cores need; the work that counts is turning codes
// into operands, about half an instruction a value. So the products run as
// mma.sync m16n8k16, whose operands are registers (codes become the A operand
// where they were loaded; tcgen05 would want them written to shared memory
// again), transposed: M = 16 slots (then 16 dimensions), N = 8 query rows.
//
// A CTA takes one chunk of the slots of one (sequence, key/value head, block
// of 8 or 16 query rows), in tiles of 128 slots, 32 for each of its four
// warps, which keep running maxima, sums and outputs of their own, joined in
// shared memory at the end. Up to kStages tiles are in flight: a tile's codes
// and metadata are four contiguous pieces, which one lane asks for with bulk
// copies that land on the stage's barrier, once all warps have read the stage.
// (A ring for each warp cost 60 of 420 instructions on 16 slots.) Chunks of a
// long axis are joined by kv4_join_kernel (launched early: its CTAs are there
// when the last chunk ends). Everything is summed in a fixed order: results
// repeat bit for bit.
//
// Measured, 8 sequences x 8 key/value heads x 131072 slots, D = 128, 32 query
// heads, replayed from a graph: 231 us, 5.2 TB/s of the 6.8 of a copy (59 % of the
// issue slots, 55 % of the integer pipe). With one power of two a warp in place of
// each row's own (Roundings, below) it was 227: loads alone 173 us, arithmetic
// alone 199 us. 16 ragged sequences of up to 8192 slots, with scores: 45 us, the
// chunks, then the join, then the scores. (One wave of CTAs, each an equal run of
// tiles across the sequences' borders, measured 236 instead of 227 and 43.5
// instead of 46 us then.)
//
// Roundings: q is scaled by a power of two a row and becomes half precision
// (exact for bf16 values down to 2^-17 of the row's largest; queries beyond
// 2^90 are out of range); p times the value scale becomes half precision, 11
// bits, brought into its range by a power of two that each row keeps for each
// group: the largest product of the row's own met so far becomes 1 or more. A
// weight is off by at most 2^-11 of itself, or 2^-25 of the group's largest where
// it is a subnormal half. Sums are float32, but for one cut: the matrix unit lines
// products up by their operands' exponents, a subnormal's being its type's least,
// so what lies below 2^-16 (high nibbles 2^-20) of the largest weight of 16 slots
// falls off a product with a code (measured on two slots, one of them with the
// code 8 and so without a product of its own). Nothing of this is shared between
// rows: what a row does not see (a later drafted token's infinite value, a slot
// that another row's window still holds) changes no bit of its results. (Asking
// of the products themselves whether one leaves the range, by a second vote a
// tile, instead of the scales' bound: 251 instead of 243 us a call.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "checks.cuh"
#include "early_launch.cuh"
#include "fastmath.cuh"
#include "kv4_internal.h"
#include "sm100.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpSlots = kKv4Tile / kWarps;
static_assert(kWarpSlots == 32, "two 16-slot products a warp and tile");
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kRescaleLog2 = 4;           // p stays below 2^4
constexpr int kFlush = 8;
constexpr int kLiftMax = 112;             // p 2^112 is finite
constexpr int kWeightLog2 = 13;           // weights stay below 2^13; half ends at 2^16, but
                                          // bounds on logits past 2^24 are rounded
constexpr float kLn2 = 0.69314718055994531f;
constexpr float k2P24 = 16777216.f, k2Pm24 = 1.f / k2P24;

// The visible tiles of one block of query rows.
struct Span {
  int hi;              // slots from here on are invisible to every row
  int pmin, pmax;      // positions of the block's first and last token
  int n_sink_tiles;    // tiles of the first slots that the windows left behind
  int w0;              // first tile of the windows
  int n;               // tiles in all
  __device__ __forceinline__ int tile(int v) const {
    return v < n_sink_tiles ? v : v - n_sink_tiles + w0;
  }
};

__device__ __forceinline__ Span span_of(const Kv4AttnArgs& a, int b, int rb) {
  Span s;
  const int grp = a.H_q / a.H_kv;
  const int len = min(max(__ldg(a.lens + b), 0), a.max_len);
  const int r0 = rb * a.rows, r1 = min(r0 + a.rows, a.S_q * grp) - 1;
  s.pmin = len - a.S_q + r0 / grp;
  s.pmax = len - a.S_q + r1 / grp;
  s.hi = max(s.pmax + 1, 0);
  const int lo = a.window > 0 ? max(s.pmin - a.window + 1, 0) : 0;
  s.w0 = lo / kKv4Tile;
  s.n_sink_tiles = min((min(a.n_sink, s.hi) + kKv4Tile - 1) / kKv4Tile, s.w0);
  s.n = s.n_sink_tiles + max((s.hi + kKv4Tile - 1) / kKv4Tile - s.w0, 0);
  return s;
}

// Whether the row at position p sees slot j.
__device__ __forceinline__ bool sees(const Kv4AttnArgs& a, int p, int j) {
  return j <= p && (a.window <= 0 || j > p - a.window || j < a.n_sink);
}

// d += a b, or d = a b.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b + c, c the same in every row.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1, const float (&c)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]));
}
// Transposes an 8 x 8 matrix of 16-bit values held by a warp, two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Nibbles 0 and 4 (kHigh: 1 and 5) of x as two halves, times 2^-24 (2^-20).
template <bool kHigh>
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
  return x & (kHigh ? 0x00f000f0u : 0x000f000fu);
}

__device__ __forceinline__ float pow2_field(int f) { return __uint_as_float((uint32_t)f << 23); }
__device__ __forceinline__ int exponent_field(float x) { return (int)(__float_as_uint(x) >> 23); }

// The stages, and what the warps leave for the join over the same memory
// once all are done.
template <int D, int NT>
struct Smem {
  static constexpr int kStages = 3;
  static constexpr int kCodes = kKv4Tile * (D / 2);
  static constexpr int kMeta = kKv4Tile * (D / kKv4Group) * 4;
  static constexpr int kVc = kCodes, kKm = 2 * kCodes, kVm = kKm + kMeta;   // K codes at 0
  static constexpr int kStage = kVm + kMeta;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kOut = kWarps * 8 * NT * D * 4;
  static constexpr int kData = kRing > kOut ? kRing : kOut;
  static constexpr int kMl = kData;                             // [2][kWarps][8 NT]
  static constexpr int kFull = kMl + 2 * kWarps * 8 * NT * 4;   // [kStages] a tile has landed
  static constexpr int kFree = kFull + kStages * 8;             // [kStages] every warp has read it
  static constexpr int kAbort = kFree + kStages * 8;            // abort flag, then a 0
  static constexpr int kBytes = kAbort + 8;
  static_assert(kStage % 128 == 0, "stages keep the bulk copies' 16-byte alignment");
};

// D: head size; NT: blocks of 8 query rows; kScore: keep the logits.
template <int D, int NT, bool kScore>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 2)
kv4_attn_kernel(const Kv4AttnArgs a) {
  using S = Smem<D, NT>;
  constexpr int NG = D / kKv4Group;         // groups a row
  constexpr int RB = 8 * NT;                // query rows of the block
  extern __shared__ __align__(128) uint8_t smem[];
  float* sO = reinterpret_cast<float*>(smem);                   // [kWarps][RB][D]
  float* sM = reinterpret_cast<float*>(smem + S::kMl);          // [kWarps][RB]
  float* sL = sM + kWarps * RB;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kAbort);
  volatile int* never = abort_flag + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int grp = a.H_q / a.H_kv, R = a.S_q * grp;
  int blk = blockIdx.x;
  const int split = blk % a.n_split;
  blk /= a.n_split;                          // (b, hk, rb)
  const int rb = blk % a.n_rb;
  const int bh = blk / a.n_rb;               // b * H_kv + hk
  const int hk = bh % a.H_kv, b = bh / a.H_kv;
  const Span sp = span_of(a, b, rb);
  const int v_begin = split * a.chunk;
  const int v_end = min(sp.n, v_begin + a.chunk);
  if (v_begin >= v_end && a.n_split > 1) return;      // the join knows how many chunks there are
  let_dependents_start();

  // ---- the ring of tiles; lane 0 of warp 0 fills it
  const uint32_t ring = sm100::smem_u32(smem);
  const uint32_t full = ring + S::kFull, free_ = ring + S::kFree;
  const size_t row0 = (size_t)bh * a.C;
  const int n_tiles = v_end - v_begin;
  auto fill = [&](int stage, int i) {
    const int j0 = sp.tile(v_begin + i) * kKv4Tile;
    const int n = min(kKv4Tile, a.C - j0);             // less only at the capacity's end
    const uint32_t dst = ring + stage * S::kStage, bar = full + 8 * stage;
    const size_t row = row0 + j0;
    if (!in_range((long long)row, n, (long long)a.B * a.H_kv * a.C, a.status)) return;
    sm100::mbar_arrive_expect_tx(bar, n * (D + 2 * NG * 4));
    sm100::bulk_load(dst, a.c.kc + row * (D / 2), n * (D / 2), bar);
    sm100::bulk_load(dst + S::kKm, a.c.km + row * NG, n * NG * 4, bar);
    sm100::bulk_load(dst + S::kVc, a.c.vc + row * (D / 2), n * (D / 2), bar);
    sm100::bulk_load(dst + S::kVm, a.c.vm + row * NG, n * NG * 4, bar);
  };
  int filled = 0;                            // tiles asked for (lane 0 of warp 0)
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      sm100::mbar_init(full + 8 * i, 1);
      sm100::mbar_init(free_ + 8 * i, kWarps);
    }
    *abort_flag = *never = 0;
    sm100::fence_mbar_init();
    for (; filled < min(S::kStages, n_tiles); ++filled) fill(filled, filled);
  }
  __syncthreads();

  // ---- the block's query rows as B operands: lane (g, c) holds row g's
  // dimensions in the order in which the codes come out of a word
  uint32_t qf[NT][NG][2][2][2];              // [rows][group][word][half][operand]
  float qsum[NT][NG][2], minus8[NT][NG][2], sl2[NT][2];   // of rows 2c and 2c + 1
  int pos[NT][2];                            // their positions; below 0: sees nothing
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rb * RB + nt * 8 + g;
    const bool row_ok = r < R;
    float x[NG][16];
    float top = 0.f;
    const long long off = row_ok ? (((long long)b * a.S_q + r / grp) * a.H_q + hk * grp + r % grp) * D : 0;
    const bool ok = row_ok && in_range(off, D, (long long)a.B * a.S_q * a.H_q * D, a.status);
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (ok)
          u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + off +
                                              gr * kKv4Group + 16 * c + 8 * w);
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[gr][8 * w + 2 * i] = __uint_as_float(uw[i] << 16);
          x[gr][8 * w + 2 * i + 1] = __uint_as_float(uw[i] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[gr][i]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the largest x becomes 2^14 to 2^15
    const int e = min(max((int)(__float_as_uint(top) >> 23), 16), 217);
    const float down = pow2_field(268 - e), up = pow2_field(e - 14);
    float sums[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      sums[gr] = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[gr][i] *= down;
        sums[gr] += x[gr][i];
      }
      sums[gr] += __shfl_xor_sync(0xffffffffu, sums[gr], 1);
      sums[gr] += __shfl_xor_sync(0xffffffffu, sums[gr], 2);
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int o = 0; o < 2; ++o)
            qf[nt][gr][w][h][o] = pack_half2(x[gr][8 * w + 2 * h + o] * (o ? 0.0625f : 1.f),
                                             x[gr][8 * w + 2 * h + o + 4] * (o ? 0.0625f : 1.f));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = 4 * (2 * c + i);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        qsum[nt][gr][i] = __shfl_sync(0xffffffffu, sums[gr], src) * k2Pm24;
        minus8[nt][gr][i] = -8.f * qsum[nt][gr][i];
      }
      sl2[nt][i] = __shfl_sync(0xffffffffu, up, src) * a.scale_log2 * k2P24;
      const int rr = rb * RB + nt * 8 + 2 * c + i;
      pos[nt][i] = rr < R ? sp.pmin + rr / grp - (rb * RB) / grp : -1;
    }
  }

  // Running state of rows 2c and 2c + 1: what the exponent subtracts (the running
  // maximum in base 2, rounded down, so that raising it scales sums by a power of
  // two), and the bound that a score (before sl2) has to pass to raise it; -inf
  // until the row has seen a slot.
  float o[NT][NG][4][4];
  float bound[NT][2], sub[NT][2], l[NT][2], zo[NT][NG][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][gr][e][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bound[nt][i] = -INFINITY;
      sub[nt][i] = l[nt][i] = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) zo[nt][gr][i] = 0.f;
    }
  }
  // The power of two that a row's products p sv of a group are multiplied by
  // for half precision (o is in its units; 2^112 until the first), and the largest
  // scale, as bf16 bits, that no product of this lane's rows leaves the range with.
  float lift[NT][2][NG];
  uint32_t sv_bound[NG];
#pragma unroll
  for (int gr = 0; gr < NG; ++gr) sv_bound[gr] = 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) lift[nt][h][gr] = pow2_field(127 + kLiftMax);
  // -8 2^-24 times the rows' weights not yet taken off o: of group 0 (rows 0-7
  // of the product) in the first two, of group 1 in the others
  float off[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 4; ++x) off[nt][x] = 0.f;
  auto flush_row = [&](int nt, int h, int gr) {
    const float y = off[nt][2 * gr + h];
    off[nt][2 * gr + h] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[nt][gr][e][h] += y;                                     // low nibbles
      o[nt][gr][e][2 + h] = fmaf(16.f, y, o[nt][gr][e][2 + h]);  // high ones
    }
  };
  auto flush = [&] {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) flush_row(nt, h, gr);
  };
  // A row's sums of a group times mul; all lanes of the row together.
  auto scale_row = [&](int nt, int h, int gr, float mul) {
    flush_row(nt, h, gr);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[nt][gr][e][h] *= mul;
      o[nt][gr][e][2 + h] *= mul;
    }
  };

  int stage = 0;
  uint32_t phase = 0;
  for (int it = 0; it < n_tiles; ++it) {   // tiles
    // most tiles have landed: one test, and the bounded wait only when not
    if (!__all_sync(0xffffffffu, sm100::mbar_test_wait(full + 8 * stage, phase)) &&
        !sm100::mbar_wait_warp(full + 8 * stage, phase, abort_flag, kTimeoutNs))
      break;
    // this warp's 32 slots of the tile
    const int j0 = sp.tile(v_begin + it) * kKv4Tile + kWarpSlots * warp;
    const uint8_t* tile = smem + stage * S::kStage;
    const uint8_t* kc = tile + warp * (S::kCodes / kWarps);
    const uint8_t* vc = kc + S::kVc;
    const uint32_t* km =
        reinterpret_cast<const uint32_t*>(tile + S::kKm + warp * (S::kMeta / kWarps));
    const uint32_t* vm = km + S::kMeta / 4;
    // ---- metadata: lane (g, c) holds slots g, g + 8, g + 16 and g + 24
    uint32_t mk[4][NG], mv[4][NG];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        mk[i][gr] = km[(8 * i + g) * NG + gr];
        mv[i][gr] = vm[(8 * i + g) * NG + gr];
      }
    // ---- scores: rows of S are slots, columns query rows
    float s[4][NT][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        uint32_t kw[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint2 u = *reinterpret_cast<const uint2*>(kc + (16 * t + 8 * i + g) * (D / 2) +
                                                          32 * gr + 8 * c);
          kw[i][0] = u.x;
          kw[i][1] = u.y;
        }
        float acc[NT][4];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = kw[0][w] >> (8 * h), x1 = kw[1][w] >> (8 * h);
            const uint32_t af[4] = {codes2<false>(x0), codes2<false>(x1),
                                    codes2<true>(x0), codes2<true>(x1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (w + h == 0)
                mma16816_first(acc[nt], af, qf[nt][gr][w][h][0], qf[nt][gr][w][h][1],
                               minus8[nt][gr]);
              else
                mma16816(acc[nt], af, qf[nt][gr][w][h][0], qf[nt][gr][w][h][1]);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float sk = __uint_as_float(mk[2 * t + i][gr] << 16);
          const float zk = __uint_as_float(mk[2 * t + i][gr] & 0xffff0000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float z = gr == 0 ? zk * qsum[nt][0][h]
                                      : fmaf(zk, qsum[nt][gr][h], s[2 * t + i][nt][h]);
              s[2 * t + i][nt][h] = fmaf(sk, acc[nt][2 * i + h], z);
            }
        }
      }
    }
    if constexpr (kScore) {
      float* lg = a.logits + ((size_t)blk * a.slots + j0) * a.log_rows;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int at = (8 * i + g) * a.log_rows + nt * 8 + 2 * c;
          if (nt * 8 + 2 * c < a.log_rows &&
              in_range(((long long)blk * a.slots + j0) * a.log_rows + at, 2,
                       (long long)a.B * a.H_kv * a.n_rb * a.slots * a.log_rows, a.status))
            *reinterpret_cast<float2*>(lg + at) =
                make_float2(s[i][nt][0] * sl2[nt][0], s[i][nt][1] * sl2[nt][1]);
        }
    }
    // ---- tiles that some row does not see in full
    const bool whole = j0 + kWarpSlots - 1 <= sp.pmin &&
                       (a.window <= 0 || j0 > sp.pmax - a.window || j0 + kWarpSlots <= a.n_sink);
    uint32_t hidden = 0;                     // a bit for each score of a slot that its row does not see
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (!sees(a, pos[nt][h], j0 + 8 * i + g)) {
              s[i][nt][h] = -INFINITY;
              hidden |= 1u << ((i * NT + nt) * 2 + h);
            }
    }
    // ---- raise the running maxima, and lower lifts, only when a score or a scale
    // passes its bound: rare after the first tile. Which rows are changed, and
    // how, goes by what each of them sees.
    bool raise = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[nt][h] = fmaxf(fastmath::fmax3(s[0][nt][h], s[1][nt][h], s[2][nt][h]), s[3][nt][h]);
        raise |= top[nt][h] > bound[nt][h];
      }
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      uint32_t sv_top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sv_top = max(sv_top, mv[i][gr] & 0x7fffu);
      raise |= sv_top > sv_bound[gr];
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = top[nt][h];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          if (x > bound[nt][h]) {
            // whole numbers: the sums so far take a power of two, exactly
            const float to = floorf(x * sl2[nt][h]);
            const float alpha = bound[nt][h] == -INFINITY ? 0.f : exp2f(sub[nt][h] - to);
            sub[nt][h] = to;
            bound[nt][h] = (to + (float)kRescaleLog2) / sl2[nt][h];
            l[nt][h] *= alpha;
            // the products met so far shrink by alpha, so what brings them to 1
            // grows by 1 / alpha and o stays as it is, but at the end of the range
            const int grow = 127 - exponent_field(alpha);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              const int f = exponent_field(lift[nt][h][gr]), up = min(grow, 127 + kLiftMax - f);
              const float mul = alpha * pow2_field(127 + up);
              lift[nt][h][gr] = pow2_field(f + up);
              if (mul != 1.f) scale_row(nt, h, gr, mul);
              zo[nt][gr][h] *= alpha;
            }
          }
        }
      // A scale that is not finite goes to the zero point as NaN, which reaches the
      // rows that see the slot, in this group alone; a product would take it to the
      // other group, as 0 times NaN in the constant operand's other rows.
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
          if ((mv[i][gr] & 0x7f80u) == 0x7f80u) mv[i][gr] = 0x7fc00000u;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        int most = 0;                        // exponent field of the lane's largest lift
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = 0.f;                   // the row's largest product, times 2^-16
#pragma unroll
            for (int i = 0; i < 4; ++i)      // NaN and hidden slots are passed over
              x = fmaxf(x, fabsf(sm100::ex2_approx(fmaf(s[i][nt][h], sl2[nt][h], -sub[nt][h])) *
                                 (__uint_as_float(mv[i][gr] << 16) * (1.f / 65536.f))));
#pragma unroll
            for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            // 2^(to - 127) brings it to 1 to 2
            const int f = exponent_field(lift[nt][h][gr]), to = max(238 - exponent_field(x), 1);
            if (to < f) {
              lift[nt][h][gr] = pow2_field(to);
              scale_row(nt, h, gr, lift[nt][h][gr] * pow2_field(254 - f));
            }
            if (bound[nt][h] > -INFINITY) most = max(most, min(to, f));
          }
        // scales below 2^(kWeightLog2 - kRescaleLog2) / lift
        const int below = 127 + kWeightLog2 - kRescaleLog2 - (most - 127);
        sv_bound[gr] = ((uint32_t)min(below, 255) << 7) - 1;
      }
    }
    // ---- weights, and their products with the value codes
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p = sm100::ex2_approx(fmaf(s[i][nt][h], sl2[nt][h], -sub[nt][h]));
          s[i][nt][h] = p;
          l[nt][h] += p;
        }
    // masked: a row takes nothing from a slot that it does not see, whatever the
    // slot's value (0 times NaN is not 0)
    auto add_values = [&](auto masked) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          uint32_t vw[4];                    // codes of slots 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vw[i] = *reinterpret_cast<const uint32_t*>(
                vc + (16 * t + 8 * (i >> 1) + 2 * c + (i & 1)) * (D / 2) + 32 * gr + 4 * g);
          uint32_t pf[NT][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float sv = __uint_as_float(mv[2 * t + i][gr] << 16);
            const float zv = __uint_as_float(mv[2 * t + i][gr] & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float w[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float p = s[2 * t + i][nt][h];
                w[h] = p * lift[nt][h][gr] * sv;
                float z = fmaf(p, zv, zo[nt][gr][h]);
                if (decltype(masked)::value && (hidden >> (((2 * t + i) * NT + nt) * 2 + h) & 1u)) {
                  w[h] = 0.f;
                  z = zo[nt][gr][h];
                }
                zo[nt][gr][h] = z;
              }
              pf[nt][i] = transpose8x8(pack_half2(w[0], w[1]));
            }
          }
          const uint32_t minus8_rows[4] = {gr == 0 ? 0x80088008u : 0u, gr == 1 ? 0x80088008u : 0u,
                                           gr == 0 ? 0x80088008u : 0u, gr == 1 ? 0x80088008u : 0u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(off[nt], minus8_rows, pf[nt][0], pf[nt][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // two dimensions, nibbles 0 and 1 of byte e, of two slots a register
            const uint32_t sel = (uint32_t)(e | e << 4 | (4 + e) << 8 | (4 + e) << 12);
            const uint32_t x0 = __byte_perm(vw[0], vw[1], sel), x1 = __byte_perm(vw[2], vw[3], sel);
            const uint32_t af[4] = {codes2<false>(x0), codes2<true>(x0), codes2<false>(x1),
                                    codes2<true>(x1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][gr][e], af, pf[nt][0], pf[nt][1]);
          }
        }
    };
    if (whole) add_values(std::false_type());
    else add_values(std::true_type());
    if (it % kFlush == kFlush - 1) flush();
    // this warp has read the stage; the stage of the tile before, which the
    // other warps have most likely left too, takes the next tile
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(free_ + 8 * stage);
    if (threadIdx.x == 0 && it > 0 && filled < n_tiles) {
      const int s0 = stage == 0 ? S::kStages - 1 : stage - 1;
      // the free barrier's phases are the full one's
      if (sm100::mbar_wait(free_ + 8 * s0, stage == 0 ? phase ^ 1 : phase, abort_flag, kTimeoutNs)) {
        fill(s0, filled);
        ++filled;
      }
    }
    __syncwarp();
    if (++stage == S::kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  flush();
  // what was asked for lands before the CTA leaves (it has, unless a wait ran out)
  if (threadIdx.x == 0)
    for (int i = max(filled - S::kStages, 0); i < filled; ++i)
      sm100::mbar_wait(full + 8 * (i % S::kStages), (uint32_t)(i / S::kStages) & 1, never, kTimeoutNs);
  __syncwarp();

  // ---- the warps' parts meet in shared memory, in true units
  __syncthreads();                           // every ring is read
  if (threadIdx.x == 0 && (*abort_flag || *never) && a.status)
    atomicExch(a.status, (int)RA_ERR_TIMEOUT);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float ls = l[nt][h];
      float z[NG];
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) z[gr] = zo[nt][gr][h];
#pragma unroll
      for (int x = 4; x < 32; x *= 2) {
        ls += __shfl_xor_sync(0xffffffffu, ls, x);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) z[gr] += __shfl_xor_sync(0xffffffffu, z[gr], x);
      }
      const int r = nt * 8 + 2 * c + h;
      if (g == 0) {
        // in base 2 now; -inf where the row saw nothing
        sM[warp * RB + r] = bound[nt][h] == -INFINITY ? -INFINITY : sub[nt][h];
        sL[warp * RB + r] = ls;
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const float down = pow2_field(254 - exponent_field(lift[nt][h][gr]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // low and high nibbles
          float2 y = make_float2(fmaf(o[nt][gr][e][h] * k2P24, down, z[gr]),
                                 fmaf(o[nt][gr][e][2 + h] * (k2P24 / 16.f), down, z[gr]));
          *reinterpret_cast<float2*>(sO + (warp * RB + r) * D + gr * kKv4Group + 8 * g + 2 * e) = y;
        }
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < RB * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    const int row = rb * RB + r;
    if (row >= R) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sM[w * RB + r]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sM[w * RB + r], lw = sL[w * RB + r];
      if (mw == -INFINITY && lw == 0.f) continue;     // a warp that saw nothing
      const float f = mw == mx ? 1.f : exp2f(mw - mx);
      const float4 x = *reinterpret_cast<const float4*>(sO + (w * RB + r) * D + d);
      y.x = fmaf(f, x.x, y.x);
      y.y = fmaf(f, x.y, y.y);
      y.z = fmaf(f, x.z, y.z);
      y.w = fmaf(f, x.w, y.w);
      ls = fmaf(f, lw, ls);
    }
    if (a.n_split > 1) {
      const long long part = ((long long)blk * a.n_split + split) * RB + r;
      if (d == 0) {
        a.part_ml[2 * part] = mx;
        a.part_ml[2 * part + 1] = ls;
      }
      *reinterpret_cast<float4*>(a.part_o + part * D + d) = y;
    } else {
      const int t = row / grp, h = hk * grp + row % grp;
      const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);   // 0: no slot; NaN stays
      const long long off = (((long long)b * a.S_q + t) * a.H_q + h) * D + d;
      if (in_range(off, 4, (long long)a.B * a.S_q * a.H_q * D, a.status))
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + off) =
            make_uint2(sm100::pack_bf16x2(y.x * inv, y.y * inv),
                       sm100::pack_bf16x2(y.z * inv, y.w * inv));
      if (d == 0) {
        const float lse2 = ls == 0.f ? -INFINITY : mx + log2f(ls);
        if (kScore) a.row_lse2[(long long)blk * RB + r] = lse2;
        if (a.lse) a.lse[((long long)b * a.H_q + h) * a.S_q + t] = lse2 * kLn2;
      }
    }
  }
}

// Joins the chunks of one query row: 8 warps share the chunks, a warp's
// lanes the row's D values.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
kv4_join_kernel(const Kv4AttnArgs a) {
  constexpr int V = D / 32;                  // values a lane
  __shared__ float sO[kJoinWarps][D], sM[kJoinWarps], sL[kJoinWarps];
  const int grp = a.H_q / a.H_kv, R = a.S_q * grp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x % R, bh = blockIdx.x / R;
  const int b = bh / a.H_kv, hk = bh % a.H_kv;
  const int rb = row / a.rows, r = row % a.rows;
  const Span sp = span_of(a, b, rb);
  const int n = (sp.n + a.chunk - 1) / a.chunk;       // chunks that hold a visible tile
  let_dependents_start();
  wait_for_prior_grid();
  const long long base = ((long long)bh * a.n_rb + rb) * a.n_split;
  float y[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.f;
  for (int s = warp; s < n; s += kJoinWarps) {
    const long long part = (base + s) * a.rows + r;
    const float pm = a.part_ml[2 * part], pl = a.part_ml[2 * part + 1];
    if (pm == -INFINITY && pl == 0.f) continue;
    const float mn = fmaxf(m, pm);
    const float f0 = m == -INFINITY ? 0.f : exp2f(m - mn), f1 = pm == mn ? 1.f : exp2f(pm - mn);
    l = l * f0 + pl * f1;
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = y[i] * f0 + a.part_o[part * D + i * 32 + lane] * f1;
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sO[warp][i * 32 + lane] = y[i];
  if (lane == 0) {
    sM[warp] = m;
    sL[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D) return;
  float mx = -INFINITY, ls = 0.f, z = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, sM[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (sM[w] == -INFINITY && sL[w] == 0.f) continue;
    const float f = sM[w] == mx ? 1.f : exp2f(sM[w] - mx);
    ls = fmaf(f, sL[w], ls);
    z = fmaf(f, sO[w][threadIdx.x], z);
  }
  const int t = row / grp, h = hk * grp + row % grp;
  const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);
  const long long off = (((long long)b * a.S_q + t) * a.H_q + h) * D + threadIdx.x;
  if (in_range(off, 1, (long long)a.B * a.S_q * a.H_q * D, a.status))
    static_cast<__nv_bfloat16*>(a.out)[off] = __float2bfloat16_rn(z * inv);
  if (threadIdx.x == 0) {
    const float lse2 = ls == 0.f ? -INFINITY : mx + log2f(ls);
    if (a.score) a.row_lse2[((long long)bh * a.n_rb + rb) * a.rows + r] = lse2;
    if (a.lse) a.lse[((long long)b * a.H_q + h) * a.S_q + t] = lse2 * kLn2;
  }
}

// Adds every visible slot's weight to its running sum: kScorePer slots a
// thread, whose loads are in flight together.
constexpr int kScoreThreads = 128, kScorePer = 4;
__global__ void __launch_bounds__(kScoreThreads)
kv4_score_kernel(const Kv4AttnArgs a, int blocks_per_head) {
  const int bh = blockIdx.x / blocks_per_head;
  const int j0 = (blockIdx.x % blocks_per_head) * (kScoreThreads * kScorePer) + threadIdx.x;
  const int b = bh / a.H_kv;
  const int grp = a.H_q / a.H_kv, R = a.S_q * grp;
  // what this call does not write is read while the grid before still runs
  const Span first = span_of(a, b, 0);
  float old[kScorePer];
#pragma unroll
  for (int e = 0; e < kScorePer; ++e) {
    const int j = j0 + e * kScoreThreads;
    old[e] = j < a.max_len ? a.score[(long long)bh * a.C + j] : 0.f;
  }
  wait_for_prior_grid();
  float sum[kScorePer] = {};
  bool seen[kScorePer] = {};
  for (int rb = 0; rb < a.n_rb; ++rb) {
    const Span sp = rb == 0 ? first : span_of(a, b, rb);
    if (j0 >= sp.hi) continue;
    const long long blk = (long long)bh * a.n_rb + rb;
    const float* lse2 = a.row_lse2 + blk * a.rows;
    for (int r4 = 0; r4 < a.log_rows; r4 += 4) {
      float4 x4[kScorePer];
#pragma unroll
      for (int e = 0; e < kScorePer; ++e) {
        // rows past the last and hidden slots are read and never used
        const int j = min(j0 + e * kScoreThreads, sp.hi - 1);
        x4[e] = *reinterpret_cast<const float4*>(a.logits + (blk * a.slots + j) * a.log_rows + r4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = rb * a.rows + r4 + i;
        if (row >= R) break;
        const float l2 = lse2[r4 + i];
        const int p = sp.pmin + row / grp - (rb * a.rows) / grp;
#pragma unroll
        for (int e = 0; e < kScorePer; ++e) {
          const float x[4] = {x4[e].x, x4[e].y, x4[e].z, x4[e].w};
          if (sees(a, p, j0 + e * kScoreThreads)) {
            sum[e] += sm100::ex2_approx(x[i] - l2);
            seen[e] = true;
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kScorePer; ++e) {
    const long long at = (long long)bh * a.C + j0 + e * kScoreThreads;
    if (seen[e] && in_range(at, 1, (long long)a.B * a.H_kv * a.C, a.status)) a.score[at] = old[e] + sum[e];
  }
}

template <int D, int NT>
ra_status launch_nt(const Kv4AttnArgs& a, cudaStream_t stream) {
  const long long grid = (long long)a.B * a.H_kv * a.n_rb * a.n_split;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  auto kern = a.score ? kv4_attn_kernel<D, NT, true> : kv4_attn_kernel<D, NT, false>;
  constexpr int smem = Smem<D, NT>::kBytes;
  static std::atomic<uint64_t> allowed[2];
  if (!allow_smem(kern, smem, allowed[a.score ? 1 : 0])) return RA_ERR_LAUNCH;
  kern<<<(unsigned)grid, kThreads, smem, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return RA_ERR_LAUNCH;
  if (a.n_split > 1) {
    const long long rows = (long long)a.B * a.H_q * a.S_q;
    if (rows > 0x7fffffffLL) return RA_ERR_RANGE;
    if (!launch_early(kv4_join_kernel<D>, rows, 32 * kJoinWarps, 0, stream, a)) return RA_ERR_LAUNCH;
  }
  if (a.score) {
    const int per = (a.max_len + kScoreThreads * kScorePer - 1) / (kScoreThreads * kScorePer);
    const long long blocks = (long long)a.B * a.H_kv * per;
    if (blocks > 0x7fffffffLL) return RA_ERR_RANGE;
    if (!launch_early(kv4_score_kernel, blocks, kScoreThreads, 0, stream, a, per))
      return RA_ERR_LAUNCH;
  }
  return RA_OK;
}

}  // namespace

// Chunks: as many as fill whole waves of resident CTAs best, two waves by
// preference (sequences of different lengths then even out), but none under
// kMinChunk tiles, where joining would cost more than it spreads.
ra_status kv4_attn_plan(Kv4AttnArgs* a, bool score, size_t* bytes) {
  constexpr int kMinChunk = 2;
  const long long R = (long long)a->S_q * (a->H_q / a->H_kv);
  a->rows = R <= 8 ? 8 : 16;
  const long long n_rb = (R + a->rows - 1) / a->rows;
  const long long blocks = (long long)a->B * a->H_kv * n_rb;
  long long tiles = ((long long)a->max_len + kKv4Tile - 1) / kKv4Tile;
  if (a->window > 0) {
    const long long seen = ((long long)a->n_sink + kKv4Tile - 1) / kKv4Tile +
                           ((long long)a->window + a->S_q - 1 + kKv4Tile - 1) / kKv4Tile + 1;
    if (seen < tiles) tiles = seen;
  }
  // CTAs resident at a time on a GB300: a constant, as the workspace's size has to
  // be the same where there is no device to ask
  const long long wave = 152 * (a->rows == 8 ? 4 : 2);
  long long best = 1, best_full = 0;                        // chunks, and what they fill of their waves
  for (int w = 2; w >= 1; --w) {
    const long long n = wave * w / blocks;
    const long long full = n * blocks * 1000 / (wave * w);
    if (full > best_full + 20) {
      best = n;
      best_full = full;
    }
  }
  long long chunk = (tiles + best - 1) / best;
  if (chunk < kMinChunk) chunk = kMinChunk;
  const long long n_split = tiles > chunk ? (tiles + chunk - 1) / chunk : 1;
  if (blocks * n_split > 0x7fffffffLL) return RA_ERR_RANGE;
  a->n_rb = (int)n_rb;
  a->chunk = (int)chunk;
  a->n_split = (int)n_split;
  a->slots = (a->max_len + kKv4Tile - 1) / kKv4Tile * kKv4Tile;
  const size_t parts = (size_t)blocks * n_split * a->rows;
  const size_t n_o = n_split > 1 ? parts * a->D : 0;
  const size_t n_ml = n_split > 1 ? parts * 2 : 0;
  a->log_rows = n_rb == 1 ? (int)(R + 3) / 4 * 4 : a->rows;
  const size_t n_lg = score ? (size_t)blocks * ((size_t)a->slots * a->log_rows + a->rows) : 0;
  *bytes = (n_o + n_ml + n_lg) * sizeof(float);
  return RA_OK;
}

ra_status launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  if (a.D == 64)
    return a.rows == 8 ? launch_nt<64, 1>(a, stream) : launch_nt<64, 2>(a, stream);
  return a.rows == 8 ? launch_nt<128, 1>(a, stream) : launch_nt<128, 2>(a, stream);
}

}  // namespace ra
