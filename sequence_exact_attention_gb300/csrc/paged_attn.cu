// Attention of a few query rows a sequence over its pages.
//
// For a query row (token t, head h) at slot p of its sequence, over the visible
// slots j <= p (with a window: and j > p - window or j < n_sink):
//   s_j = scale <q, k_j>,  lse = log sum exp(s_j),  out = sum exp(s_j - lse) v_j
// in one pass, with a running maximum and sum. What bounds it: the bytes of the
// visible slots, read once. A slot's rows meet some 4 to 16 query rows, far less
// than tensor cores need, so the products run as mma.sync m16n8k16, whose operands
// are registers, transposed: M = 16 slots (then 16 dimensions), N = 8 query rows.
//
// 8 bits. A code is a half (exact). The scale of a key multiplies its scores.
// The scale 2^e of a value would leave half's range in a weight, so weights are
//   w_j = 2^(s_j + e_j - m'),  out = sum w_j c_j 2^(m' - m) / sum 2^(s_j - m)
// in base 2, with a maximum m' of their own: the row's largest weight is between
// 2^10 and 2^15, whatever the scales. Where slots' scales lie far apart, though, one
// maximum over s + e leaves the others nothing: a row's one value of 2^30 would round
// the weights of all slots around 1 to 0, and with them the dimensions in which it is 0
// itself. So a row whose m' - m passes some visible slot's e by 10 takes that step of 16
// slots apart, its weights as two bf16 numbers. Every other weight is 2^(s_j - m) or
// more. Queries become halves times a power of two a row, exact for values down to
// 2^-31 of the row's largest; rows with smaller ones are multiplied as bf16 numbers.
// Roundings: weights to half, 2^-11 of a weight at most, or 2^-25 of the row's largest
// 2^(s - m), whatever the values. A bf16 page's values may pass half's range, so there,
// and in steps taken apart, a weight is the sum of two bf16 numbers (2^-16) in two
// products (one, rounded at 2^-8, made the error against 64 bits 2.3e-3 where the
// outputs' rounding alone makes 1.7e-3). Sums and statistics are float32.
//
// For up to 16 query rows a sequence and key/value head (new tokens times the heads
// that share it), over 8-bit pages up to 48 in blocks of 16; more: paged_tiles.cu. (Of
// packed sequences of both kinds over 8-bit pages each kernel takes its own.) A
// CTA takes one chunk of the slots that a block sees. A producer warp looks the pages
// up, a lane for each, and asks for their boxes (TMA, swizzled, so that ldmatrix meets
// no bank conflict; a page's row is one box, as some 30 cycles a box are what small
// pages cost); four warps share a tile's slots and keep running maxima, sums and
// outputs of their own, joined in shared memory at the end. Chunks of a long axis are
// joined by a second kernel. Everything is summed in a fixed order: results repeat bit
// for bit. (CTAs that each take an equal run of all tiles, across blocks' borders, with
// loads going on from one block to the next: 32 ragged sequences 115 instead of 110 us,
// 8 x 128K slots of 8 bits 364 instead of 310, one CTA of eight warps a multiprocessor;
// two with four warps each 6 % slower on equal lengths.)
//
// Slots that a row does not see change no bit of its results, whatever they hold:
// scores are replaced, and in tiles that are not whole the values' operands are
// masked, too (0 times a NaN is not 0); where tokens differ in what they see and a
// value is not finite, such a tile is multiplied once for each of them (always doing
// so took 26 instead of 20 us for 4 x 4 tokens under a window of 4096).
//
// Measured, replayed from a graph: 8 x 128K slots of 8 heads, D = 128, 8 bits 309 us,
// 7.0 TB/s; 32 ragged sequences up to 8K slots, bf16 in pages of 16 109.5 us, 6.1 TB/s.
// (Telling what has to be taken apart costs blocks of 8 rows nothing; blocks of 16, whose
// registers are used up, 2 %: 8 x 32K slots of 4 heads, D = 128, 25 rows 127.4 us instead
// of 124.8; 8 x 64K of 8, D = 64, 16 rows 159.8 instead of 155.7.)
#include <cuda_bf16.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "checks.cuh"
#include "early_launch.cuh"
#include "fastmath.cuh"
#include "kv4_internal.h"
#include "paged_internal.h"
#include "paged_ops.cuh"
#include "sm100.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;                 // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kRescaleLog2 = 4.f;       // weights stay below 2^5,
constexpr float kHalfUp = 10.f;           // halves below 2^15
constexpr float kLn2 = 0.69314718055994531f;

// d += a b.
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held by a warp, two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float pow2_field(int f) { return __uint_as_float((uint32_t)f << 23); }

// Shared memory: the ring of tiles, over which the warps leave their parts for
// the join once all are done.
template <int D, int NT, bool kQuant>
struct Smem {
  static constexpr int kTile = paged_rows_tile(D, kQuant);         // slots
  static constexpr int kRowBytes = kQuant ? D : 128;               // of a part of a row
  static constexpr int kParts = kQuant ? 1 : D / 64;               // a page's, one after the other
  static constexpr int kKv = kTile * kParts * kRowBytes;           // keys, or values, of a tile
  static constexpr int kKs = 2 * kKv, kVs = kKs + (kQuant ? kTile : 0);
  static constexpr int kStage = (kVs + (kQuant ? kTile : 0) + 1023) / 1024 * 1024;
  static constexpr int kStages = 100 * 1024 / kStage;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kOut = kWarps * 8 * NT * D * 4;
  static constexpr int kData = kRing > kOut ? kRing : kOut;
  static constexpr int kMl = kData;                                // [2][kWarps][8 NT]
  static constexpr int kFar = kMl + 2 * kWarps * 8 * NT * 4;       // [2][kWarps][8 NT]
  static constexpr int kFull = kFar + 2 * kWarps * 8 * NT * 4;     // [kStages]
  static constexpr int kFree = kFull + kStages * 8;                // [kStages]
  static constexpr int kGone = kFree + kStages * 8;                // [kStages] pages not there
  static constexpr int kAbort = kGone + kStages * 4;               // abort flag, then a 0
  static constexpr int kBytes = kAbort + 8 + 1024;                 // and alignment
};

// Byte offset of 16-byte chunk c of row r in a swizzled box.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return kRowBytes == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4))
                          : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// D: head size; NT: blocks of 8 query rows; kQuant: 8-bit pages.
template <int D, int NT, bool kQuant>
__global__ void __launch_bounds__(kThreads, 2)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PagedAttnArgs a) {
  using S = Smem<D, NT, kQuant>;
  constexpr int kTile = S::kTile;
  constexpr int WS = kTile / kWarps;        // slots a warp
  static_assert(WS % 16 == 0, "products of 16 slots");
  constexpr int RB = 8 * NT;                // query rows, at most
  constexpr int KS = D / 16;                // steps of 16 dimensions
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = sm100::smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (ring - raw);
  float* sO = reinterpret_cast<float*>(smem);                   // [kWarps][RB][D]
  float* sM = reinterpret_cast<float*>(smem + S::kMl);          // [kWarps][RB]
  float* sL = sM + kWarps * RB;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kAbort);
  volatile int* never = abort_flag + 1;
  uint32_t* gone = reinterpret_cast<uint32_t*>(smem + S::kGone);
  const uint32_t full = ring + S::kFull, free_ = ring + S::kFree;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int H_kv = a.p.H_kv, grp = a.H_q / H_kv;
  // the blocks of a sequence and head run side by side: what one of them reads the others
  // find in L2. All first chunks come first, as the last ones are shorter where lengths
  // differ (a sequence's chunks in a row: 111 instead of 109.5 us for 32 ragged
  // sequences, 310.5 instead of 308.7 for 8 x 128K slots)
  const int item = blockIdx.x % a.n_items, split = blockIdx.x / a.n_items;
  const int rb = item % a.n_rb, bh = item / a.n_rb;
  const int b = bh / H_kv, hk = bh % H_kv;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      sm100::mbar_init(full + 8 * i, 1);
      sm100::mbar_init(free_ + 8 * i, kWarps);
    }
    *abort_flag = *never = 0;
    sm100::fence_mbar_init();
  }
  let_dependents_start();
  wait_for_prior_grid();
  const PagedSeq sq = paged_seq(a, b);
  const int r0 = rb * RB;                   // the block's first of the head's query rows
  const int R = min(sq.n * grp - r0, RB);   // and how many
  if (R <= 0 || !paged_mine(a, sq)) return; // a sequence of fewer new tokens, or of many
  const int first = sq.len - sq.n;          // position of the first new token
  PagedSpan<kTile> sp;
  sp.init(a, first + r0 / grp, first + (r0 + R - 1) / grp);
  const int v_begin = split * a.chunk;
  const int n_tiles = max(min(sp.n, v_begin + a.chunk) - v_begin, 0);
  __syncthreads();

  if (warp == kWarps) {
    // ======================= producer =======================
    // A lane for each page's box looks the page up, a tile ahead, and asks for its keys,
    // values and scales. (Scales through registers, loaded a tile ahead and stored by
    // the lanes, took 332 instead of 314 us for 8 x 128K slots.)
    const int box_rows = min(a.p.page, kTile);
    const int shift = 31 - __clz(a.p.page);
    const int n_box = kTile / box_rows;     // at most 8
    const int at = lane * box_rows;
    struct Box {
      bool wanted;                          // some row sees some of it
      int id, row;                          // id below 0: no such page
    };
    auto look_up = [&](int i) -> Box {
      Box x = {false, -1, 0};
      if (i >= n_tiles || lane >= n_box) return x;
      const int j = sp.tile(v_begin + i) * kTile + at;
      if (j >= sp.hi || !sp.meets(a, j, box_rows)) return x;
      x.wanted = true;
      x.row = j & (a.p.page - 1);
      x.id = paged_entry(a, b, j >> shift);
      return x;
    };
    Box next = look_up(0);
    int i = 0, stage = 0;
    uint32_t phase = 0;
    bool bad = false;
    for (; i < n_tiles; ++i) {
      const Box cur = next;
      next = look_up(i + 1);
      if (i >= S::kStages &&
          !sm100::mbar_wait_warp(free_ + 8 * stage, phase ^ 1, abort_flag, kTimeoutNs))
        break;
      const long long row = ((long long)cur.id * H_kv + hk) * a.p.page + cur.row;
      const bool held =
          paged_held(a, cur.id) && in_range(row, box_rows, paged_pool_rows(a.p), a.status);
      const uint32_t boxes = __ballot_sync(0xffffffffu, held);
      const uint32_t missing = __ballot_sync(0xffffffffu, cur.wanted && !held);
      const uint32_t dst = ring + stage * S::kStage, bar = full + 8 * stage;
      if (lane == 0) {
        gone[stage] = missing;                // a bit for each box
        sm100::mbar_arrive_expect_tx(
            bar, __popc(boxes) * box_rows * (2 * S::kParts * S::kRowBytes + (kQuant ? 2 : 0)));
      }
      bad |= missing != 0;
      __syncwarp();
      if (held) {
        const uint32_t to = dst + at * (S::kParts * S::kRowBytes);
        const int z = cur.id * H_kv + hk;
        sm100::tma_load_4d(to, &tm_k, bar, 0, cur.row, 0, z);
        sm100::tma_load_4d(to + S::kKv, &tm_v, bar, 0, cur.row, 0, z);
        if (kQuant) {
          sm100::bulk_load(dst + S::kKs + at, a.p.ks + row, box_rows, bar);
          sm100::bulk_load(dst + S::kVs + at, a.p.vs + row, box_rows, bar);
        }
      }
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // what was asked for lands before the CTA leaves (it has, unless a wait ran out)
    for (int x = max(i - S::kStages, 0); x < i; ++x)
      sm100::mbar_wait(full + 8 * (x % S::kStages), (uint32_t)(x / S::kStages) & 1, never,
                       kTimeoutNs);
    if (bad && lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    __syncwarp();
    __syncthreads();                         // every warp has read the ring
  } else {
    // ======================= the warps that compute =======================
    // the query rows as B operands: lane (g, c) holds row g's dimensions
    // 16 k + 2 c, + 1, + 8, + 9 of step k; codes come four to a lane, 16 k + 4 c on
    uint32_t qf[NT][KS][2];
    float sl2[NT][2];                        // of rows 2c and 2c + 1
    // 8 bits: rows with a value too small beside the largest for a half: what their values
    // are multiplied by, 0 of the others, and where they lie, in rows of D (volatile: read
    // where they are needed, and nothing of it kept in registers)
    volatile float* far_down = reinterpret_cast<float*>(smem + S::kFar) + warp * RB;
    volatile int* far_row = reinterpret_cast<int*>(smem + S::kFar) + (kWarps + warp) * RB;
    bool any_far = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const bool row_ok = r < R;
      const int row = row_ok ? (sq.row0 + (r0 + r) / grp) * a.H_q + hk * grp + (r0 + r) % grp : 0;
      const long long off = (long long)row * D;
      const bool ok = row_ok && in_range(off, D, (long long)a.rows * a.H_q * D, a.status);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + off;
      if constexpr (kQuant) {
        uint2 u[KS];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          u[k] = ok ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * c) : make_uint2(0, 0);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(u[k].x << 16)),
                                       fabsf(__uint_as_float(u[k].x & 0xffff0000u))),
                                 fmaxf(fabsf(__uint_as_float(u[k].y << 16)),
                                       fabsf(__uint_as_float(u[k].y & 0xffff0000u)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest value becomes 2^14 to 2^15
        const int e = max((int)(__float_as_uint(top) >> 23), 16);
        const float down = pow2_field(268 - e), up = pow2_field(e - 14);
        bool lost = false;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          auto halves = [&](uint32_t x) -> uint32_t {
            const float lo = __uint_as_float(x << 16) * down;
            const float hi = __uint_as_float(x & 0xffff0000u) * down;
            const uint32_t h = pack_half2(lo, hi);
            const float2 back = half2_values(h);
            lost |= back.x != lo || back.y != hi;
            return h;
          };
          qf[nt][k][0] = halves(u[k].x);
          qf[nt][k][1] = halves(u[k].y);
        }
        const bool far = (__ballot_sync(0xffffffffu, lost) >> (4 * g) & 15u) != 0;
        any_far |= __any_sync(0xffffffffu, lost);
        if (c == 0) {
          far_down[r] = far ? down : 0.f;
          far_row[r] = row;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sl2[nt][h] = __shfl_sync(0xffffffffu, up, 4 * (2 * c + h)) * a.scale_log2;
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qf[nt][k][x] =
                ok ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * x + 2 * c) : 0u;
        sl2[nt][0] = sl2[nt][1] = a.scale_log2;
      }
    }
    __syncwarp();
    // the position of row 2c + h; below 0: sees nothing
    auto pos = [&](int nt, int h) -> int {
      const int r = nt * 8 + 2 * c + h;
      return r < R ? first + (r0 + r) / grp : -1;
    };

    // Running state of rows 2c and 2c + 1. What the exponents subtract: the running
    // maximum in base 2, rounded down, so that raising it scales sums by a power of
    // two, -inf until the row has seen a slot; a score kRescaleLog2 above raises it.
    // (sub2: that of the weights, with the values' scales, less kHalfUp.)
    float o[NT][KS][4];
    float sub[NT][2], sub2[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[nt][h] = 0.f;
        sub[nt][h] = sub2[nt][h] = -INFINITY;
      }
    }
    // 8 bits: value scales below 2^low are too far below what one of this lane's rows has met
    float low = -INFINITY;
    auto scale_row = [&](int nt, int h, float mul) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        o[nt][k][h] *= mul;
        o[nt][k][2 + h] *= mul;
      }
    };

    // the largest of a row's values, which the lanes of equal c hold
    auto row_max = [](float x) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
      return x;
    };
    constexpr int kSteps = kQuant ? KS / 2 : KS, kPer = kQuant ? 2 : 1;

    int stage = 0, it = 0, w0 = WS * warp;
    uint32_t phase = 0;
    // The walk over the tiles, of 8-bit pages in two forms: the plain one stops (true) before
    // the first step in which a row has to be taken apart, and the other goes on from there;
    // queries with far smaller values begin with it. (One loop with both: what it
    // never runs costs it registers, blocks of 16 rows 2 to 6 %.)
    auto walk = [&](auto both) -> bool {
      constexpr bool kBoth = decltype(both)::value;
      for (; it < n_tiles; ++it) {
        // most tiles have landed: one test, and the bounded wait only when not
        if (!__all_sync(0xffffffffu, sm100::mbar_test_wait(full + 8 * stage, phase)) &&
            !sm100::mbar_wait_warp(full + 8 * stage, phase, abort_flag, kTimeoutNs))
          return false;
        const uint32_t tile = ring + stage * S::kStage;
        const uint32_t missing = gone[stage];
        const int box_rows = min(a.p.page, kTile), box_shift = 31 - __clz(box_rows);
        // 16 slots at a time, in a loop that is not unrolled: code that a short call runs
        // once or twice costs it more to fetch than to run (two at a time side by side:
        // 31 instead of 25 us for 4 x 4 tokens under a window of 4096, and no less for 8
        // x 128K slots)
#pragma unroll 1
        for (; w0 < WS * (warp + 1); w0 += 16) {
          const int j0 = sp.tile(v_begin + it) * kTile + w0;
          // where the first row of 16 lies, of the keys; from one part of it to the next
          const uint32_t rows =
              tile + (uint32_t)((w0 & ~(box_rows - 1)) * S::kParts * S::kRowBytes +
                                (w0 & (box_rows - 1)) * S::kRowBytes);
          const uint32_t next_part = (uint32_t)(box_rows * S::kRowBytes);
          // ---- scores: rows of s are slots, columns query rows
          float s[NT][4];
          float ev[2];                     // the value scales' exponents
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
          if constexpr (kQuant) {
            float ks[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint8_t* at = smem + stage * S::kStage + w0 + 8 * i + g;
              ks[i] = pow2_byte(at[S::kKs]);
              ev[i] = (float)((int)at[S::kVs] - 127);
            }
#pragma unroll
            for (int x = 0; x < KS / 2; ++x) {   // two chunks of 16 dimensions
              uint32_t w[4];
              ldmatrix4(w, rows + swizzled<S::kRowBytes>(lane & 15, 2 * x + (lane >> 4)));
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t af[4] = {e4m3x2_half2(w[2 * y]), e4m3x2_half2(w[2 * y + 1]),
                                        e4m3x2_half2(w[2 * y] >> 16),
                                        e4m3x2_half2(w[2 * y + 1] >> 16)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<true>(s[nt], af, qf[nt][2 * x + y][0], qf[nt][2 * x + y][1]);
              }
            }
            if (kBoth && any_far) {
              // those rows' products anew: values and codes as bf16 numbers, both exact
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float down = far_down[nt * 8 + g];
                const uint2* q = reinterpret_cast<const uint2*>(
                    static_cast<const __nv_bfloat16*>(a.q) + (long long)far_row[nt * 8 + g] * D);
                float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int x = 0; x < KS / 2; ++x) {
                  uint32_t w[4];
                  ldmatrix4(w, rows + swizzled<S::kRowBytes>(lane & 15, 2 * x + (lane >> 4)));
#pragma unroll
                  for (int y = 0; y < 2; ++y) {
                    const uint2 u = down > 0.f ? q[4 * (2 * x + y) + c] : make_uint2(0, 0);
                    auto times = [&](uint32_t v) -> uint32_t {
                      return sm100::pack_bf16x2(__uint_as_float(v << 16) * down,
                                                __uint_as_float(v & 0xffff0000u) * down);
                    };
                    auto bf16 = [](uint32_t codes) -> uint32_t {
                      const float2 f = half2_values(e4m3x2_half2(codes));
                      return sm100::pack_bf16x2(f.x, f.y);
                    };
                    const uint32_t af[4] = {bf16(w[2 * y]), bf16(w[2 * y + 1]),
                                            bf16(w[2 * y] >> 16), bf16(w[2 * y + 1] >> 16)};
                    mma16816<false>(t, af, times(u.x), times(u.y));
                  }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (far_down[nt * 8 + 2 * c + (i & 1)] > 0.f) s[nt][i] = t[i];
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[nt][i] *= ks[i >> 1] * sl2[nt][i & 1];
          } else {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t af[4];
              ldmatrix4(af, rows + (k / 4) * next_part +
                                swizzled<S::kRowBytes>(lane & 15, 2 * (k % 4) + (lane >> 4)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<false>(s[nt], af, qf[nt][k][0], qf[nt][k][1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[nt][i] *= sl2[nt][i & 1];
          }
          // ---- slots that some row does not see
          const bool whole = missing == 0 && sp.whole(a, j0, 16);
          auto lost = [&](int x) { return (missing >> ((w0 + x) >> box_shift) & 1u) != 0; };
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int x = 8 * i + g;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (lost(x) || !paged_sees(a, pos(nt, h), j0 + x)) s[nt][2 * i + h] = -INFINITY;
            }
          }
          // the halves of slots 2c, 2c + 1, and + 8 to keep: those that the row at p, or
          // (kAny) any row, sees
          constexpr int kAny = -1;
          auto keep_slots = [&](int p, uint32_t (&keep)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              keep[i] = 0;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int x = 8 * i + 2 * c + y;
                const bool see = p == kAny ? j0 + x < sp.hi && sp.meets(a, j0 + x, 1)
                                           : paged_sees(a, p, j0 + x);
                if (see && !lost(x)) keep[i] |= 0xffffu << (16 * y);
              }
            }
          };
          // the operand of 16 slots and of 16 dimensions (8 bits: two steps' at once)
          auto load_values = [&](int k, uint32_t (&af)[kPer][4]) {
            if constexpr (kQuant) {
              uint32_t w[4];
              ldmatrix4_trans(w, rows + S::kKv +
                                     swizzled<S::kRowBytes>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                // bytes: (slot 2c, dimensions 2g, 2g + 1), (slot 2c + 1, the same)
                const uint32_t lo = __byte_perm(w[2 * y], 0, 0x3120);
                const uint32_t hi = __byte_perm(w[2 * y + 1], 0, 0x3120);
                af[y][0] = e4m3x2_half2(lo);
                af[y][1] = e4m3x2_half2(lo >> 16);
                af[y][2] = e4m3x2_half2(hi);
                af[y][3] = e4m3x2_half2(hi >> 16);
              }
            } else {
              const int row = (lane & 7) + ((lane & 16) >> 1);
              const int chunk = 2 * (k % 4) + ((lane >> 3) & 1);
              ldmatrix4_trans(af[0], rows + S::kKv + (k / 4) * next_part +
                                         swizzled<S::kRowBytes>(row, chunk));
            }
          };
          auto mask = [&](const uint32_t (&keep)[2], uint32_t (&af)[kPer][4]) {
#pragma unroll
            for (int x = 0; x < kPer; ++x)
#pragma unroll
              for (int i = 0; i < 4; ++i) af[x][i] &= keep[i >> 1];
          };
          // ---- raise the maxima when a score passes its bound: rare after the first tile
          float top[NT][2], top2[NT][2];
          bool raise = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              top[nt][h] = top2[nt][h] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                top[nt][h] = fmaxf(top[nt][h], s[nt][2 * i + h]);
                if (kQuant) top2[nt][h] = fmaxf(top2[nt][h], s[nt][2 * i + h] + ev[i]);
              }
              raise |= top[nt][h] > sub[nt][h] + kRescaleLog2;
              if (kQuant) raise |= top2[nt][h] > sub2[nt][h] + (kRescaleLog2 + kHalfUp);
            }
          if (kQuant) raise |= fminf(ev[0], ev[1]) < low;
          if (__any_sync(0xffffffffu, raise)) {
            low = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // (to x rounded down, less `up`); what sums are multiplied by
                auto raise_to = [&](float x, float up, float& sub_) -> float {
                  if (!(x > sub_ + (kRescaleLog2 + up))) return 1.f;
                  const float to = floorf(x) - up;
                  const float alpha = sub_ == -INFINITY ? 0.f : exp2f(sub_ - to);
                  sub_ = to;
                  return alpha;
                };
                const float alpha = raise_to(row_max(top[nt][h]), 0.f, sub[nt][h]);
                l[nt][h] *= alpha;
                scale_row(nt, h,
                          kQuant ? raise_to(row_max(top2[nt][h]), kHalfUp, sub2[nt][h]) : alpha);
                if (kQuant) low = fmaxf(low, sub2[nt][h] - sub[nt][h]);    // (NaN: nothing seen)
              }
            // the rows (bit 2 nt + h) that have met too much for a slot that they see, as all
            // lanes that hold the row know
            uint32_t wide = 0;
            if (kQuant && __any_sync(0xffffffffu, fminf(ev[0], ev[1]) < low)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  bool far = false;
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    far |= s[nt][2 * i + h] > -INFINITY && ev[i] < sub2[nt][h] - sub[nt][h];
                  uint32_t of_c = __ballot_sync(0xffffffffu, far);
                  of_c |= of_c >> 16;
                  of_c |= of_c >> 8;
                  of_c |= of_c >> 4;
                  wide |= (of_c >> c & 1u) << (2 * nt + h);
                }
            }
            if (!kBoth && __any_sync(0xffffffffu, wide)) return true;
            if (kBoth && __any_sync(0xffffffffu, wide)) {
              // Rows to which a slot's value scale is too small for a half's range: their
              // products of this step, weights in two bf16 numbers, codes in one (exact). What
              // follows finds them without scores: weights of 0, which NaN codes, here left to
              // it, make NaN.
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t wh[2], wl[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float w[2] = {0.f, 0.f};
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float& x = s[nt][2 * i + h];
                    if (wide >> (2 * nt + h) & 1u) {
                      l[nt][h] += sm100::ex2_approx(x - sub[nt][h]);
                      w[h] = sm100::ex2_approx(x + (ev[i] - sub2[nt][h]));
                      x = -INFINITY;
                    }
                  }
                  const uint32_t u = sm100::pack_bf16x2(w[0], w[1]);
                  wh[i] = transpose8x8(u);
                  wl[i] = transpose8x8(sm100::pack_bf16x2(
                      w[0] - __uint_as_float(u << 16), w[1] - __uint_as_float(u & 0xffff0000u)));
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                  uint32_t af[kPer][4];
                  load_values(k, af);
#pragma unroll
                  for (int x = 0; x < kPer; ++x) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      const float2 f = half2_values(af[x][i]);
                      af[x][i] = sm100::pack_bf16x2(f.x == f.x ? f.x : 0.f, f.y == f.y ? f.y : 0.f);
                    }
                    mma16816<false>(o[nt][kPer * k + x], af[x], wh[0], wh[1]);
                    mma16816<false>(o[nt][kPer * k + x], af[x], wl[0], wl[1]);
                  }
                }
              }
            }
          }
          // ---- weights, as B operands: one half, or two bf16 numbers, what the first
          // leaves being the second
          uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // (a row that has seen nothing has scores of -inf alone)
            const float less[2] = {fmaxf(sub[nt][0], -FLT_MAX), fmaxf(sub[nt][1], -FLT_MAX)};
            const float less2[2] = {fmaxf(sub2[nt][0], -FLT_MAX), fmaxf(sub2[nt][1], -FLT_MAX)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float w[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x = s[nt][2 * i + h];
                const float p = sm100::ex2_approx(x - less[h]);
                l[nt][h] += p;
                w[h] = kQuant ? sm100::ex2_approx(x + (ev[i] - less2[h])) : p;
              }
              if constexpr (kQuant) {
                pf[nt][i] = transpose8x8(pack_half2(w[0], w[1]));
              } else {
                // the first below the weight, so that both are above 0, and infinite values
                // times both keep their sign
                const uint32_t b0 = max(__float_as_uint(w[0]), 1u) - 1u;
                const uint32_t b1 = max(__float_as_uint(w[1]), 1u) - 1u;
                const uint32_t u = __byte_perm(b0, b1, 0x7632);
                pf[nt][i] = transpose8x8(u);
                pl[nt][i] = transpose8x8(sm100::pack_bf16x2(
                    w[0] - __uint_as_float(u << 16), w[1] - __uint_as_float(u & 0xffff0000u)));
              }
            }
          }
          // ---- their products with the values: rows of o are dimensions
          auto multiply = [&](float (&acc)[4], const uint32_t (&af)[4], int nt) {
            mma16816<kQuant>(acc, af, pf[nt][0], pf[nt][1]);
            if (!kQuant) mma16816<kQuant>(acc, af, pl[nt][0], pl[nt][1]);
          };
          if (whole) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              uint32_t af[kPer][4];
              load_values(k, af);
#pragma unroll
              for (int x = 0; x < kPer; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) multiply(o[nt][kPer * k + x], af[x], nt);
            }
          } else {
            // where tokens differ in what they see, a value that is not finite would reach
            // the rows that do not see it
            bool apart = false;
            if (sp.pmin != sp.pmax) {
              uint32_t keep[2];
              keep_slots(kAny, keep);
#pragma unroll 1
              for (int k = 0; k < kSteps; ++k) {
                uint32_t af[kPer][4];
                load_values(k, af);
                mask(keep, af);
                constexpr uint32_t ones = kQuant ? 0x7c007c00u : 0x7f807f80u;   // exponents
#pragma unroll
                for (int x = 0; x < kPer; ++x)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t u = af[x][i] & ones;
                    apart |= (u & 0xffffu) == (ones & 0xffffu) || (u >> 16) == (ones >> 16);
                  }
              }
              apart = __any_sync(0xffffffffu, apart);
            }
            if (!apart) {
              uint32_t keep[2];
              keep_slots(kAny, keep);
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                uint32_t af[kPer][4];
                load_values(k, af);
                mask(keep, af);
#pragma unroll
                for (int x = 0; x < kPer; ++x)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) multiply(o[nt][kPer * k + x], af[x], nt);
              }
            }
            for (int p = max(sp.pmin, 0); apart && p <= sp.pmax; ++p) {
              uint32_t keep[2];
              keep_slots(p, keep);
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                uint32_t af[kPer][4];
                load_values(k, af);
                mask(keep, af);
#pragma unroll
                for (int x = 0; x < kPer; ++x)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    float(&acc)[4] = o[nt][kPer * k + x];
                    float y[4] = {acc[0], acc[1], acc[2], acc[3]};
                    multiply(y, af[x], nt);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                      if (pos(nt, i & 1) == p) acc[i] = y[i];
                  }
              }
            }
          }
        }
        w0 = WS * warp;
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(free_ + 8 * stage);
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      return false;
    };
    if constexpr (kQuant) {
      if (any_far || walk(std::false_type())) walk(std::true_type());
    } else {
      walk(std::false_type());
    }
    __syncthreads();                         // every warp has read the ring

    // ---- the warps' parts meet in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float ls = l[nt][h];
#pragma unroll
        for (int x = 4; x < 32; x *= 2) ls += __shfl_xor_sync(0xffffffffu, ls, x);
        const int r = nt * 8 + 2 * c + h;
        if (g == 0) {
          sM[warp * RB + r] = sub[nt][h];    // -inf where the row saw nothing
          sL[warp * RB + r] = ls;
        }
        const float mul = kQuant && sub[nt][h] > -INFINITY ? exp2f(sub2[nt][h] - sub[nt][h]) : 1.f;
        float* row = sO + (warp * RB + r) * D;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if constexpr (kQuant) {
            *reinterpret_cast<float2*>(row + 16 * k + 2 * g) =
                make_float2(o[nt][k][h] * mul, o[nt][k][2 + h] * mul);
          } else {
            row[16 * k + g] = o[nt][k][h];
            row[16 * k + 8 + g] = o[nt][k][2 + h];
          }
        }
      }
  }
  __syncthreads();
  if (threadIdx.x == 0 && (*abort_flag || *never) && a.status)
    atomicExch(a.status, (int)RA_ERR_TIMEOUT);
  for (int i = threadIdx.x; i < RB * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    if (r >= R) continue;
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
    const int t = (r0 + r) / grp, h = hk * grp + (r0 + r) % grp;
    const long long row = (long long)(sq.row0 + t) * a.H_q + h;
    if (a.n_split > 1) {
      const long long part = paged_part(a, item, split, r);
      if (!in_range(part, 1, paged_part_rows(a), a.status)) continue;
      if (d == 0) {
        a.part_ml[2 * part] = mx;
        a.part_ml[2 * part + 1] = ls;
      }
      if (n_tiles > 0) *reinterpret_cast<float4*>(a.part_o + part * D + d) = y;
    } else {
      const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);   // 0: no slot; NaN stays
      if (in_range(row * D + d, 4, (long long)a.rows * a.H_q * D, a.status))
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + d) =
            make_uint2(sm100::pack_bf16x2(y.x * inv, y.y * inv),
                       sm100::pack_bf16x2(y.z * inv, y.w * inv));
      if (d == 0 && a.lse) {
        const long long at = paged_lse_at(a, b, sq.row0 + t, t, h);
        if (in_range(at, 1, (long long)a.rows * a.H_q, a.status))
          a.lse[at] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * kLn2;
      }
    }
  }
}

// ---- Joining chunks. A chunk without a visible slot has the sum 0, and outputs that
// nobody wrote: they may be read, never used. Every CTA waits for the grid before it,
// as the next one takes this one's end for the end of both, and before it reads
// offsets, which may come from a grid that that one has waited for.

__device__ __forceinline__ float chunk_weight(float2 ml, float m) {     // below 0: nothing there
  if (ml.x == -INFINITY && ml.y == 0.f) return -1.f;
  return ml.x == m ? 1.f : exp2f(ml.x - m);
}

// Four outputs of row `row` of q and of head h, from d on.
template <int D>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, int row, int h, int d, float4 y,
                                          float m, float l) {
  const long long at = ((long long)row * a.H_q + h) * D + d;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);     // 0: no slot; NaN stays
  if (in_range(at, 4, (long long)a.rows * a.H_q * D, a.status))
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(sm100::pack_bf16x2(y.x * inv, y.y * inv), sm100::pack_bf16x2(y.z * inv, y.w * inv));
  if (d == 0 && a.lse) {
    const long long to = paged_lse_at(a, a.cu ? 0 : row / a.T, row, a.cu ? 0 : row % a.T, h);
    if (in_range(to, 1, (long long)a.rows * a.H_q, a.status))
      a.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// Few rows: a CTA joins one row, whose chunks may be hundreds: its parts, each D / 4
// threads, a float4 of the output a thread, take every kParts-th chunk.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_few_kernel(const PagedAttnArgs a, int rows) {
  constexpr int kLanes = D / 4, kParts = kJoinThreads / kLanes, kPre = 4;
  __shared__ float4 sO[kParts][kLanes];
  __shared__ float sM[kParts], sL[kParts];
  let_dependents_start();
  if (a.cu) wait_for_prior_grid();
  const int item = (int)(blockIdx.x / (uint32_t)rows), r = (int)(blockIdx.x % (uint32_t)rows);
  const PagedBlock blk = paged_block(a, item);
  const int grp = a.H_q / a.p.H_kv;
  const PagedSeq sq = paged_seq(a, blk.b);
  if (!a.cu) wait_for_prior_grid();
  const int r_head = blk.rb * a.block_rows + r;        // of the head's rows
  if (r_head >= sq.n * grp || !paged_mine(a, sq)) return;
  const int part = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  if (!in_range(paged_part(a, item, 0, r), (long long)(a.n_split - 1) * a.block_rows + 1,
                paged_part_rows(a), a.status))
    return;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + paged_part(a, item, 0, r);
  const float* o = a.part_o + paged_part(a, item, 0, r) * D + d;
  float m = -INFINITY, l = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  auto chunk = [&](int s) -> float2 { return ml[s * a.block_rows]; };
  auto outputs = [&](int s) -> float4 {
    return *reinterpret_cast<const float4*>(o + (size_t)s * a.block_rows * D);
  };
  auto add = [&](float2 x, float4 f) {
    const float w = chunk_weight(x, m);
    if (w < 0.f) return;
    l = fmaf(w, x.y, l);
    y.x = fmaf(w, f.x, y.x);
    y.y = fmaf(w, f.y, y.y);
    y.z = fmaf(w, f.z, y.z);
    y.w = fmaf(w, f.w, y.w);
  };
  // the first ones' loads all at once
  float2 pre_ml[kPre];
  float4 pre_o[kPre];
#pragma unroll
  for (int x = 0; x < kPre; ++x) {
    const int s = part + x * kParts;
    pre_ml[x] = s < a.n_split ? chunk(s) : make_float2(-INFINITY, 0.f);
    pre_o[x] = s < a.n_split ? outputs(s) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int x = 0; x < kPre; ++x) m = fmaxf(m, pre_ml[x].x);
  for (int s = part + kPre * kParts; s < a.n_split; s += kParts) m = fmaxf(m, chunk(s).x);
#pragma unroll
  for (int x = 0; x < kPre; ++x) add(pre_ml[x], pre_o[x]);
#pragma unroll 4
  for (int s = part + kPre * kParts; s < a.n_split; s += kParts) add(chunk(s), outputs(s));
  sO[part][d / 4] = y;
  if (d == 0) {
    sM[part] = m;
    sL[part] = l;
  }
  __syncthreads();
  if (part > 0) return;
#pragma unroll
  for (int w = 1; w < kParts; ++w) m = fmaxf(m, sM[w]);
  l = 0.f;
  y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kParts; ++w) {
    const float f = chunk_weight(make_float2(sM[w], sL[w]), m);
    if (f < 0.f) continue;
    const float4 x = sO[w][d / 4];
    l = fmaf(f, sL[w], l);
    y.x = fmaf(f, x.x, y.x);
    y.y = fmaf(f, x.y, y.y);
    y.z = fmaf(f, x.z, y.z);
    y.w = fmaf(f, x.w, y.w);
  }
  store_row<D>(a, sq.row0 + r_head / grp, blk.hk * grp + r_head % grp, d, y, m, l);
}

// Many rows: a warp joins kAtOnce rows (D = 64: pairs of rows) of one block, a float4 of
// the output a lane. Its lanes look at the chunks' maxima and sums, 32 at a time, while
// the first kPre chunks' outputs are on their way; which rows they are the block's first
// chunk has noted, as looking a packed block up would take as long as the rest. What
// bounds it is that way, and code that runs once. Attention of 64 tokens behind 100000
// slots (19 chunks of 2048 rows) 90.5 us, of two sequences under a window of 2048 (2
// chunks of 18432) 85 (weights made for the whole CTA first, in shared memory: 96.5 and
// 88; four rows a warp and four chunks: 91 and 90; one row: 91 and 89).
template <int D, int kAtOnce>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_many_kernel(const PagedAttnArgs a) {
  constexpr int kLanes = D / 4, kPer = 32 / kLanes;           // lanes a row, rows side by side
  constexpr int kRows = kAtOnce * kPer * (kJoinThreads / 32);  // of a CTA
  constexpr int kPre = kAtOnce == 1 ? 8 : 2;
  let_dependents_start();
  wait_for_prior_grid();
  const int cut = blockIdx.x / (256 / kRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane / kLanes;
  const int d = lane % kLanes * 4;
  const int r0 = blockIdx.x % (256 / kRows) * kRows + warp * (kAtOnce * kPer);   // the warp's first
  if (!in_range(cut, 1, a.n_cut, a.status)) return;
  const int4 blk = a.part_block[cut];
  if (a.cu && blk.y <= 0) return;                  // no such block (packed calls alone)
  // chunk s of row r is part s * 256 + r of the block's
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + (size_t)cut * a.n_split * 256;
  const float* o = a.part_o + ((size_t)cut * a.n_split * 256 + r0 + half) * D + d;
  float4 pre[kPre][kAtOnce];
#pragma unroll
  for (int s = 0; s < kPre; ++s)
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (s < a.n_split)
        pre[s][e] = *reinterpret_cast<const float4*>(o + ((size_t)s * 256 + e * kPer) * D);
  float m[kAtOnce][kPer], l[kAtOnce][kPer], w[kAtOnce][kPer];
  float4 y[kAtOnce];
  auto chunk = [&](int s, int e, int p) -> float2 {
    return s < a.n_split ? ml[(size_t)s * 256 + r0 + e * kPer + p] : make_float2(-INFINITY, 0.f);
  };
#pragma unroll
  for (int e = 0; e < kAtOnce; ++e) {
    y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      l[e][p] = 0.f;
      m[e][p] = -INFINITY;
      for (int s = lane; s < a.n_split; s += 32) m[e][p] = fmaxf(m[e][p], chunk(s, e, p).x);
#pragma unroll
      for (int x = 16; x > 0; x /= 2)
        m[e][p] = fmaxf(m[e][p], __shfl_xor_sync(0xffffffffu, m[e][p], x));
    }
  }
  auto add = [&](int s, int e, float4 f) {
    float x = __shfl_sync(0xffffffffu, w[e][0], s & 31);
    if (kPer == 2) {
      const float x1 = __shfl_sync(0xffffffffu, w[e][kPer - 1], s & 31);
      if (half) x = x1;
    }
    if (x < 0.f) return;
    y[e].x = fmaf(x, f.x, y[e].x);
    y[e].y = fmaf(x, f.y, y[e].y);
    y[e].z = fmaf(x, f.z, y[e].z);
    y[e].w = fmaf(x, f.w, y[e].w);
  };
  for (int s0 = 0; s0 < a.n_split; s0 += 32) {
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const float2 x = chunk(s0 + lane, e, p);
        w[e][p] = chunk_weight(x, m[e][p]);
        if (!(w[e][p] < 0.f)) l[e][p] = fmaf(w[e][p], x.y, l[e][p]);
      }
    if (s0 == 0) {
#pragma unroll
      for (int s = 0; s < kPre; ++s)
        if (s < a.n_split)
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) add(s, e, pre[s][e]);
    }
    const int end = min(s0 + 32, a.n_split);
#pragma unroll 4
    for (int s = s0 > 0 ? s0 : kPre; s < end; ++s)
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e)
        add(s, e, *reinterpret_cast<const float4*>(o + ((size_t)s * 256 + e * kPer) * D));
  }
  const int grp = a.H_q / a.p.H_kv, tt = 128 / grp;
#pragma unroll
  for (int e = 0; e < kAtOnce; ++e) {
    float lr = 0.f, mr = -INFINITY;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
#pragma unroll
      for (int x = 16; x > 0; x /= 2) l[e][p] += __shfl_xor_sync(0xffffffffu, l[e][p], x);
      if (p == half) {
        lr = l[e][p];
        mr = m[e][p];
      }
    }
    const int r = r0 + e * kPer + half, in = r & 127;
    const int t = (r >> 7) * tt + in / grp;
    if (in >= tt * grp || t >= blk.y) continue;                // no token's
    store_row<D>(a, blk.x + t, blk.z * grp + in % grp, d, y[e], mr, lr);
  }
}

template <int D, int NT, bool kQuant>
ra_status launch_rows(const PagedAttnArgs& a, cudaStream_t stream) {
  using S = Smem<D, NT, kQuant>;
  CUtensorMap mk, mv;
  const int box_rows = a.p.page < S::kTile ? a.p.page : S::kTile;
  if (!make_page_map(&mk, a.p, a.p.k, box_rows, S::kParts) ||
      !make_page_map(&mv, a.p, a.p.v, box_rows, S::kParts))
    return RA_ERR_LAUNCH;
  const long long grid = (long long)a.n_items * a.n_split;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  auto kern = paged_attn_kernel<D, NT, kQuant>;
  static std::atomic<uint64_t> allowed;
  if (!allow_smem(kern, S::kBytes, allowed)) return RA_ERR_LAUNCH;
  return launch_early(kern, grid, kThreads, S::kBytes, stream, mk, mv, a) ? RA_OK : RA_ERR_LAUNCH;
}

}  // namespace

ra_status launch_paged_rows(const PagedAttnArgs& a, cudaStream_t stream) {
  auto launch = [&](auto few, auto more) { return a.block_rows == 8 ? few(a, stream) : more(a, stream); };
  if (a.p.D == 64)
    return a.p.quant ? launch(launch_rows<64, 1, true>, launch_rows<64, 2, true>)
                     : launch(launch_rows<64, 1, false>, launch_rows<64, 2, false>);
  return a.p.quant ? launch(launch_rows<128, 1, true>, launch_rows<128, 2, true>)
                   : launch(launch_rows<128, 1, false>, launch_rows<128, 2, false>);
}

ra_status launch_paged_join(const PagedAttnArgs& a, cudaStream_t stream) {
  const long long items = a.n_cut;
  if (a.block_rows <= 16) {
    const long long R = a.few_rows > 0 ? a.few_rows : (long long)a.T * (a.H_q / a.p.H_kv);
    const int rows = R < a.block_rows ? (int)R : a.block_rows;    // those that may hold a token
    const long long grid = items * rows;
    if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
    auto kern = a.p.D == 64 ? paged_join_few_kernel<64> : paged_join_few_kernel<128>;
    return launch_early(kern, grid, kJoinThreads, 0, stream, a, rows) ? RA_OK : RA_ERR_LAUNCH;
  }
  // half the rows a CTA where CTAs would be few
  int rows = 2 * kJoinThreads / (a.p.D / 4);
  auto kern = a.p.D == 64 ? paged_join_many_kernel<64, 2> : paged_join_many_kernel<128, 2>;
  if (items * (256 / rows) < 2 * 152) {
    rows /= 2;
    kern = a.p.D == 64 ? paged_join_many_kernel<64, 1> : paged_join_many_kernel<128, 1>;
  }
  const long long grid = items * (256 / rows);
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  return launch_early(kern, grid, kJoinThreads, 0, stream, a) ? RA_OK : RA_ERR_LAUNCH;
}

}  // namespace ra
