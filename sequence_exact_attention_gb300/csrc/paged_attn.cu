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
// 1 and 2^5, whatever the scales. Queries become halves times a power of two a row
// (exact for values down to 2^-17 of the row's largest).
// Roundings: weights to half (2^-12) or, in bf16 pages, to bf16 (2^-9); sums and
// statistics are float32.
//
// For up to 16 query rows a sequence and key/value head (new tokens times the heads
// that share it; more: paged_tiles.cu). A CTA takes one chunk of the slots of one
// sequence and key/value head. A producer warp looks the pages up, a lane for each, and asks
// for their boxes (TMA, swizzled, so that ldmatrix meets no bank conflict); four
// warps share a tile's slots and keep running maxima, sums and outputs of their own,
// joined in shared memory at the end. Chunks of a long axis are joined by a second
// kernel. Everything is summed in a fixed order: results repeat bit for bit.
//
// Slots that a row does not see change no bit of its results, whatever they hold:
// scores are replaced, and in tiles that are not whole the values' operands are
// masked, too (0 times a NaN is not 0); where the block's tokens differ in what
// they see, such a tile is multiplied once for each of them.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <cstdint>

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
constexpr float kRescaleLog2 = 4.f;       // weights stay below 2^5
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
  static constexpr int kTile = !kQuant && D == 128 ? 64 : 128;     // slots
  static constexpr int kRowBytes = kQuant ? D : 128;               // of a box's row
  static constexpr int kBoxes = kQuant ? 1 : D / 64;               // boxes a row takes
  static constexpr int kPart = kTile * kRowBytes;
  static constexpr int kKv = kBoxes * kPart;                       // keys, or values, of a tile
  static constexpr int kKs = 2 * kKv, kVs = kKs + (kQuant ? kTile : 0);
  static constexpr int kStage = (kVs + (kQuant ? kTile : 0) + 1023) / 1024 * 1024;
  static constexpr int kStages = kStage <= 18 * 1024 ? 4 : 3;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kOut = kWarps * 8 * NT * D * 4;
  static constexpr int kData = kRing > kOut ? kRing : kOut;
  static constexpr int kMl = kData;                                // [2][kWarps][8 NT]
  static constexpr int kFull = kMl + 2 * kWarps * 8 * NT * 4;      // [kStages]
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
  constexpr int MB = WS / 16;
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
  const int split = blockIdx.x % a.n_split;
  const int bh = blockIdx.x / a.n_split;
  const int hk = bh % H_kv, b = bh / H_kv;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      sm100::mbar_init(full + 8 * i, 1);
      sm100::mbar_init(free_ + 8 * i, kWarps);
    }
    *abort_flag = *never = 0;
    sm100::fence_mbar_init();
  }
  const PagedSeq sq = paged_seq(a, b);
  const int R = sq.n * grp;                 // query rows of this head
  if (R == 0) return;                       // a sequence without new tokens
  const int first = sq.len - sq.n;          // position of the first new token
  PagedSpan<kTile> sp;
  sp.init(a, first, first + sq.n - 1);
  const int v_begin = split * a.chunk;
  const int n_tiles = max(min(sp.n, v_begin + a.chunk) - v_begin, 0);
  let_dependents_start();
  __syncthreads();

  if (warp == kWarps) {
    // ======================= producer =======================
    const int box_rows = min(a.p.page, kTile);
    const int shift = 31 - __clz(a.p.page);
    const int n_box = kTile / box_rows;     // at most 8: a lane for each
    const int at = lane * box_rows;
    auto look_up = [&](int i) -> int {      // -1: nothing to load; -2: no such page
      if (i >= n_tiles || lane >= n_box) return -1;
      const int j = sp.tile(v_begin + i) * kTile + at;
      if (j >= sp.hi || !sp.meets(a, j, box_rows)) return -1;
      const int at_page = j >> shift;
      if (at_page >= a.width) return -2;
      const int id = __ldg(a.table + (size_t)b * a.width + at_page);
      return id >= 0 && id < a.p.n_pages ? id : -2;
    };
    int id = look_up(0);
    int i = 0, stage = 0;
    uint32_t phase = 0;
    bool bad = false;
    for (; i < n_tiles; ++i) {
      const int next = look_up(i + 1);
      if (i >= S::kStages &&
          !sm100::mbar_wait_warp(free_ + 8 * stage, phase ^ 1, abort_flag, kTimeoutNs))
        break;
      const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
      const uint32_t missing = __ballot_sync(0xffffffffu, id == -2);
      const uint32_t dst = ring + stage * S::kStage, bar = full + 8 * stage;
      if (lane == 0) {
        gone[stage] = missing;
        sm100::mbar_arrive_expect_tx(
            bar, __popc(there) * box_rows * (2 * S::kBoxes * S::kRowBytes + (kQuant ? 2 : 0)));
      }
      bad |= missing != 0;
      __syncwarp();
      if (id >= 0) {
        const int row = (sp.tile(v_begin + i) * kTile + at) & (a.p.page - 1);
        const int z = id * H_kv + hk;
#pragma unroll
        for (int x = 0; x < S::kBoxes; ++x)
          tma_load_3d(dst + x * S::kPart + at * S::kRowBytes, &tm_k, bar, x * 64, row, z);
#pragma unroll
        for (int x = 0; x < S::kBoxes; ++x)
          tma_load_3d(dst + S::kKv + x * S::kPart + at * S::kRowBytes, &tm_v, bar, x * 64, row, z);
        if (kQuant) {
          const size_t from = (size_t)z * a.p.page + row;
          sm100::bulk_load(dst + S::kKs + at, a.p.ks + from, box_rows, bar);
          sm100::bulk_load(dst + S::kVs + at, a.p.vs + from, box_rows, bar);
        }
      }
      id = next;
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
    int pos[NT][2];                          // their positions; below 0: sees nothing
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const bool row_ok = r < R;
      const long long off =
          row_ok ? ((long long)(sq.row0 + r / grp) * a.H_q + hk * grp + r % grp) * D : 0;
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
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[nt][k][0] = pack_half2(__uint_as_float(u[k].x << 16) * down,
                                    __uint_as_float(u[k].x & 0xffff0000u) * down);
          qf[nt][k][1] = pack_half2(__uint_as_float(u[k].y << 16) * down,
                                    __uint_as_float(u[k].y & 0xffff0000u) * down);
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
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rr = nt * 8 + 2 * c + h;
        pos[nt][h] = rr < R ? first + rr / grp : -1;
      }
    }

    // Running state of rows 2c and 2c + 1. What the exponents subtract: the running
    // maximum in base 2, rounded down, so that raising it scales sums by a power of
    // two; a score that passes `bound` raises it. (sub2, bound2: those of the
    // weights, with the values' scales.)
    float o[NT][KS][4];
    float sub[NT][2], bound[NT][2], sub2[NT][2], bound2[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sub[nt][h] = sub2[nt][h] = l[nt][h] = 0.f;
        bound[nt][h] = bound2[nt][h] = -INFINITY;
      }
    }
    auto scale_row = [&](int nt, int h, float mul) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        o[nt][k][h] *= mul;
        o[nt][k][2 + h] *= mul;
      }
    };

    int stage = 0;
    uint32_t phase = 0;
    for (int it = 0; it < n_tiles; ++it) {
      // most tiles have landed: one test, and the bounded wait only when not
      if (!__all_sync(0xffffffffu, sm100::mbar_test_wait(full + 8 * stage, phase)) &&
          !sm100::mbar_wait_warp(full + 8 * stage, phase, abort_flag, kTimeoutNs))
        break;
      const int w0 = WS * warp;              // the warp's first slot in the tile
      const int j0 = sp.tile(v_begin + it) * kTile + w0;
      const uint32_t tile = ring + stage * S::kStage;
      const uint32_t missing = gone[stage];
      // ---- scores: rows of s are slots, columns query rows
      float s[MB][NT][4];
      int ev[MB][2];                         // the value scales' exponents
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int slot = w0 + 16 * m + (lane & 15);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][nt][i] = 0.f;
        if constexpr (kQuant) {
          float ks[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ks[i] = pow2_byte(smem[stage * S::kStage + S::kKs + w0 + 16 * m + 8 * i + g]);
            ev[m][i] = (int)smem[stage * S::kStage + S::kVs + w0 + 16 * m + 8 * i + g] - 127;
          }
#pragma unroll
          for (int x = 0; x < KS / 2; ++x) {   // two chunks of 16 dimensions
            uint32_t w[4];
            ldmatrix4(w, tile + swizzled<S::kRowBytes>(slot, 2 * x + (lane >> 4)));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t af[4] = {e4m3x2_half2(w[2 * y]), e4m3x2_half2(w[2 * y + 1]),
                                      e4m3x2_half2(w[2 * y] >> 16),
                                      e4m3x2_half2(w[2 * y + 1] >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(s[m][nt], af, qf[nt][2 * x + y][0], qf[nt][2 * x + y][1]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[m][nt][i] *= ks[i >> 1] * sl2[nt][i & 1];
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t af[4];
            ldmatrix4(af, tile + (k / 4) * S::kPart +
                              swizzled<S::kRowBytes>(slot, 2 * (k % 4) + (lane >> 4)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<false>(s[m][nt], af, qf[nt][k][0], qf[nt][k][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[m][nt][i] *= sl2[nt][i & 1];
        }
      }
      // ---- tiles that some row does not see in full
      const int box_shift = 31 - __clz(min(a.p.page, kTile));
      const bool whole = missing == 0 && sp.whole(a, j0, WS);
      if (!whole) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int x = 16 * m + 8 * i + g;
            const bool lost = missing >> ((w0 + x) >> box_shift) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (lost || !paged_sees(a, pos[nt][h], j0 + x)) s[m][nt][2 * i + h] = -INFINITY;
          }
      }
      // ---- raise the maxima when a score passes its bound: rare after the first tile
      float top[NT][2], top2[NT][2];
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[nt][h] = top2[nt][h] = -INFINITY;
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = s[m][nt][2 * i + h];
              top[nt][h] = fmaxf(top[nt][h], x);
              if (kQuant) top2[nt][h] = fmaxf(top2[nt][h], x + (float)ev[m][i]);
            }
          raise |= top[nt][h] > bound[nt][h];
          if (kQuant) raise |= top2[nt][h] > bound2[nt][h];
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = top[nt][h], y = top2[nt][h];
#pragma unroll
            for (int d = 4; d < 32; d *= 2) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
              if (kQuant) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
            }
            if (x > bound[nt][h]) {
              const float to = floorf(x);
              const float alpha = bound[nt][h] == -INFINITY ? 0.f : exp2f(sub[nt][h] - to);
              sub[nt][h] = to;
              bound[nt][h] = to + kRescaleLog2;
              l[nt][h] *= alpha;
              if (!kQuant) scale_row(nt, h, alpha);
            }
            if (kQuant && y > bound2[nt][h]) {
              const float to = floorf(y);
              const float alpha = bound2[nt][h] == -INFINITY ? 0.f : exp2f(sub2[nt][h] - to);
              sub2[nt][h] = to;
              bound2[nt][h] = to + kRescaleLog2;
              scale_row(nt, h, alpha);
            }
          }
      }
      // ---- weights, as B operands
      uint32_t pf[MB][NT][2];
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = s[m][nt][2 * i + h];
              const float p = sm100::ex2_approx(x - sub[nt][h]);
              l[nt][h] += p;
              w[h] = kQuant ? sm100::ex2_approx(x + ((float)ev[m][i] - sub2[nt][h])) : p;
            }
            pf[m][nt][i] = transpose8x8(kQuant ? pack_half2(w[0], w[1])
                                               : sm100::pack_bf16x2(w[0], w[1]));
          }
      // ---- their products with the values: rows of o are dimensions. p: the
      // position whose rows alone count, with the slots that it sees; below 0: all
      auto add_values = [&](int p) {
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};     // slots 2c, 2c + 1, and + 8
          // o += v w of one product, for the rows that count
          auto add = [&](int nt, int k, const uint32_t (&af)[4]) {
            if (p < 0) {
              mma16816<kQuant>(o[nt][k], af, pf[m][nt][0], pf[m][nt][1]);
            } else {
              float y[4] = {o[nt][k][0], o[nt][k][1], o[nt][k][2], o[nt][k][3]};
              mma16816<kQuant>(y, af, pf[m][nt][0], pf[m][nt][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (pos[nt][i & 1] == p) o[nt][k][i] = y[i];
            }
          };
          if (p >= 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              keep[i] = 0;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int x = 16 * m + 8 * i + 2 * c + y;
                if (!(missing >> ((w0 + x) >> box_shift) & 1u) && paged_sees(a, p, j0 + x))
                  keep[i] |= 0xffffu << (16 * y);
              }
            }
          }
          if constexpr (kQuant) {
            const int slot = w0 + 16 * m + (lane & 15);
#pragma unroll
            for (int x = 0; x < KS / 2; ++x) {
              uint32_t w[4];
              ldmatrix4_trans(w, tile + S::kKv +
                                     swizzled<S::kRowBytes>(slot, 2 * x + (lane >> 4)));
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                // bytes: (slot 2c, dimensions 2g, 2g + 1), (slot 2c + 1, the same)
                const uint32_t lo = __byte_perm(w[2 * y], 0, 0x3120);
                const uint32_t hi = __byte_perm(w[2 * y + 1], 0, 0x3120);
                const uint32_t af[4] = {e4m3x2_half2(lo) & keep[0], e4m3x2_half2(lo >> 16) & keep[0],
                                        e4m3x2_half2(hi) & keep[1], e4m3x2_half2(hi >> 16) & keep[1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  add(nt, 2 * x + y, af);
              }
            }
          } else {
            const int slot = w0 + 16 * m + (lane & 7) + ((lane & 16) >> 1);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t af[4];
              ldmatrix4_trans(af, tile + S::kKv + (k / 4) * S::kPart +
                                      swizzled<S::kRowBytes>(slot, 2 * (k % 4) + ((lane >> 3) & 1)));
#pragma unroll
              for (int x = 0; x < 4; ++x) af[x] &= keep[x >> 1];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) add(nt, k, af);
            }
          }
        }
      };
      if (whole) {
        add_values(-1);
      } else {
        for (int p = max(sp.pmin, 0); p <= sp.pmax; ++p) add_values(p);
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(free_ + 8 * stage);
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
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
          // -inf where the row saw nothing
          sM[warp * RB + r] = bound[nt][h] == -INFINITY ? -INFINITY : sub[nt][h];
          sL[warp * RB + r] = ls;
        }
        const float mul = kQuant ? exp2f(sub2[nt][h] - sub[nt][h]) : 1.f;
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
    const int t = r / grp, h = hk * grp + r % grp;
    const long long row = (long long)(sq.row0 + t) * a.H_q + h;
    if (a.n_split > 1) {
      const long long part = (long long)split * a.rows * a.H_q + row;
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

// Joins the chunks of one query row: the warps share the chunks, a warp's lanes
// the row's D values. A chunk without a visible slot has the sum 0.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
paged_join_kernel(const PagedAttnArgs a) {
  constexpr int V = D / 32;                  // values a lane
  __shared__ float sO[kJoinWarps][D], sM[kJoinWarps], sL[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x;          // (token row, head)
  const int tok = (int)(row / a.H_q), h = (int)(row % a.H_q);
  let_dependents_start();
  wait_for_prior_grid();
  // the token's sequence; rows behind the last one stay as they are
  int b, t;
  if (a.cu) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= tok) lo = mid;
      else hi = mid;
    }
    b = lo;
    const PagedSeq sq = paged_seq(a, b);
    t = tok - sq.row0;
    if (t < 0 || t >= sq.n) return;
  } else {
    b = tok / a.T;
    t = tok % a.T;
  }
  const long long stride = (long long)a.rows * a.H_q;
  float y[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.f;
  for (int s = warp; s < a.n_split; s += kJoinWarps) {
    const long long part = s * stride + row;
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
  const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);
  if (in_range(row * D + threadIdx.x, 1, (long long)a.rows * a.H_q * D, a.status))
    static_cast<__nv_bfloat16*>(a.out)[row * D + threadIdx.x] = __float2bfloat16_rn(z * inv);
  if (threadIdx.x == 0 && a.lse) {
    const long long at = paged_lse_at(a, b, tok, t, h);
    if (in_range(at, 1, (long long)a.rows * a.H_q, a.status))
      a.lse[at] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * kLn2;
  }
}

template <int D, int NT, bool kQuant>
ra_status launch_rows(const PagedAttnArgs& a, cudaStream_t stream) {
  using S = Smem<D, NT, kQuant>;
  CUtensorMap mk, mv;
  const int box_rows = a.p.page < S::kTile ? a.p.page : S::kTile;
  if (!make_page_map(&mk, a.p, a.p.k, box_rows) || !make_page_map(&mv, a.p, a.p.v, box_rows))
    return RA_ERR_LAUNCH;
  const long long grid = (long long)a.B * a.p.H_kv * a.n_split;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  auto kern = paged_attn_kernel<D, NT, kQuant>;
  static std::atomic<uint64_t> allowed;
  if (!allow_smem(kern, S::kBytes, allowed)) return RA_ERR_LAUNCH;
  kern<<<(unsigned)grid, kThreads, S::kBytes, stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
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
  auto kern = a.p.D == 64 ? paged_join_kernel<64> : paged_join_kernel<128>;
  return launch_early(kern, (long long)a.rows * a.H_q, 32 * kJoinWarps, 0, stream, a) ? RA_OK
                                                                                      : RA_ERR_LAUNCH;
}

}  // namespace ra
