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
//   <q, k_j> = sum_groups sk <q, c_j - 8> + zk <q, 1>
//   out      = sum_j (p_j sv) (c_j - 8) + sum_j p_j zv
// so the matrix units see the codes themselves, integers in [-8, 7] that
// half precision holds exactly, and scales and zero points are applied in
// float32: nothing is lost to a dequantised copy, and none is written.
//
// What bounds it: the cache's bytes, 144 a slot and head at D = 128, read
// once. A row has 2 * 2 * D flops a slot, some 4 to 16 rows share a slot, far
// below what the tensor cores need; the work that counts is turning codes
// into operands, about 1.2 instructions a value. So the products run as
// mma.sync m16n8k16, whose operands are registers (codes become the A operand
// where they were loaded; tcgen05 would want them written to shared memory
// again), transposed: M = 16 slots (then 16 dimensions), N = 8 query rows.
//
// A CTA takes one chunk of the slots of one (sequence, key/value head, block
// of 8 or 16 query rows). Its warps take the chunk's tiles of 32 slots in
// turn, each with its own running maximum, sum and output, joined in shared
// memory at the end. Chunks of a long axis are joined by kv4_join_kernel.
// Everything is summed in a fixed order: results repeat bit for bit.
//
// Roundings: q is scaled by a power of two a row and becomes half precision
// (exact for bf16 values down to 2^-14 of the row's largest); p times the
// value scale becomes half precision, 11 bits, relative to the largest value
// scale met so far (a power of two, raised like the running maximum), so a
// weight is off by at most 2^-12 of itself. Sums are float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "checks.cuh"
#include "kv4_internal.h"
#include "sm100.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kRescaleLog2 = 8.0f;      // p stays below 2^8
constexpr float kLn2 = 0.69314718055994531f;

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

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
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
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes of nibbles 0 and 4 (kHigh: 1 and 5) of x, minus 8, as half2. Set
// into the mantissa of 1024 a nibble n reads 1024 + n (1024 + 16 n), from
// which one exact operation makes n - 8.
template <bool kHigh>
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
  const uint32_t u = (x & (kHigh ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
  __half2 h = *reinterpret_cast<const __half2*>(&u);
  if (kHigh)
    h = __hfma2(h, __floats2half2_rn(0.0625f, 0.0625f), __floats2half2_rn(-72.f, -72.f));
  else
    h = __hsub2(h, __floats2half2_rn(1032.f, 1032.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float pow2_field(int f) { return __uint_as_float((uint32_t)f << 23); }

// D: head size; NT: blocks of 8 query rows; kScore: keep the logits.
template <int D, int NT, bool kScore>
__global__ void __launch_bounds__(kThreads)
kv4_attn_kernel(const Kv4AttnArgs a) {
  constexpr int NG = D / kKv4Group;         // groups a row
  constexpr int RB = 8 * NT;                // query rows of the block
  __shared__ float sO[kWarps][RB][D];
  __shared__ float sM[kWarps][RB], sL[kWarps][RB];

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

  // ---- the block's query rows as B operands: lane (g, c) holds row g's
  // dimensions in the order in which the codes come out of a word
  uint32_t qf[NT][NG][2][2][2];              // [rows][group][word][half][operand]
  float qsum[NT][NG][2], sl2[NT][2];         // of rows 2c and 2c + 1
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
    // x * 2^-e in [-2, 2]
    const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 253);
    const float down = pow2_field(254 - e), up = pow2_field(e);
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
            qf[nt][gr][w][h][o] = pack_half2(x[gr][8 * w + 2 * h + o], x[gr][8 * w + 2 * h + o + 4]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = 4 * (2 * c + i);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) qsum[nt][gr][i] = __shfl_sync(0xffffffffu, sums[gr], src);
      sl2[nt][i] = __shfl_sync(0xffffffffu, up, src) * a.scale_log2;
      const int rr = rb * RB + nt * 8 + 2 * c + i;
      pos[nt][i] = rr < R ? sp.pmin + rr / grp - (rb * RB) / grp : -1;
    }
  }

  float o[NT][NG][4][4];
  float m[NT][2], l[NT][2], zo[NT][NG][2];
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
      m[nt][i] = -INFINITY;
      l[nt][i] = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) zo[nt][gr][i] = 0.f;
    }
  }
  int vfield = 0;                            // exponent field of the largest value scale so far
  float v_down = pow2_field(253);            // 2^-(that + 1)

  const size_t row0 = (size_t)bh * a.C;
  const uint8_t* kc = a.c.kc + row0 * (D / 2);
  const uint8_t* vc = a.c.vc + row0 * (D / 2);
  const uint32_t* km = a.c.km + row0 * NG;
  const uint32_t* vm = a.c.vm + row0 * NG;

  for (int v = v_begin + warp; v < v_end; v += kWarps) {
    const int j0 = sp.tile(v) * kKv4Tile;
    // ---- scores of 32 slots: rows of S are slots, columns query rows
    float s[2][NT][4];
    float sv[2][2][NG], zv[2][2][NG];        // value scales and zero points of slots g, g + 8
    uint32_t vw[2][4][NG];                   // value codes of slots 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t kw[2][NG][2];
      float sk[2][NG], zk[2][NG];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // slots past the capacity are read as its last (and masked below)
        const size_t j = (size_t)min(j0 + 16 * t + 8 * i + g, a.C - 1);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const uint2 u = *reinterpret_cast<const uint2*>(kc + j * (D / 2) + 32 * gr + 8 * c);
          kw[i][gr][0] = u.x;
          kw[i][gr][1] = u.y;
          const uint32_t mk = km[j * NG + gr], mv = vm[j * NG + gr];
          sk[i][gr] = __uint_as_float(mk << 16);
          zk[i][gr] = __uint_as_float(mk & 0xffff0000u);
          sv[t][i][gr] = __uint_as_float(mv << 16);
          zv[t][i][gr] = __uint_as_float(mv & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t j = (size_t)min(j0 + 16 * t + 8 * (i >> 1) + 2 * c + (i & 1), a.C - 1);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
          vw[t][i][gr] = *reinterpret_cast<const uint32_t*>(vc + j * (D / 2) + 32 * gr + 4 * g);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][nt][i] = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = kw[0][gr][w] >> (8 * h), x1 = kw[1][gr][w] >> (8 * h);
            const uint32_t af[4] = {codes2<false>(x0), codes2<false>(x1), codes2<true>(x0),
                                    codes2<true>(x1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(acc[nt], af, qf[nt][gr][w][h][0], qf[nt][gr][w][h][1]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[t][nt][i] += fmaf(sk[i >> 1][gr], acc[nt][i], zk[i >> 1][gr] * qsum[nt][gr][i & 1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][nt][i] *= sl2[nt][i & 1];
    }
    if constexpr (kScore) {
      float* lg = a.logits + ((size_t)blk * a.slots + j0) * RB;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int at = (16 * t + 8 * i + g) * RB + nt * 8 + 2 * c;
            if (in_range(((long long)blk * a.slots + j0) * RB + at, 2,
                         (long long)a.B * a.H_kv * a.n_rb * a.slots * RB, a.status))
              *reinterpret_cast<float2*>(lg + at) =
                  make_float2(s[t][nt][2 * i], s[t][nt][2 * i + 1]);
          }
    }
    // ---- tiles that some row does not see in full
    const bool whole = j0 + kKv4Tile - 1 <= sp.pmin &&
                       (a.window <= 0 || j0 > sp.pmax - a.window || j0 + kKv4Tile <= a.n_sink);
    if (!whole) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = j0 + 16 * t + 8 * i + g;
          bool any = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool ok = sees(a, pos[nt][h], j);
              any |= ok;
              if (!ok) s[t][nt][2 * i + h] = -INFINITY;
            }
          // a slot that none of this lane's rows sees may hold anything
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
            if (!any) sv[t][i][gr] = zv[t][i][gr] = 0.f;
        }
    }
    // ---- running maximum of every row and largest value scale
    bool raise = false;
    float mt[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(fmaxf(s[0][nt][h], s[0][nt][2 + h]), fmaxf(s[1][nt][h], s[1][nt][2 + h]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        mt[nt][h] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        raise |= mt[nt][h] > m[nt][h] + kRescaleLog2;
      }
    uint32_t vtop = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
          vtop = max(vtop, __float_as_uint(sv[t][i][gr]) & 0x7fffffffu);
    const int field = (int)(__reduce_max_sync(0xffffffffu, vtop) >> 23);
    raise |= field > vfield;
    if (__any_sync(0xffffffffu, raise)) {
      float shrink = 1.f;
      if (field > vfield) {
        const float down = pow2_field(max(253 - field, 1));
        shrink = down / v_down;
        v_down = down;
        vfield = field;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float alpha = 1.f;
          if (mt[nt][h] > m[nt][h] + kRescaleLog2) {
            alpha = exp2f(m[nt][h] - mt[nt][h]);        // 0 from -inf
            m[nt][h] = mt[nt][h];
          }
          l[nt][h] *= alpha;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            zo[nt][gr][h] *= alpha;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[nt][gr][e][h] *= alpha * shrink;
              o[nt][gr][e][2 + h] *= alpha * shrink;
            }
          }
        }
    }
    // ---- weights, and their products with the value codes
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t pf[NT][NG][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mu = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
          p[i] = sm100::ex2_approx(s[t][nt][i] - mu);
          l[nt][i & 1] += p[i];
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // a weight of 0 in a tile with masked slots takes nothing from its value
            const bool off = !whole && p[i] == 0.f;
            w[i] = off ? 0.f : p[i] * (sv[t][i >> 1][gr] * v_down);
            zo[nt][gr][i & 1] += off ? 0.f : p[i] * zv[t][i >> 1][gr];
          }
          pf[nt][gr][0] = transpose8x8(pack_half2(w[0], w[1]));
          pf[nt][gr][1] = transpose8x8(pack_half2(w[2], w[3]));
        }
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // two dimensions of four slots: (2c, 2c + 1), (2c + 8, 2c + 9)
          const uint32_t sel = e < 2 ? 0x5410u : 0x7632u;
          const uint32_t x0 = __byte_perm(vw[t][0][gr], vw[t][1][gr], sel) >> (8 * (e & 1));
          const uint32_t x1 = __byte_perm(vw[t][2][gr], vw[t][3][gr], sel) >> (8 * (e & 1));
          const uint32_t af[4] = {codes2<false>(x0), codes2<true>(x0), codes2<false>(x1),
                                  codes2<true>(x1)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][gr][e], af, pf[nt][gr][0], pf[nt][gr][1]);
        }
    }
  }

  // ---- the warps' parts meet in shared memory, in true units
  const float v_up = pow2_field(254 - (int)(__float_as_uint(v_down) >> 23));
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
        sM[warp][r] = m[nt][h];
        sL[warp][r] = ls;
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 y = make_float2(fmaf(o[nt][gr][e][h], v_up, z[gr]),
                                 fmaf(o[nt][gr][e][2 + h], v_up, z[gr]));
          *reinterpret_cast<float2*>(&sO[warp][r][gr * kKv4Group + 8 * g + 2 * e]) = y;
        }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < RB * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    const int row = rb * RB + r;
    if (row >= R) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sM[w][r]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (sM[w][r] == -INFINITY && sL[w][r] == 0.f) continue;     // a warp that saw nothing
      const float f = sM[w][r] == mx ? 1.f : exp2f(sM[w][r] - mx);
      const float4 x = *reinterpret_cast<const float4*>(&sO[w][r][d]);
      y.x = fmaf(f, x.x, y.x);
      y.y = fmaf(f, x.y, y.y);
      y.z = fmaf(f, x.z, y.z);
      y.w = fmaf(f, x.w, y.w);
      ls = fmaf(f, sL[w][r], ls);
    }
    if (a.n_split > 1 || kScore) {
      const long long part = ((long long)blk * a.n_split + split) * RB + r;
      if (d == 0) {
        a.part_ml[2 * part] = mx;
        a.part_ml[2 * part + 1] = ls;
      }
      if (a.n_split > 1) *reinterpret_cast<float4*>(a.part_o + part * D + d) = y;
    }
    if (a.n_split == 1) {
      const int t = row / grp, h = hk * grp + row % grp;
      const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);   // 0: no slot; NaN stays
      const long long off = (((long long)b * a.S_q + t) * a.H_q + h) * D + d;
      if (in_range(off, 4, (long long)a.B * a.S_q * a.H_q * D, a.status))
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + off) =
            make_uint2(sm100::pack_bf16x2(y.x * inv, y.y * inv),
                       sm100::pack_bf16x2(y.z * inv, y.w * inv));
      if (d == 0 && a.lse)
        a.lse[((long long)b * a.H_q + h) * a.S_q + t] =
            ls == 0.f ? -INFINITY : (mx + log2f(ls)) * kLn2;
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
  if (threadIdx.x == 0 && a.lse)
    a.lse[((long long)b * a.H_q + h) * a.S_q + t] =
        ls == 0.f ? -INFINITY : (mx + log2f(ls)) * kLn2;
}

// Adds every visible slot's weight to its running sum, one thread a slot; the
// rows' log-sums come from the chunks' partial sums again.
constexpr int kScoreSlots = 256;
__global__ void __launch_bounds__(kScoreSlots)
kv4_score_kernel(const Kv4AttnArgs a, int blocks_per_head) {
  __shared__ float lse2[16];
  __shared__ int pos[16];
  const int bh = blockIdx.x / blocks_per_head;
  const int j = (blockIdx.x % blocks_per_head) * kScoreSlots + threadIdx.x;
  const int b = bh / a.H_kv;
  const int grp = a.H_q / a.H_kv, R = a.S_q * grp;
  float sum = 0.f;
  for (int rb = 0; rb < a.n_rb; ++rb) {
    const Span sp = span_of(a, b, rb);
    const int n = (sp.n + a.chunk - 1) / a.chunk;
    const long long blk = (long long)bh * a.n_rb + rb;
    __syncthreads();
    if (threadIdx.x < a.rows) {
      const int r = threadIdx.x;
      float m = -INFINITY, l = 0.f;
      for (int s = 0; s < n; ++s) {
        const long long part = (blk * a.n_split + s) * a.rows + r;
        if (rb * a.rows + r >= R) break;
        const float pm = a.part_ml[2 * part], pl = a.part_ml[2 * part + 1];
        if (pm == -INFINITY && pl == 0.f) continue;
        const float mn = fmaxf(m, pm);
        l = l * (m == -INFINITY ? 0.f : exp2f(m - mn)) + pl * (pm == mn ? 1.f : exp2f(pm - mn));
        m = mn;
      }
      lse2[r] = m + log2f(l);
      pos[r] = rb * a.rows + r < R ? sp.pmin + (rb * a.rows + r) / grp - (rb * a.rows) / grp : -1;
    }
    __syncthreads();
    if (j < sp.hi) {
      const float* lg = a.logits + (blk * a.slots + j) * a.rows;
      for (int r = 0; r < a.rows; ++r)
        if (sees(a, pos[r], j)) sum += exp2f(lg[r] - lse2[r]);
    }
  }
  if (j < a.C && sum != 0.f) a.score[(long long)bh * a.C + j] += sum;
}

template <int D, int NT>
ra_status launch_nt(const Kv4AttnArgs& a, cudaStream_t stream) {
  const long long grid = (long long)a.B * a.H_kv * a.n_rb * a.n_split;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  if (a.score)
    kv4_attn_kernel<D, NT, true><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  else
    kv4_attn_kernel<D, NT, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return RA_ERR_LAUNCH;
  if (a.n_split > 1) {
    const long long rows = (long long)a.B * a.H_q * a.S_q;
    if (rows > 0x7fffffffLL) return RA_ERR_RANGE;
    kv4_join_kernel<D><<<(unsigned)rows, 32 * kJoinWarps, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return RA_ERR_LAUNCH;
  }
  if (a.score) {
    const int per = (a.max_len + kScoreSlots - 1) / kScoreSlots;
    const long long blocks = (long long)a.B * a.H_kv * per;
    if (blocks > 0x7fffffffLL) return RA_ERR_RANGE;
    kv4_score_kernel<<<(unsigned)blocks, kScoreSlots, 0, stream>>>(a, per);
    if (cudaGetLastError() != cudaSuccess) return RA_ERR_LAUNCH;
  }
  return RA_OK;
}

}  // namespace

// Chunks: enough CTAs for three waves of four a multiprocessor (sequences of
// different lengths then even out), but no chunk under kMinChunk tiles, where
// joining would cost more than it spreads.
ra_status kv4_attn_plan(Kv4AttnArgs* a, bool score, size_t* bytes) {
  constexpr long long kTargetCtas = 152 * 4 * 3;
  constexpr int kMinChunk = 2 * kWarps;
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
  long long chunk = (tiles * blocks + kTargetCtas - 1) / kTargetCtas;
  chunk = (chunk + kWarps - 1) / kWarps * kWarps;
  if (chunk < kMinChunk) chunk = kMinChunk;
  const long long n_split = tiles > chunk ? (tiles + chunk - 1) / chunk : 1;
  if (blocks * n_split > 0x7fffffffLL) return RA_ERR_RANGE;
  a->n_rb = (int)n_rb;
  a->chunk = (int)chunk;
  a->n_split = (int)n_split;
  a->slots = (a->max_len + kKv4Tile - 1) / kKv4Tile * kKv4Tile;
  const size_t parts = (size_t)blocks * n_split * a->rows;
  const size_t n_o = n_split > 1 ? parts * a->D : 0;
  const size_t n_ml = n_split > 1 || score ? parts * 2 : 0;
  const size_t n_lg = score ? (size_t)blocks * a->slots * a->rows : 0;
  *bytes = (n_o + n_ml + n_lg) * sizeof(float);
  return RA_OK;
}

ra_status launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  if (a.D == 64)
    return a.rows == 8 ? launch_nt<64, 1>(a, stream) : launch_nt<64, 2>(a, stream);
  return a.rows == 8 ? launch_nt<128, 1>(a, stream) : launch_nt<128, 2>(a, stream);
}

}  // namespace ra
