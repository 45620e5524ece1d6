// Exact float32 attention with a sliding window and a few first tokens that
// stay visible, on the CUDA cores (FMA pipe). As in the float32 kernel without
// a window every product and sum is IEEE float32 and exponentials are the
// accurate exp2f, for a tolerance of 1e-4.
//
// A block owns 32 query rows of one (batch, head) and walks the key tiles of
// 64 that some row sees, in position order (window_iter.cuh), folding each into
// the rows' running maximum, sum and unnormalised output. Windows make short
// walks, so rows a block are few (more blocks) and the next tile's keys and
// values are copied (cp.async, two buffers) while this one is worked on.
//
// Mapping: 128 threads = 8 groups of 4 rows x 16 threads. A thread makes the
// scores of its 4 rows against keys kc, kc + 16, kc + 32, kc + 48 and then its
// 4 rows' outputs at dimensions 4 kc .. 4 kc + 3 (and 64 further at D = 128):
// 64 FMA on 8 16-byte shared loads in either product. Probabilities pass
// between the two through shared memory that only the group's half warp
// touches. What bounds it: those shared loads, at long walks; one block's own
// latency at short ones. Two sequences of 4096, 16 heads, window 1024: 0.97 ms, 31
// TFLOP/s of the visible pairs, at D = 64, 2.13 ms, 28 at D = 128, where a block's
// 160 KB leave one of four warps a multiprocessor. 2 x 777 tokens, 4 heads, D = 64, window 100: 20 us (45
// with the mapping of the kernel without a window, 4 threads a row).
#include <cmath>
#include <cstdint>

#include "checks.cuh"
#include "ra_internal.h"
#include "window_iter.cuh"

namespace ra {
namespace {

constexpr int kQ = 32;           // query rows a block
constexpr int kK = 64;           // keys a tile (the geometry's tile)
constexpr int kThreads = 128;

template <int D>
struct Smem {
  static constexpr int kStride = D + 4;        // floats a row: rows start 4 banks apart
  static constexpr int kQs = 0;
  static constexpr int kPs = kQs + kQ * kStride;
  static constexpr int kPStride = kK + 4;
  static constexpr int kBuf = kPs + kQ * kPStride;
  static constexpr int kBufFloats = 2 * kK * kStride;   // keys, then values
  static constexpr int kBytes = (kBuf + 2 * kBufFloats) * 4;
};

__device__ __forceinline__ void copy16(float* dst, const float* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int D, bool kVarlen>
__global__ void __launch_bounds__(kThreads, 2)
attn_f32_window_kernel(const WinGeometry gp, const float* __restrict__ q,
                       const float* __restrict__ k, const float* __restrict__ v,
                       float* __restrict__ out, float* __restrict__ lse,
                       int* __restrict__ status) {
  using S = Smem<D>;
  constexpr int V4 = D / 4;                    // 16-byte vectors a row
  constexpr int ND = D / 64;                   // a thread's 4-dimension pieces
  extern __shared__ __align__(16) float smem[];
  float* Qs = smem + S::kQs;
  float* Ps = smem + S::kPs;

  const int BH = gp.B * gp.H_q;
  const int bh = blockIdx.x % BH, b = bh / gp.H_q, h = bh % gp.H_q;
  const int hk = h / (gp.H_q / gp.H_kv);
  const int n_qt = gp.n_seg * gp.nt * (kK / kQ);
  const int qid = n_qt - 1 - blockIdx.x / BH;
  const int seg = qid / (gp.nt * (kK / kQ)), ti = qid % (gp.nt * (kK / kQ));
  WinGeometry gv;
  int row0 = 0;
  if constexpr (kVarlen) varlen_window_geometry(gp, b, gv, row0, threadIdx.x == 0 ? status : nullptr);
  const WinGeometry& g = kVarlen ? gv : gp;
  const int q_lo = seg * g.seg_len + ti * kQ;
  const int q_valid = min(kQ, seg_tokens(g, seg) - ti * kQ);
  if (q_valid <= 0) return;                    // padding only
  const size_t srow = kVarlen ? (size_t)row0 : (size_t)b * gp.S;
  const size_t lrow = kVarlen ? (size_t)h * gp.total + row0 : (size_t)bh * gp.S;

  const int rg = threadIdx.x >> 4, kc = threadIdx.x & 15;
  const int r_lo = 4 * rg;                     // this thread's first row

  for (int i = threadIdx.x; i < kQ * V4; i += kThreads) {
    const int r = i / V4, c = i % V4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t off = ((srow + q_lo + r) * g.H_q + h) * D + 4 * c;
    if (r < q_valid && in_range((long long)off, 4, extent_q(gp), status))
      x = *reinterpret_cast<const float4*>(q + off);
    *reinterpret_cast<float4*>(Qs + r * S::kStride + 4 * c) = x;
  }
  // rows of the tile past its keys are zeroed: their scores are masked, and their
  // weights of 0 would meet what the buffer held before, where NaN survives them
  auto fetch = [&](const KvTile& t, int buf) {
    float* Ks = smem + S::kBuf + buf * S::kBufFloats;
    float* Vs = Ks + kK * S::kStride;
    for (int i = threadIdx.x; i < kK * V4; i += kThreads) {
      const int r = i / V4, c = i % V4;
      const size_t off = ((srow + t.lo + r) * g.H_kv + hk) * D + 4 * c;
      float* kd = Ks + r * S::kStride + 4 * c;
      float* vd = Vs + r * S::kStride + 4 * c;
      if (r < t.valid && in_range((long long)off, 4, extent_kv(gp), status)) {
        copy16(kd, k + off);
        copy16(vd, v + off);
      } else {
        *reinterpret_cast<float4*>(kd) = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(vd) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  };

  WinKvIter it;
  it.init(g, seg_owner(g, seg), q_lo, q_valid);
  KvTile kv, next;
  bool have = it.next(g, kv);                  // every row sees itself: at least one tile
  if (have) fetch(kv, 0);
  copies_commit();

  float m[4], l[4], o[4][ND][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int n = 0; n < ND; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][n][e] = 0.f;
  }

  for (int buf = 0; have; buf ^= 1) {
    const bool more = it.next(g, next);
    __syncthreads();                           // the other buffer is read
    if (more) fetch(next, buf ^ 1);
    copies_commit();
    copies_wait<1>();                          // this tile's own
    __syncthreads();
    const float* Ks = smem + S::kBuf + buf * S::kBufFloats;
    const float* Vs = Ks + kK * S::kStride;

    float s[4][4] = {};
#pragma unroll 4
    for (int c = 0; c < V4; ++c) {
      float4 x[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = *reinterpret_cast<const float4*>(Qs + (r_lo + r) * S::kStride + 4 * c);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = *reinterpret_cast<const float4*>(Ks + (kc + 16 * j) * S::kStride + 4 * c);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[r][j] = fmaf(x[r].x, y[j].x, s[r][j]);
          s[r][j] = fmaf(x[r].y, y[j].y, s[r][j]);
          s[r][j] = fmaf(x[r].z, y[j].z, s[r][j]);
          s[r][j] = fmaf(x[r].w, y[j].w, s[r][j]);
        }
    }
    if (kv.work == kMask) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = kc + 16 * j, kp = kv.lo + key;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int qp = q_lo + r_lo + r;
          if (key >= kv.valid || kp > qp || (kp >= g.n_sink && kp <= qp - g.window))
            s[r][j] = -INFINITY;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float mx = fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]));
#pragma unroll
      for (int d = 1; d < 16; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float m_new = fmaxf(m[r], mx * g.scale_log2);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = m[r] == -INFINITY ? 0.f : exp2f(m[r] - m_new);
      m[r] = m_new;
      l[r] *= alpha;
#pragma unroll
      for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][n][e] *= alpha;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(fmaf(s[r][j], g.scale_log2, -m_use));
        l[r] += p;
        Ps[(r_lo + r) * S::kPStride + kc + 16 * j] = p;
      }
    }
    __syncwarp();
#pragma unroll 2
    for (int c = 0; c < kK / 4; ++c) {
      float4 p[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        p[r] = *reinterpret_cast<const float4*>(Ps + (r_lo + r) * S::kPStride + 4 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          const float4 y =
              *reinterpret_cast<const float4*>(Vs + (4 * c + e) * S::kStride + 64 * n + 4 * kc);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = e == 0 ? p[r].x : (e == 1 ? p[r].y : (e == 2 ? p[r].z : p[r].w));
            o[r][n][0] = fmaf(w, y.x, o[r][n][0]);
            o[r][n][1] = fmaf(w, y.y, o[r][n][1]);
            o[r][n][2] = fmaf(w, y.z, o[r][n][2]);
            o[r][n][3] = fmaf(w, y.w, o[r][n][3]);
          }
        }
    }
    __syncwarp();
    kv = next;
    have = more;
  }

#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
    if (r_lo + r >= q_valid) continue;
    const int pos = q_lo + r_lo + r;
    const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
    const size_t off = ((srow + pos) * g.H_q + h) * D;
    if (in_range((long long)off, D, extent_q(gp), status))
#pragma unroll
      for (int n = 0; n < ND; ++n)
        *reinterpret_cast<float4*>(out + off + 64 * n + 4 * kc) =
            make_float4(o[r][n][0] * inv, o[r][n][1] * inv, o[r][n][2] * inv, o[r][n][3] * inv);
    if (kc == 0 && lse && in_range((long long)(lrow + pos), 1, extent_lse(gp), status))
      // 0 only where every score is -inf; the NaN of a row that sees one stays
      lse[lrow + pos] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * 0.69314718055994531f;
  }
}

template <int D, bool kVarlen>
ra_status launch_d(const WinGeometry& g, const float* q, const float* k, const float* v,
                   float* out, float* lse, int* status, cudaStream_t stream) {
  if (cudaFuncSetAttribute(attn_f32_window_kernel<D, kVarlen>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Smem<D>::kBytes) != cudaSuccess)
    return RA_ERR_LAUNCH;
  const long long grid = (long long)g.n_seg * g.nt * (kK / kQ) * g.B * g.H_q;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  attn_f32_window_kernel<D, kVarlen><<<(unsigned)grid, kThreads, Smem<D>::kBytes, stream>>>(
      g, q, k, v, out, lse, status);
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

}  // namespace

ra_status launch_attn_f32_window(const WinGeometry& g, const float* q, const float* k,
                                 const float* v, float* out, float* lse, int* dev_status,
                                 cudaStream_t stream) {
  if (g.cu_seqlens)
    return g.D == 64 ? launch_d<64, true>(g, q, k, v, out, lse, dev_status, stream)
                     : launch_d<128, true>(g, q, k, v, out, lse, dev_status, stream);
  return g.D == 64 ? launch_d<64, false>(g, q, k, v, out, lse, dev_status, stream)
                   : launch_d<128, false>(g, q, k, v, out, lse, dev_status, stream);
}

}  // namespace ra
