// The paged key/value cache: writing new tokens to their pages and reading
// slots back (format: paged_internal.h).
//
// In 8 bits a row x of D values has the scale 2^e, e the least number from -117
// on with max |x| / 2^e <= 448, the largest e4m3 number; its codes are
// e4m3(x / 2^e), to nearest, half to even. A power of two costs a floating
// format nothing (its steps are relative), makes x / 2^e and c 2^e exact, and
// c 2^e a bfloat16 number: from -117 on the least step, 2^-9 2^e, is 2^-126. An
// infinity or a NaN becomes a NaN of its own value alone, and the scale goes by
// the finite ones.
//
// Both kernels move rows and do little else: their bytes bound them, if enough are in
// flight and what a row costs besides is little. Eight lanes (four at D = 64) share a
// row, sixteen values each, of its key and its value, loaded before their place is
// looked up. Measured, 8 x 8192 tokens of 8 heads, D = 128, 8 bits: append
// 66 us, read 67 us, 6.1 and 6.0 TB/s, one behind the other 129 (eight values a lane and
// one row: 95 and 72).
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "checks.cuh"
#include "divisor.cuh"
#include "early_launch.cuh"
#include "paged_internal.h"
#include "paged_ops.cuh"
#include "sm100.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kVals = 16;            // values a lane

// A lane's values of a row as they come: bfloat16 two to a word, or float32.
template <typename T>
struct Lane {
  static constexpr int kWords = kVals * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  // The bits of the largest magnitude: float32's order is that of its bits.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
};
__device__ __forceinline__ bool finite_bits(uint32_t u) { return (u & 0x7fffffffu) < 0x7f800000u; }

template <int N>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(
        sm100::pack_bf16x2(x[8 * i], x[8 * i + 1]), sm100::pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
        sm100::pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), sm100::pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
}
template <int N>
__device__ __forceinline__ void store(float* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}

struct Divisors {
  Divisor heads, tokens;
};

// One row of the token tensors (fewer than 2^25 rows: they hold fewer than 2^31
// values).
struct Place {
  long long row;       // its row in the pool: (page id * H_kv + head) * page + place in it
  bool counts;         // not padding (append)
  bool held;           // its slot has a page
};

__device__ __forceinline__ Place locate(const PagedRowArgs& a, const Divisors& by, uint32_t i) {
  const uint32_t token = by.heads.of(i), h = i - token * by.heads.d;
  Place x = {0, true, false};
  int b, t;
  if (a.cu) {
    // the last sequence that starts at or before the token (empty ones share starts)
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= (int)token) lo = mid;
      else hi = mid;
    }
    b = lo;
    t = (int)token - a.cu[b];
    x.counts = t >= 0 && (int)token < a.cu[b + 1];
  } else {
    b = (int)by.tokens.of(token);
    t = (int)(token - (uint32_t)b * by.tokens.d);
    x.counts = !a.n_new || t < a.n_new[b];
  }
  if (!x.counts) return x;
  const long long slot = (long long)(a.start ? a.start[b] : 0) + t;
  const int shift = 31 - __clz(a.p.page);
  if (slot < 0 || (slot >> shift) >= a.width) return x;
  const long long entry = (long long)b * a.width + (slot >> shift);
  if (!in_range(entry, 1, (long long)a.B * a.width, a.status)) return x;
  const int id = a.table[entry];
  if (id < 0 || id >= a.p.n_pages) return x;
  x.row = ((((long long)id * a.p.H_kv + h) << shift)) + (slot & (a.p.page - 1));
  x.held = in_range(x.row, 1, paged_pool_rows(a.p), a.status);
  return x;
}

// A row's scale byte and this lane's codes of it.
template <int kLanes, typename T>
__device__ __forceinline__ uint4 encode(const Lane<T>& x, uint32_t mask, int& byte) {
  auto row_max = [&](uint32_t u) {
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) u = max(u, __shfl_xor_sync(mask, u, o));
    return u;
  };
  uint32_t top = row_max(x.top());
  const bool fine = finite_bits(top);
  if (!fine) {                                       // the whole row together
    top = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const uint32_t u = __float_as_uint(x.value(i)) & 0x7fffffffu;
      top = max(top, finite_bits(u) ? u : 0u);
    }
    top = row_max(top);
  }
  // 448 = 1.75 2^8; biased as the field is. 10 is 2^-117
  byte = max((int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u), 10);
  const float down = __uint_as_float((uint32_t)(254 - byte) << 23);
  uint32_t c[kVals / 4];
#pragma unroll
  for (int i = 0; i < kVals / 4; ++i) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = x.value(4 * i + e);
      y[e] = fine || finite_bits(__float_as_uint(v)) ? v * down : __uint_as_float(0x7fc00000u);
    }
    c[i] = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

template <typename T, int kLanes, bool kQuant>
__global__ void __launch_bounds__(kThreads)
paged_append_kernel(const PagedRowArgs a, const Divisors by, uint32_t rows) {
  constexpr int D = kLanes * kVals;
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  let_dependents_start();
  wait_for_prior_grid();
  // a row's lanes leave or stay together: the shuffles name only them
  const uint32_t mask = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
  if (i >= rows) return;
  const size_t elem = (size_t)i * D + lane * kVals;
  if (!in_range((long long)elem, kVals, a.rows * a.p.H_kv * D, a.status)) return;
  Lane<T> k, v;
  k.load(static_cast<const T*>(a.k) + elem);
  v.load(static_cast<const T*>(a.v) + elem);
  const Place r = locate(a, by, i);
  if (!r.counts) return;
  if (!r.held) {
    if (lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    return;
  }
  const size_t to = (size_t)r.row * D + lane * kVals;
  if constexpr (kQuant) {
    int bk, bv;
    const uint4 ck = encode<kLanes>(k, mask, bk), cv = encode<kLanes>(v, mask, bv);
    *reinterpret_cast<uint4*>(a.p.k + to) = ck;
    *reinterpret_cast<uint4*>(a.p.v + to) = cv;
    if (lane == 0) {
      a.p.ks[r.row] = (uint8_t)bk;
      a.p.vs[r.row] = (uint8_t)bv;
    }
  } else {
    float x[kVals];
#pragma unroll
    for (int e = 0; e < kVals; ++e) x[e] = k.value(e);
    store(reinterpret_cast<__nv_bfloat16*>(a.p.k) + to, x);
#pragma unroll
    for (int e = 0; e < kVals; ++e) x[e] = v.value(e);
    store(reinterpret_cast<__nv_bfloat16*>(a.p.v) + to, x);
  }
}

// Reading: eight values a lane, so that a warp's stores fill whole sectors, and
// kReadRows rows, whose loads are in flight together.
constexpr int kReadVals = 8, kReadRows = 2;
__device__ __forceinline__ void decode(uint2 c, int byte, float (&x)[kReadVals]) {
  const float scale = pow2_byte(byte);
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < kReadVals / 2; ++i) {
    const float2 f = half2_values(e4m3x2_half2(w[i / 2] >> (16 * (i % 2))));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}
__device__ __forceinline__ void decode(uint4 u, float (&x)[kReadVals]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <typename T, int kLanes, bool kQuant>
__global__ void __launch_bounds__(kThreads)
paged_read_kernel(const PagedRowArgs a, const Divisors by, uint32_t rows) {
  constexpr int D = kLanes * kReadVals, kAtOnce = kThreads / kLanes;
  const uint32_t first = blockIdx.x * (kAtOnce * kReadRows) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes, d = lane * kReadVals;
  let_dependents_start();
  wait_for_prior_grid();
  Place r[kReadRows];
#pragma unroll
  for (int x = 0; x < kReadRows; ++x) {
    const uint32_t i = first + x * kAtOnce;
    r[x] = {0, false, false};
    if (i < rows) r[x] = locate(a, by, i);
  }
  using Word = typename std::conditional<kQuant, uint2, uint4>::type;
  Word wk[kReadRows], wv[kReadRows];
  int bk[kReadRows], bv[kReadRows];
#pragma unroll
  for (int x = 0; x < kReadRows; ++x) {
    wk[x] = wv[x] = Word();                          // no such slot: zeros
    bk[x] = bv[x] = 0;
    if (!r[x].held) continue;
    const size_t from = ((size_t)r[x].row * D + d) * (kQuant ? 1 : 2);
    wk[x] = *reinterpret_cast<const Word*>(a.p.k + from);
    wv[x] = *reinterpret_cast<const Word*>(a.p.v + from);
    if (kQuant) {
      bk[x] = a.p.ks[r[x].row];
      bv[x] = a.p.vs[r[x].row];
    }
  }
#pragma unroll
  for (int x = 0; x < kReadRows; ++x) {
    const uint32_t i = first + x * kAtOnce;
    if (i >= rows) break;
    if (!r[x].held && lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    float k[kReadVals], v[kReadVals];
    if constexpr (kQuant) {
      decode(wk[x], bk[x], k);
      decode(wv[x], bv[x], v);
    } else {
      decode(wk[x], k);
      decode(wv[x], v);
    }
    const size_t elem = (size_t)i * D + d;
    if (!in_range((long long)elem, kReadVals, a.rows * a.p.H_kv * D, a.status)) continue;
    if (a.k) store(static_cast<T*>(a.k) + elem, k);
    if (a.v) store(static_cast<T*>(a.v) + elem, v);
  }
}

// `per`: rows a CTA takes.
ra_status launch_rows(void (*kern)(PagedRowArgs, Divisors, uint32_t), const PagedRowArgs& a,
                      int per, cudaStream_t stream) {
  const long long rows = a.rows * a.p.H_kv;
  const long long blocks = (rows + per - 1) / per;
  const Divisors by = {Divisor((uint32_t)a.p.H_kv), Divisor((uint32_t)a.T)};
  return launch_early(kern, blocks, kThreads, 0, stream, a, by, (uint32_t)rows) ? RA_OK
                                                                                : RA_ERR_LAUNCH;
}

template <typename T, int D>
ra_status append(const PagedRowArgs& a, cudaStream_t stream) {
  constexpr int kLanes = D / kVals, kPer = kThreads / kLanes;
  return a.p.quant ? launch_rows(paged_append_kernel<T, kLanes, true>, a, kPer, stream)
                   : launch_rows(paged_append_kernel<T, kLanes, false>, a, kPer, stream);
}
template <typename T, int D>
ra_status read(const PagedRowArgs& a, cudaStream_t stream) {
  constexpr int kLanes = D / kReadVals, kPer = kThreads / kLanes * kReadRows;
  return a.p.quant ? launch_rows(paged_read_kernel<T, kLanes, true>, a, kPer, stream)
                   : launch_rows(paged_read_kernel<T, kLanes, false>, a, kPer, stream);
}

}  // namespace

ra_status launch_paged_append(const PagedRowArgs& a, int dtype, cudaStream_t stream) {
  if (dtype == RA_F32) return a.p.D == 64 ? append<float, 64>(a, stream) : append<float, 128>(a, stream);
  return a.p.D == 64 ? append<__nv_bfloat16, 64>(a, stream) : append<__nv_bfloat16, 128>(a, stream);
}

ra_status launch_paged_read(const PagedRowArgs& a, int dtype, cudaStream_t stream) {
  if (dtype == RA_F32) return a.p.D == 64 ? read<float, 64>(a, stream) : read<float, 128>(a, stream);
  return a.p.D == 64 ? read<__nv_bfloat16, 64>(a, stream) : read<__nv_bfloat16, 128>(a, stream);
}

}  // namespace ra
