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
// Both kernels move rows and do little else: their bytes bound them. Sixteen
// lanes (eight at D = 64) share a row, eight values each, of its key and its
// value; the float side moves in 16-byte vectors.
#include <cuda_bf16.h>

#include <cstdint>

#include "checks.cuh"
#include "divisor.cuh"
#include "paged_internal.h"
#include "paged_ops.cuh"
#include "sm100.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kVals = 8;             // values a lane

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[kVals]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[kVals]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[kVals]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(sm100::pack_bf16x2(x[0], x[1]), sm100::pack_bf16x2(x[2], x[3]),
                 sm100::pack_bf16x2(x[4], x[5]), sm100::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[kVals]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
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
      if (__ldg(a.cu + mid) <= (int)token) lo = mid;
      else hi = mid;
    }
    b = lo;
    t = (int)token - __ldg(a.cu + b);
    x.counts = t >= 0 && (int)token < __ldg(a.cu + b + 1);
  } else {
    b = (int)by.tokens.of(token);
    t = (int)(token - (uint32_t)b * by.tokens.d);
    x.counts = !a.n_new || t < __ldg(a.n_new + b);
  }
  if (!x.counts) return x;
  const long long slot = (long long)(a.start ? __ldg(a.start + b) : 0) + t;
  const int shift = 31 - __clz(a.p.page);
  if (slot < 0 || (slot >> shift) >= a.width) return x;
  const int id = __ldg(a.table + (size_t)b * a.width + (slot >> shift));
  if (id < 0 || id >= a.p.n_pages) return x;
  x.row = ((((long long)id * a.p.H_kv + h) << shift)) + (slot & (a.p.page - 1));
  x.held = in_range(x.row, 1, (long long)a.p.n_pages * a.p.H_kv * a.p.page, a.status);
  return x;
}

// A row's scale byte and this lane's eight codes of it.
template <int kLanes>
__device__ __forceinline__ uint2 encode(const float (&x)[kVals], uint32_t mask, int& byte) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
    top = max(top, u < 0x7f800000u ? u : 0u);
  }
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) top = max(top, __shfl_xor_sync(mask, top, o));
  // 448 = 1.75 2^8; biased as the field is. 10 is 2^-117
  byte = max((int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u), 10);
  const float down = __uint_as_float((uint32_t)(254 - byte) << 23);
  float y[kVals];
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    const bool fine = (__float_as_uint(x[e]) & 0x7fffffffu) < 0x7f800000u;
    y[e] = fine ? x[e] * down : __uint_as_float(0x7fc00000u);
  }
  return make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16,
                    e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
}

__device__ __forceinline__ void decode(uint2 c, int byte, float (&x)[kVals]) {
  const float scale = pow2_byte(byte);
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_values(e4m3x2_half2(w[i]));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

template <typename T, int kLanes, bool kQuant>
__global__ void __launch_bounds__(kThreads)
paged_append_kernel(const PagedRowArgs a, const Divisors by, uint32_t rows) {
  constexpr int D = kLanes * kVals;
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  // a row's lanes leave or stay together: the shuffles name only them
  const uint32_t mask = (kLanes == 16 ? 0xffffu : 0xffu) << (threadIdx.x & 31 & ~(kLanes - 1));
  if (i >= rows) return;
  const Place r = locate(a, by, i);
  if (!r.counts) return;
  if (!r.held) {
    if (lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    return;
  }
  const size_t elem = (size_t)i * D + lane * kVals;
  float k[kVals], v[kVals];
  load8(static_cast<const T*>(a.k) + elem, k);
  load8(static_cast<const T*>(a.v) + elem, v);
  const size_t to = (size_t)r.row * D + lane * kVals;
  if constexpr (kQuant) {
    int bk, bv;
    const uint2 ck = encode<kLanes>(k, mask, bk), cv = encode<kLanes>(v, mask, bv);
    *reinterpret_cast<uint2*>(a.p.k + to) = ck;
    *reinterpret_cast<uint2*>(a.p.v + to) = cv;
    if (lane == 0) {
      a.p.ks[r.row] = (uint8_t)bk;
      a.p.vs[r.row] = (uint8_t)bv;
    }
  } else {
    store8(reinterpret_cast<__nv_bfloat16*>(a.p.k) + to, k);
    store8(reinterpret_cast<__nv_bfloat16*>(a.p.v) + to, v);
  }
}

template <typename T, int kLanes, bool kQuant>
__global__ void __launch_bounds__(kThreads)
paged_read_kernel(const PagedRowArgs a, const Divisors by, uint32_t rows) {
  constexpr int D = kLanes * kVals;
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (i >= rows) return;
  const Place r = locate(a, by, i);
  float k[kVals] = {}, v[kVals] = {};                // no such slot: zeros
  if (r.held) {
    const size_t from = (size_t)r.row * D + lane * kVals;
    if constexpr (kQuant) {
      const uint2 ck = *reinterpret_cast<const uint2*>(a.p.k + from);
      const uint2 cv = *reinterpret_cast<const uint2*>(a.p.v + from);
      decode(ck, a.p.ks[r.row], k);
      decode(cv, a.p.vs[r.row], v);
    } else {
      load8(reinterpret_cast<const __nv_bfloat16*>(a.p.k) + from, k);
      load8(reinterpret_cast<const __nv_bfloat16*>(a.p.v) + from, v);
    }
  } else if (lane == 0 && a.status) {
    atomicExch(a.status, (int)RA_ERR_RANGE);
  }
  const size_t elem = (size_t)i * D + lane * kVals;
  if (a.k) store8(static_cast<T*>(a.k) + elem, k);
  if (a.v) store8(static_cast<T*>(a.v) + elem, v);
}

template <int kLanes, typename Kernel>
ra_status launch_rows(Kernel kern, const PagedRowArgs& a, cudaStream_t stream) {
  const long long rows = a.rows * a.p.H_kv;
  const int per = kThreads / kLanes;
  const long long blocks = (rows + per - 1) / per;
  const Divisors by = {Divisor((uint32_t)a.p.H_kv), Divisor((uint32_t)a.T)};
  kern<<<(unsigned)blocks, kThreads, 0, stream>>>(a, by, (uint32_t)rows);
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

template <typename T, int kLanes>
ra_status append(const PagedRowArgs& a, cudaStream_t stream) {
  return a.p.quant ? launch_rows<kLanes>(paged_append_kernel<T, kLanes, true>, a, stream)
                   : launch_rows<kLanes>(paged_append_kernel<T, kLanes, false>, a, stream);
}
template <typename T, int kLanes>
ra_status read(const PagedRowArgs& a, cudaStream_t stream) {
  return a.p.quant ? launch_rows<kLanes>(paged_read_kernel<T, kLanes, true>, a, stream)
                   : launch_rows<kLanes>(paged_read_kernel<T, kLanes, false>, a, stream);
}

}  // namespace

ra_status launch_paged_append(const PagedRowArgs& a, int dtype, cudaStream_t stream) {
  if (dtype == RA_F32)
    return a.p.D == 64 ? append<float, 8>(a, stream) : append<float, 16>(a, stream);
  return a.p.D == 64 ? append<__nv_bfloat16, 8>(a, stream) : append<__nv_bfloat16, 16>(a, stream);
}

ra_status launch_paged_read(const PagedRowArgs& a, int dtype, cudaStream_t stream) {
  if (dtype == RA_F32) return a.p.D == 64 ? read<float, 8>(a, stream) : read<float, 16>(a, stream);
  return a.p.D == 64 ? read<__nv_bfloat16, 8>(a, stream) : read<__nv_bfloat16, 16>(a, stream);
}

}  // namespace ra
