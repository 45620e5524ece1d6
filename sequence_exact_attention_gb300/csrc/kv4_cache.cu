// The 4-bit key/value cache: quantising new tokens into it and reading slots
// back (format: kv4_internal.h).
//
// A group of 64 values x has lo = min x, hi = max x,
//   scale = bf16(hi / 15 - lo / 15)     sixteen levels over the range
//   zero  = bf16(lo + 8 scale)          the ninth level
//   code  = clamp(rint((x - zero) / scale) + 8, 0, 15), or 8 where scale = 0
// in float32 with one rounding a step (half to even), so a value is off by at
// most half a step and what the two roundings to bfloat16 move the levels by.
// scale and zero take two bytes each to keep a row at 4.5 bits a value; bf16
// holds the range of any input. A group that holds an infinity or a NaN reads
// back as NaN.
//
// Reading is bound by the bytes moved, once the instructions a value are few
// (below); appending by its instructions, an IEEE division a value among them: a
// prompt of 8 x 8192 tokens of 8 heads, D = 128, 152 us from bfloat16 (2.3 TB/s) and
// 150 us from float32 (4.1 TB/s). Eight lanes share a group, eight values each: the float side
// moves in 16-byte vectors, a group's codes are one 32-byte sector. Measured,
// reading 4096 slots of 64 heads, D = 128, as bfloat16: 31 us, 5.6 TB/s (with two
// divisions a thread and float32 arithmetic 33 us, 76 % of the issue slots).
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "checks.cuh"
#include "divisor.cuh"
#include "kv4_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;            // lanes a group
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
// One group of the token rows [B, T, H_kv, D]. Token tensors hold fewer than
// 2^31 elements, and so fewer than 2^25 groups.
struct Group {
  long long word;      // the group's word in meta: ((b H_kv + h) C + slot) (D / 64) + group
  bool counts;         // not padding (append)
  bool in_cache;       // its slot exists
};

struct Divisors {
  Divisor heads, tokens;
};

__device__ __forceinline__ Group locate(const Kv4RowArgs& a, const Divisors& by, uint32_t i) {
  const uint32_t two = a.D == 128;                   // groups a row: 1 or 2
  const uint32_t gr = i & two, row = i >> two;
  const uint32_t bt = by.heads.of(row), h = row - bt * by.heads.d;
  const uint32_t b = by.tokens.of(bt), t = bt - b * by.tokens.d;
  Group x;
  const long long slot = (long long)(a.start ? __ldg(a.start + b) : 0) + t;
  x.counts = !a.n_new || (int)t < __ldg(a.n_new + b);
  x.in_cache = slot >= 0 && slot < a.C;
  x.word = ((((long long)b * a.H_kv + h) * a.C + slot) << two) + gr;
  if (x.in_cache)
    x.in_cache = in_range(x.word, 1, (long long)a.B * a.H_kv * a.C << two, a.status);
  return x;
}

// Eight values of a group whose other lanes are the mask's: its codes as one
// word, its scale and zero point.
__device__ __forceinline__ uint32_t encode(const float (&x)[kVals], uint32_t mask,
                                           uint32_t& meta) {
  float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    bad += x[e] * 0.f;                // NaN as soon as one value is not finite
  }
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
    bad += __shfl_xor_sync(mask, bad, o);
  }
  const __nv_bfloat16 sb =
      __float2bfloat16_rn(__fadd_rn(__fsub_rn(__fdiv_rn(hi, 15.f), __fdiv_rn(lo, 15.f)), bad));
  const float scale = __bfloat162float(sb);
  const __nv_bfloat16 zb = __float2bfloat16_rn(__fadd_rn(__fadd_rn(lo, __fmul_rn(8.f, scale)), bad));
  const float zero = __bfloat162float(zb);
  meta = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    const float n = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(x[e], zero), scale)) : 0.f;
    const int c = (int)fminf(fmaxf(n, -8.f), 7.f) + 8;
    w |= (uint32_t)c << (4 * e);
  }
  return w;
}

// The eight values of a word of codes, stored as float32 (one rounding) ...
__device__ __forceinline__ void store_values(float* p, uint32_t w, uint32_t meta) {
  const float scale = __uint_as_float(meta << 16), zero = __uint_as_float(meta & 0xffff0000u);
  float x[kVals];
#pragma unroll
  for (int e = 0; e < kVals; ++e)      // 2^23 + c, exact as everything up to the sum
    x[e] = fmaf(scale, __uint_as_float(((w >> (4 * e)) & 15u) | 0x4b000000u) - 8388616.f, zero);
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// ... or as bfloat16 (one rounding, two values an operation: 128 + c and c - 8
// are bfloat16 numbers).
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t w, uint32_t meta) {
  auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
  const __nv_bfloat162 scale = pair(__byte_perm(meta, 0, 0x1010));
  const __nv_bfloat162 zero = pair(__byte_perm(meta, 0, 0x3232));
  uint32_t r[4];                       // values e and e + 4
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t u = ((w >> (4 * e)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 x = __hfma2(scale, __hsub2(pair(u), pair(0x43084308u)), zero);
    r[e] = *reinterpret_cast<const uint32_t*>(&x);
  }
  *reinterpret_cast<uint4*>(p) =
      make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                 __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
}

// Both kernels: eight lanes a group, of the keys and of the values.
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const Kv4RowArgs a, const Divisors by, uint32_t groups) {
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  // eight lanes leave or stay together: the shuffles name only them
  const uint32_t mask = 0xffu << (threadIdx.x & 24);
  if (i >= groups) return;
  const Group r = locate(a, by, i);
  if (!r.counts) return;
  if (!r.in_cache) {
    if (lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    return;
  }
  const size_t elem = (size_t)i * kKv4Group + lane * kVals;
  float k[kVals], v[kVals];
  load8(static_cast<const T*>(a.k) + elem, k);
  load8(static_cast<const T*>(a.v) + elem, v);
  uint32_t mk, mv;
  const uint32_t wk = encode(k, mask, mk), wv = encode(v, mask, mv);
  reinterpret_cast<uint32_t*>(a.c.kc)[r.word * kLanes + lane] = wk;
  reinterpret_cast<uint32_t*>(a.c.vc)[r.word * kLanes + lane] = wv;
  if (lane == 0) {
    a.c.km[r.word] = mk;
    a.c.vm[r.word] = mv;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4RowArgs a, const Divisors by, uint32_t groups) {
  const uint32_t i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (i >= groups) return;
  const Group r = locate(a, by, i);
  uint32_t wk = 0, wv = 0, mk = 0, mv = 0;           // no such slot: zeros
  if (r.in_cache) {
    wk = __ldg(reinterpret_cast<const uint32_t*>(a.c.kc) + r.word * kLanes + lane);
    wv = __ldg(reinterpret_cast<const uint32_t*>(a.c.vc) + r.word * kLanes + lane);
    mk = __ldg(a.c.km + r.word);
    mv = __ldg(a.c.vm + r.word);
  } else if (lane == 0 && a.status) {
    atomicExch(a.status, (int)RA_ERR_RANGE);
  }
  const size_t elem = (size_t)i * kKv4Group + lane * kVals;
  if (a.k) store_values(static_cast<T*>(a.k) + elem, wk, mk);
  if (a.v) store_values(static_cast<T*>(a.v) + elem, wv, mv);
}

template <typename Kernel>
ra_status launch_rows(Kernel kern, const Kv4RowArgs& a, cudaStream_t stream) {
  const long long groups = (long long)a.B * a.T * a.H_kv * (a.D / kKv4Group);
  const int per = kThreads / kLanes;
  const long long blocks = (groups + per - 1) / per;
  const Divisors by = {Divisor((uint32_t)a.H_kv), Divisor((uint32_t)a.T)};
  kern<<<(unsigned)blocks, kThreads, 0, stream>>>(a, by, (uint32_t)groups);
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

}  // namespace

ra_status launch_kv4_append(const Kv4RowArgs& a, int dtype, cudaStream_t stream) {
  return dtype == RA_F32 ? launch_rows(kv4_append_kernel<float>, a, stream)
                         : launch_rows(kv4_append_kernel<__nv_bfloat16>, a, stream);
}

ra_status launch_kv4_read(const Kv4RowArgs& a, int dtype, cudaStream_t stream) {
  return dtype == RA_F32 ? launch_rows(kv4_read_kernel<float>, a, stream)
                         : launch_rows(kv4_read_kernel<__nv_bfloat16>, a, stream);
}

}  // namespace ra
