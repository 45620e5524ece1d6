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
// Both kernels are bound by the bytes they move. Eight lanes share a group,
// eight values each: the float side moves in 16-byte vectors, a group's codes
// are one 32-byte sector.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "checks.cuh"
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
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[kVals]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[kVals]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// One group of the token rows [B, T, H_kv, D]: its token's sequence and slot.
struct Group {
  long long elem;      // first element of the group in the token tensor
  long long word;      // the group's word in meta: ((b H_kv + h) C + slot) (D / 64) + group
  int b, t, slot;
};

__device__ __forceinline__ Group locate(const Kv4RowArgs& a, long long i) {
  Group r;
  const int ng = a.D / kKv4Group;
  r.elem = i * kKv4Group;
  const int gr = (int)(i % ng);
  i /= ng;
  const int h = (int)(i % a.H_kv);
  i /= a.H_kv;
  r.t = (int)(i % a.T);
  r.b = (int)(i / a.T);
  // a start so large that slot overflows is out of range in any case
  const long long slot = (long long)(a.start ? __ldg(a.start + r.b) : 0) + r.t;
  r.slot = slot >= 0 && slot < a.C ? (int)slot : -1;
  r.word = (((long long)r.b * a.H_kv + h) * a.C + slot) * ng + gr;
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const Kv4RowArgs a, long long groups) {
  const long long i = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  // eight lanes leave or stay together: the shuffles below name only them
  const uint32_t mask = 0xffu << (threadIdx.x & 24);
  if (i >= groups) return;
  const Group r = locate(a, i);
  if (a.n_new && r.t >= __ldg(a.n_new + r.b)) return;    // padding of this sequence
  if (r.slot < 0) {
    if (lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    return;
  }
  const bool is_v = blockIdx.y != 0;
  float x[kVals];
  load8(static_cast<const T*>(is_v ? a.v : a.k) + r.elem + lane * kVals, x);
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
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < kVals; ++e) {
    const float n = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(x[e], zero), scale)) : 0.f;
    const int c = (int)fminf(fmaxf(n, -8.f), 7.f) + 8;
    w |= (uint32_t)c << (4 * e);
  }
  const long long word = r.word;
  const long long n_words = (long long)a.B * a.H_kv * a.C * (a.D / kKv4Group);
  if (!in_range(word, 1, n_words, a.status)) return;
  reinterpret_cast<uint32_t*>(is_v ? a.c.vc : a.c.kc)[word * kLanes + lane] = w;
  if (lane == 0)
    (is_v ? a.c.vm : a.c.km)[word] =
        (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4RowArgs a, long long groups) {
  const long long i = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (i >= groups) return;
  const bool is_v = blockIdx.y != 0;
  T* dst = static_cast<T*>(is_v ? a.v : a.k);
  if (!dst) return;
  const Group r = locate(a, i);
  float x[kVals];
  const long long n_words = (long long)a.B * a.H_kv * a.C * (a.D / kKv4Group);
  if (r.slot < 0 || !in_range(r.word, 1, n_words, a.status)) {
    // no such slot: zeros, and the status says so
    if (lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
#pragma unroll
    for (int e = 0; e < kVals; ++e) x[e] = 0.f;
  } else {
    const uint32_t m = __ldg((is_v ? a.c.vm : a.c.km) + r.word);
    const uint32_t w =
        __ldg(reinterpret_cast<const uint32_t*>(is_v ? a.c.vc : a.c.kc) + r.word * kLanes + lane);
    const float scale = __uint_as_float(m << 16), zero = __uint_as_float(m & 0xffff0000u);
#pragma unroll
    for (int e = 0; e < kVals; ++e)      // the product is exact in float32
      x[e] = fmaf(scale, (float)((int)((w >> (4 * e)) & 15u) - 8), zero);
  }
  store8(dst + r.elem + lane * kVals, x);
}

template <typename Kernel>
ra_status launch_rows(Kernel kern, const Kv4RowArgs& a, cudaStream_t stream) {
  const long long groups = (long long)a.B * a.T * a.H_kv * (a.D / kKv4Group);
  const int per = kThreads / kLanes;
  const long long blocks = (groups + per - 1) / per;
  if (blocks > 0x7fffffffLL) return RA_ERR_RANGE;
  kern<<<dim3((unsigned)blocks, 2), kThreads, 0, stream>>>(a, groups);
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
