// Eviction from a 4-bit cache by accumulated attention weight.
//
// A sequence that uses n > budget slots keeps `budget` of them, a head at a
// time: the first n_sink, the last n_recent and, of those between, the
// need = budget - n_sink - n_recent with the largest scores; among equal
// scores the lowest slot, NaN below every number. Kept slots keep their
// order. n <= budget keeps all. The kept rows go to another cache, so no copy
// waits for another and the source stays as it was.
//
// The threshold score is found by radix selection: the scores' bits, mapped
// so that their order is the numbers', eight bits a pass from the top; a
// histogram of the digit among the slots that match the threshold so far
// tells the next digit. Accumulated weights share their leading bits, so the
// lanes of a warp that hold one digit add to it once, together. (Eleven bits
// in three passes measured slower: a cluster then moves eight times the
// histogram through its shared memories.)
//
// Long caches: a cluster of eight CTAs shares one (sequence, head), every
// warp a contiguous run of its slots, whose keys it keeps in shared memory.
// Histograms and the counts before a run are read through distributed shared
// memory; then every warp lists the slots that its own run keeps, and, when
// the list is whole, the cluster shares the rows evenly (the last n_recent
// slots, all kept, lie in a few runs: runs that copied their own rows took 90
// us of 130 at 8 x 8 heads of 32K slots). Up to kAloneSlots slots one CTA does
// it, without the cluster's barriers. One launch either way.
//
// What bounds it: the passes' barriers and round trips first, then the bytes
// copied (read and written once). Measured, 8 sequences of 8K to 32K slots x 8
// heads, D = 128, 4096 kept: 35 us; of the longest's time 2 us load its scores, 15
// are the four passes, 6 the lists and 9 the copy (92 MB).
#include <cooperative_groups.h>

#include <cstdint>
#include <type_traits>

#include "checks.cuh"
#include "kv4_internal.h"

namespace cg = cooperative_groups;

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAloneSlots = 2048;
constexpr int kClusterCtas = 8;
constexpr int kPasses = 4, kBins = 256;
constexpr int kSmemSlots = 50000;        // a CTA's keys in shared memory (200 KB)
constexpr int kListRows = 1024;
static_assert(kThreads == kBins, "one bin a thread");

// Unsigned order = the scores' order; NaN 0, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A warp's run of n slots: whole chunks of 32.
template <int kCtas>
__host__ __device__ __forceinline__ int run_slots(int n) {
  return ((n + kCtas * kWarps - 1) / (kCtas * kWarps) + 31) / 32 * 32;
}

// kCtas: CTAs a (sequence, head); D: head size. in_smem: the keys of a CTA's
// runs are in `slice` (else they are made from the scores each time), and the
// first two words of a chunk then hold which of its slots are kept for sure
// and which are at the threshold.
template <int kCtas, int D>
__global__ void __launch_bounds__(kThreads)
kv4_evict_kernel(const Kv4EvictArgs a, int in_smem) {
  extern __shared__ uint32_t slice[];
  __shared__ int hist[kPasses][kBins];     // one a pass: no pass waits for the last one's readers
  __shared__ int digit, rest;
  __shared__ int sums[2][kWarps];
  __shared__ int counts[kWarps][2];        // a warp's slots kept for sure, at the threshold
  __shared__ int list[kListRows];          // kept slots being copied
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCtas == 1 ? 0 : (int)cluster.block_rank();
  auto all_here = [&] {
    if constexpr (kCtas == 1) __syncthreads();
    else cluster.sync();
  };
  auto peer = [&](int* p, int r) -> const int* {
    if constexpr (kCtas == 1) return p;
    else return cluster.map_shared_rank(p, r);
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = blockIdx.x / kCtas, b = bh / a.H_kv;
  const int n = min(max(__ldg(a.lens + b), 0), a.C);
  const int keep = min(n, a.budget);
  const bool all = n <= a.budget;
  // this warp's run of slots, and where its CTA's first run starts
  const int run = run_slots<kCtas>(n);
  const int base = min(rank * kWarps * run, n);
  const int s0 = min((rank * kWarps + warp) * run, n), s1 = min(s0 + run, n);
  // the slots between the protected ones
  const int c0 = a.n_sink, c1 = n - a.n_recent;
  const int need = a.budget - a.n_sink - a.n_recent;
  const bool pick = !all && need > 0;
  const float* score = a.score + (size_t)bh * a.C;

  for (int i = threadIdx.x; i < kPasses * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  if (pick && in_smem)
    for (int j = s0 + lane; j < s1; j += 32) slice[j - base] = order_key(__ldg(score + j));
  __syncthreads();
  auto key = [&](int j) { return in_smem ? slice[j - base] : order_key(__ldg(score + j)); };

  uint32_t thr = 0;                        // the threshold's digits so far
  int left = need;                         // slots to take among those that match them
  if (pick) {
    const int lo = max(s0, c0), hi = min(s1, c1);
    for (int pass = 0; pass < kPasses; ++pass) {
      const int shift = 24 - 8 * pass;
      // four chunks at a time: after the first pass few of them match at all
      for (int j0 = lo; j0 < hi; j0 += 4 * 32) {
        uint32_t d[4];                     // kBins: no digit
        bool any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + 32 * e + lane;
          const uint32_t k = j < hi ? key(j) : 0u;
          const bool in = j < hi && (pass == 0 || ((k ^ thr) >> (shift + 8)) == 0);
          d[e] = in ? (k >> shift) & (kBins - 1) : kBins;
          any |= in;
        }
        if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t same = __match_any_sync(0xffffffffu, d[e]);
          if (d[e] < kBins && lane == __ffs(same) - 1) atomicAdd(&hist[pass][d[e]], __popc(same));
        }
      }
      all_here();
      // thread t: bin 255 - t of all slices
      int count = 0;
#pragma unroll
      for (int r = 0; r < kCtas; ++r) count += peer(&hist[pass][0], r)[kBins - 1 - threadIdx.x];
      int upto = count;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) sums[pass & 1][warp] = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += sums[pass & 1][w];
      if (upto - count < left && upto >= left) {
        digit = kBins - 1 - threadIdx.x;
        rest = left - (upto - count);
      }
      __syncthreads();
      thr |= (uint32_t)digit << shift;
      left = rest;
    }
  }
  // ---- what each run keeps: protected slots and scores above the threshold
  // for sure, and of those at it the first `left` of all runs
  auto classify = [&](int j) -> int {      // 1 kept for sure, 2 at the threshold, 0 not
    if (j >= s1) return 0;
    if (all || j < c0 || j >= c1) return 1;
    if (!pick) return 0;
    const uint32_t k = key(j);
    return k > thr ? 1 : (k == thr ? 2 : 0);
  };
  {
    int sure = 0, equal = 0;
#pragma unroll 4
    for (int j0 = s0; j0 < s1; j0 += 32) {
      const int k = classify(j0 + lane);
      const uint32_t is_sure = __ballot_sync(0xffffffffu, k == 1);
      const uint32_t is_equal = __ballot_sync(0xffffffffu, k == 2);
      sure += __popc(is_sure);
      equal += __popc(is_equal);
      if (in_smem && lane < 2) slice[j0 - base + lane] = lane ? is_equal : is_sure;
    }
    if (lane == 0) {
      counts[warp][0] = sure;
      counts[warp][1] = equal;
    }
  }
  all_here();
  // the runs before this one, in order: lane l of each step one run
  int out = 0, quota = left;               // first row written, slots at the threshold still to take
  const int before = rank * kWarps + warp;
  {
    int sure = 0, equal = 0;
    for (int r = lane; r < before; r += 32) {
      const int* c = peer(&counts[0][0], r / kWarps) + 2 * (r % kWarps);
      sure += c[0];
      equal += c[1];
    }
    sure = __reduce_add_sync(0xffffffffu, sure);
    equal = min(__reduce_add_sync(0xffffffffu, equal), quota);
    out = sure + equal;
    quota -= equal;
  }
  int* kept = a.kept + (size_t)bh * a.budget;
  for (int j0 = s0; j0 < s1; j0 += 32) {
    uint32_t is_sure, is_equal;
    if (in_smem) {
      is_sure = slice[j0 - base];
      is_equal = slice[j0 - base + 1];
    } else {
      const int k = classify(j0 + lane);
      is_sure = __ballot_sync(0xffffffffu, k == 1);
      is_equal = __ballot_sync(0xffffffffu, k == 2);
    }
    const uint32_t below = (1u << lane) - 1;
    const int equal_before = __popc(is_equal & below);
    if ((is_sure >> lane & 1) || ((is_equal >> lane & 1) && equal_before < quota)) {
      const int at = out + __popc(is_sure & below) + min(equal_before, quota);
      if (in_range(at, 1, a.budget, a.status)) kept[at] = j0 + lane;
    }
    const int taken = min(__popc(is_equal), quota);
    out += __popc(is_sure) + taken;
    quota -= taken;
  }
  for (int i = keep + rank * kThreads + threadIdx.x; i < a.budget; i += kCtas * kThreads) kept[i] = -1;
  if (rank == 0 && threadIdx.x == 0 && bh % a.H_kv == 0) a.dst_lens[b] = keep;
  all_here();                              // the list is whole; no peer's counts are read after
  // ---- copy this CTA's share of the rows, four loads in flight a thread
  const int share = (keep + kCtas - 1) / kCtas;
  const int r_end = min((rank + 1) * share, keep);
  const size_t src = (size_t)bh * a.C, dst = (size_t)bh * a.C_dst;
  for (int r0 = rank * share; r0 < r_end; r0 += kListRows) {
    const int rows = min(kListRows, r_end - r0);
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += kThreads) list[r] = kept[r0 + r];
    __syncthreads();
    auto copy = [&](auto* to_k, auto* to_v, const auto* from_k, const auto* from_v, auto width_c) {
      constexpr int width = decltype(width_c)::value;
      const int items = rows * 2 * width;
      for (int i0 = threadIdx.x; i0 < items; i0 += 4 * kThreads) {
        std::remove_const_t<std::remove_reference_t<decltype(*from_k)>> u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * kThreads, w = i % width;
          if (i < items)
            u[e] = __ldg((i & width ? from_v : from_k) + (src + list[i / (2 * width)]) * width + w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + e * kThreads, w = i % width;
          if (i < items)
            (i & width ? to_v : to_k)[(dst + r0 + i / (2 * width)) * width + w] = u[e];
        }
      }
    };
    // 16-byte vectors of codes, and a row's words of metadata
    copy(reinterpret_cast<uint4*>(a.dst.kc), reinterpret_cast<uint4*>(a.dst.vc),
         reinterpret_cast<const uint4*>(a.src.kc), reinterpret_cast<const uint4*>(a.src.vc),
         std::integral_constant<int, D / 32>());
    copy(a.dst.km, a.dst.vm, const_cast<const uint32_t*>(a.src.km),
         const_cast<const uint32_t*>(a.src.vm), std::integral_constant<int, D / kKv4Group>());
    if (a.dst_score)
      for (int r = threadIdx.x; r < rows; r += kThreads)
        a.dst_score[dst + r0 + r] = __ldg(score + list[r]);
  }
}

template <int kCtas, int D>
ra_status launch_ctas(const Kv4EvictArgs& a, cudaStream_t stream) {
  const long long grid = (long long)a.B * a.H_kv * kCtas;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  const int per = run_slots<kCtas>(a.C) * kWarps;     // slots a CTA at most
  const bool in_smem = per <= kSmemSlots;
  const int smem = in_smem ? per * 4 : 0;
  static std::atomic<uint64_t> allowed;
  if (!allow_smem(kv4_evict_kernel<kCtas, D>, kSmemSlots * 4, allowed)) return RA_ERR_LAUNCH;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCtas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_evict_kernel<kCtas, D>, a, in_smem ? 1 : 0) == cudaSuccess
             ? RA_OK
             : (cudaGetLastError(), RA_ERR_LAUNCH);
}

}  // namespace

ra_status launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  if (a.D == 64)
    return a.C <= kAloneSlots ? launch_ctas<1, 64>(a, stream) : launch_ctas<kClusterCtas, 64>(a, stream);
  return a.C <= kAloneSlots ? launch_ctas<1, 128>(a, stream) : launch_ctas<kClusterCtas, 128>(a, stream);
}

}  // namespace ra
