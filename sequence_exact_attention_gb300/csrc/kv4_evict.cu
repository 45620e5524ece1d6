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
// tells the next digit. A cluster of kCtas CTAs shares one (sequence, head):
// each counts a contiguous slice of the slots, the histograms and the counts
// before a slice are read through distributed shared memory, and each copies
// the rows that its own slice keeps. One launch.
//
// What bounds it: at large sizes the bytes copied (read and written once) and
// the scores; at small ones the passes' barriers.
#include <cooperative_groups.h>

#include <cstdint>

#include "checks.cuh"
#include "kv4_internal.h"

namespace cg = cooperative_groups;

namespace ra {
namespace {

constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Unsigned order = the scores' order; NaN 0, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
kv4_evict_kernel(const Kv4EvictArgs a) {
  __shared__ int hist[4][256];             // one a pass: no pass waits for the last one's readers
  __shared__ int total[256];
  __shared__ int digit, rest;
  __shared__ int my_sure, my_equal;        // slots kept for sure, slots at the threshold
  __shared__ int wsum[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / kCtas, b = bh / a.H_kv;
  const int n = min(max(__ldg(a.lens + b), 0), a.C);
  const int keep = min(n, a.budget);
  const bool all = n <= a.budget;
  const int per = (n + kCtas - 1) / kCtas;
  const int s0 = min(rank * per, n), s1 = min(s0 + per, n);
  // the slots between the protected ones
  const int c0 = a.n_sink, c1 = n - a.n_recent;
  const int need = a.budget - a.n_sink - a.n_recent;
  const float* score = a.score + (size_t)bh * a.C;

  for (int i = threadIdx.x; i < 4 * 256; i += kThreads) hist[i / 256][i % 256] = 0;
  __syncthreads();
  uint32_t thr = 0;                        // the threshold's digits so far
  int left = need;                         // slots to take among those that match them
  if (!all && need > 0) {
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int j = max(s0, c0) + threadIdx.x; j < min(s1, c1); j += kThreads) {
        const uint32_t k = order_key(__ldg(score + j));
        if (pass == 0 || (k >> (shift + 8)) == (thr >> (shift + 8)))
          atomicAdd(&hist[pass][(k >> shift) & 255u], 1);
      }
      cluster.sync();
      if (threadIdx.x < 256) {
        int t = 0;
        for (int r = 0; r < kCtas; ++r) t += cluster.map_shared_rank(&hist[pass][0], r)[threadIdx.x];
        total[threadIdx.x] = t;
      }
      __syncthreads();
      if (threadIdx.x < 32) {
        // lane i: digits 255 - 8i down to 248 - 8i; the first whose running
        // count reaches `left` is the threshold's digit
        const int top = 255 - 8 * threadIdx.x;
        int sum = 0;
        for (int i = 0; i < 8; ++i) sum += total[top - i];
        int before = sum;
        for (int o = 1; o < 32; o *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if ((int)threadIdx.x >= o) before += y;
        }
        before -= sum;
        if (before < left && before + sum >= left) {
          int d = top;
          while (before + total[d] < left) before += total[d--];
          digit = d;
          rest = left - before;
        }
      }
      __syncthreads();
      thr |= (uint32_t)digit << shift;
      left = rest;
    }
  }
  // ---- what this slice keeps: protected slots and scores above the
  // threshold for sure, and of those at it the first `left` of all slices
  const bool pick = !all && need > 0;
  auto classify = [&](int j) -> int {      // 1 kept for sure, 2 at the threshold, 0 not
    if (all || j < c0 || j >= c1) return 1;
    if (!pick) return 0;
    const uint32_t k = order_key(__ldg(score + j));
    return k > thr ? 1 : (k == thr ? 2 : 0);
  };
  if (threadIdx.x == 0) my_sure = my_equal = 0;
  __syncthreads();
  {
    int sure = 0, equal = 0;
    for (int j = s0 + threadIdx.x; j < s1; j += kThreads) {
      const int k = classify(j);
      sure += k == 1;
      equal += k == 2;
    }
    sure = __reduce_add_sync(0xffffffffu, sure);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if ((threadIdx.x & 31) == 0) {
      atomicAdd(&my_sure, sure);
      atomicAdd(&my_equal, equal);
    }
  }
  cluster.sync();
  int out = 0, quota = left;               // first row written, slots at the threshold still to take
  for (int r = 0; r < rank; ++r) {
    const int e = min(*cluster.map_shared_rank(&my_equal, r), quota);
    out += *cluster.map_shared_rank(&my_sure, r) + e;
    quota -= e;
  }
  const int first = out;
  int* kept = a.kept + (size_t)bh * a.budget;
  // ---- the kept slots in order: a running count over the slice
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j0 = s0; j0 < s1; j0 += kThreads) {
    const int j = j0 + threadIdx.x;
    const int k = j < s1 ? classify(j) : 0;
    // low half: kept for sure, high half: at the threshold
    int x = k == 1 ? 1 : (k == 2 ? 1 << 16 : 0);
    const int mine = x;
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();                       // the last round's sums are read
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int pre = x - mine, tot = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += wsum[w];
      tot += wsum[w];
    }
    const int equal_before = pre >> 16;
    if (k == 1 || (k == 2 && equal_before < quota)) {
      const int at = out + (pre & 0xffff) + min(equal_before, quota);
      if (in_range(at, 1, a.budget, a.status)) kept[at] = j;
    }
    out += (tot & 0xffff) + min(tot >> 16, quota);
    quota -= min(tot >> 16, quota);
  }
  __syncthreads();
  // ---- copy the rows
  const int rows = out - first;
  const int vecs = a.D / 32;               // 16-byte vectors of a row's codes
  const int ng = a.D / kKv4Group;
  const size_t src = (size_t)bh * a.C, dst = (size_t)bh * a.C_dst + first;
  const int* from = kept + first;
  for (int i = threadIdx.x; i < rows * 2 * vecs; i += kThreads) {
    const int r = i / (2 * vecs), w = i % (2 * vecs);
    const bool is_v = w >= vecs;
    const int e = is_v ? w - vecs : w;
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(is_v ? a.src.vc : a.src.kc) +
                          (src + from[r]) * vecs + e);
    reinterpret_cast<uint4*>(is_v ? a.dst.vc : a.dst.kc)[(dst + r) * vecs + e] = u;
  }
  for (int i = threadIdx.x; i < rows * 2 * ng; i += kThreads) {
    const int r = i / (2 * ng), w = i % (2 * ng);
    const bool is_v = w >= ng;
    const int e = is_v ? w - ng : w;
    (is_v ? a.dst.vm : a.dst.km)[(dst + r) * ng + e] =
        __ldg((is_v ? a.src.vm : a.src.km) + (src + from[r]) * ng + e);
  }
  if (a.dst_score)
    for (int r = threadIdx.x; r < rows; r += kThreads) a.dst_score[dst + r] = score[from[r]];
  for (int i = keep + rank * kThreads + threadIdx.x; i < a.budget; i += kCtas * kThreads) kept[i] = -1;
  if (rank == 0 && threadIdx.x == 0 && bh % a.H_kv == 0) a.dst_lens[b] = keep;
  cluster.sync();                          // no CTA leaves while another reads its counts
}

}  // namespace

ra_status launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t stream) {
  const long long grid = (long long)a.B * a.H_kv * kCtas;
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  kv4_evict_kernel<<<(unsigned)grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? RA_OK : RA_ERR_LAUNCH;
}

}  // namespace ra
