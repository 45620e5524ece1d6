// Attention of many query rows a sequence (pieces of prompts) over its pages, on
// the tcgen05 tensor cores; definitions as in paged_attn.cu.
//
// A query tile is 128 rows of one key/value head: the rows of a group's heads
// side by side, 128 / group tokens of them, so that a key/value tile is loaded once
// for the whole group and a short piece still fills a tile. (A group that does not
// divide 128 leaves the last rows unused.) One CTA owns two query tiles and walks
// the tiles of 128 slots that some row of them sees; each tile of keys and values
// serves both. Of the blocks that do not fill a wave of CTAs the walks are cut into
// chunks, joined by paged_join_many_kernel (paged_plan.cpp).
//
// bf16 pages are read where they lie: the producer warp looks a tile's pages up, a
// lane for each, and asks for their boxes; a page that is not there, or that holds
// nothing that the block sees, comes as zeros (a coordinate past the tensor). 8-bit
// pages are expanded first, by a kernel of their own, to bf16 tiles in the
// workspace: exact, as a code times its row's power of two is a bf16 number. It
// moves 5 bytes a value where the products take 4 D flops a row and value pair.
//
// Roles (384 threads): warps 0-7 softmax, two threads a query row, 64 columns each,
// for Q0 and then Q1 at every tile; a producer warp; an issuer warp whose elected
// lane issues every MMA; two warps that keep values that are not finite from rows that
// do not see them (in the softmax warps' hands this took 4 to 8 us of 90 under a
// window). Tensor memory: S_i (128 f32 columns) at 128 i, over whose first 64 the
// weights are written as bf16; O_i (D columns) at 256 + D i. Per tile j the tensor core
// runs PV0(j) S0(j+1) PV1(j) S1(j+1), one tile's products under the other's softmax.
//
// What bounds it: the softmax, as in the forward kernel (attn_tc.cu), some 1.55 us a
// tile of two times 128 x 128 scores at D = 128 where the products take 1.1; and 7 us a
// CTA outside its tiles (look-ups 1.2, the first tile's way 2 to 3, the end 3). Measured,
// replayed from a graph: 4096 tokens behind 12288 slots, 32 heads on 8, D = 128: 647 us,
// 1490 TFLOP/s; 64 tokens behind 100000 slots: 90 us.
//
// Roundings: weights to bf16 (2^-8 of a weight at most); sums and statistics float32.
// Barriers:
//   qfull[i]         Q_i landed
//   kfull/vfull[s]   keys / values of a tile landed in slot s
//   done[j mod kKBuf] every MMA up to S1(j) is done: K_j's and V_{j-1}'s slots are free
//   sfull[i]         S_i(j) done; it covers PV_i(j-1)
//   pfull[i]         P_i(j) written, O_i rescaled (256 arrivals), V_j checked (64, i = 0)
//   odone[i]         the last PV_i done
// Every wait is bounded: after kTimeoutNs a thread raises the CTA's abort flag, all
// roles fall through to the teardown, which waits (bounded) for copies and MMAs in
// flight and frees the tensor memory, and the status word says RA_ERR_TIMEOUT.
#include <cuda.h>
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
#include "tc_tiles.cuh"

namespace ra {
namespace {

using namespace sm100;
using namespace fastmath;
using tc::kBoxBytes;
using tc::kTile;

constexpr int kSoftmaxWarps = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kCheckWarp = 10, kCheckWarps = 2;
constexpr int kThreads = 32 * (kCheckWarp + kCheckWarps);
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;
constexpr float kRescaleLog2 = 8.0f;       // O is rescaled when the maximum grows by more
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kBoxes = D / 64;
  static constexpr int kKBuf = D == 128 ? 2 : 3;
  static constexpr int kVBuf = kKBuf;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kKBuf * kTileBytes;
  static constexpr int kBarOff = kVOff + kVBuf * kTileBytes;
  static constexpr int kBarBytes = 256;
  // maxima [2 parities][2 parts][128 rows], sums [2 tiles][2 parts][128 rows]
  static constexpr int kRedOff = kBarOff + kBarBytes;
  static constexpr int kRedBytes = (512 + 512) * 4;
  // values that are not finite, of tiles that rows differ in: a bit each, [kEdges][128
  // slots][2][D / 32], first infinity or NaN, then minus infinity or NaN. The block's 256
  // positions make at most three such tiles at each end of a window, the first slots' last
  // tile one more.
  static constexpr int kEdges = 7;
  static constexpr int kOddOff = kRedOff + kRedBytes;
  static constexpr int kOddBytes = kEdges * kTile * 2 * (D / 32) * 4;
  static constexpr int kUsed = kOddOff + kOddBytes + 1024;   // + alignment slack
  // more than half an SM's shared memory: one CTA an SM, so the allocation of all
  // tensor memory never waits for another CTA
  static constexpr int kSmemBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static constexpr int bQFull = 0;                  // [2]
  static constexpr int bKFull = 2;                  // [kKBuf]
  static constexpr int bVFull = bKFull + kKBuf;     // [kVBuf]
  static constexpr int bDone = bVFull + kVBuf;      // [kKBuf]
  static constexpr int bSFull = bDone + kKBuf;      // [2]
  static constexpr int bPFull = bSFull + 2;         // [2]
  static constexpr int bODone = bPFull + 2;         // [2]
  static constexpr int bFinal = bODone + 2;
  static constexpr int kNumBars = bFinal + 1;
  static constexpr int kGoneOff = kBarBytes - 88;     // [8] pages not there, of tile j at j mod 8
  static constexpr int kEdgeOff = kBarBytes - 56;     // [kEdges] first slots of the tiles of kOddOff
  static constexpr int kAnyOff = kBarBytes - 24;      // how many of them have a bit set, or 0
  static constexpr int kHolderOff = kBarBytes - 16;   // tensor memory's address
  static constexpr int kNeverOff = kBarBytes - 12;    // stays 0: waits that ignore aborts
  static constexpr int kAbortOff = kBarBytes - 8;     // abort flag
  static_assert(kNumBars * 8 <= kGoneOff, "barrier area overflow");
  static_assert(kSmemBytes > 116 * 1024, "must not fit two CTAs per SM");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(kOCol + 2 * D <= kTmemCols, "tensor memory budget");
};

// Notes the values of a tile's first `to` rows that are not finite, but not those of rows
// [skip_from, skip_to), in `odd` and makes them 0: a row that does
// not see them has the weight 0 for them. (`odd`: a tile's part of Cfg::kOddOff.) By the
// checking threads. Says whether this thread found any.
template <int D>
__device__ __forceinline__ bool take_odd_values(uint8_t* tile, int to, int skip_from, int skip_to,
                                                uint32_t* odd, int thread) {
  constexpr uint32_t kOnes = 0x7f807f80u;              // two exponents
  // first whether there are any: an exponent of ones carries into its sign
  constexpr int kEach = kTile * (D / 8) / (32 * kCheckWarps);
  uint32_t found = 0;
#pragma unroll 8
  for (int x = 0; x < kEach; ++x) {
    const uint4 v = reinterpret_cast<const uint4*>(tile)[thread + x * 32 * kCheckWarps];
    found |= ((v.x & kOnes) + 0x00800080u) | ((v.y & kOnes) + 0x00800080u) |
             ((v.z & kOnes) + 0x00800080u) | ((v.w & kOnes) + 0x00800080u);
  }
  if (!__any_sync(0xffffffffu, found & 0x80008000u)) return false;
  bool noted = false;
  for (int x = 0; x < kEach; ++x) {
    const int i = thread + x * 32 * kCheckWarps;       // 16 bytes, eight values
    const int row = i / 8 % kTile, chunk = i / (8 * kTile) * 8 + ((i ^ row) & 7);
    if (row >= to || (row >= skip_from && row < skip_to)) continue;
    uint4* at = reinterpret_cast<uint4*>(tile) + i;
    const uint4 v = *at;
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, up = 0, down = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t u = w[k] >> (16 * y) & 0xffffu;
        if ((u & 0x7f80u) != 0x7f80u) continue;
        if (u != 0xff80u) up |= 1u << (2 * k + y);           // infinity or NaN
        if (u != 0x7f80u) down |= 1u << (2 * k + y);         // minus infinity or NaN
        w[k] &= y ? 0x0000ffffu : 0xffff0000u;
      }
    if (up | down) {
      *at = make_uint4(w[0], w[1], w[2], w[3]);
      uint32_t* to_bits = odd + row * (2 * (D / 32)) + chunk / 4;
      atomicOr(to_bits, up << (8 * (chunk % 4)));
      atomicOr(to_bits + D / 32, down << (8 * (chunk % 4)));
      noted = true;
    }
  }
  return noted;
}

// Rows [from, to) of a tile of 64-column boxes, as 0, by the checking threads.
__device__ __forceinline__ void zero_rows(uint32_t tile, int boxes, int from, int to, int thread) {
  for (int bx = 0; bx < boxes; ++bx)
    for (int i = thread; i < (to - from) * 8; i += 32 * kCheckWarps)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                       tile + (uint32_t)(bx * kBoxBytes + from * 128 + i * 16)),
                   "r"(0)
                   : "memory");
}

// The columns below x, a bit each of 64.
__device__ __forceinline__ uint64_t below(int x) {
  return x <= 0 ? 0 : x >= 64 ? ~0ull : (1ull << x) - 1;
}

// The tiles of 128 slots that a sequence's new tokens see, all of them: their
// places among the expanded ones.
__device__ __forceinline__ PagedSpan<kTile> sequence_span(const PagedAttnArgs& a,
                                                          const PagedSeq& sq) {
  PagedSpan<kTile> s;
  s.init(a, sq.len - sq.n, sq.len - 1);
  return s;
}

template <int D, bool kExpanded>
__global__ void __launch_bounds__(kThreads, 1)
paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PagedAttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + C::kBarOff + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + C::kBarOff + C::kAbortOff);
  volatile int* never = reinterpret_cast<volatile int*>(base_ptr + C::kBarOff + C::kNeverOff);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + C::kBarOff + C::kHolderOff);
  volatile uint32_t* gone = reinterpret_cast<volatile uint32_t*>(base_ptr + C::kBarOff + C::kGoneOff);

  uint32_t* odd = reinterpret_cast<uint32_t*>(base_ptr + C::kOddOff);
  volatile int* edge_lo = reinterpret_cast<volatile int*>(base_ptr + C::kBarOff + C::kEdgeOff);
  volatile int* any_odd = reinterpret_cast<volatile int*>(base_ptr + C::kBarOff + C::kAnyOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  let_dependents_start();
  wait_for_prior_grid();
  // ---- work item: two query tiles of one key/value head, all of their walk or one
  // chunk of it
  const int H_kv = a.p.H_kv, grp = a.H_q / H_kv;
  const int tt = kTile / grp;                     // tokens a query tile
  const PagedWork work = paged_work(a, blockIdx.x);
  const PagedBlock blk = paged_block(a, work.item);
  const int b = blk.b, hk = blk.hk;
  const PagedSeq sq = b >= 0 ? paged_seq(a, b) : PagedSeq{0, 0, 0};
  const int t0 = blk.rb * 2 * tt;                 // the block's first new token
  const int n_tok = min(2 * tt, sq.n - t0);
  if (work.split == 0 && threadIdx.x == 0 &&      // for the join
      in_range(work.item - a.n_whole, 1, a.n_cut, a.status))
    a.part_block[work.item - a.n_whole] = make_int4(sq.row0 + t0, max(n_tok, 0), hk, 0);
  if (n_tok <= 0) return;                         // past the last block of the batch
  const bool two = n_tok > tt;
  const int first = sq.len - sq.n + t0;           // its position
  PagedSpan<kTile> sp;
  sp.init(a, first, first + n_tok - 1);
  const int v_begin = max(work.split, 0) * a.chunk;
  const int n = max((work.split < 0 ? sp.n : min(sp.n, v_begin + a.chunk)) - v_begin, 0);  // tiles
  auto tile_lo = [&](int j) -> int { return sp.tile(v_begin + j) * kTile; };

  // ---- set-up: barriers, abort flag, TMEM
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::bQFull + i), 1);
      mbar_init(bar(C::bSFull + i), 1);
      mbar_init(bar(C::bPFull + i), 32 * (kSoftmaxWarps + (i == 0 ? kCheckWarps : 0)));
      mbar_init(bar(C::bODone + i), 1);
    }
    for (int i = 0; i < C::kKBuf; ++i) {
      mbar_init(bar(C::bKFull + i), 1);
      mbar_init(bar(C::bVFull + i), 1);
      mbar_init(bar(C::bDone + i), 1);
    }
    mbar_init(bar(C::bFinal), 1);
    *abort_flag = 0;
    *never = 0;
    *any_odd = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < C::kOddBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(base_ptr + C::kOddOff)[i] = make_uint4(0, 0, 0, 0);
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == kProducerWarp) {
    // ======================= TMA producer =======================
    if (lane == 0) {
      for (int i = 0; i < (two ? 2 : 1); ++i) {
        mbar_arrive_expect_tx(bar(C::bQFull + i), (uint32_t)(C::kBoxes * tt * grp * 128));
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_3d(base + C::kQOff + i * C::kTileBytes + bx * kBoxBytes, &tm_q,
                      bar(C::bQFull + i), bx * 64, hk * grp, sq.row0 + t0 + i * tt);
      }
    }
    __syncwarp();
    // done(x) is phase x / kKBuf of ring barrier x mod kKBuf. It is waited for only
    // while K_{x + kKBuf}, which done(x + kKBuf) needs, is not loaded, so the barrier
    // is never two phases ahead.
    auto wait_done = [&](int x) -> bool {
      return mbar_wait_warp(bar(C::bDone + x % C::kKBuf), (uint32_t)(x / C::kKBuf) & 1, abort_flag,
                            kTimeoutNs);
    };
    const int shift = 31 - __clz(a.p.page);
    const int n_box = kTile >> shift;             // pages a tile
    const int at = lane << shift;                 // this lane's page's first slot in the tile
    const PagedSpan<kTile> whole = sequence_span(a, sq);
    const int past = kExpanded ? 0 : a.p.n_pages * H_kv;      // past the tensor: zeros
    auto look_up = [&](int j) -> int {            // -1: nothing to load; -2: no such page
      if (j >= n || lane >= n_box) return -1;
      const int slot = tile_lo(j) + at;
      if (slot >= sp.hi || !sp.meets(a, slot, a.p.page)) return -1;
      const int id = paged_entry(a, b, slot >> shift);
      return paged_held(a, id) ? id : -2;
    };
    auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t full, int id, int j) {
      if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
      __syncwarp();
      if constexpr (kExpanded) {
        const int t = sp.tile(v_begin + j);
        const int v = t < whole.n_sink_tiles ? t : t - whole.w0 + whole.n_sink_tiles;
        if (lane < C::kBoxes)
          tma_load_4d(dst + lane * kBoxBytes, m, full, 0, 0, lane,
                      (b * a.n_expanded + v) * H_kv + hk);
      } else if (lane < n_box) {
        const int z = id >= 0 ? id * H_kv + hk : past;
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(dst + bx * kBoxBytes + at * 128, m, full, 0, 0, bx, z);
      }
    };
    int id = look_up(0);
    int nk = 0, nv = 0, s = 0;                    // tiles of keys, of values asked for; slot
    bool bad = false;
    for (int j = 0; j < n; ++j) {
      const int next = look_up(j + 1);
      const uint32_t missing = __ballot_sync(0xffffffffu, id == -2);
      bad |= missing != 0;
      // K_j reuses the slot of K_{j-kKBuf}: free at done(j - kKBuf)
      if (j >= C::kKBuf && !wait_done(j - C::kKBuf)) break;
      if (lane == 0) gone[j & 7] = missing;       // tile j - 8's has been read long since
      load(base + C::kKOff + s * C::kTileBytes, &tm_k, bar(C::bKFull + s), id, j);
      ++nk;
      // V_j reuses the slot of V_{j-kVBuf}: free at done(j - kVBuf + 1)
      if (j >= C::kVBuf && !wait_done(j - C::kVBuf + 1)) break;
      load(base + C::kVOff + s * C::kTileBytes, &tm_v, bar(C::bVFull + s), id, j);
      ++nv;
      id = next;
      if (++s == C::kKBuf) s = 0;
    }
    // what was asked for lands before the CTA leaves (it has, unless it aborted)
    for (int x = max(nk - C::kKBuf, 0); x < nk; ++x)
      mbar_wait(bar(C::bKFull + x % C::kKBuf), (uint32_t)(x / C::kKBuf) & 1, never, kTimeoutNs);
    for (int x = max(nv - C::kVBuf, 0); x < nv; ++x)
      mbar_wait(bar(C::bVFull + x % C::kVBuf), (uint32_t)(x / C::kVBuf) & 1, never, kTimeoutNs);
    for (int i = 0; i < (two ? 2 : 1); ++i) mbar_wait(bar(C::bQFull + i), 0, never, kTimeoutNs);
    if (bad && lane == 0 && a.status) atomicExch(a.status, (int)RA_ERR_RANGE);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ======================= MMA issuer =======================
    // The whole warp runs the loop, so its descriptor arithmetic is warp-uniform;
    // one elected lane issues the MMAs and commits.
    const bool leader = elect_one_sync();
    const uint64_t q_desc = sw128_desc(base + C::kQOff, 16, 1024);
    const uint64_t k_desc = sw128_desc(base + C::kKOff, 16, 1024);
    const uint64_t v_desc = sw128_desc(base + C::kVOff, kBoxBytes, 1024);
    const uint64_t q1_off = (uint64_t)(C::kTileBytes >> 4);
    const uint32_t tS0 = tmem, tS1 = tmem + kTile;
    const uint32_t tO0 = tmem + kOCol, tO1 = tmem + kOCol + D;
    bool ok = mbar_wait_warp(bar(C::bQFull), 0, abort_flag, kTimeoutNs) &&
              (!two || mbar_wait_warp(bar(C::bQFull + 1), 0, abort_flag, kTimeoutNs));
    if (ok && n > 0) {
      ok = mbar_wait_warp(bar(C::bKFull), 0, abort_flag, kTimeoutNs);
      if (ok) {
        tc_fence_after();
        if (leader) {
          tc::issue_s<D>(tS0, q_desc, k_desc);
          umma_commit(bar(C::bSFull));
          if (two) {
            tc::issue_s<D>(tS1, q_desc + q1_off, k_desc);
            umma_commit(bar(C::bSFull + 1));
          }
        }
        __syncwarp();
      }
    }
    int ks = 0, kn = 0;                           // slot and use of tile j
    for (int j = 0; ok && j < n; ++j) {
      const bool last = j + 1 == n;
      int nks = ks + 1, nkn = kn;
      if (nks == C::kKBuf) { nks = 0; ++nkn; }
      const uint64_t vd = v_desc + (uint64_t)((ks * C::kTileBytes) >> 4);
      const uint64_t kd = k_desc + (uint64_t)((nks * C::kTileBytes) >> 4);
      // V_j and K_{j+1} have almost always landed long before P0(j): test all three
      // at once and wait one by one only when one is missing
      const uint32_t kb = bar(C::bKFull + (last ? ks : nks));
      const uint32_t kp = (uint32_t)(last ? kn : nkn) & 1;
      if (!__all_sync(0xffffffffu,
                      tc::mbar_test3(bar(C::bVFull + ks), (uint32_t)kn & 1, kb, kp,
                                     bar(C::bPFull), (uint32_t)j & 1)))
        ok = mbar_wait_warp(bar(C::bVFull + ks), (uint32_t)kn & 1, abort_flag, kTimeoutNs) &&
             mbar_wait_warp(kb, kp, abort_flag, kTimeoutNs) &&
             mbar_wait_warp(bar(C::bPFull), (uint32_t)j & 1, abort_flag, kTimeoutNs);
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        tc::issue_pv<D, false>(tO0, tS0, vd, j > 0);
        if (last) {
          umma_commit(bar(C::bODone));
        } else {
          tc::issue_s<D>(tS0, q_desc, kd);
          umma_commit(bar(C::bSFull));
        }
      }
      __syncwarp();
      if (two) {
        ok = mbar_wait_warp(bar(C::bPFull + 1), (uint32_t)j & 1, abort_flag, kTimeoutNs);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          tc::issue_pv<D, false>(tO1, tS1, vd, j > 0);
          if (last) {
            umma_commit(bar(C::bODone + 1));
          } else {
            tc::issue_s<D>(tS1, q_desc + q1_off, kd);
            umma_commit(bar(C::bSFull + 1));
          }
        }
        __syncwarp();
      }
      ks = nks;
      kn = nkn;
    }
    // all tensor-core work this warp issued has completed before teardown
    if (leader) {
      umma_commit(bar(C::bFinal));
      mbar_wait(bar(C::bFinal), 0, never, kTimeoutNs);
    }
    __syncwarp();
  } else if (warp >= kCheckWarp) {
    // ======================= values that rows must not see =======================
    // Where rows differ in what they see, hidden values have weight 0, which NaN and
    // infinities would survive: those that no row of the block sees are made 0, others
    // that are not finite are noted for the rows that see them.
    const int thread = threadIdx.x - 32 * kCheckWarp;
    // no row sees the slots from n_sink to dead_to, nor from sp.hi on
    const int dead_to = a.window > 0 ? first - a.window + 1 : 0;
    int n_edges = 0;
    bool found = false;
    for (int j = 0; j < n; ++j) {
      const int lo = tile_lo(j);
      if (!sp.whole(a, lo, kTile)) {
        const int vs = j % C::kVBuf;
        if (!mbar_wait_warp(bar(C::bVFull + vs), (uint32_t)(j / C::kVBuf) & 1, abort_flag,
                            kTimeoutNs))
          break;
        const int z0 = max(a.n_sink - lo, 0), z1 = min(dead_to - lo, kTile);
        const int z2 = min(max(sp.hi - lo, 0), kTile);
        uint8_t* tile = base_ptr + C::kVOff + vs * C::kTileBytes;
        if (z0 < z1) zero_rows(smem_u32(tile), C::kBoxes, z0, z1, thread);
        if (z2 < kTile) zero_rows(smem_u32(tile), C::kBoxes, z2, kTile, thread);
        if (n_edges < C::kEdges) {
          found |= take_odd_values<D>(tile, z2, z0, z1, odd + n_edges * kTile * 2 * (D / 32),
                                      thread);
          if (thread == 0) edge_lo[n_edges] = lo;
          ++n_edges;
        }
        fence_proxy_async_smem();
      }
      // an arrival a phase: the next one's follows when this one is over
      mbar_arrive(bar(C::bPFull));
      if (j + 1 < n && !mbar_wait_warp(bar(C::bPFull), (uint32_t)j & 1, abort_flag, kTimeoutNs))
        break;
    }
    if (found) *any_odd = n_edges;                // of those noted, one writes at least
    tc::named_bar_sync(5, 32 * (kSoftmaxWarps + kCheckWarps));
  } else {
    // ============ softmax: two threads a query row, Q0 and Q1 in turn ============
    // Warps w and w + 4 share TMEM lane quarter w % 4 (the same 32 rows of each
    // query tile); part p = w / 4 takes columns [64p, 64p + 64) of S_i and
    // [pD/2, (p + 1)D/2) of O_i. A row's two partial maxima meet in shared memory at a
    // named barrier of the pair, which also orders both parts' loads of S before
    // either writes P over it.
    const int wq = warp & 3, part = warp >> 2;
    const int row = wq * 32 + lane;
    const uint32_t t_lane = (uint32_t)(wq * 32) << 16;
    const int ntile = two ? 2 : 1;
    const float sl2 = a.scale_log2;
    const uint64_t sl2x2 = pack2(sl2, sl2);
    const uint32_t pair_bar = 1 + wq;
    float* red = reinterpret_cast<float*>(base_ptr + C::kRedOff);
    const int tok = row / grp;                    // the row's token in its tile
    const int shift = 31 - __clz(a.p.page);
    int ex = 0;                                   // exchanges so far (buffer parity)
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    bool ok = true;
    const bool relay = warp == 0 && lane == 0;
    int rd = 0;
    for (int j = 0; j < n; ++j) {
      const int lo = tile_lo(j);
#pragma unroll
      for (int qi = 0; qi < 2; ++qi) {
        if (qi >= ntile) break;
        const uint32_t tS = tmem + t_lane + (uint32_t)(qi * kTile);
        const int p_first = first + qi * tt;      // the tile's first position
        float* red_e = red + (ex & 1) * 256;
        ++ex;
        if (ok) ok = mbar_wait_warp(bar(C::bSFull + qi), (uint32_t)j & 1, abort_flag, kTimeoutNs);
        if (!ok) {
          // keep meeting the partner at every exchange so it never waits alone
          tc::named_bar_sync(pair_bar, 64);
          continue;
        }
        tc_fence_after();
        uint32_t uu[2][32];
        tmem_ld32(tS + part * 64, uu[0]);
        tmem_ld32(tS + part * 64 + 32, uu[1]);
        // (the keys have landed: the test makes the producer's note of their pages visible)
        mbar_test_wait(bar(C::bKFull + j % C::kKBuf), (uint32_t)(j / C::kKBuf) & 1);
        const uint32_t missing = gone[j & 7];
        if (relay && qi == ntile - 1) {
          mbar_arrive(bar(C::bDone + rd));
          if (++rd == C::kKBuf) rd = 0;
        }
        tmem_ld_wait();
        reg_fence(uu[0]);
        reg_fence(uu[1]);
        const bool all = lo + kTile - 1 <= p_first &&
                         (a.window <= 0 || lo > p_first + tt - 1 - a.window ||
                          lo + kTile <= a.n_sink);
        if (!all || missing) {
          // a bit for each of this part's 64 columns that the row sees
          const int q_pos = p_first + tok, c0 = lo + part * 64;
          uint64_t see = below(q_pos + 1 - c0);
          if (a.window > 0) see &= ~below(q_pos - a.window + 1 - c0) | below(a.n_sink - c0);
          for (uint32_t rest = missing; rest; rest &= rest - 1) {
            const int x = ((__ffs(rest) - 1) << shift) - part * 64;     // a page that is not there
            see &= ~below(x + a.p.page) | below(x);
          }
          const uint32_t bits[2] = {(uint32_t)see, (uint32_t)(see >> 32)};
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(bits[c / 32] >> (c % 32) & 1u)) uu[c / 32][c % 32] = __float_as_uint(-INFINITY);
        }
        float m8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
        tc::max_chunk(uu[0], m8);
        tc::max_chunk(uu[1], m8);
        red_e[part * 128 + row] = tc::max8(m8);
        tc_fence_before();
        tc::named_bar_sync(pair_bar, 64);
        tc_fence_after();
        const float mx = fmaxf(red_e[row], red_e[128 + row]);
        const float m_new = fmaxf(m_run[qi], mx * sl2);
        const bool resc = m_new > m_run[qi] + kRescaleLog2;
        float alpha = 1.f;
        if (resc) {
          alpha = ex2_approx(m_run[qi] - m_new);     // 0 when m_run = -inf
          m_run[qi] = m_new;
          l_run[qi] *= alpha;
        }
        const float m_use = (m_run[qi] == -INFINITY) ? 0.f : m_run[qi];
        const uint64_t neg_m2 = pack2(-m_use, -m_use);
        uint64_t sum2a = pack2(0.f, 0.f), sum2b = sum2a;
        tc::exp_chunk(uu[0], sl2x2, neg_m2, sum2a, sum2b, tS + part * 32);
        tc::exp_chunk(uu[1], sl2x2, neg_m2, sum2a, sum2b, tS + part * 32 + 16);
        {
          float a0, a1;
          unpack2(fadd2(sum2a, sum2b), a0, a1);
          l_run[qi] += a0 + a1;
        }
        // O_i is scaled before P_i(j) V_j is added to it; PV_i(j-1) is done. Both
        // parts take the same decision for a row.
        if (__any_sync(0xffffffffu, resc) && j > 0)
          tc::scale_cols<D / 2>(tmem + t_lane + kOCol + (uint32_t)(qi * D + part * (D / 2)), alpha);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::bPFull + qi));
      }
    }

    // ---- epilogue: out = O / l, lse = ln2 (m + log2 l), l = sum of both parts
    float* red_l = red + 512;
    for (int qi = 0; qi < ntile; ++qi) red_l[(qi * 2 + part) * 128 + row] = l_run[qi];
    tc::named_bar_sync(5, 32 * (kSoftmaxWarps + kCheckWarps));     // what those noted is there
    for (int qi = 0; qi < ntile; ++qi) {
      const float ls = red_l[qi * 256 + row] + red_l[qi * 256 + 128 + row];
      const int t = t0 + qi * tt + tok;
      const bool valid = tok < tt && t < t0 + n_tok;
      if (ok && n > 0) {
        ok = mbar_wait_warp(bar(C::bODone + qi), 0, abort_flag, kTimeoutNs);
        tc_fence_after();
      }
      if (!ok) break;
      const int h = hk * grp + row % grp;
      const long long orow = (long long)(sq.row0 + t) * a.H_q + h;
      const uint32_t tO = tmem + t_lane + kOCol + (uint32_t)(qi * D + part * (D / 2));
      const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);   // 0: no slot; NaN stays
      // this part's dimensions in which the row sees an infinity or NaN, and the other one
      uint32_t up[D / 64] = {}, down[D / 64] = {};
      if (*any_odd) {
        const int q_pos = first + qi * tt + tok;
        for (int i = 0; i < *any_odd * kTile; ++i) {
          if (!paged_sees(a, q_pos, edge_lo[i / kTile] + i % kTile)) continue;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            up[c] |= odd[2 * i * (D / 32) + part * (D / 64) + c];
            down[c] |= odd[(2 * i + 1) * (D / 32) + part * (D / 64) + c];
          }
        }
      }
      const long long prow = paged_part(a, work.item, work.split, qi * kTile + row);
      // The warp's 32 rows go through shared memory (the keys', which every MMA has
      // read), so that they leave as whole runs of D / 2 values: float32 parts, or bf16
      // outputs. (Each thread storing its own row: two sequences under a window of 2048
      // 89 instead of 84 us, a piece of 4096 tokens 652 instead of 646.)
      const bool whole = work.split < 0;
      uint8_t* stage = base_ptr + C::kKOff + warp * (32 * (D / 2) * 4);
      const uint32_t swap = whole ? (D == 128 ? 7 : 3) : 7;      // conflict-free 16-byte chunks
      const uint32_t row_bytes = (D / 2) * (whole ? 2 : 4);
      uint8_t* own = stage + lane * row_bytes;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t uo[32];
        if (n > 0) {
          tmem_ld32(tO + c * 32, uo);
          tmem_ld_wait(uo);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) uo[i] = 0u;
        }
        if (up[c] | down[c]) {                   // infinities of both signs: NaN
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (up[c] >> i & 1u) uo[i] = __float_as_uint(__uint_as_float(uo[i]) + INFINITY);
            if (down[c] >> i & 1u) uo[i] = __float_as_uint(__uint_as_float(uo[i]) - INFINITY);
          }
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = pack_bf16x2(__uint_as_float(uo[8 * i + 2 * x]) * inv,
                                 __uint_as_float(uo[8 * i + 2 * x + 1]) * inv);
            *reinterpret_cast<uint4*>(own + (((4 * c + i) ^ (lane & swap)) * 16)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(own + (((8 * c + i) ^ (lane & swap)) * 16)) =
                make_uint4(uo[4 * i], uo[4 * i + 1], uo[4 * i + 2], uo[4 * i + 3]);
        }
      }
      __syncwarp();
      // where this thread's row goes, in bytes; below 0: nowhere
      const long long at_row = (whole ? orow * 2 : prow * 4) * D + part * row_bytes;
      const bool in = !valid || (whole ? in_range(orow * D, D, (long long)a.rows * a.H_q * D, a.status)
                                       : in_range(prow, 1, paged_part_rows(a), a.status));
      const bool store = valid && in && (whole || n > 0);
      uint8_t* to = whole ? static_cast<uint8_t*>(a.out) : reinterpret_cast<uint8_t*>(a.part_o);
      const int chunks = row_bytes / 16;                         // a row's: 4, 8 or 16
      for (int i = lane; i < 32 * chunks; i += 32) {
        const int r = i / chunks, k = i & (chunks - 1);
        const long long off = __shfl_sync(0xffffffffu, store ? at_row : -1LL, r);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * row_bytes + ((k ^ (r & swap)) * 16));
        if (off >= 0) *reinterpret_cast<uint4*>(to + off + k * 16) = v;
      }
      __syncwarp();                                              // the next tile's rows go there, too
      if (valid && in && part == 0) {
        if (work.split >= 0) {
          a.part_ml[2 * prow] = ls == 0.f ? -INFINITY : m_run[qi];
          a.part_ml[2 * prow + 1] = ls;
        } else if (a.lse) {
          const long long at = paged_lse_at(a, b, sq.row0 + t, t, h);
          if (in_range(at, 1, (long long)a.rows * a.H_q, a.status))
            a.lse[at] = ls == 0.f ? -INFINITY : (m_run[qi] + log2f(ls)) * kLn2;
        }
      }
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && (*abort_flag || *never) && a.status)
    atomicExch(a.status, (int)RA_ERR_TIMEOUT);
}

// 8-bit pages to bf16 tiles [B][n_expanded][H_kv][128][D], keys and values: the
// tiles that the sequences' new tokens see, in order; slots past the last and those
// that no token sees as zeros. (Or, a.by_page, the pages of the slots that they see, to as
// many bf16 pages; sequences that share one write it alike.) A CTA makes some rows of one tile and head, 16 values a
// thread, and goes on where there are more of them than the card has places: a launch
// for all that there may be takes 100 us of CTAs that only leave, for 64 sequences of 8K
// slots. Bound by the bytes, and by the chain of look-ups before them.
constexpr int kExpandThreads = 256;
constexpr long long kExpandCtas = 2 * 8 * 152;
template <int D>
__global__ void __launch_bounds__(kExpandThreads)
paged_expand_kernel(const PagedAttnArgs a, uint32_t shares) {
  constexpr int kLanes = D / 16, kRows = kExpandThreads / kLanes, kShares = kTile / kRows;
  static_assert(kShares == D / kPagedShare, "what the plan counts");
  let_dependents_start();
  wait_for_prior_grid();
  const int shift = 31 - __clz(a.p.page), lane = threadIdx.x & 31;
  const int d = threadIdx.x % kLanes * 16;
  for (uint32_t share = blockIdx.x; share < shares; share += gridDim.x) {
    // which tile of which sequence and head: looked up among their numbers of tiles
    const int x = (int)(share / kShares);
    int b0 = 0, before = 0;                        // tiles of the sequences before these 32
    uint32_t past = 0;
    int sum, nv;
    for (;; b0 += 32) {
      if (b0 >= a.B) return;                       // past the last
      nv = 0;
      if (b0 + lane < a.B) {
        const PagedSeq sq = paged_seq(a, b0 + lane);
        if (sq.n > 0 && paged_mine(a, sq)) nv = min(sequence_span(a, sq).n, a.n_expanded);
      }
      sum = warp_prefix(nv, lane);
      past = __ballot_sync(0xffffffffu, x < (before + sum) * a.p.H_kv);
      if (past) break;
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    const int src = __ffs(past) - 1, b = b0 + src;
    const int in = x - (before + __shfl_sync(0xffffffffu, sum - nv, src)) * a.p.H_kv;
    const int v = in / a.p.H_kv, hk = in % a.p.H_kv;
    const size_t tile = ((size_t)b * a.n_expanded + v) * a.p.H_kv + hk;
    const PagedSpan<kTile> sp = sequence_span(a, paged_seq(a, b));
    const int r = share % kShares * kRows + threadIdx.x / kLanes;
    const int slot = sp.tile(v) * kTile + r;
    long long from = -1;
    if (slot < sp.hi && sp.meets(a, slot, 1)) {
      const int id = paged_entry(a, b, slot >> shift);
      if (paged_held(a, id)) from = (((long long)id * a.p.H_kv + hk) << shift) + (slot & (a.p.page - 1));
      if (from >= 0 && !in_range(from, 1, paged_pool_rows(a.p), a.status)) from = -1;
    }
    if (a.by_page && from < 0) continue;             // (the tiles' kernel finds no page, either)
    const size_t to = a.by_page ? (size_t)from : tile * kTile + r;
    if (!in_range((long long)to, 1,
                  a.by_page ? paged_pool_rows(a.p) : (long long)a.B * a.n_expanded * a.p.H_kv * kTile,
                  a.status))
      continue;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint32_t w[8] = {};
      if (from >= 0) {
        const uint4 c = *reinterpret_cast<const uint4*>((side ? a.p.v : a.p.k) + from * D + d);
        const float scale = pow2_byte((side ? a.p.vs : a.p.ks)[from]);
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float2 f = half2_values(e4m3x2_half2(cw[x / 2] >> (16 * (x % 2))));
          w[x] = pack_bf16x2(f.x * scale, f.y * scale);
        }
      }
      uint4* dst = reinterpret_cast<uint4*>((side ? a.expanded_v : a.expanded_k) + to * D + d);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int D, bool kExpanded>
ra_status launch_tiles(const PagedAttnArgs& a, cudaStream_t stream) {
  const int grp = a.H_q / a.p.H_kv, tt = kTile / grp;
  CUtensorMap mq, mk, mv;
  PagePool p = a.p;
  if (kExpanded) {
    const long long shares = (long long)a.B * a.n_expanded * a.p.H_kv * (D / kPagedShare);
    const long long ctas = shares < kExpandCtas ? shares : kExpandCtas;
    if (!launch_early(paged_expand_kernel<D>, ctas, kExpandThreads, 0, stream, a, (uint32_t)shares))
      return RA_ERR_LAUNCH;
    p.k = reinterpret_cast<uint8_t*>(a.expanded_k);
    p.v = reinterpret_cast<uint8_t*>(a.expanded_v);
    p.quant = 0;
    if (a.by_page) {
      PagedAttnArgs pages = a;
      pages.p = p;
      return launch_tiles<D, false>(pages, stream);
    }
    p.n_pages = a.B * a.n_expanded;
    p.page = kTile;
  }
  if (!make_query_map(&mq, a.q, a.rows, a.H_q, D, grp, tt) ||
      !make_page_map(&mk, p, p.k, p.page, 1) || !make_page_map(&mv, p, p.v, p.page, 1))
    return RA_ERR_LAUNCH;
  const long long grid = a.n_items + (long long)a.n_cut * (a.n_split - 1);
  if (grid > 0x7fffffffLL) return RA_ERR_RANGE;
  auto kern = paged_tiles_kernel<D, kExpanded>;
  static std::atomic<uint64_t> allowed;
  if (!allow_smem(kern, Cfg<D>::kSmemBytes, allowed)) return RA_ERR_LAUNCH;
  return launch_early(kern, grid, kThreads, Cfg<D>::kSmemBytes, stream, mq, mk, mv, a)
             ? RA_OK : RA_ERR_LAUNCH;
}

}  // namespace

ra_status launch_paged_tiles(const PagedAttnArgs& a, cudaStream_t stream) {
  if (a.p.D == 64)
    return a.p.quant ? launch_tiles<64, true>(a, stream) : launch_tiles<64, false>(a, stream);
  return a.p.quant ? launch_tiles<128, true>(a, stream) : launch_tiles<128, false>(a, stream);
}

}  // namespace ra
