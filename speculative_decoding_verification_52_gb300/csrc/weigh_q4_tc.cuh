// weigh_q4_tc.cuh -- the weights of cached tokens (weigh_q4.cuh) for many rows, on the
// tcgen05 tensor cores: chunks of prompts, whose rows meet every cached token.
//
//   S[128 tokens x 64 rows] = K[128 x D] Q^T    (A = K in tensor memory, B = Q in shared memory)
//
// in bf16: a code times its scale has 6 significant bits, the queries are bf16 as they
// come, and one factor takes all products to the log2 domain.  With the tokens as M a
// thread has one token and adds up its row of S; nothing crosses threads.  The unit of
// work is a tile of 128 tokens of a head, whose keys are unpacked once and stay in
// tensor memory while the rows pass by, 64 at a time, two tiles of rows under way in S
// and four or six in shared memory.
//
// Roles of a CTA (two an SM): four warps that add up, four that unpack a unit's keys and
// bring the rows' lse, one that has the queries copied, one that issues the products.
// The queries come by tensor-map copies of 64 / G nodes with their G query heads, in the
// 128-byte swizzle that the tensor cores read.  (Asynchronous copies of 16 bytes by a
// warp took 2,200 clocks a tile, three times what adding it up takes.)  A path's nodes do
// not lie side by side: its rows are few, and weigh_q4.cuh's.
//
// Bound, 2 chunks of 1,024 tokens behind 2,048 and 14,336, 16 query and 2 kv heads of 64
// (285 million scores): 78 us.  Products of 128 x 64 x 16, which take as long as ones of
// 128 x 128 x 16, keep the tensor cores busy most of it; the exponentials take 31 us at 32
// a clock and SM, the adding warps' instructions about as long.  (A second set of adding
// warps changed 75 to 72 us, and units of few tiles by a tenth for the worse.)  A unit
// costs about 2 us by itself (its place in the list, its keys' way from memory).
#pragma once

#include <cuda.h>

#include "tcgen05.cuh"
#include "weigh_q4.cuh"

namespace sv {

constexpr int WT_TILE = 128;      // tokens of a unit
constexpr int WT_ROWS = 64;       // rows of a tile, the last of which stay empty where G does not divide it
constexpr int WT_WARPS = 10, WT_THREADS = 32 * WT_WARPS;
constexpr uint32_t WT_COLS = 256; // tensor memory: two buffers of S, two of K

template <int D>
struct WtShared {
  static constexpr uint32_t q_bytes = WT_ROWS * D * 2;
  static constexpr int STAGES = D == 64 ? 6 : 4;   // tiles of queries
  unsigned char q[STAGES][q_bytes];                // [D / 64][64 rows][128 bytes], swizzled
  float neg_lse[STAGES][WT_ROWS];         // -lse log2(e); -inf: the row adds nothing
  uint64_t qfull[STAGES], qempty[STAGES], kfull[2], kempty[2], sready[2], sfree[2], drain;
  uint32_t tmem;
  int dead;                                  // a wait ran out of time
};

__device__ __noinline__ bool wt_wait_long(uint64_t* bar, uint32_t parity, int* dead, unsigned long long limit);

// Bounded wait, as tc_wait of attend_q4_tc.cuh.
__device__ __forceinline__ bool wt_wait(uint64_t* bar, uint32_t parity, int* dead, unsigned long long limit) {
  if (__builtin_expect(tc_poll(bar, parity), 1)) return true;
  return wt_wait_long(bar, parity, dead, limit);
}
__device__ __noinline__ bool wt_wait_long(uint64_t* bar, uint32_t parity, int* dead, unsigned long long limit) {
  if (*reinterpret_cast<volatile int*>(dead)) return false;   // (at once: the others go on in step)
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1; i < (1u << 28); ++i) {
    if (tc_poll(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*reinterpret_cast<volatile int*>(dead)) return false;
      if (global_ns() - t0 > limit) break;
    }
  }
  *reinterpret_cast<volatile int*>(dead) = 1;
  return false;
}

// Waits for a barrier's phase whatever the flag says: for copies on their way.
__device__ __noinline__ void wt_drain(uint64_t* bar, uint32_t parity, unsigned long long limit) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1; i < (1u << 28) && !tc_poll(bar, parity); ++i)
    if ((i & 63u) == 0u && global_ns() - t0 > limit) break;
}

// A unit: 128 tokens from t0 on of a head of sequence b, and the row tiles that see any
// of them.
struct WtUnit {
  int b, h, t0, old, end, rows, first, last;
};
__device__ __forceinline__ WtUnit wt_unit(const WeighArgs& a, int per, const long long* prefix, const int* all_rows, long long u) {
  WtUnit x;
  int lo = 0, hi = a.B - 1;   // last b with prefix[b] * Hkv <= u that has tiles
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] * a.Hkv <= u) lo = mid;
    else hi = mid - 1;
  }
  x.b = lo;
  const int tiles = static_cast<int>(prefix[lo + 1] - prefix[lo]);
  const long long rem = u - prefix[lo] * a.Hkv;
  x.h = static_cast<int>(rem / tiles);
  x.t0 = static_cast<int>(rem - static_cast<long long>(x.h) * tiles) * WT_TILE;
  x.old = a.lengths[lo];
  const int n = all_rows[lo];
  x.end = x.old + n;
  x.rows = n * a.G;
  x.first = max(0, x.t0 - x.old) * a.G / per;
  x.last = (x.rows + per - 1) / per;
  return x;
}

template <int D>
__global__ void __launch_bounds__(WT_THREADS, 2) weigh_q4_tc_kernel(const WeighArgs a, const __grid_constant__ CUtensorMap map) {
  using S = WtShared<D>;
  extern __shared__ __align__(128) unsigned char wt_raw[];
  __shared__ long long scratch[WT_WARPS];
  unsigned char* aligned = wt_raw + ((1024u - (smem_addr(wt_raw) & 1023u)) & 1023u);
  S& sh = *reinterpret_cast<S*>(aligned);
  long long* prefix = reinterpret_cast<long long*>(aligned + (sizeof(S) + 15) / 16 * 16);   // [B + 1], in tiles
  int* all_rows = reinterpret_cast<int*>(prefix + a.B + 1);                               // [B]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3;
  const unsigned long long limit = a.timeout_ns;
  const int nodes = WT_ROWS / a.G, per = nodes * a.G;   // nodes and rows of a tile

  if (per < WT_ROWS) {   // (rows that no copy writes)
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(sh.q) / 16); i += WT_THREADS) reinterpret_cast<uint4*>(sh.q)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc_proxy_fence();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&sh.qfull[i], 2);
      mbar_init(&sh.qempty[i], 5);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kfull[i], 4);
      mbar_init(&sh.kempty[i], 1);
      mbar_init(&sh.sready[i], 1);
      mbar_init(&sh.sfree[i], 4);
    }
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    mbar_fence_init();
  }
  wg_prefix<WT_THREADS>(a, WT_TILE, prefix, all_rows, scratch);   // (synchronises the CTA)
  const long long units = prefix[a.B] * a.Hkv;
  if (blockIdx.x >= units) return;
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "r"(WT_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, t_k = tmem + 2 * WT_ROWS;   // S: columns 0..127; K: D / 2 each from 128 on

  if (warp < 4) {
    // ---- sums: a thread a token -------------------------------------------------------
    const uint32_t lane_at = static_cast<uint32_t>(32 * quad) << 16;
    const float f = a.scale_log2 * a.k_mul;
    int c = 0;   // tiles of rows so far
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
      const WtUnit x = wt_unit(a, per, prefix, all_rows, u);
      const int pos = x.t0 + 32 * quad + lane;
      long long at = -1;
      float old = 0.f;
      if (pos < x.end) {
        const int e = pos / a.P, page = a.table[static_cast<long long>(x.b) * a.W + e];
        if (page >= 0 && page < a.pages) at = (static_cast<long long>(page) * a.Hkv + x.h) * a.P + (pos - e * a.P);
        if (at >= 0 && pos < x.old) old = a.weights[at];
      }
      float sum = 0.f;
      for (int i = x.first; i < x.last; ++i, ++c) {
        const int buf = c & 1, s = c % S::STAGES;
        wt_wait(&sh.sready[buf], (c >> 1) & 1, &sh.dead, limit);
        wt_wait(&sh.qfull[s], (c / S::STAGES) & 1, &sh.dead, limit);   // (long since: what brought the lse is seen here, too)
        tc_fence_after();
        const float* nl = sh.neg_lse[s];
        const int hidden = max(0, pos - x.old) * a.G - i * per;   // rows of the tile that do not see the token (its distance times G may pass 32 bits)
        const uint32_t s_at = tmem + lane_at + buf * WT_ROWS;
        float part = 0.f;
        bool odd = __any_sync(0xffffffffu, hidden > 0);
        if (!odd) {
          const unsigned long long ff = f2_pack(f, f);
          unsigned long long t0 = 0ull, t1 = 0ull;
          uint32_t r[2][32];
          tc_ld32_start(s_at, r[0]);
#pragma unroll
          for (int k = 0; k < WT_ROWS; k += 32) {   // (the second half comes beside the first one's sums)
            float y[32];
            tc_ld32_end(r[k / 32], y);
            if (k == 0) tc_ld32_start(s_at + 32, r[1]);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 l = *reinterpret_cast<const float4*>(nl + k + j);
              float z0, z1, z2, z3;
              f2_unpack(f2_fma(f2_pack(y[j], y[j + 1]), ff, f2_pack(l.x, l.y)), z0, z1);
              f2_unpack(f2_fma(f2_pack(y[j + 2], y[j + 3]), ff, f2_pack(l.z, l.w)), z2, z3);
              t0 = f2_add(t0, f2_pack(ex2_approx(z0), ex2_approx(z1)));
              t1 = f2_add(t1, f2_pack(ex2_approx(z2), ex2_approx(z3)));
            }
          }
          float p0, p1;
          f2_unpack(f2_add(t0, t1), p0, p1);
          part = p0 + p1;
          odd = __any_sync(0xffffffffu, !(part == part));   // (some score is no number)
        }
        if (TC_RARE(odd)) {   // rows that do not see the token, and scores that are no numbers, weigh nothing
          part = 0.f;
#pragma unroll 1
          for (int k = 0; k < WT_ROWS; k += 8) {
            float y[8];
            __syncwarp();
            tc_ld<8>(s_at + k, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) part += k + j < hidden ? 0.f : ex2_approx(fmaxf(__fmaf_rn(y[j], f, nl[k + j]), kNegInf));
          }
        }
        sum += part;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.sfree[buf]);
          mbar_arrive(&sh.qempty[s]);
        }
      }
      if (at >= 0) {
        if (*reinterpret_cast<volatile int*>(&sh.dead)) sum = __int_as_float(0x7fc00000);
        a.new_weights[at] = pos < x.old ? __fmaf_rn(a.decay, old, sum) : sum;
        if (a.positions && pos >= x.old) a.positions[at] = (a.first ? a.first[x.b] : x.old) + (pos - x.old);
      }
    }
  } else if (warp < 8) {
    // ---- keys: a thread a token; then lse: a warp every fourth tile ---------------------------------------------------------
    const uint32_t lane_at = static_cast<uint32_t>(32 * quad) << 16;
    int n = 0, c = 0;   // units with rows, tiles of rows so far
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
      const WtUnit x = wt_unit(a, per, prefix, all_rows, u);
      if (x.first >= x.last) continue;
      const int pos = x.t0 + 32 * quad + lane;
      uint4 code[D / 32];
      uint64_t sc = 0ull;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) code[i] = make_uint4(0u, 0u, 0u, 0u);
      if (pos < x.end) {
        const int e = pos / a.P, page = a.table[static_cast<long long>(x.b) * a.W + e];
        if (page >= 0 && page < a.pages) {
          const unsigned char* blk = q4_block(const_cast<unsigned char*>(a.cache), page, x.h, pos - e * a.P, a.Hkv, a.P, D);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) code[i] = __ldg(reinterpret_cast<const uint4*>(blk + lane * (D / 2)) + i);
          if constexpr (D == 128) sc = __ldg(reinterpret_cast<const unsigned long long*>(blk + 32 * D + lane * 8));
          else sc = __ldg(reinterpret_cast<const uint32_t*>(blk + 32 * D + lane * 4));
        }
      }
      if (n >= 2) wt_wait(&sh.kempty[n & 1], ((n >> 1) & 1) ^ 1, &sh.dead, limit);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t r[16];
        tc_widen(code[i].x, code[i].y, tc_scale(static_cast<uint32_t>(sc), 0), r);
        tc_widen(code[i].z, code[i].w, tc_scale(static_cast<uint32_t>(sc), 1), r + 8);
        sc >>= 16;
#pragma unroll
        for (int k = 0; k < 16; ++k) r[k] = f16x2_to_bf16x2(r[k]);   // (exact)
        tc_st16(t_k + lane_at + (n & 1) * (D / 2) + i * 16, r);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.kfull[n & 1]);
      ++n;
      const float* lse = a.lse + static_cast<long long>(x.b) * a.N * (a.Hkv * a.G) + x.h * a.G;
      for (int i = x.first; i < x.last; ++i, ++c) {
        if ((c & 3) != quad) continue;
        float l[WT_ROWS / 32];
#pragma unroll
        for (int k = 0; k < WT_ROWS / 32; ++k) {
          const int r = 32 * k + lane, row = i * per + r, node = row / a.G;
          l[k] = r < per && row < x.rows ? __ldg(lse + static_cast<long long>(node) * (a.Hkv * a.G) + (row - node * a.G)) : __builtin_huge_valf();
        }
        const int s = c % S::STAGES;
        if (c >= S::STAGES) wt_wait(&sh.qempty[s], ((c / S::STAGES) & 1) ^ 1, &sh.dead, limit);
#pragma unroll
        for (int k = 0; k < WT_ROWS / 32; ++k)
          sh.neg_lse[s][32 * k + lane] = fabsf(l[k]) < __builtin_huge_valf() ? l[k] * -1.44269504088896f : kNegInf;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.qfull[s]);
      }
    }
  } else if (warp == 8) {
    // ---- queries: one thread ------------------------------------------------------------------
    int c = 0;
    bool go = lane == 0;
    for (long long u = blockIdx.x; go && u < units; u += gridDim.x) {
      const WtUnit x = wt_unit(a, per, prefix, all_rows, u);
      for (int i = x.first; i < x.last; ++i, ++c) {
        const int s = c % S::STAGES;
        // (Warps whose wait has failed go on in step and release stages whose copies may
        // still be on their way; the flag was set before they did.)
        if (c >= S::STAGES) go = wt_wait(&sh.qempty[s], ((c / S::STAGES) & 1) ^ 1, &sh.dead, limit) && !*reinterpret_cast<volatile int*>(&sh.dead);
        if (!go) break;
        mbar_arrive_expect_tx(&sh.qfull[s], static_cast<uint32_t>(per) * D * 2);
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                  smem_addr(sh.q[s]) + k * (WT_ROWS * 128)),
              "l"(&map), "r"(64 * k), "r"(x.h * a.G), "r"(i * nodes), "r"(x.b), "r"(smem_addr(&sh.qfull[s]))
              : "memory");
      }
    }
    // what was started has arrived before the CTA ends
    if (lane == 0)
      for (int t = max(0, c - S::STAGES); t < c; ++t) wt_drain(&sh.qfull[t % S::STAGES], (t / S::STAGES) & 1, limit);
  } else if (lane == 0) {
    // ---- products: one thread ---------------------------------------------------------------
    constexpr uint32_t id = tc_idesc(WT_ROWS, true, false, false);
    int c = 0, n = 0;
    bool ok = true;
    for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const WtUnit x = wt_unit(a, per, prefix, all_rows, u);
      if (x.first >= x.last) continue;
      ok = wt_wait(&sh.kfull[n & 1], (n >> 1) & 1, &sh.dead, limit);
      for (int i = x.first; ok && i < x.last; ++i, ++c) {
        const int buf = c & 1, s = c % S::STAGES;
        ok = wt_wait(&sh.qfull[s], (c / S::STAGES) & 1, &sh.dead, limit);
        if (ok && c >= 2) ok = wt_wait(&sh.sfree[buf], ((c >> 1) & 1) ^ 1, &sh.dead, limit);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = tc_desc_128(smem_addr(sh.q[s]));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)   // (16 elements: 32 bytes on; 64: the next part)
          tc_mma_ts(tmem + buf * WT_ROWS, t_k + (n & 1) * (D / 2) + k * 8, qd + (k / 4) * (WT_ROWS * 128 / 16) + (k % 4) * 2, id, k > 0);
        tc_commit(&sh.sready[buf]);
        tc_commit(&sh.qempty[s]);
      }
      tc_commit(&sh.kempty[n & 1]);
      ++n;
    }
    tc_commit(&sh.drain);
    mbar_wait(&sh.drain, 0, limit);   // nothing is in flight when tensor memory is given back
  }
  __syncwarp();
  __syncthreads();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(WT_COLS) : "memory");
}

}  // namespace sv
