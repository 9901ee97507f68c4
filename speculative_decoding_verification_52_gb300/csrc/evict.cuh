// evict.cuh -- which tokens leave a paged cache by the weight that attention gave
// them, and the entries that fill their places.
//
// The plan.  Of the n cached tokens of a (sequence, kv head), the K = budget with the
// largest keys stay; a key is the token's accumulated weight, above all others for the
// first and the latest positions, equal keys by the lower slot.  What stays at a place
// below K is not touched; the j-th token that stays at a place from K on moves to the
// j-th place below K that becomes free.  So a step that drops 6 of 2,054 tokens moves
// at most 6 entries of a head, where closing the gaps in order would move all that lie
// behind the first.
//
// A CTA or a cluster of up to 8 takes a (sequence, head), each CTA a contiguous part of
// its tokens.  The K-th largest key comes from a radix selection, eight bits a pass, over
// keys that stay in shared memory (those beyond its size are read again): a histogram
// for each warp, added up over the CTA and the cluster.  It ends early in a pass whose
// last bin is needed whole.  (Three passes of 2,048 bins read 64 KB of the other CTAs'
// shared memory a CTA and pass, which took 15,000 clocks.)
//
// Bound: 8 bytes a token read (weight and position).  256 sequences of 8 heads that drop
// up to 6 of 2,054 tokens take 18 us, 1.9 TB/s: a warp a head, 13 warps an SM, about 4,000
// instructions each.  64 heads of 8,192 to 57,344 tokens cut to 4,096 take 31 us, 22 of
// them in the CTAs of the longest: keys 6, four passes of the selection 9, the moves 5,
// most of it barriers of the cluster and of the CTAs.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "kv_q4.cuh"

namespace sv {

constexpr int EV_THREADS = 256;
constexpr int EV_BINS = 256;    // of a pass, eight bits; a bin a thread
constexpr int EV_HISTS = EV_THREADS / 32 + 2;
constexpr int EV_CAP = 8192;    // keys of a CTA in shared memory, at most
constexpr int EV_CLUSTER = 8;   // CTAs of a cluster, at most

struct PlanArgs {
  const float* weights;       // [pages, Hkv, P]
  const int32_t* positions;   // [pages, Hkv, P]
  const int32_t* table;       // [B, W]
  const int32_t* lengths;     // [B]
  const int32_t* budgets;     // [B]
  const int32_t* next;        // [B]
  int B, Hkv, P, pages, W, max_moves, sinks, recent;
  int cap;                    // keys of a CTA, or of a pair, in shared memory (a multiple of 128)
  int rows;                   // pairs of a CTA
  int C;                      // CTAs of a cluster
  int32_t* moves;             // [B, Hkv, max_moves, 2]
  int32_t* counts;            // [B, Hkv]
  int32_t* new_lengths;       // [B]
};

// integers that compare as the weights do; NaN below everything
__device__ __forceinline__ uint32_t ev_ordered(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);   // (-0 becomes 0)
  return w != w ? 0u : u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// a value that k of the warp's lanes reach, the largest such; 0 if fewer have one above 0
__device__ __forceinline__ uint32_t warp_kth(uint32_t v, int k) {
  uint32_t m;
  do {
    m = __reduce_max_sync(0xffffffffu, v);
    const bool top = v == m;
    k -= __popc(__ballot_sync(0xffffffffu, top));
    if (top) v = 0u;
  } while (k > 0 && m != 0u);
  return m;
}

constexpr int EV_FEW = 32;      // tokens to drop, up to which they are looked for themselves
constexpr int EV_LIST = 128;    // places for candidates then
constexpr int EV_ROWS = 4;      // (sequence, head) pairs of a CTA, at most

struct EvShared {
  int warp[2][EV_THREADS / 32];
  int total[3];                // of this CTA: equal keys, free places, tokens to move
  int bad;
  uint32_t bin, need, equal;
  int later[EV_ROWS];          // what the few tokens' search left to the selection
  unsigned long long list[EV_ROWS][EV_LIST];
  int dropped[EV_ROWS][EV_FEW];
};

// exclusive scan of x over the CTA; the sum comes back in `all`
__device__ __forceinline__ int ev_scan(int x, int* warp_sums, int& all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();   // (the array is free)
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < EV_THREADS / 32; ++i) {
    const int s = warp_sums[i];
    if (i < w) before += s;
    all += s;
  }
  return before + v - x;
}

template <bool CLUSTER>
__device__ __forceinline__ void ev_sync() {
  if constexpr (CLUSTER) cluster_sync_all();
  else __syncthreads();
}

// what a (sequence, head) asks for
struct EvRow {
  int pair, b, h, n, K;
  const int32_t* table;
  int from;          // positions from here on stay
  bool ok, cut;      // the length is in range; there is something to drop
};
__device__ __forceinline__ EvRow ev_row(const PlanArgs& a, int pair) {
  EvRow r;
  r.pair = pair;
  r.b = pair / a.Hkv;
  r.h = pair - r.b * a.Hkv;
  r.n = a.lengths[r.b];
  r.K = a.budgets[r.b];
  r.table = a.table + static_cast<long long>(r.b) * a.W;
  r.from = static_cast<int>(max(static_cast<long long>(a.next[r.b]) - a.recent, static_cast<long long>(INT_MIN)));
  r.ok = r.n >= 0 && static_cast<long long>(r.n) <= static_cast<long long>(a.W) * a.P;
  r.cut = r.ok && r.K >= 0 && r.n > r.K;
  if (r.cut && min(r.K, r.n - r.K) > a.max_moves) r.ok = r.cut = false;
  return r;
}
__device__ __forceinline__ void ev_uncut(const PlanArgs& a, const EvRow& r, bool ok) {   // one thread
  a.counts[r.pair] = 0;
  if (r.h == 0) a.new_lengths[r.b] = ok ? r.n : -1;
}
__device__ __forceinline__ int ev_slot(const PlanArgs& a, const EvRow& r, int i) {
  const int e = i / a.P;
  return r.table[e] * a.P + (i - e * a.P);
}
__device__ __forceinline__ uint32_t ev_key(const PlanArgs& a, const EvRow& r, float w, int pos) {
  return pos < a.sinks || pos >= r.from ? 0xffffffffu : ev_ordered(w);
}

// A warp's run of blocks [k0, k1): their tokens' keys, bits turned by `flip`, to keys[]
// (tokens before `cap` of it; those behind the sequence's end count as kept), EV_AHEAD
// blocks under way at a time, the places of 32 blocks looked up by a lane each; true if
// a page is none.  worst: the complement of the thread's least key.
constexpr int EV_AHEAD = 8;
__device__ __forceinline__ bool ev_load(const PlanArgs& a, const EvRow& r, int k0, int k1, uint32_t flip, uint32_t* keys, int cap, uint32_t& worst) {
  const int lane = threadIdx.x & 31, per = a.P / Q4_BLOCK;
  bool bad = false;
  for (int c0 = k0; c0 < k1; c0 += 32) {
    uint32_t blk = 0u;   // of the chunk's lane-th block among the pool's
    bool none = false;
    if (c0 + lane < k1) {
      const int e = (c0 + lane) / per, page = r.table[e];
      none = page < 0 || page >= a.pages;
      blk = (static_cast<uint32_t>(page) * a.Hkv + r.h) * per + (c0 + lane - e * per);
    }
    if (__any_sync(0xffffffffu, none)) {
      bad = true;
      continue;
    }
    const int c1 = min(k1, c0 + 32);
    for (int k = c0; k < c1; k += EV_AHEAD) {
      float w[EV_AHEAD];
      int pos[EV_AHEAD];
#pragma unroll
      for (int u = 0; u < EV_AHEAD; ++u) {
        // (behind the end the last block again: loads without a branch between them)
        const unsigned long long at = static_cast<unsigned long long>(__shfl_sync(0xffffffffu, blk, min(k + u, c1 - 1) - c0)) * Q4_BLOCK + lane;
        w[u] = __ldg(a.weights + at);
        pos[u] = __ldg(a.positions + at);
      }
#pragma unroll
      for (int u = 0; u < EV_AHEAD; ++u) {
        const int i = (k + u) * Q4_BLOCK + lane;
        if (k + u < c1) {
          const uint32_t x = i >= r.n ? 0xffffffffu : ev_key(a, r, w[u], pos[u]);
          if (i - k0 * Q4_BLOCK < cap) keys[i - k0 * Q4_BLOCK] = x ^ flip;
          worst = max(worst, ~x);
        }
      }
    }
  }
  return bad;
}

// Few tokens to drop, as when a step's tokens push out as many: a warp looks for the
// least keys themselves, much as the largest logits of a row are found
// (token_logprobs.cuh): what the drop-th worst of its threads' worst reaches is listed,
// and the list is put in order.  False where that does not do (a list that runs over, of
// many equal keys).  (256 sequences of 8 heads that drop up to 6 of 2,054: the radix
// selection, with a CTA for each, takes 39 us; this with a CTA's eight warps 24.)
__device__ __forceinline__ bool ev_few(const PlanArgs& a, const EvRow& r, uint32_t* keys, unsigned long long* list, int* dropped) {
  const int lane = threadIdx.x & 31, drop = r.n - r.K;
  uint32_t worst = 0u;   // (of complements: the largest)
  const bool bad = ev_load(a, r, 0, (r.n + Q4_BLOCK - 1) / Q4_BLOCK, 0xffffffffu, keys, a.cap, worst);
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) ev_uncut(a, r, false);
    return true;
  }
  const uint32_t bound = warp_kth(worst, drop);
  if (bound == 0u) return false;
  __syncwarp();
  int m = 0;
  for (int i0 = 0; i0 < r.n; i0 += 128) {
    const uint4 x = *reinterpret_cast<const uint4*>(keys + i0 + 4 * lane);   // (there is room for 128 at a time)
    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 4 * lane + j;
      const uint32_t all = __ballot_sync(0xffffffffu, y[j] >= bound && i < r.n);
      if (all == 0u) continue;
      const int p = m + __popc(all & ((1u << lane) - 1u));
      if ((all >> lane & 1u) && p < EV_LIST) list[p] = (static_cast<unsigned long long>(y[j]) << 32) | static_cast<uint32_t>(i);
      m += __popc(all);
    }
  }
  if (m > EV_LIST) return false;
  __syncwarp();
  for (int i = lane; i < m; i += 32) {
    const unsigned long long x = list[i];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < m; ++j) before += list[j] > x;
    if (before < drop) dropped[before] = static_cast<int>(x & 0xffffffffu);   // (equal keys: the last place goes first)
  }
  __syncwarp();
  int32_t* moves = a.moves + 2 * static_cast<long long>(r.pair) * a.max_moves;
  const int t = lane < drop ? dropped[lane] : r.n;
  const uint32_t gone = __reduce_or_sync(0xffffffffu, t >= r.K && t < r.n ? 1u << (t - r.K) : 0u);   // of the places behind
  int before = 0;
  for (int j = 0; j < drop; ++j) before += __shfl_sync(0xffffffffu, t, j) < t;
  if (t < r.K) moves[2 * before + 1] = ev_slot(a, r, t);
  if (lane < drop && !(gone >> lane & 1u)) moves[2 * __popc(~gone & ((1u << lane) - 1u))] = ev_slot(a, r, r.K + lane);
  if (lane == 0) {
    a.counts[r.pair] = drop - __popc(gone);
    if (r.h == 0) a.new_lengths[r.b] = r.K;
  }
  return true;
}

// Any number of tokens to drop: the selection, by a CTA or a cluster.
template <bool CLUSTER>
__device__ __forceinline__ void ev_select(const PlanArgs& a, const EvRow& row, EvShared& sh, uint32_t* hist, uint32_t* keys) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = CLUSTER ? a.C : 1;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0u;
  const bool first = rank == 0 && tid == 0;
  const int n = row.n, K = row.K;
  const int32_t* table = row.table;

  // this CTA's tokens, and of them a warp's
  const int blocks = (n + Q4_BLOCK - 1) / Q4_BLOCK;
  const int blk0 = static_cast<int>(static_cast<long long>(blocks) * rank / C);
  const int blk1 = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / C);
  const int base = blk0 * Q4_BLOCK, mine = max(0, min(n, blk1 * Q4_BLOCK) - base);
  const int w0 = blk0 + (blk1 - blk0) * warp / (EV_THREADS / 32), w1 = blk0 + (blk1 - blk0) * (warp + 1) / (EV_THREADS / 32);
  uint32_t worst = 0u;
  bool bad = ev_load(a, row, w0, w1, 0u, keys + (w0 - blk0) * Q4_BLOCK, a.cap - (w0 - blk0) * Q4_BLOCK, worst);
  const bool here = mine <= a.cap;   // all keys are in shared memory
  auto slot_of = [&](int i) { return ev_slot(a, row, i); };
  auto key_at = [&](int i) {   // i: of this CTA's tokens
    if (i < a.cap) return keys[i];
    const int t = base + i, e = t / a.P;
    const long long at = (static_cast<long long>(table[e]) * a.Hkv + row.h) * a.P + (t - e * a.P);
    return ev_key(a, row, __ldg(a.weights + at), __ldg(a.positions + at));
  };
  bad = __syncthreads_or(bad);
  if constexpr (CLUSTER) {
    if (tid == 0) sh.bad = bad;
    cluster_sync_all();
    bad = __any_sync(0xffffffffu, lane < C && ld_peer_u32(&sh.bad, lane) != 0u);
  }
  if (bad) {
    if (first) ev_uncut(a, row, false);
    if constexpr (CLUSTER) cluster_sync_all();   // (its shared memory was read)
    return;
  }
  int32_t* moves = a.moves + 2 * static_cast<long long>(row.pair) * a.max_moves;

  // the K-th largest key
  uint32_t prefix = 0, need = static_cast<uint32_t>(K);
  uint32_t tau = K > 0 ? 0u : 0xffffffffu;   // what is above it stays (nothing, for a budget of 0),
  uint32_t take = 0;                         // and the first `take` of what equals it
  static_assert(EV_BINS == EV_THREADS, "a bin a thread");
  uint32_t* mine_hist = hist + warp * EV_BINS;
#pragma unroll 1
  for (int pass = K > 0 ? 0 : 4; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll
    for (int i = 0; i < EV_BINS / 32; ++i) mine_hist[32 * i + lane] = 0u;
    __syncwarp();
    auto count = [&](uint32_t k) {
      if (pass == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&mine_hist[(k >> shift) & 255u], 1u);
    };
    if (here) {
      for (int i = 4 * tid; i < mine; i += 4 * EV_THREADS) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        count(k.x);
        if (i + 1 < mine) count(k.y);
        if (i + 2 < mine) count(k.z);
        if (i + 3 < mine) count(k.w);
      }
    } else {
      for (int i = tid; i < mine; i += EV_THREADS) count(key_at(i));
    }
    __syncthreads();
    // thread t has the bin 255 - t: of the warps, then of the cluster
    const int bin = EV_BINS - 1 - tid;
    uint32_t c = 0u;
#pragma unroll
    for (int i = 0; i < EV_THREADS / 32; ++i) c += hist[i * EV_BINS + bin];
    if constexpr (CLUSTER) {
      uint32_t* sums = hist + (EV_THREADS / 32 + (pass & 1)) * EV_BINS;   // (two, as the next pass's come before the last one's are read)
      sums[bin] = c;
      cluster_sync_all();
      uint32_t x[EV_CLUSTER];
#pragma unroll
      for (int r = 0; r < EV_CLUSTER; ++r) x[r] = ld_peer_u32(sums + bin, r < C ? r : 0);   // (all under way before the first sum)
      c = 0u;
#pragma unroll
      for (int r = 0; r < EV_CLUSTER; ++r) c += r < C ? x[r] : 0u;
    }
    int all;
    const uint32_t above = static_cast<uint32_t>(ev_scan(static_cast<int>(c), sh.warp[0], all));
    if (above < need && need <= above + c) {
      sh.bin = static_cast<uint32_t>(bin);
      sh.need = need - above;
      sh.equal = c;
    }
    __syncthreads();
    prefix = (prefix << 8) | sh.bin;
    need = sh.need;
    const uint32_t equal = sh.equal;
    if (equal == need) {   // all that share these bits stay (some token does not, so they are not zero)
      tau = (prefix << shift) - 1u;
      break;
    }
    if (pass == 3) {
      tau = prefix;
      take = need;
    }
  }

  // Consecutive tokens a thread, an odd number of fours, so that the threads' vectors lie in
  // different banks: equal keys are counted first, then free places and tokens to move.
  const int per = 4 * (((mine + 4 * EV_THREADS - 1) / (4 * EV_THREADS)) | 1);
  const int i0 = min(mine, tid * per), i1 = min(mine, i0 + per);
  auto each = [&](auto&& f) {   // f(token, key)
    if (here) {
      for (int i = i0; i < i1; i += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        f(i, k.x);
        if (i + 1 < i1) f(i + 1, k.y);
        if (i + 2 < i1) f(i + 2, k.z);
        if (i + 3 < i1) f(i + 3, k.w);
      }
    } else {
      for (int i = i0; i < i1; ++i) f(i, key_at(i));
    }
  };
  int equal_before = 0, all = 0;
  if (take > 0) {
    int x = 0;
    each([&](int, uint32_t k) { x += k == tau; });
    equal_before = ev_scan(x, sh.warp[1], all);
    if constexpr (CLUSTER) {
      if (tid == 0) sh.total[0] = all;
      cluster_sync_all();
      equal_before += __reduce_add_sync(0xffffffffu, lane < static_cast<int>(rank) ? static_cast<int>(ld_peer_u32(&sh.total[0], lane)) : 0);
    }
  }
  int holes = 0, movers = 0, e = equal_before;
  each([&](int i, uint32_t k) {
    const bool kept = k > tau || (k == tau && e++ < static_cast<int>(take));
    if (base + i < K) holes += !kept;
    else movers += kept;
  });
  int all_holes, all_movers;
  int hole = ev_scan(holes, sh.warp[0], all_holes), mover = ev_scan(movers, sh.warp[1], all_movers);
  if constexpr (CLUSTER) {
    if (tid == 0) {
      sh.total[1] = all_holes;
      sh.total[2] = all_movers;
    }
    cluster_sync_all();
    const int x = lane < C ? static_cast<int>(ld_peer_u32(&sh.total[1], lane)) : 0, y = lane < C ? static_cast<int>(ld_peer_u32(&sh.total[2], lane)) : 0;
    hole += __reduce_add_sync(0xffffffffu, lane < static_cast<int>(rank) ? x : 0);
    mover += __reduce_add_sync(0xffffffffu, lane < static_cast<int>(rank) ? y : 0);
    all_holes = __reduce_add_sync(0xffffffffu, x);
  }
  if (holes + movers > 0) {
    e = equal_before;
    each([&](int i, uint32_t k) {
      const bool kept = k > tau || (k == tau && e++ < static_cast<int>(take));
      if (kept == (base + i < K)) return;
      int32_t* at = moves + (kept ? 2 * mover++ : 2 * hole++ + 1);
      *at = slot_of(base + i);
    });
  }
  if (first) {
    a.counts[row.pair] = all_holes;
    if (row.h == 0) a.new_lengths[row.b] = K;
  }
  ev_sync<CLUSTER>();   // (nobody ends, or goes on, while shared memory is read)
}

// CLUSTER: a cluster a pair.  Else a CTA has `rows` pairs: a warp for each looks for few
// tokens to drop, and the CTA takes the others one after the other.
template <bool CLUSTER>
__global__ void __launch_bounds__(EV_THREADS, 4) evict_plan_kernel(const PlanArgs a) {
  extern __shared__ uint4 ev_dynamic[];
  __shared__ EvShared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(ev_dynamic);   // the warps', and two of the CTA
  uint32_t* keys = hist + EV_HISTS * EV_BINS;                 // [rows][cap]
  if constexpr (CLUSTER) {
    const EvRow row = ev_row(a, blockIdx.x / a.C);
    if (!row.cut) {   // (the same for all CTAs of a sequence)
      if (cluster_rank() == 0 && threadIdx.x == 0) ev_uncut(a, row, row.ok);
      return;
    }
    ev_select<true>(a, row, sh, hist, keys);
  } else {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pair = blockIdx.x * a.rows + warp;
    if (warp < a.rows) {
      bool later = false;
      if (pair < a.B * a.Hkv) {
        const EvRow row = ev_row(a, pair);
        if (!row.cut) {
          if (lane == 0) ev_uncut(a, row, row.ok);
        } else {
          later = row.n - row.K > EV_FEW || row.n > a.cap;
          if (!later) later = !ev_few(a, row, keys + warp * a.cap, sh.list[warp], sh.dropped[warp]);
        }
      }
      if (lane == 0) sh.later[warp] = later;
    }
    __syncthreads();
    for (int r = 0; r < a.rows; ++r)
      if (sh.later[r]) ev_select<false>(a, ev_row(a, blockIdx.x * a.rows + r), sh, hist, keys);
  }
}

// ---------------------------------------------------------------------------
// The moves.  A warp takes 32: a lane looks up where one of them goes, then sixteen lanes
// carry one, its codes in 16-byte pieces, its two groups of scales, its weight and its
// position, MV_AHEAD of them under way at a time.  No place that a plan names is source
// and destination, so there is no order.  Bound: the bus, by sectors of 32 bytes, of
// which the scales, the weight and the position fill an eighth or a quarter: 256 bytes
// read and 256 written for a move of 152 (D = 128).  (With the places' divisions done by
// all lanes of a move, they were two thirds of 40 us for 64 heads of about 3,500 moves.)
// ---------------------------------------------------------------------------
constexpr int MV_THREADS = 256;
constexpr int MV_AHEAD = 4;

struct MoveArgs {
  unsigned char* cache;       // [pages, Hkv, P / 32, 36 D]
  float* weights;             // [pages, Hkv, P] or null
  int32_t* positions;         // [pages, Hkv, P] or null
  const int32_t* moves;       // [B, Hkv, max_moves, 2]
  const int32_t* counts;      // [B, Hkv]
  int Hkv, P, pages, max_moves;
};

template <int D>
__global__ void __launch_bounds__(MV_THREADS) kv_move_q4_kernel(const MoveArgs a) {
  constexpr int PIECES = D / 32;   // of a token's key or value codes
  const int pair = blockIdx.x, h = pair % a.Hkv, lane = threadIdx.x & 31, l = lane & 15;
  const uint32_t count = max(0, min(a.counts[pair], a.max_moves));   // (a step of the loop below may pass 31 bits)
  const int per = a.P / Q4_BLOCK;
  const long long slots = static_cast<long long>(a.pages) * a.P;
  const int2* moves = reinterpret_cast<const int2*>(a.moves) + static_cast<long long>(pair) * a.max_moves;
  // what the lane carries: its bytes, and where they are: in a block, or in the weights or positions
  int bytes = 0, at = 0, each = 0;
  unsigned char* base = a.cache;
  unsigned long long block = q4_block_bytes(D);
  if (l < 2 * PIECES) {
    bytes = 16;
    at = (l / PIECES) * (Q4_BLOCK * D / 2) + (l % PIECES) * 16;
    each = D / 2;
  } else if (l == 8 || l == 9) {
    bytes = D / 16;
    at = Q4_BLOCK * D + (l - 8) * (Q4_BLOCK * D / 16);
    each = D / 16;
  } else if (l == 10 || l == 11) {
    base = l == 10 ? reinterpret_cast<unsigned char*>(a.weights) : reinterpret_cast<unsigned char*>(a.positions);
    bytes = base ? 4 : 0;
    block = 4 * Q4_BLOCK;
    each = 4;
  }
  for (uint32_t i0 = 32 * (blockIdx.y * (MV_THREADS / 32) + (threadIdx.x >> 5)); i0 < count; i0 += 32 * gridDim.y * (MV_THREADS / 32)) {
    // the lane's move: numbers of the blocks among the pool's, rows in them; ~0: none
    uint32_t from = ~0u, to = 0u, rows = 0u;
    if (i0 + lane < count) {
      const int2 m = __ldg(moves + i0 + lane);
      if (m.x >= 0 && m.y >= 0 && m.x < slots && m.y < slots) {
        const int b0 = m.x / Q4_BLOCK, p0 = b0 / per, b1 = m.y / Q4_BLOCK, p1 = b1 / per;
        from = (static_cast<uint32_t>(p0) * a.Hkv + h) * per + (b0 - p0 * per);
        to = (static_cast<uint32_t>(p1) * a.Hkv + h) * per + (b1 - p1 * per);
        rows = (m.x % Q4_BLOCK) | (m.y % Q4_BLOCK) << 8;
      }
    }
    const int n = min(32u, count - i0);
    for (int j0 = 0; j0 < n; j0 += 2 * MV_AHEAD) {
      uint4 x[MV_AHEAD];
      unsigned char* dst[MV_AHEAD];
#pragma unroll
      for (int u = 0; u < MV_AHEAD; ++u) {
        const int j = j0 + 2 * u + (lane >> 4);
        const uint32_t b0 = __shfl_sync(0xffffffffu, from, j), b1 = __shfl_sync(0xffffffffu, to, j), r = __shfl_sync(0xffffffffu, rows, j);
        const bool go = b0 != ~0u && bytes;
        const unsigned char* src = base + b0 * block + at + (r & 255u) * each;
        dst[u] = go ? base + b1 * block + at + (r >> 8) * each : nullptr;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (go) {
          if (bytes == 16) x[u] = *reinterpret_cast<const uint4*>(src);
          else if (bytes == 8) *reinterpret_cast<uint2*>(&x[u]) = *reinterpret_cast<const uint2*>(src);
          else x[u].x = *reinterpret_cast<const uint32_t*>(src);
        }
      }
#pragma unroll
      for (int u = 0; u < MV_AHEAD; ++u) {
        if (!dst[u]) continue;
        if (bytes == 16) *reinterpret_cast<uint4*>(dst[u]) = x[u];
        else if (bytes == 8) *reinterpret_cast<uint2*>(dst[u]) = make_uint2(x[u].x, x[u].y);
        else *reinterpret_cast<uint32_t*>(dst[u]) = x[u].x;
      }
    }
  }
}

}  // namespace sv
