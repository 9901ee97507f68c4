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
// A cluster of 1 to 8 CTAs takes a (sequence, head), each a contiguous part of its
// tokens.  The K-th largest key comes from a radix selection, 11 + 11 + 10 bits, over
// keys that stay in shared memory (those beyond its size are read again): a histogram
// a pass, added up over the cluster.  Most selections end early, in a pass whose last
// bin is needed whole.
//
// Bound: 8 bytes a token read (weight and position); in the steady state the passes'
// barriers, of which there are enough CTAs an SM to cover.
#pragma once

#include "common.cuh"
#include "kv_q4.cuh"

namespace sv {

constexpr int EV_THREADS = 256;
constexpr int EV_BINS = 2048;
constexpr int EV_CAP = 8192;    // keys of a CTA in shared memory, at most

struct PlanArgs {
  const float* weights;       // [pages, Hkv, P]
  const int32_t* positions;   // [pages, Hkv, P]
  const int32_t* table;       // [B, W]
  const int32_t* lengths;     // [B]
  const int32_t* budgets;     // [B]
  const int32_t* next;        // [B]
  int B, Hkv, P, pages, W, max_moves, sinks, recent;
  int cap;                    // keys of a CTA in shared memory
  int C;                      // CTAs of a cluster
  int32_t* moves;             // [B, Hkv, max_moves, 2]
  int32_t* counts;            // [B, Hkv]
  int32_t* new_lengths;       // [B]
};

// integers that compare as the weights do; NaN below everything
__device__ __forceinline__ uint32_t ev_ordered(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);   // (-0 becomes 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct EvShared {
  int warp[2][EV_THREADS / 32];
  int total[3];                // of this CTA: equal keys, free places, tokens to move
  int bad;
  uint32_t bin, need, equal;
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

template <bool CLUSTER>
__global__ void __launch_bounds__(EV_THREADS) evict_plan_kernel(const PlanArgs a) {
  extern __shared__ uint4 ev_dynamic[];
  __shared__ EvShared sh;
  uint32_t* hist0 = reinterpret_cast<uint32_t*>(ev_dynamic);   // [CLUSTER ? 2 : 1][EV_BINS]
  uint32_t* keys = hist0 + (CLUSTER ? 2 : 1) * EV_BINS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = CLUSTER ? a.C : 1;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0u;
  const int pair = blockIdx.x / C, b = pair / a.Hkv, h = pair - b * a.Hkv;
  const bool first = rank == 0 && tid == 0;
  const int n = a.lengths[b], budget = a.budgets[b];
  // (the same for all CTAs of a sequence)
  if (n < 0 || static_cast<long long>(n) > static_cast<long long>(a.W) * a.P || budget < 0 || n <= budget ||
      min(budget, n - budget) > a.max_moves) {
    if (first) {
      const bool ok = n >= 0 && static_cast<long long>(n) <= static_cast<long long>(a.W) * a.P && (budget < 0 || n <= budget);
      a.counts[pair] = 0;
      if (h == 0) a.new_lengths[b] = ok ? n : -1;
    }
    return;
  }
  const int32_t* table = a.table + static_cast<long long>(b) * a.W;
  const long long from = static_cast<long long>(a.next[b]) - a.recent;   // positions from here on stay

  // this CTA's tokens
  const int blocks = (n + Q4_BLOCK - 1) / Q4_BLOCK;
  const int blk0 = static_cast<int>(static_cast<long long>(blocks) * rank / C);
  const int blk1 = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / C);
  const int base = blk0 * Q4_BLOCK, mine = max(0, min(n, blk1 * Q4_BLOCK) - base);

  auto key_of = [&](long long at) {
    const int pos = __ldg(a.positions + at);
    const float w = __ldg(a.weights + at);
    return pos < a.sinks || pos >= from ? 0xffffffffu : ev_ordered(w);
  };
  // keys into shared memory, a block a warp, four at a time; pages that are none are noted
  bool bad = false;
  for (int k0 = blk0 + warp; k0 < blk1; k0 += 4 * (EV_THREADS / 32)) {
    int page[4], in[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = (k0 + u * (EV_THREADS / 32)) * Q4_BLOCK;
      page[u] = 0;
      if (t < n && k0 + u * (EV_THREADS / 32) < blk1) {
        const int e = t / a.P;
        in[u] = t - e * a.P;
        page[u] = table[e];
      }
    }
    float w[4];
    int pos[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * (EV_THREADS / 32), i = k * Q4_BLOCK + lane - base;
      if (k >= blk1) break;
      if (page[u] < 0 || page[u] >= a.pages) {
        bad = true;
      } else if (i < mine && i < a.cap) {
        const long long at = (static_cast<long long>(page[u]) * a.Hkv + h) * a.P + in[u] + lane;
        w[u] = __ldg(a.weights + at);
        pos[u] = __ldg(a.positions + at);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * (EV_THREADS / 32), i = k * Q4_BLOCK + lane - base;
      if (k >= blk1) break;
      if (page[u] >= 0 && page[u] < a.pages && i < mine && i < a.cap)
        keys[i] = pos[u] < a.sinks || pos[u] >= from ? 0xffffffffu : ev_ordered(w[u]);
    }
  }
  auto slot_of = [&](int i) {
    const int e = i / a.P;
    return table[e] * a.P + (i - e * a.P);
  };
  auto key_at = [&](int i) {   // i: of this CTA's tokens
    if (i < a.cap) return keys[i];
    const int t = base + i, e = t / a.P;
    return key_of((static_cast<long long>(table[e]) * a.Hkv + h) * a.P + (t - e * a.P));
  };
  bad = __syncthreads_or(bad);
  if constexpr (CLUSTER) {
    if (tid == 0) sh.bad = bad;
    cluster_sync_all();
    for (int r = 0; r < C; ++r) bad |= ld_peer_u32(&sh.bad, r) != 0u;
  }
  if (bad) {
    if (first) {
      a.counts[pair] = 0;
      if (h == 0) a.new_lengths[b] = -1;
    }
    if constexpr (CLUSTER) cluster_sync_all();   // (its shared memory was read)
    return;
  }

  // the K-th largest key
  const int K = budget;
  uint32_t prefix = 0, need = static_cast<uint32_t>(K);
  uint32_t tau = K > 0 ? 0u : 0xffffffffu;   // what is above it stays (nothing, for a budget of 0),
  uint32_t take = 0;                         // and the first `take` of what equals it
#pragma unroll 1
  for (int pass = K > 0 ? 0 : 3; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* hist = hist0 + (CLUSTER && (pass & 1) ? EV_BINS : 0);
    for (int i = tid; i < EV_BINS; i += EV_THREADS) hist[i] = 0u;
    __syncthreads();
    for (int i = tid; i < mine; i += EV_THREADS) {
      const uint32_t k = key_at(i);
      if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    ev_sync<CLUSTER>();
    // thread t has the eight bins below 2048 - 8 t
    constexpr int EACH = EV_BINS / EV_THREADS;
    static_assert(EACH == 8, "two vectors a thread");
    const int lo = EV_BINS - EACH * (tid + 1);
    uint32_t c[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) c[i] = 0u;
    for (int r = 0; r < C; ++r) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint4 x;
        if constexpr (CLUSTER) x = ld_peer_u128(hist + lo + 4 * v, r);
        else x = *reinterpret_cast<const uint4*>(hist + lo + 4 * v);
        c[4 * v] += x.x;
        c[4 * v + 1] += x.y;
        c[4 * v + 2] += x.z;
        c[4 * v + 3] += x.w;
      }
    }
    int sum = 0, all;
#pragma unroll
    for (int i = 0; i < EACH; ++i) sum += static_cast<int>(c[i]);
    uint32_t above = static_cast<uint32_t>(ev_scan(sum, sh.warp[0], all));
    if (above < need && need <= above + sum) {
      bool found = false;
#pragma unroll
      for (int i = EACH - 1; i >= 0; --i) {
        if (!found && need <= above + c[i]) {
          found = true;
          sh.bin = static_cast<uint32_t>(lo + i);
          sh.need = need - above;
          sh.equal = c[i];
        }
        if (!found) above += c[i];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | sh.bin;
    need = sh.need;
    const uint32_t equal = sh.equal;
    if (equal == need) {   // all that share these bits stay (some token does not, so they are not zero)
      tau = (prefix << shift) - 1u;
      break;
    }
    if (pass == 2) {
      tau = prefix;
      take = need;
    }
  }

  // Consecutive tokens a thread (an odd number, which lie in different banks): equal
  // keys are counted first, then free places and tokens to move.
  const int per = ((mine + EV_THREADS - 1) / EV_THREADS) | 1;
  const int i0 = min(mine, tid * per), i1 = min(mine, i0 + per);
  int equal_before = 0, all = 0;
  if (take > 0) {
    int x = 0;
    for (int i = i0; i < i1; ++i) x += key_at(i) == tau;
    equal_before = ev_scan(x, sh.warp[1], all);
    if constexpr (CLUSTER) {
      if (tid == 0) sh.total[0] = all;
      cluster_sync_all();
      for (uint32_t r = 0; r < rank; ++r) equal_before += static_cast<int>(ld_peer_u32(&sh.total[0], r));
    }
  }
  int holes = 0, movers = 0, e = equal_before;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    const bool kept = k > tau || (k == tau && e++ < static_cast<int>(take));
    if (base + i < K) holes += !kept;
    else movers += kept;
  }
  int all_holes, all_movers;
  int hole = ev_scan(holes, sh.warp[0], all_holes), mover = ev_scan(movers, sh.warp[1], all_movers);
  if constexpr (CLUSTER) {
    if (tid == 0) {
      sh.total[1] = all_holes;
      sh.total[2] = all_movers;
    }
    cluster_sync_all();
    all_holes = 0;
    for (uint32_t r = 0; r < static_cast<uint32_t>(C); ++r) {
      const int x = static_cast<int>(ld_peer_u32(&sh.total[1], r)), y = static_cast<int>(ld_peer_u32(&sh.total[2], r));
      if (r < rank) {
        hole += x;
        mover += y;
      }
      all_holes += x;
    }
  }
  int32_t* moves = a.moves + 2 * static_cast<long long>(pair) * a.max_moves;
  if (holes + movers > 0) {
    e = equal_before;
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = key_at(i);
      const bool kept = k > tau || (k == tau && e++ < static_cast<int>(take));
      if (base + i < K) {
        if (!kept) moves[2 * hole++ + 1] = slot_of(base + i);
      } else if (kept) {
        moves[2 * mover++] = slot_of(base + i);
      }
    }
  }
  if (first) {
    a.counts[pair] = all_holes;
    if (h == 0) a.new_lengths[b] = K;
  }
  if constexpr (CLUSTER) cluster_sync_all();   // nobody ends while its shared memory is read
}

// ---------------------------------------------------------------------------
// The moves.  Sixteen lanes take one: its codes in 16-byte pieces, its two groups of
// scales, its weight and its position.  No place that a plan names is source and
// destination, so there is no order.  Bound: the bus, by sectors of 32 bytes, of which
// the scales, the weight and the position fill an eighth or a quarter: 256 bytes read
// and 256 written for a move of 152 (D = 128).
// ---------------------------------------------------------------------------
constexpr int MV_THREADS = 256;

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
  const int pair = blockIdx.x, h = pair % a.Hkv, l = threadIdx.x & 15;
  const int count = min(a.counts[pair], a.max_moves);
  const long long slots = static_cast<long long>(a.pages) * a.P;
  const int2* moves = reinterpret_cast<const int2*>(a.moves) + static_cast<long long>(pair) * a.max_moves;
  // what the lane carries: its bytes, and where they are in a block
  int bytes = 0, at = 0, each = 0;
  if (l < 2 * PIECES) {
    bytes = 16;
    at = (l / PIECES) * (Q4_BLOCK * D / 2) + (l % PIECES) * 16;
    each = D / 2;
  } else if (l == 8 || l == 9) {
    bytes = D / 16;
    at = Q4_BLOCK * D + (l - 8) * (Q4_BLOCK * D / 16);
    each = D / 16;
  }
  const bool weight = l == 10 && a.weights, position = l == 11 && a.positions;
  for (int i = blockIdx.y * (MV_THREADS / 16) + (threadIdx.x >> 4); i < count; i += gridDim.y * (MV_THREADS / 16)) {
    const int2 m = __ldg(moves + i);
    if (m.x < 0 || m.y < 0 || m.x >= slots || m.y >= slots) continue;
    const int p0 = m.x / a.P, t0 = m.x - p0 * a.P, p1 = m.y / a.P, t1 = m.y - p1 * a.P;
    if (bytes) {
      const unsigned char* src = q4_block(a.cache, p0, h, t0, a.Hkv, a.P, D) + at + (t0 % Q4_BLOCK) * each;
      unsigned char* dst = q4_block(a.cache, p1, h, t1, a.Hkv, a.P, D) + at + (t1 % Q4_BLOCK) * each;
      if (bytes == 16) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
      else if (bytes == 8) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
      else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
    } else if (weight || position) {
      const long long from = (static_cast<long long>(p0) * a.Hkv + h) * a.P + t0, to = (static_cast<long long>(p1) * a.Hkv + h) * a.P + t1;
      if (weight) a.weights[to] = a.weights[from];
      else a.positions[to] = a.positions[from];
    }
  }
}

}  // namespace sv
