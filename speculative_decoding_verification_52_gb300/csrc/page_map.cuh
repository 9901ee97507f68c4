// page_map.cuh -- block tables and slot maps of a paged cache, built on the GPU
// from the requests' lengths.
//
// Sequence b holds held[b] pages (its row of the block table), has lengths[b]
// tokens in the cache and asks for places for count[b] more:
//   need = ceil((lengths + count) / P),  take = max(0, need - held),
// and the pages come from a ring of free page ids, in sequence order; a
// negative count gives the sequence's pages back to the ring's end.  Token j of
// the request goes to slot table[b, pos / P] * P + pos % P, pos = lengths[b] + j.
//
// What bounds it: 8 bytes written per token (slot and position) against a few
// bytes per sequence, and for one decoding step the launch itself.  So there is
// one launch and no hand-over between CTAs: every CTA scans the (small) request
// arrays itself, 512 sequences a pass, and keeps only the pass at hand in
// shared memory; a CTA owns a tile of 2048 tokens of the packed map, and the
// pages to hand out or take back are dealt to the CTAs by their number.  The
// scan's results never meet through memory: pages taken are read from
// [head, head + available) of the ring, pages given back are written behind it
// (the two cannot overlap: a release that does not fit is refused), and the
// state that a call reads is never the state that it writes.
#pragma once

#include "common.cuh"

namespace sv {

constexpr int PM_THREADS = 512;
constexpr int PM_TILE = 4 * PM_THREADS;   // tokens of the packed map per CTA: four a thread

struct PageMapArgs {
  const int32_t* lengths;     // [B]
  const int32_t* count;       // [B]
  const int32_t* held;        // [B]
  int32_t* ring;              // [F] free page ids, circular
  const int32_t* ring_state;  // [2] head, available
  int32_t* table;             // [B, W]
  int B, F, P, W, T;
  int32_t* offsets;           // [B + 1]
  int32_t* slots;             // [T]
  int32_t* positions;         // [T]
  int32_t* new_held;          // [B]
  int32_t* new_ring_state;    // [2]
  int32_t* status;            // [B]
  bool vec;                   // 16-byte stores of slots and positions
};

struct Sum3 {
  long long n, take, put;
};

__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return {a.n + b.n, a.take + b.take, a.put + b.put};
}

// inclusive scan over the CTA; the CTA's sum comes back in `all`
__device__ __forceinline__ Sum3 pm_scan(Sum3 v, Sum3* warp_sums, Sum3& all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum3 u = {__shfl_up_sync(0xffffffffu, v.n, o), __shfl_up_sync(0xffffffffu, v.take, o),
                    __shfl_up_sync(0xffffffffu, v.put, o)};
    if (lane >= o) v = v + u;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  Sum3 before = {0, 0, 0};
  all = before;
#pragma unroll
  for (int i = 0; i < PM_THREADS / 32; ++i) {
    const Sum3 s = warp_sums[i];
    if (i < w) before = before + s;
    all = all + s;
  }
  return v + before;
}

// first index whose end lies past x (ends[] does not decrease)
__device__ __forceinline__ int pm_find(const long long* ends, int n, long long x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PM_THREADS) page_map_kernel(const PageMapArgs a) {
  __shared__ Sum3 warp_sums[PM_THREADS / 32];
  __shared__ long long tok_end[PM_THREADS], take_end[PM_THREADS], put_end[PM_THREADS];
  __shared__ int s_len[PM_THREADS], s_held[PM_THREADS], s_count[PM_THREADS];
  __shared__ signed char s_status[PM_THREADS];

  const int head = a.ring_state[0], avail = a.ring_state[1];
  const bool ring_ok = head >= 0 && head < a.F && avail >= 0 && avail <= a.F;
  const long long t0 = static_cast<long long>(blockIdx.x) * PM_TILE;
  const long long t1 = min(t0 + PM_TILE, static_cast<long long>(a.T));
  const long long item0 = static_cast<long long>(blockIdx.x) * PM_THREADS + threadIdx.x;
  const long long item_step = static_cast<long long>(gridDim.x) * PM_THREADS;
  Sum3 base = {0, 0, 0};      // of the passes so far: places, demanded pages, released pages
  long long granted_take = 0, granted_put = 0;

  for (int b0 = 0; b0 < a.B; b0 += PM_THREADS) {
    const int b = b0 + threadIdx.x, nb = min(PM_THREADS, a.B - b0);
    int len = 0, n = 0, held = 0;
    if (b < a.B) {
      len = a.lengths[b];
      n = a.count[b];
      held = a.held[b];
    }
    const long long last = static_cast<long long>(len) + n;
    bool ok = ring_ok && len >= 0 && held >= 0 && held <= a.W && (n < 0 || last <= static_cast<long long>(a.W) * a.P);
    // the places a request takes in the map do not depend on whether it is granted
    Sum3 v = {b < a.B && n > 0 ? n : 0, 0, 0}, all;
    {
      // whether the places fit decides what is demanded, so the places are scanned first
      const Sum3 s = pm_scan(v, warp_sums, all);
      ok = ok && (n < 0 || base.n + s.n <= a.T);
      __syncthreads();
      v = {v.n, 0, 0};
      if (b < a.B && ok) {
        if (n < 0) v.put = held;
        else v.take = max(0LL, (last + a.P - 1) / a.P - held);
      }
    }
    const Sum3 s = pm_scan(v, warp_sums, all);
    int st = 0;
    if (!ok) st = -1;
    else if ((v.take > 0 && base.take + s.take > avail) || (v.put > 0 && avail + base.put + s.put > a.F)) st = -3;
    tok_end[threadIdx.x] = base.n + s.n;
    take_end[threadIdx.x] = base.take + s.take;
    put_end[threadIdx.x] = base.put + s.put;
    s_len[threadIdx.x] = len;
    s_held[threadIdx.x] = held;
    s_count[threadIdx.x] = n;
    s_status[threadIdx.x] = static_cast<signed char>(st);
    if (st == 0) {
      granted_take += v.take;
      granted_put += v.put;
    }
    if (blockIdx.x == 0 && b < a.B) {
      a.status[b] = st;
      a.new_held[b] = st != 0 ? held : n < 0 ? 0 : held + static_cast<int>(v.take);
      a.offsets[b + 1] = static_cast<int32_t>(min(base.n + s.n, static_cast<long long>(a.T)));
    }
    __syncthreads();

    // pages handed out: entries held .. held + take - 1 of the sequence's row.
    // (demands past what is available are not visited: the granted ones come first)
    for (long long i = item0; i < min(all.take, avail - base.take); i += item_step) {
      const int k = pm_find(take_end, nb, base.take + i);
      if (s_status[k] != 0) continue;
      const long long first = k ? take_end[k - 1] : base.take;
      const long long e = s_held[k] + (base.take + i - first);
      a.table[static_cast<long long>(b0 + k) * a.W + e] = a.ring[(head + base.take + i) % a.F];
    }
    // pages given back, behind the ring's free ones
    for (long long i = item0; i < min(all.put, a.F - avail - base.put); i += item_step) {
      const int k = pm_find(put_end, nb, base.put + i);
      if (s_status[k] != 0) continue;
      const long long first = k ? put_end[k - 1] : base.put;
      a.ring[(head + static_cast<long long>(avail) + base.put + i) % a.F] =
          a.table[static_cast<long long>(b0 + k) * a.W + (base.put + i - first)];
    }
    // the part of this CTA's tile that belongs to the pass
    const long long p1 = base.n + all.n;
    if (p1 > t0 && base.n < t1) {
      const long long t = t0 + 4 * static_cast<long long>(threadIdx.x);
      int k = -1;
      int slot[4], pos_of[4];
      bool mine[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const long long x = t + u;
        mine[u] = x >= base.n && x < p1 && x < t1;
        slot[u] = pos_of[u] = -1;
        if (!mine[u]) continue;
        if (k < 0) k = pm_find(tok_end, nb, x);
        while (tok_end[k] <= x) ++k;   // ends: x < p1 = the last end
        if (s_status[k] != 0) continue;
        const long long pos = s_len[k] + (x - (tok_end[k] - s_count[k]));
        const long long e = pos / a.P;
        const int page = e < s_held[k]
                             ? a.table[static_cast<long long>(b0 + k) * a.W + e]
                             : a.ring[(head + (k ? take_end[k - 1] : base.take) + (e - s_held[k])) % a.F];
        pos_of[u] = static_cast<int>(pos);
        if (page >= 0 && page < a.F) slot[u] = page * a.P + static_cast<int>(pos - e * a.P);
      }
      if (a.vec && mine[0] && mine[3]) {
        *reinterpret_cast<int4*>(a.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos_of[0], pos_of[1], pos_of[2], pos_of[3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (mine[u]) {
            a.slots[t + u] = slot[u];
            a.positions[t + u] = pos_of[u];
          }
      }
    }
    base = base + all;
    __syncthreads();   // the shared arrays are reused by the next pass
  }

  // places that no request took
  for (long long x = max(t0, base.n) + threadIdx.x; x < t1; x += PM_THREADS) {
    a.slots[x] = -1;
    a.positions[x] = -1;
  }
  if (blockIdx.x == 0) {
    const Sum3 s = {0, granted_take, granted_put};
    Sum3 all;
    pm_scan(s, warp_sums, all);
    if (threadIdx.x == 0) {
      a.offsets[0] = 0;
      if (ring_ok) {
        a.new_ring_state[0] = static_cast<int32_t>((head + all.take) % a.F);
        a.new_ring_state[1] = static_cast<int32_t>(avail - all.take + all.put);
      } else {
        a.new_ring_state[0] = head;
        a.new_ring_state[1] = avail;
      }
    }
  }
}

}  // namespace sv
