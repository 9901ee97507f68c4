// page_trim.cuh -- pages that sequences no longer need go back to a paged cache's ring
// of free page ids: of the held[b] pages of sequence b, those behind the first
// ceil(tokens[b] / P), in sequence order.
//
// Built like the page map (page_map.cuh): one launch, every CTA scans the requests
// itself, 512 sequences a pass, and the pages given back are dealt to the CTAs by their
// number.  What bounds it: the launch, and 8 bytes a page that is given back.
#pragma once

#include "page_map.cuh"

namespace sv {

struct PageTrimArgs {
  const int32_t* tokens;      // [B]
  const int32_t* held;        // [B]
  int32_t* ring;              // [F] free page ids, circular
  const int32_t* ring_state;  // [2] head, available
  const int32_t* table;       // [B, W]
  int B, F, P, W;
  int32_t* new_held;          // [B]
  int32_t* new_ring_state;    // [2]
  int32_t* status;            // [B]
};

__global__ void __launch_bounds__(PM_THREADS) page_trim_kernel(const PageTrimArgs a) {
  __shared__ long long warp_sums[PM_THREADS / 32], put_end[PM_THREADS];
  __shared__ int s_need[PM_THREADS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = a.ring_state[0], avail = a.ring_state[1];
  const bool ring_ok = head >= 0 && head < a.F && avail >= 0 && avail <= a.F;
  const long long room = ring_ok ? a.F - avail : 0;
  const long long item0 = static_cast<long long>(blockIdx.x) * PM_THREADS + threadIdx.x;
  const long long item_step = static_cast<long long>(gridDim.x) * PM_THREADS;
  long long base = 0, granted = 0;   // pages of the passes so far: to be given back, given back
  for (int b0 = 0; b0 < a.B; b0 += PM_THREADS) {
    const int b = b0 + threadIdx.x, nb = min(PM_THREADS, a.B - b0);
    int tokens = 0, held = 0;
    if (b < a.B) {
      tokens = a.tokens[b];
      held = a.held[b];
    }
    const bool ok = ring_ok && tokens >= 0 && held >= 0 && held <= a.W;
    const int need = static_cast<int>((static_cast<long long>(tokens) + a.P - 1) / a.P);
    const long long put = b < a.B && ok ? max(0, held - need) : 0;
    long long v = put;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int i = 0; i < PM_THREADS / 32; ++i) {
      const long long s = warp_sums[i];
      if (i < warp) v += s;
      all += s;
    }
    const int st = !ok ? -1 : put > 0 && base + v > room ? -3 : 0;
    put_end[threadIdx.x] = base + v;
    s_need[threadIdx.x] = st == 0 ? need : -1;
    if (blockIdx.x == 0) {
      granted += st == 0 ? put : 0;
      if (b < a.B) {
        a.status[b] = st;
        a.new_held[b] = st == 0 ? min(held, need) : held;
      }
    }
    __syncthreads();
    // (once a sequence's pages find no room, nobody's behind it do)
    for (long long i = item0; i < min(all, room - base); i += item_step) {
      const int k = pm_find(put_end, nb, base + i);
      if (s_need[k] < 0) continue;
      const long long first = k ? put_end[k - 1] : base;
      a.ring[(head + static_cast<long long>(avail) + base + i) % a.F] =
          a.table[static_cast<long long>(b0 + k) * a.W + s_need[k] + (base + i - first)];
    }
    base += all;
    __syncthreads();   // the shared arrays are reused by the next pass
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) granted += __shfl_xor_sync(0xffffffffu, granted, o);
    if (lane == 0) warp_sums[warp] = granted;
    __syncthreads();
    if (threadIdx.x == 0) {
      long long sum = 0;
      for (int i = 0; i < PM_THREADS / 32; ++i) sum += warp_sums[i];
      a.new_ring_state[0] = head;
      a.new_ring_state[1] = static_cast<int32_t>(avail + sum);
    }
  }
}

}  // namespace sv
