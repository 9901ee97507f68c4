// token_logprobs.cuh -- log probabilities of the tokens a verification emitted, their
// ranks, the rows' entropies and their most probable tokens.
//
// A row's logits l at temperature T, z = l / T, m = max z, S = sum e^(z - m):
//   logprob(t) = z_t - m - log S,   entropy = log S - (sum e^(z - m) (z - m)) / S,
//   rank(t) = 1 + #{v: l_v > l_t, or l_v = l_t and v < t}.
// Everything comes from one pass over the row, in the log2 domain (c = log2(e) / T),
// with a running reference a thread; when it moves by d <= 0,
//   S' = 2^d S,  X' = 2^d (X + d S)   for X = sum 2^z z.
//
// The largest n.  A thread that has seen elements knows the largest of its own; in a
// team of `WARPS` warps, the ceil(n / WARPS)-th largest of a warp's 32, taken as the
// least over the warps, has n elements at or above it.  Only what reaches that bound
// goes into a list: a few dozen elements beside the first tile's, since the bound is
// taken anew after 1, 2, 4, ... tiles.  Equal elements are told apart by their index in
// the bound, too, so that a row of equal logits fills no list.  Where a list runs over all
// the same (a row whose logits rise to its end), the team searches the row once for each
// of its n largest.  Elements that the bound or the token's logit concerns are looked for
// by the vector's maximum, which the references need anyway.
//
// Bound: one read of the row; beside it about 5 instructions an element.
#pragma once

#include "common.cuh"
#include "evict.cuh"

namespace sv {

constexpr int LP_THREADS = 256;
constexpr int LP_MAX_TOP = 32;
constexpr float LP_FAR = 1.2676506002282294e30f;   // 2^100: logits of this size count as infinities

struct LogprobArgs {
  const unsigned char* logits;  // [B, R, V]
  const int32_t* tokens;        // [B, M]
  const int32_t* path;          // [B, W] or null
  int B, R, V, M, W, top;
  int C;                        // CTAs that share a row (a cluster)
  float c;                      // log2(e) / T
  float* logprobs;              // [B, M], each of the outputs or null
  float* entropy;               // [B, M]
  int32_t* ranks;               // [B, M]
  int32_t* top_tokens;          // [B, M, top]
  float* top_logprobs;          // [B, M, top]
};

// a logit with its place, so that a larger one is a better one: larger logit, then
// smaller index.  0: none.
__device__ __forceinline__ unsigned long long lp_key(float x, int i) {
  return (static_cast<unsigned long long>(ev_ordered(x)) << 32) | static_cast<uint32_t>(~i);
}
__device__ __forceinline__ float lp_value(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int lp_index(unsigned long long k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// A thread's part of a row.  Exponents are (l - m) c, which is 0 for m itself however
// large it is; l c - fl(m c), an instruction less, is off by what the product lost.
struct LpAcc {
  float m, s, x;       // reference (a logit), sum 2^z, sum 2^z z
  int at;              // index of m
  __device__ __forceinline__ void init() {
    m = -LP_FAR;
    s = x = 0.f;
    at = -1;
  }
  // to a reference of `to` (above the present one) at index i
  __device__ __forceinline__ void raise(float to, float c, int i) {
    if (s > 0.f) {
      const float d = __fmul_rn(__fsub_rn(m, to), c), f = ex2_approx(d);   // (d <= 0)
      x = f * __fmaf_rn(d, s, x);
      s *= f;
    }
    m = to;
    at = i;
  }
  __device__ __forceinline__ void merge(float m2, float s2, float x2, float c) {
    if (!(s2 > 0.f)) return;
    if (!(s > 0.f)) {
      m = m2, s = s2, x = x2;
      return;
    }
    if (m2 > m) {
      const float t0 = m, t1 = s, t2 = x;
      m = m2, s = s2, x = x2;
      m2 = t0, s2 = t1, x2 = t2;
    }
    const float d = __fmul_rn(__fsub_rn(m2, m), c), f = ex2_approx(d);
    x += f * __fmaf_rn(d, s2, x2);
    s += f * s2;
  }
};

template <class T>
__device__ __forceinline__ float lp_vec_max(const uint4& q);
template <>
__device__ __forceinline__ float lp_vec_max<BF16T>(const uint4& q) {
  const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(q.x, q.y), bf16x2_max_nan(q.z, q.w));
  return fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
template <>
__device__ __forceinline__ float lp_vec_max<F32T>(const uint4& q) {
  return fmax_nan(fmax_nan(__uint_as_float(q.x), __uint_as_float(q.y)), fmax_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
}
// elements not below -2^100 (a NaN stays one)
template <class T>
__device__ __forceinline__ uint4 lp_clamp(uint4 q);
template <>
__device__ __forceinline__ uint4 lp_clamp<BF16T>(uint4 q) {
  const uint32_t lo = 0xf180f180u;   // twice -2^100
  return make_uint4(bf16x2_max_nan(q.x, lo), bf16x2_max_nan(q.y, lo), bf16x2_max_nan(q.z, lo), bf16x2_max_nan(q.w, lo));
}
template <>
__device__ __forceinline__ uint4 lp_clamp<F32T>(uint4 q) {
  auto f = [](uint32_t u) { return __float_as_uint(fmax_nan(__uint_as_float(u), -LP_FAR)); };
  return make_uint4(f(q.x), f(q.y), f(q.z), f(q.w));
}
template <class T>
__device__ __forceinline__ uint4 lp_nothing() {
  const uint32_t x = T::esz == 2 ? 0xf180f180u : __float_as_uint(-LP_FAR);
  return make_uint4(x, x, x, x);
}
__device__ __forceinline__ uint4 lp_load(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// value of the k-th largest of the warp's lanes (k = 1..32), as an ordered integer
__device__ __forceinline__ uint32_t lp_kth(uint32_t v, int k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const uint32_t u = __shfl_xor_sync(0xffffffffu, v, d);
      const bool larger = ((lane & d) == 0) == ((lane & size) == 0);   // this lane keeps the larger one
      v = larger ? max(u, v) : min(u, v);
    }
  }
  return __shfl_sync(0xffffffffu, v, k - 1);
}

template <int WARPS>
struct LpShared {
  static constexpr int CAP = WARPS == 1 ? 256 : 2048;   // places of a team's list
  static constexpr int CAP2 = WARPS == 1 ? 1 : 256;     // of those that reach the last bound
  unsigned long long list[CAP], list2[CAP2];
  unsigned long long bound[2][WARPS];   // two, so that a warp that is a step ahead does not change what another reads
  unsigned long long top[LP_MAX_TOP];
  float m[WARPS], s[WARPS], x[WARPS];
  int ahead[WARPS], bad[WARPS];
  int count, count2;
};

template <int WARPS>
__device__ __forceinline__ void lp_sync() {
  if constexpr (WARPS == 1) __syncwarp();
  else __syncthreads();
}

// One team a row, or a part of it: the CTA (WARPS = 8), or a warp.
template <class T, int WARPS, bool TOP>
__global__ void __launch_bounds__(LP_THREADS, 4) token_logprobs_kernel(const LogprobArgs a) {
  using S = LpShared<WARPS>;
  constexpr int TEAM = 32 * WARPS, TEAMS = LP_THREADS / TEAM, U = 4, E = T::vpe;
  extern __shared__ uint4 lp_dynamic[];
  const int tid = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x, lane = threadIdx.x & 31, warp = tid >> 5;
  const int team = WARPS == 1 ? threadIdx.x >> 5 : 0;
  S& sh = reinterpret_cast<S*>(lp_dynamic)[team];
  const int C = WARPS == 1 ? 1 : a.C;
  const uint32_t part = C > 1 ? cluster_rank() : 0u;
  const long long place = static_cast<long long>(blockIdx.x) * TEAMS / C + team;
  if (place >= static_cast<long long>(a.B) * a.M) return;
  const int b = static_cast<int>(place / a.M), mth = static_cast<int>(place - static_cast<long long>(b) * a.M);
  const int token = a.tokens[place];
  int row = mth;
  if (a.path) row = mth == 0 ? 0 : a.path[static_cast<long long>(b) * a.W + mth - 1];
  const bool there = token >= 0, ok = there && token < a.V && row >= 0 && row < a.R;
  const int n = TOP ? a.top : 0;
  if (!ok) {   // (alike in the whole cluster)
    if (part == 0) {
      const float none = there ? __int_as_float(0x7fc00000) : 0.f;
      if (tid == 0) {
        a.logprobs[place] = none;
        if (a.entropy) a.entropy[place] = none;
        if (a.ranks) a.ranks[place] = there ? -1 : 0;
      }
      if (tid < n) {
        a.top_tokens[place * n + tid] = -1;
        a.top_logprobs[place * n + tid] = there ? none : kNegInf;
      }
    }
    return;
  }
  const unsigned char* base = a.logits + (static_cast<long long>(b) * a.R + row) * a.V * T::esz;
  // the row: elements before the first 16-byte border, vectors, and a rest
  const int head = min(a.V, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(base) & 15u)) & 15u) / T::esz);
  const int vectors = (a.V - head) / E, rest = a.V - head - vectors * E;
  const int v0 = static_cast<int>(static_cast<long long>(vectors) * part / C), v1 = static_cast<int>(static_cast<long long>(vectors) * (part + 1) / C);
  const uint4* body = reinterpret_cast<const uint4*>(base + head * T::esz);
  const float xt = fmax_nan(T::load(base, token), -LP_FAR);
  // (what equals the token's logit counts before it, not behind it)
  const float below = xt == 0.f ? -1.401298464e-45f : __uint_as_float(__float_as_uint(xt) + (xt > 0.f ? 0xffffffffu : 1u));

  if (tid == 0) sh.count = sh.count2 = 0;
  LpAcc acc;
  acc.init();
  int ahead = 0;       // elements before the token's in the order
  bool bad = false;
  // the odd elements, one a thread
  float odd = -LP_FAR;
  int odd_at = -1;
  if (part == 0 && tid < head + rest) {
    odd_at = tid < head ? tid : a.V - rest + tid - head;
    odd = fmax_nan(T::load(base, odd_at), -LP_FAR);
    bad = !(odd < LP_FAR);
    if (odd > -LP_FAR && !bad) {
      acc.raise(odd, a.c, odd_at);
      acc.s = 1.f;
    }
    ahead = odd > xt || (odd == xt && odd_at < token);
  }

  // The bound of the largest n: the least of the warps' keys that ceil(n / WARPS) of their
  // threads' largest elements reach; 0 while some warp has none.
  unsigned long long bound = 0ull;
  float bound_v = -LP_FAR;
  int turn = 0;
  auto publish = [&]() {
    const int k = (n + WARPS - 1) / WARPS;
    const uint32_t mine = acc.at >= 0 ? ev_ordered(acc.m) : 0u, v = lp_kth(mine, k);
    const uint32_t last = __reduce_max_sync(0xffffffffu, mine == v ? static_cast<uint32_t>(acc.at) : 0u);
    turn ^= 1;
    if (lane == 0) sh.bound[turn][warp] = v == 0u ? 0ull : (static_cast<unsigned long long>(v) << 32) | static_cast<uint32_t>(~last);
  };
  auto refresh = [&]() {
    bound = sh.bound[turn][0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) bound = min(bound, sh.bound[turn][w]);
    bound_v = bound ? lp_value(bound) : -LP_FAR;
  };
  auto push = [&](float x, int i) {
    const unsigned long long k = lp_key(x, i);
    if (x > -LP_FAR && k >= bound) {
      const int p = atomicAdd(&sh.count, 1);
      if (p < S::CAP) sh.list[p] = k;
    }
  };

  const int tiles = (v1 - v0 + TEAM * U - 1) / (TEAM * U);
  uint4 q[U];
  auto fetch = [&](int tile) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int v = v0 + tile * (TEAM * U) + j * TEAM + tid;
      q[j] = v < v1 ? lp_load(body + v) : lp_nothing<T>();
    }
  };
  fetch(0);
#pragma unroll 1
  for (int tile = 0; tile < max(tiles, 1); ++tile) {
    uint4 w[U];
    float top[U];
#pragma unroll
    for (int j = 0; j < U; ++j) w[j] = lp_clamp<T>(q[j]);
    if (tile + 1 < tiles) fetch(tile + 1);
    const int first = v0 + tile * (TEAM * U) + tid;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      top[j] = lp_vec_max<T>(w[j]);
      bad |= !(top[j] < LP_FAR);
      float x[E];
      T::unpack(w[j], x);
      if (top[j] > acc.m) {
        int f = E - 1;
#pragma unroll
        for (int k = E - 2; k >= 0; --k)
          if (x[k] == top[j]) f = k;
        acc.raise(top[j], a.c, head + (first + j * TEAM) * E + f);
      }
      if (acc.at < 0) continue;   // nothing with a weight so far
      const unsigned long long cc = f2_pack(a.c, a.c), mm = f2_pack(-acc.m, -acc.m);
      unsigned long long s2 = 0ull, x2 = 0ull;
#pragma unroll
      for (int k = 0; k < E; k += 2) {
        const unsigned long long z = f2_mul(f2_add(f2_pack(x[k], x[k + 1]), mm), cc);
        float z0, z1;
        f2_unpack(z, z0, z1);
        const unsigned long long e = f2_pack(ex2_approx(z0), ex2_approx(z1));
        s2 = f2_add(s2, e);
        x2 = f2_fma(e, z, x2);
      }
      float s0, s1, x0, x1;
      f2_unpack(s2, s0, s1);
      f2_unpack(x2, x0, x1);
      acc.s += s0 + s1;
      acc.x += x0 + x1;
    }
    // what stands before the token
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int v = first + j * TEAM, i = head + v * E;
      if (top[j] >= xt && v < v1) {
        float x[E];
        T::unpack(w[j], x);
        const float t = i < token ? below : xt;
#pragma unroll
        for (int k = 0; k < E; ++k) ahead += x[k] > t;
        if (i < token && token < i + E) {   // (what equals it behind it, and itself)
#pragma unroll
          for (int k = 0; k < E; ++k) ahead -= x[k] == xt && i + k >= token;
        }
      }
    }
    if constexpr (TOP) {
      if ((tile & (tile + 1)) == 0 || bound == 0ull) {   // (alike in the whole team)
        publish();
        lp_sync<WARPS>();
        refresh();
        if (tile == 0 && odd_at >= 0) push(odd, odd_at);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (top[j] >= bound_v && top[j] > -LP_FAR) {
          float x[E];
          T::unpack(w[j], x);
          uint32_t hits = 0u;
#pragma unroll
          for (int k = 0; k < E; ++k) hits |= x[k] >= bound_v ? 1u << k : 0u;
          for (; hits; hits &= hits - 1u) {
            const int i = head + (first + j * TEAM) * E + __ffs(hits) - 1;
            push(T::load(base, i), i);
          }
        }
      }
    }
  }

  if constexpr (TOP) publish();   // the last bound
  if (TOP && tid < n) sh.top[tid] = 0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    acc.merge(__shfl_down_sync(0xffffffffu, acc.m, o), __shfl_down_sync(0xffffffffu, acc.s, o), __shfl_down_sync(0xffffffffu, acc.x, o), a.c);
  ahead = __reduce_add_sync(0xffffffffu, ahead);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.m[warp] = acc.m;
    sh.s[warp] = acc.s;
    sh.x[warp] = acc.x;
    sh.ahead[warp] = ahead;
    sh.bad[warp] = bad;
  }
  lp_sync<WARPS>();

  if constexpr (TOP) {
    refresh();
    const int count = sh.count;
    if (count <= S::CAP) {
      // those that reach the last bound, each to the place that its rank among them is
      const unsigned long long* list = sh.list;
      int m = count;
      if constexpr (WARPS == 1) {
        m = 0;
        for (int i0 = 0; i0 < count; i0 += 32) {
          const unsigned long long k = i0 + lane < count ? sh.list[i0 + lane] : 0ull;
          const bool in = k != 0ull && k >= bound;
          const uint32_t all = __ballot_sync(0xffffffffu, in);
          if (in) sh.list[m + __popc(all & ((1u << lane) - 1u))] = k;   // (not past what has been read)
          m += __popc(all);
          __syncwarp();
        }
      } else {
        for (int i = tid; i < count; i += TEAM) {
          const unsigned long long k = sh.list[i];
          if (k >= bound) {
            const int p = atomicAdd(&sh.count2, 1);
            if (p < S::CAP2) sh.list2[p] = k;
          }
        }
        __syncthreads();
        if (sh.count2 <= S::CAP2) {
          list = sh.list2;
          m = sh.count2;
        }
      }
      for (int i = tid; i < m; i += TEAM) {
        const unsigned long long k = list[i];
        int r = 0;
        for (int j = 0; j < m; ++j) r += list[j] > k;
        if (r < n) sh.top[r] = k;
      }
    } else {
      // the list ran over: the largest below the last found, n times
      unsigned long long last = ~0ull;
      for (int r = 0; r < n; ++r) {
        unsigned long long best = 0ull;
        auto take = [&](float x, int i) {
          const unsigned long long k = lp_key(x, i);
          if (x > -LP_FAR && k < last) best = max(best, k);
        };
        if (odd_at >= 0) take(odd, odd_at);
        for (int v = v0 + tid; v < v1; v += TEAM) {
          const uint4 w = __ldg(body + v);
          float x[E];
          T::unpack(w, x);
#pragma unroll
          for (int k = 0; k < E; ++k) take(x[k], head + v * E + k);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if constexpr (WARPS > 1) {
          __syncthreads();
          if (lane == 0) sh.bound[0][warp] = best;
          __syncthreads();
          for (int w = 0; w < WARPS; ++w) best = max(best, sh.bound[0][w]);
        }
        if (tid == 0) sh.top[r] = best;
        last = best;
        if (best == 0ull) break;
      }
    }
  }
  if constexpr (WARPS > 1) {
    __syncthreads();
    if (warp == 0) {   // the CTA's sums, in the first place
      const bool in = lane < WARPS;
      LpAcc t;
      t.init();
      if (in) t.m = sh.m[lane], t.s = sh.s[lane], t.x = sh.x[lane];
      int before = in ? sh.ahead[lane] : 0;
      bool any = in && sh.bad[lane];
      __syncwarp();
#pragma unroll
      for (int o = WARPS / 2; o > 0; o >>= 1)
        t.merge(__shfl_down_sync(0xffffffffu, t.m, o), __shfl_down_sync(0xffffffffu, t.s, o), __shfl_down_sync(0xffffffffu, t.x, o), a.c);
      before = __reduce_add_sync(0xffffffffu, before);
      any = __any_sync(0xffffffffu, any);
      if (lane == 0) {
        sh.m[0] = t.m;
        sh.s[0] = t.s;
        sh.x[0] = t.x;
        sh.ahead[0] = before;
        sh.bad[0] = any;
      }
    }
    if (C > 1) {   // the cluster's, in the first CTA
      cluster_sync_all();
      if (part == 0) {
        if (warp == 0) {
          const bool in = lane < C;
          LpAcc t;
          t.init();
          int before = 0, any = 0;
          if (in) {
            t.m = __uint_as_float(ld_peer_u32(&sh.m[0], lane));
            t.s = __uint_as_float(ld_peer_u32(&sh.s[0], lane));
            t.x = __uint_as_float(ld_peer_u32(&sh.x[0], lane));
            before = static_cast<int>(ld_peer_u32(&sh.ahead[0], lane));
            any = static_cast<int>(ld_peer_u32(&sh.bad[0], lane));
          }
          __syncwarp();
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            t.merge(__shfl_down_sync(0xffffffffu, t.m, o), __shfl_down_sync(0xffffffffu, t.s, o), __shfl_down_sync(0xffffffffu, t.x, o), a.c);
          before = __reduce_add_sync(0xffffffffu, before);
          any = __any_sync(0xffffffffu, any != 0);
          if (lane == 0) {
            sh.m[1] = t.m;
            sh.s[1] = t.s;
            sh.x[1] = t.x;
            sh.ahead[1] = before;
            sh.bad[1] = any;
          }
        }
        if constexpr (TOP) {
          for (int i = tid; i < n * C; i += TEAM) {
            const int r = i / n, j = i - r * n;
            const unsigned long long* k = &sh.top[j];
            const uint32_t lo = ld_peer_u32(k, r), hi = ld_peer_u32(reinterpret_cast<const uint32_t*>(k) + 1, r);
            sh.list[i] = (static_cast<unsigned long long>(hi) << 32) | lo;
          }
          __syncthreads();
          if (tid < n) sh.top[tid] = 0ull;
          __syncthreads();
          for (int i = tid; i < n * C; i += TEAM) {
            const unsigned long long k = sh.list[i];
            int r = 0;
            for (int j = 0; j < n * C; ++j) r += sh.list[j] > k;
            if (k != 0ull && r < n) sh.top[r] = k;
          }
        }
      }
      cluster_sync_all();   // nobody ends while its shared memory is read
      if (part != 0) return;
    }
  }
  lp_sync<WARPS>();
  const int at = C > 1 ? 1 : 0;
  const float m = sh.m[at], s = sh.s[at];
  const bool valid = !sh.bad[at] && s > 0.f;
  const float nan = __int_as_float(0x7fc00000), log_s = log2f(s), ln2 = 0.693147180559945f;
  auto logprob = [&](float x) { return x > -LP_FAR ? (__fmul_rn(__fsub_rn(x, m), a.c) - log_s) * ln2 : kNegInf; };
  if (tid == 0) {
    a.logprobs[place] = valid ? logprob(xt) : nan;
    if (a.entropy) a.entropy[place] = valid ? fmaxf(log_s - sh.x[at] / s, 0.f) * ln2 : nan;
    if (a.ranks) a.ranks[place] = valid ? sh.ahead[at] + 1 : -1;
  }
  if (TOP && tid < n) {
    const unsigned long long k = sh.top[tid];
    a.top_tokens[place * n + tid] = valid && k ? lp_index(k) : -1;
    a.top_logprobs[place * n + tid] = !valid ? nan : k ? logprob(lp_value(k)) : kNegInf;
  }
}

}  // namespace sv
