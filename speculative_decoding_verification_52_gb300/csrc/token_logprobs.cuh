// token_logprobs.cuh -- log probabilities of the tokens a verification emitted, their
// ranks, the rows' entropies and their most probable tokens.
//
// A row's logits l at temperature T, z = l / T, m = max z, S = sum e^(z - m):
//   logprob(t) = z_t - m - log S,   entropy = log S - (sum e^(z - m) (z - m)) / S,
//   rank(t) = 1 + #{v: l_v > l_t, or l_v = l_t and v < t}.
// Everything comes from one pass over the row, in the log2 domain (c = log2(e) / T),
// with a running reference a warp; when it moves by d <= 0,
//   S' = 2^d S,  X' = 2^d (X + d S)   for X = sum 2^z z.
//
// The largest n.  A thread that has seen elements knows the largest of its own; in a
// team of `WARPS` warps, the ceil(n / WARPS)-th largest of a warp's 32, taken as the
// least over the warps, has n elements at or above it.  Only what reaches that bound
// goes into a list: some dozens of elements, since the bound is taken anew after 1, 2,
// 4, ... tiles.  Equal elements are told apart by their index in
// the bound, too, so that a row of equal logits fills no list.  Where a list runs over all
// the same (a row whose logits rise to its end), the team searches the row once for each
// of its n largest.  Elements that the bound or the token's logit concerns are looked for
// by the vector's maximum, which the references need anyway.
//
// Bound: one read of the row.  842 rows of 128,256 bf16 with 20 alternatives take 56 us,
// 3.9 TB/s; 2,432 rows 117 (5.3 TB/s), without alternatives 98 (6.4 TB/s): 12 instructions
// an element, of which 8 for the sums, issue 72 % busy.  What the smaller batch loses is
// the tail: a CTA a row, four an SM, makes 608 rows at a time.  (Two CTAs a row as a cluster
// 72 us, sixteen warps a CTA 72, four 68.)  One row, on eight CTAs, takes 7.5 us, of which
// the cluster's two meetings 3.
#pragma once

#include "common.cuh"
#include "evict.cuh"

namespace sv {

constexpr int LP_WARPS = 8;        // of the CTA that takes a long row
constexpr int LP_TEAMS = 8;        // warps of a CTA that take a short row each
__host__ __device__ constexpr int lp_threads(int warps) { return warps == 1 ? 32 * LP_TEAMS : 32 * warps; }
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

// Sums of a part of a row against a reference (a logit; -2^100: nothing with a weight
// yet).  Exponents are (l - m) c, which is 0 for m itself however large it is; l c -
// fl(m c), an instruction less, is off by what the product lost.
struct LpAcc {
  float m, s, x;       // reference, sum 2^z, sum 2^z z
  // to a reference of `to` (above the present one)
  __device__ __forceinline__ void raise(float to, float c) {
    if (s > 0.f) {
      const float d = __fmul_rn(__fsub_rn(m, to), c), f = ex2_approx(d);   // (d <= 0)
      x = f * __fmaf_rn(d, s, x);
      s *= f;
    }
    m = to;
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

// elements of a vector above t
template <class T>
__device__ __forceinline__ int lp_above(const uint4& q, float t) {
  float x[T::vpe];
  T::unpack(q, x);
  int n = 0;
#pragma unroll
  for (int k = 0; k < T::vpe; ++k) n += x[k] > t;
  return n;
}
template <>   // (t is a bf16, and so is the next number below one)
__device__ __forceinline__ int lp_above<BF16T>(const uint4& q, float t) {
  const uint32_t u = __byte_perm(__float_as_uint(t), 0u, 0x3232);
  auto set = [&](uint32_t x) {
    uint32_t d;
    asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(u));
    return d;
  };
  auto add = [](uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  };
  const uint32_t n = add(add(set(q.x), set(q.y)), add(set(q.z), set(q.w)));
  return static_cast<int>(__uint_as_float(n << 16) + __uint_as_float(n & 0xffff0000u));
}

template <int WARPS>
struct LpShared {
  static constexpr int CAP = WARPS == 1 ? 256 : 1024;   // a team's list
  static constexpr int CAP2 = WARPS == 1 ? 256 : 512;   // elements that reach the last bound
  uint2 list[CAP];   // of what a thread had of a tile: the largest element (ordered), the first vector
  unsigned long long list2[CAP2];
  uint32_t picked[CAP];   // of the list, what reaches the last bound: the first vectors
  unsigned long long bound[WARPS];
  unsigned long long top[LP_MAX_TOP];
  float m[WARPS], s[WARPS], x[WARPS];
  int ahead[WARPS], bad[WARPS];
  int count, count2, count3;
};

// the first n of m different keys, in order; `each` threads (a power of two) count for one
__device__ __forceinline__ void lp_order(const unsigned long long* list, int m, int n, int tid, int team, unsigned long long* top) {
  int each = 1;
  while (each < 32 && each * 2 * m <= team) each *= 2;
  const int sub = tid & (each - 1);
  for (int i0 = 0; i0 < m; i0 += team / each) {   // (whole warps go on alike)
    const int i = i0 + tid / each;
    const unsigned long long k = i < m ? list[i] : 0ull;
    int r = 0;
#pragma unroll 8
    for (int j = sub; j < m; j += each) r += list[j] > k;
    for (int o = each >> 1; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (sub == 0 && k != 0ull && r < n) top[r] = k;
  }
}

template <int WARPS>
__device__ __forceinline__ void lp_sync() {
  if constexpr (WARPS == 1) __syncwarp();
  else __syncthreads();
}

// One team a row, or a part of it: the CTA, or a warp.
template <class T, int WARPS, bool TOP>
__global__ void __launch_bounds__(lp_threads(WARPS), 1024 / lp_threads(WARPS)) token_logprobs_kernel(const LogprobArgs a) {
  using S = LpShared<WARPS>;
  constexpr int TEAM = 32 * WARPS, TEAMS = lp_threads(WARPS) / TEAM, U = 4, E = T::vpe;
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
  constexpr uint32_t ULP = T::esz == 2 ? 0x10000u : 1u;
  const float below = __uint_as_float(xt == 0.f ? 0x80000000u + ULP : xt > 0.f ? __float_as_uint(xt) - ULP : __float_as_uint(xt) + ULP);

  if (tid == 0) sh.count = sh.count2 = sh.count3 = 0;
  LpAcc acc = {-LP_FAR, 0.f, 0.f};   // (m: the warp's)
  float most = -LP_FAR;   // the largest of the thread's elements, and the last index of its tile
  int at = 0;
  int ahead = 0;          // elements before the token's in the order
  bool bad = false;
  // the odd elements, one a thread
  float odd = -LP_FAR;
  int odd_at = -1;
  if (part == 0 && tid < head + rest) {
    odd_at = tid < head ? tid : a.V - rest + tid - head;
    odd = fmax_nan(T::load(base, odd_at), -LP_FAR);
    bad = !(odd < LP_FAR);
    if (bad) odd = -LP_FAR;
    most = odd;
    at = odd_at;
    ahead = odd > xt || (odd == xt && odd_at < token);
  }

  // The bound of the largest n: the least of the warps' keys that ceil(n / WARPS) of their
  // threads' largest elements reach; 0 while some warp has none.
  unsigned long long bound = 0ull;
  float bound_v = -LP_FAR;
  auto publish = [&]() {
    const int k = (n + WARPS - 1) / WARPS;
    const uint32_t mine = most > -LP_FAR ? ev_ordered(most) : 0u, v = warp_kth(mine, k);
    const uint32_t last = __reduce_max_sync(0xffffffffu, mine == v ? static_cast<uint32_t>(at) : 0u);
    if (lane == 0) *const_cast<volatile unsigned long long*>(&sh.bound[warp]) = v == 0u ? 0ull : (static_cast<unsigned long long>(v) << 32) | static_cast<uint32_t>(~last);
  };
  auto refresh = [&]() {
    const unsigned long long k = *const_cast<volatile unsigned long long*>(&sh.bound[lane % WARPS]);
    const uint32_t hi = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0xffffffffu);
    bound = (static_cast<unsigned long long>(hi) << 32) | lo;
    bound_v = bound ? lp_value(bound) : -LP_FAR;
  };

  const int tiles = (v1 - v0 + TEAM * U - 1) / (TEAM * U);
  uint4 q[U];
  auto fetch = [&](int tile) {
    const int v = v0 + tile * (TEAM * U) + tid;
    if (v0 + (tile + 1) * (TEAM * U) <= v1) {
#pragma unroll
      for (int j = 0; j < U; ++j) q[j] = lp_load(body + v + j * TEAM);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        q[j] = lp_nothing<T>();
        if (v + j * TEAM < v1) q[j] = lp_load(body + v + j * TEAM);
      }
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
    float all = tile == 0 ? odd : -LP_FAR;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      top[j] = lp_vec_max<T>(w[j]);
      all = fmax_nan(all, top[j]);
    }
    if (TOP && all > most) {
      most = all;
      at = head + (first + (U - 1) * TEAM) * E + E - 1;
    }
    bad |= !(all < LP_FAR);
    // The warp's reference moves when an element passes it by 8 in the exponent (and for
    // the first with a weight).  A reference for each thread that followed its largest
    // element moved in some lane at three vectors of four.
    if (__any_sync(0xffffffffu, __fmul_rn(__fsub_rn(all, acc.m), a.c) > (acc.m > -LP_FAR ? 8.f : 0.f))) {
      const uint32_t k = __reduce_max_sync(0xffffffffu, ev_ordered(all));   // (a NaN is the least)
      const float to = lp_value(static_cast<unsigned long long>(k) << 32);
      if (to > acc.m) acc.raise(to, a.c);
    }
    if (acc.m > -LP_FAR) {
      const unsigned long long cc = f2_pack(a.c, a.c), mm = f2_pack(-acc.m, -acc.m);
      if (tile == 0 && odd_at >= 0) {
        const float z = __fmul_rn(__fsub_rn(odd, acc.m), a.c), e = ex2_approx(z);
        acc.s += e;
        acc.x += e * z;
      }
      unsigned long long s2 = 0ull, x2 = 0ull;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float x[E];
        T::unpack(w[j], x);
#pragma unroll
        for (int k = 0; k < E; k += 2) {
          const unsigned long long z = f2_mul(f2_add(f2_pack(x[k], x[k + 1]), mm), cc);
          float z0, z1;
          f2_unpack(z, z0, z1);
          const unsigned long long e = f2_pack(ex2_approx(z0), ex2_approx(z1));
          s2 = f2_add(s2, e);
          x2 = f2_fma(e, z, x2);
        }
      }
      float s0, s1, x0, x1;
      f2_unpack(s2, s0, s1);
      f2_unpack(x2, x0, x1);
      acc.s += s0 + s1;
      acc.x += x0 + x1;
    }
    // what stands before the token (few tiles have any)
    if (__any_sync(0xffffffffu, all >= xt)) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int v = first + j * TEAM, i = head + v * E;
        if (top[j] >= xt && v < v1) {
          ahead += lp_above<T>(w[j], i < token ? below : xt);
          if (i < token && token < i + E) {   // (what equals it behind it, and itself)
            float x[E];
            T::unpack(w[j], x);
#pragma unroll
            for (int k = 0; k < E; ++k) ahead -= x[k] == xt && i + k >= token;
          }
        }
      }
    }
    if constexpr (TOP) {
      // (A bound only rises: one that another warp has not renewed yet serves, too.  The
      // first tile's are waited for.)
      if ((tile & (tile + 1)) == 0 || bound == 0ull) {
        publish();
        if (tile == 0) lp_sync<WARPS>();
        else __syncwarp();
        refresh();
      }
      if (all >= bound_v && all > -LP_FAR && (all > bound_v || head + first * E <= lp_index(bound))) {
        const int p = atomicAdd(&sh.count, 1);
        if (p < S::CAP) sh.list[p] = make_uint2(ev_ordered(all), static_cast<uint32_t>(first));
      }
    }
  }

  if constexpr (TOP) publish();   // the last bound
  if (TOP && tid < n) sh.top[tid] = 0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {   // (one reference)
    acc.s += __shfl_xor_sync(0xffffffffu, acc.s, o);
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
  }
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
      // the elements of the listed vectors that reach the last bound
      for (int i = tid; i < count; i += TEAM) {
        const uint2 e = sh.list[i];
        if (e.x >= static_cast<uint32_t>(bound >> 32)) sh.picked[atomicAdd(&sh.count3, 1)] = e.y;
      }
      lp_sync<WARPS>();
      // a vector a thread, so that all are loaded at once, and the odd elements' thread;
      // places for a warp's elements by one addition
      const int picked = sh.count3 * U;
      for (int i0 = 0; i0 < max(picked, 1); i0 += TEAM) {   // (whole warps go on alike)
        const int i = i0 + tid, v = i < picked ? static_cast<int>(sh.picked[i / U]) + i % U * TEAM : v1;
        float x[E];
        T::unpack(v < v1 ? __ldg(body + v) : lp_nothing<T>(), x);
        const bool more = i0 == 0 && odd_at >= 0;
        uint32_t hits = more && odd > -LP_FAR && lp_key(odd, odd_at) >= bound ? 1u << E : 0u;
#pragma unroll
        for (int k = 0; k < E; ++k) hits |= x[k] >= bound_v && x[k] > -LP_FAR && lp_key(x[k], head + v * E + k) >= bound ? 1u << k : 0u;
        const int mine = __popc(hits);
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        int p = 0;
        if (lane == 31 && before) p = atomicAdd(&sh.count2, before);
        p = __shfl_sync(0xffffffffu, p, 31) + before - mine;
        for (; hits; hits &= hits - 1u) {
          const int k = __ffs(hits) - 1;
          float y = odd;
#pragma unroll
          for (int e = 0; e < E; ++e) y = e == k ? x[e] : y;
          if (p < S::CAP2) sh.list2[p] = lp_key(y, k < E ? head + v * E + k : odd_at);
          ++p;
        }
      }
      lp_sync<WARPS>();
    }
    if (count <= S::CAP && sh.count2 <= S::CAP2) {
      lp_order(sh.list2, sh.count2, n, tid, TEAM, sh.top);
    } else {
      // a list ran over: the largest below the last found, n times
      unsigned long long last = ~0ull;
      for (int r = 0; r < n; ++r) {
        unsigned long long best = 0ull;
        auto take = [&](float x, int i) {
          const unsigned long long k = lp_key(x, i);
          if (x > -LP_FAR && k < last) best = max(best, k);
        };
        if (odd_at >= 0) take(odd, odd_at);
        for (int v = v0 + tid; v < v1; v += TEAM) {
          float x[E];
          T::unpack(__ldg(body + v), x);
#pragma unroll
          for (int k = 0; k < E; ++k) take(x[k], head + v * E + k);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if constexpr (WARPS > 1) {
          __syncthreads();
          if (lane == 0) sh.bound[warp] = best;
          __syncthreads();
          for (int w = 0; w < WARPS; ++w) best = max(best, sh.bound[w]);
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
      LpAcc t = {-LP_FAR, 0.f, 0.f};
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
          LpAcc t = {-LP_FAR, 0.f, 0.f};
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
            sh.list2[i] = ld_peer_u64(&sh.top[j], r);
          }
          __syncthreads();
          if (tid < n) sh.top[tid] = 0ull;
          __syncthreads();
          lp_order(sh.list2, n * C, n, tid, TEAM, sh.top);
        }
      }
      cluster_sync_all();   // nobody ends while its shared memory is read
      if (part != 0) return;
    }
  }
  lp_sync<WARPS>();
  const int in = C > 1 ? 1 : 0;
  const float m = sh.m[in], s = sh.s[in];
  const bool valid = !sh.bad[in] && s > 0.f;
  const float nan = __int_as_float(0x7fc00000), log_s = log2f(s), ln2 = 0.693147180559945f;
  auto logprob = [&](float x) { return x > -LP_FAR ? (__fmul_rn(__fsub_rn(x, m), a.c) - log_s) * ln2 : kNegInf; };
  if (tid == 0) {
    a.logprobs[place] = valid ? logprob(xt) : nan;
    if (a.entropy) a.entropy[place] = valid ? fmaxf(log_s - sh.x[in] / s, 0.f) * ln2 : nan;
    if (a.ranks) a.ranks[place] = valid ? sh.ahead[in] + 1 : -1;
  }
  if (TOP && tid < n) {
    const unsigned long long k = sh.top[tid];
    a.top_tokens[place * n + tid] = valid && k ? lp_index(k) : -1;
    a.top_logprobs[place * n + tid] = !valid ? nan : k ? logprob(lp_value(k)) : kNegInf;
  }
}

}  // namespace sv
