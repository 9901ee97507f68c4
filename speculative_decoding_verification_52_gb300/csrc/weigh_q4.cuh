// weigh_q4.cuh -- the weight that a step's committed rows gave to each cached token,
// added to what the token had:
//   w'[s] = decay * w[s] + sum over rows i and their query heads of e^(scale q_i.k_s - lse_i),
// row i (the i-th committed) seeing the positions up to lengths + i.  It is the first
// half of attention without its sums over tokens: every token's result is its own, so
// nothing is joined, and a row's logarithm of the sum is known.
//
// This kernel: the tokens are M of mma.m16n8k16, the rows N, eight at a time, as in
// attend_q4.cuh: a thread's part of a key operand is D / 4 consecutive elements of a
// token, unpacked in f16 exactly, the queries enter as f16 times a power of two per row.
// A warp has a share of the list of all blocks (32 tokens of a head), fetches their keys
// through a ring of its own by bulk copies, and keeps its queries in registers, up to 32
// rows; more rows are taken in turns, over the same keys.  A sequence's rows are taken
// in as many groups of eight as it commits, not as the batch might.
//
// Bound: the keys' 9/16 byte an element and 8 bytes of weights a token, 50 us of 256
// sequences of 2,048 tokens and 8 heads of 128; it takes 126 (2.7 TB/s) for chains of which
// 3.2 nodes of 4 query heads are committed on average, 530 instructions a block of 32
// tokens: 64 conversions and as many multiplications of code pairs, 16 products and 14
// exponentials a lane for each eight rows.  Sixteen warps an SM, as many as the registers
// allow (five CTAs, through local memory: 209 us; three: 128), issue 56 % of the time, by
// the latency of what depends on each other: two chains of products a sum 126 us, one 128.
// With the next block in registers instead of rings, and all rows that the batch may
// commit, it was 157 us.
#pragma once

#include "common.cuh"
#include "kv_q4.cuh"
#include "q4_ops.cuh"

namespace sv {

constexpr int WG_THREADS = 128;
constexpr int WG_MAX_B = 4096;

struct WeighArgs {
  const uint16_t* q;          // [B, N, Hkv * G, D] bf16
  const float* lse;           // [B, N, Hkv * G]
  const int32_t* path;        // [B, PW] or null
  const int32_t* count;       // [B] or null (all rows)
  const unsigned char* cache;
  const int32_t* table;       // [B, W]
  const int32_t* lengths;     // [B]
  const int32_t* first;       // [B] or null
  const float* weights;       // [pages, Hkv, P]
  float* new_weights;         // the same, or weights itself
  int32_t* positions;         // [pages, Hkv, P] or null
  int B, N, PW, most, G, Hkv, P, pages, W;   // most: rows that a sequence may commit
  float scale_log2, k_mul, decay;
  unsigned long long timeout_ns;
};

// rows that sequence b commits; -1: nothing is done for it
__device__ __forceinline__ int wg_rows(const WeighArgs& a, int b) {
  const int n = a.count ? a.count[b] : a.most, L = a.lengths[b];
  if (n < 0 || n > a.most || L < 0 || static_cast<long long>(L) + n > static_cast<long long>(a.W) * a.P) return -1;
  if (a.path)
    for (int i = 0; i < n; ++i) {
      const int j = a.path[static_cast<long long>(b) * a.PW + i];
      if (j < 0 || j >= a.N) return -1;
    }
  return n;
}

// prefix[b]: tiles (of `tile` tokens) of sequences 0..b-1 (one head), rows[b]: rows of sequence b
template <int THREADS>
__device__ void wg_prefix(const WeighArgs& a, int tile, long long* prefix, int* rows, long long* scratch) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    long long v = 0;
    if (b < a.B) {
      const int n = wg_rows(a, b);
      rows[b] = n;
      v = n < 0 ? 0 : (static_cast<long long>(a.lengths[b]) + n + tile - 1) / tile;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) scratch[w] = v;
    __syncthreads();
    long long all = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      const long long s = scratch[i];
      if (i < w) v += s;
      all += s;
    }
    if (b < a.B) prefix[b + 1] = base + v;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
}

// what a warp fetches of a block: codes, scales
__host__ __device__ constexpr int wg_stage_bytes(int D) { return 18 * D; }

// rows 8 j + g of a chunk as f16 operands, and for the columns 8 j + 2 t + e the factor to
// the log2 domain and minus the row's lse there (-inf: the row adds nothing)
template <int D, int NR>
__device__ __forceinline__ void wg_load_q(const WeighArgs& a, int b, int h, int row0, int rows, uint32_t (&q)[NR][D / 8], float4* fl) {
  constexpr int CH = D / 4;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int r = row0 + 8 * j + g;
    uint4 w[CH / 8];
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    float lse = __builtin_huge_valf();
    if (r < rows) {
      const int i = r / a.G, node = a.path ? a.path[static_cast<long long>(b) * a.PW + i] : i;
      const long long at = (static_cast<long long>(b) * a.N + node) * (a.Hkv * a.G) + h * a.G + (r - i * a.G);
      const uint4* p = reinterpret_cast<const uint4*>(a.q + at * D + t * CH);
#pragma unroll
      for (int x = 0; x < CH / 8; ++x) w[x] = __ldg(p + x);
      lse = __ldg(a.lse + at) * 1.44269504088896f;
      if (!(fabsf(lse) < __builtin_huge_valf())) lse = __builtin_huge_valf();
    }
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) {
      mx = bf16x2_max_nan(mx, bf16x2_max_nan(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu));
      mx = bf16x2_max_nan(mx, bf16x2_max_nan(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
    }
    float top = fmax_nan(__uint_as_float(mx << 16), __uint_as_float(mx & 0xffff0000u));
    top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // (a row with elements that are no numbers has no finite lse, or should not have one)
    const bool counts = top < __builtin_huge_valf() && lse < __builtin_huge_valf();
    if (!counts) lse = __builtin_huge_valf();
    // to [128, 256): what f16 then cannot hold is below 2^-32 of the largest element
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int sh = top > 0.f ? min(7 - ex, 100) : 0;
    const float mul = copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), a.scale_log2);
    const float back = fminf(fmaxf(fabsf(a.scale_log2) * a.k_mul * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23), 1.17549435e-38f), 3.402823466e+38f);
    // (in shared memory: registers are what limits the warps of an SM)
    const float4 both = make_float4(__shfl_sync(0xffffffffu, back, 8 * t), __shfl_sync(0xffffffffu, back, 8 * t + 4),
                                    -__shfl_sync(0xffffffffu, lse, 8 * t), -__shfl_sync(0xffffffffu, lse, 8 * t + 4));
    if (g == 0) fl[4 * j + t] = both;
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) q[j][4 * i + k] = counts ? f16x2_pack(__uint_as_float(x[k] << 16) * mul, __uint_as_float(x[k] & 0xffff0000u) * mul) : 0u;
    }
  }
}

// d = A B (+ d); not volatile, so that products of different sums may pass each other
template <bool ADD>
__device__ __forceinline__ void wg_mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (ADD)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}

// A block's sums over a chunk of rows, `groups` times eight of them; the lane gets that
// of its token, (t >> 1) * 16 + (t & 1) * 8 + g.  from: the block's codes and scales; see:
// it has tokens that not all rows see, the first `fresh` behind the old ones.
// (The unpacked keys of sixteen tokens stay in registers while the groups pass by, which
// a branch for each leaves out: sequences that commit fewer rows cost less.)
template <int D, int NR>
__device__ __forceinline__ float wg_block(const unsigned char* from, const uint32_t (&q)[NR][D / 8], const float4* fl,
                                          int groups, bool see, int fresh, int row0, int G) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float sum[4];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    // eight tokens' rows of codes lie side by side, a quarter a lane; so do their scales
    uint4 A[D / 16];
    {
      uint32_t code[2][D / 32], s2[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tok = 16 * m + 8 * u + g;
        const unsigned char* c = from + tok * (D / 2) + t * (D / 8);
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(c);
          code[u][0] = x.x, code[u][1] = x.y, code[u][2] = x.z, code[u][3] = x.w;
          s2[u] = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(from + 16 * D + tok * (D / 16) + t * 2));
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(c);
          code[u][0] = x.x, code[u][1] = x.y;
          s2[u] = e4m3x2_to_f16(from[16 * D + tok * (D / 16) + t]);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {   // eight codes of each of two tokens: two steps of 16
        uint32_t lo[4], hi[4];
        e2m1x8_to_f16(code[0][i], lo);
        e2m1x8_to_f16(code[1][i], hi);
        const uint32_t sel = i < 2 ? 0x1010u : 0x3232u, x0 = __byte_perm(s2[0], 0u, sel), x1 = __byte_perm(s2[1], 0u, sel);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          A[2 * i + k] = make_uint4(f16x2_mul(lo[2 * k], x0), f16x2_mul(hi[2 * k], x1), f16x2_mul(lo[2 * k + 1], x0), f16x2_mul(hi[2 * k + 1], x1));
      }
    }
    unsigned long long x[2] = {0ull, 0ull};   // of the two tokens, the even and the odd columns
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      if (j > 0 && j >= groups) break;
      const float4 c = fl[4 * j + t];
      float d[4], e[4];   // (two chains of products)
      wg_mma<false>(d, A[0], q[j][0], q[j][1]);
      wg_mma<false>(e, A[1], q[j][2], q[j][3]);
#pragma unroll
      for (int k = 2; k < D / 16; k += 2) {
        wg_mma<true>(d, A[k], q[j][2 * k], q[j][2 * k + 1]);
        wg_mma<true>(e, A[k + 1], q[j][2 * k + 2], q[j][2 * k + 3]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] += e[k];
      if (see) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((fresh + 16 * m + 8 * (k >> 1) + g) * G > row0 + 8 * j + 2 * t + (k & 1)) d[k] = kNegInf;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float z0, z1;
        f2_unpack(f2_fma(f2_pack(d[2 * k], d[2 * k + 1]), f2_pack(c.x, c.y), f2_pack(c.z, c.w)), z0, z1);
        x[k] = f2_add(x[k], f2_pack(ex2_approx(z0), ex2_approx(z1)));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x0, x1;
      f2_unpack(x[k], x0, x1);
      sum[2 * m + k] = x0 + x1;
    }
  }
  // over the four lanes of a token, each of which keeps one of the four tokens
  const bool up = t & 2, odd = t & 1;
  const float a0 = up ? sum[2] : sum[0], a1 = up ? sum[3] : sum[1], b0 = up ? sum[0] : sum[2], b1 = up ? sum[1] : sum[3];
  const float y0 = a0 + __shfl_xor_sync(0xffffffffu, b0, 2), y1 = a1 + __shfl_xor_sync(0xffffffffu, b1, 2);
  const float all = (odd ? y1 : y0) + __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
  // (the queries are numbers here: a sum that is none is a token's whose keys are none, and
  // none of whose scores weighs anything)
  return all == all ? all : 0.f;
}

__host__ __device__ constexpr int wg_ctas(int NR) { return NR == 1 ? 5 : NR <= 3 ? 4 : 3; }

template <int D, int NR>
__global__ void __launch_bounds__(WG_THREADS, wg_ctas(NR)) weigh_q4_kernel(const WeighArgs a, int stages) {
  extern __shared__ uint4 wg_dynamic[];
  __shared__ long long scratch[WG_THREADS / 32];
  constexpr int WARPS = WG_THREADS / 32;
  __shared__ float4 fl[WARPS][4 * NR];   // of the columns of a lane: factors, -lse
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  const int tok = (t >> 1) * 16 + (t & 1) * 8 + g;
  unsigned char* ring = reinterpret_cast<unsigned char*>(wg_dynamic) + warp * stages * wg_stage_bytes(D);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<unsigned char*>(wg_dynamic) + WARPS * stages * wg_stage_bytes(D));
  long long* prefix = reinterpret_cast<long long*>(bars + WARPS * stages);   // [B + 1]
  int* all_rows = reinterpret_cast<int*>(prefix + a.B + 1);                  // [B]
  for (int i = threadIdx.x; i < WARPS * stages; i += WG_THREADS) mbar_init(bars + i, 1);
  mbar_fence_init();
  bars += warp * stages;
  wg_prefix<WG_THREADS>(a, Q4_BLOCK, prefix, all_rows, scratch);   // (synchronises the CTA)
  const long long units = prefix[a.B] * a.Hkv;
  const long long warps = static_cast<long long>(gridDim.x) * WARPS;
  const long long w = static_cast<long long>(warp) * gridDim.x + blockIdx.x;   // (short lists spread over the SMs)
  long long u = units * w / warps;
  const long long u1 = units * (w + 1) / warps;
  const int per = a.P / Q4_BLOCK;
  int stage = 0;
  uint32_t parity = 0u;
  bool alive = true;
  while (u < u1) {
    int lo = 0, hi = a.B - 1;   // last b with prefix[b] * Hkv <= u that has blocks
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] * a.Hkv <= u) lo = mid;
      else hi = mid - 1;
    }
    // blocks [k0, k1) of head h of sequence b, in several passes where the rows are many
    const int b = lo, blocks = static_cast<int>(prefix[b + 1] - prefix[b]);
    const long long rem = u - prefix[b] * a.Hkv;
    const int h = static_cast<int>(rem / blocks), k0 = static_cast<int>(rem - static_cast<long long>(h) * blocks);
    const int k1 = static_cast<int>(min(static_cast<long long>(blocks), k0 + (u1 - u)));
    u += k1 - k0;
    const int n = all_rows[b], old = a.lengths[b], end = old + n, rows = n * a.G;
    const int32_t* table = a.table + static_cast<long long>(b) * a.W;
    const int first = (a.first ? a.first[b] : old) - old;
    for (int row0 = 0; row0 == 0 || row0 < rows; row0 += 8 * NR) {
      // The places of 32 blocks, a lane each (the block's number among the pool's, ~0: on
      // no page): of those from `look` on, to fetch; and of those from `have` on, to weigh.
      auto places = [&](int from) {
        uint32_t x = ~0u;
        if (from + lane < k1) {
          const int e = (from + lane) / per, page = table[e];
          if (page >= 0 && page < a.pages) x = (static_cast<uint32_t>(page) * a.Hkv + h) * per + (from + lane - e * per);
        }
        return x;
      };
      int look = k0, ahead = 0;   // ahead: blocks of the run that have been fetched
      uint32_t blk = places(k0), now = blk;
      auto fetch = [&](int s) {
        if (k0 + ahead - look == 32) {
          look += 32;
          blk = places(look);
        }
        const uint32_t x = __shfl_sync(0xffffffffu, blk, k0 + ahead - look);
        if (lane == 0) {
          if (x != ~0u) {
            const unsigned char* from = a.cache + static_cast<unsigned long long>(x) * q4_block_bytes(D);
            unsigned char* to = ring + s * wg_stage_bytes(D);
            mbar_arrive_expect_tx(bars + s, wg_stage_bytes(D));
            bulk_g2s(to, from, 16 * D, bars + s);
            bulk_g2s(to + 16 * D, from + 32 * D, 2 * D, bars + s);
          } else {
            mbar_arrive(bars + s);
          }
        }
        ++ahead;
      };
      for (int i = 0, s = stage; i < stages && k0 + i < k1 && alive; ++i) {
        fetch(s);
        if (++s == stages) s = 0;
      }
      uint32_t q[NR][D / 8];
      wg_load_q<D, NR>(a, b, h, row0, rows, q, fl[warp]);
      __syncwarp();
      const int groups = (min(rows - row0, 8 * NR) + 7) / 8;
      const float* from = row0 == 0 ? a.weights : a.new_weights;
      const int begun = row0 == 0 ? old : end;   // tokens that have a weight
      const float decay = row0 == 0 ? a.decay : 1.f;
      for (int k = k0; k < k1; ++k) {
        if (k > k0 && ((k - k0) & 31) == 0) now = look == k ? blk : places(k);
        const uint32_t x = __shfl_sync(0xffffffffu, now, (k - k0) & 31);
        const int pos = k * Q4_BLOCK + tok;
        const long long at = static_cast<long long>(x) * Q4_BLOCK + tok;
        const bool mine = x != ~0u && pos < end;
        float had = 0.f;
        if (mine && pos < begun) had = from[at];
        if (alive && !__all_sync(0xffffffffu, mbar_wait(bars + stage, parity, a.timeout_ns))) alive = false;
        float sum = wg_block<D, NR>(ring + stage * wg_stage_bytes(D), q, fl[warp], groups, (k + 1) * Q4_BLOCK > old, k * Q4_BLOCK - old, row0, a.G);
        __syncwarp();
        if (alive && k0 + ahead < k1) fetch(stage);
        if (!alive) sum = __int_as_float(0x7fc00000);
        if (mine) {
          a.new_weights[at] = pos < begun ? __fmaf_rn(decay, had, sum) : sum;
          if (row0 == 0 && a.positions && pos >= old) a.positions[at] = first + pos;
        }
        if (++stage == stages) {
          stage = 0;
          parity ^= 1u;
        }
        if (!alive) {   // copies that are still on their way
          for (int i = k + 1; i < k0 + ahead; ++i) {
            mbar_wait(bars + stage, parity, a.timeout_ns);
            if (++stage == stages) {
              stage = 0;
              parity ^= 1u;
            }
          }
          ahead = 0;
        }
      }
    }
  }
}

}  // namespace sv
