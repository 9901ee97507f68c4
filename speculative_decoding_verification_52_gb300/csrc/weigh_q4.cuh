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
// A warp has a share of the list of all blocks (32 tokens of a head) and keeps its
// queries in registers, up to 32 rows; more rows are taken in turns, over the same keys.
// A block comes by plain 16-byte loads, 64 bytes of a token side by side, the next one's
// while this one is weighed.
//
// Bound: the keys' 9/16 byte an element and 8 bytes of weights a token.  A block (D =
// 128) crosses the bus in about 110 clocks of an SM; it takes 64 conversions and 64
// multiplications (32 clocks each), 16 products per eight rows (32 clocks) and 8
// exponentials a lane per eight rows.
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

// a block as a lane loads it: D / 4 codes and their scales of four tokens
template <int D>
struct WgRaw {
  uint32_t code[4][D / 32];
  uint32_t scale[4];   // D = 128: two bytes
  float weight;
  long long at;        // of the lane's token among the weights; -1: no such page
};

template <int D>
__device__ __forceinline__ void wg_fetch(const WeighArgs& a, int h, int page, int in_page, int t0, int end, int old, const float* from, WgRaw<D>& r) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  r.at = -1;
  r.weight = 0.f;
  if (page < 0 || page >= a.pages) return;
  const unsigned char* blk = q4_block(const_cast<unsigned char*>(a.cache), page, h, in_page, a.Hkv, a.P, D);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = g + 8 * i;
    const unsigned char* c = blk + tok * (D / 2) + t * (D / 8);
    if constexpr (D == 128) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(c));
      r.code[i][0] = x.x, r.code[i][1] = x.y, r.code[i][2] = x.z, r.code[i][3] = x.w;
      r.scale[i] = __ldg(reinterpret_cast<const uint16_t*>(blk + 32 * D + tok * (D / 16) + t * 2));
    } else {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(c));
      r.code[i][0] = x.x, r.code[i][1] = x.y;
      r.scale[i] = __ldg(blk + 32 * D + tok * (D / 16) + t);
    }
  }
  // the token whose sum this lane ends up with
  const int tok = (t >> 1) * 16 + (t & 1) * 8 + g;
  if (t0 + tok < end) {
    r.at = (static_cast<long long>(page) * a.Hkv + h) * a.P + in_page + tok;
    if (t0 + tok < old) r.weight = from[r.at];
  }
}

// rows 8 j + g of a chunk as f16 operands, and for the lane's columns 8 j + 2 t + e the
// factor to the log2 domain and the row's lse there (infinite: the row adds nothing)
template <int D, int NR>
__device__ __forceinline__ void wg_load_q(const WeighArgs& a, int b, int h, int row0, int rows, uint32_t (&q)[NR][D / 8], float (&f)[NR][2], float (&l)[NR][2]) {
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
    // to [128, 256): what f16 then cannot hold is below 2^-32 of the largest element
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int sh = top > 0.f ? min(7 - ex, 100) : 0;
    const float mul = copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), a.scale_log2);
    const float back = fminf(fmaxf(fabsf(a.scale_log2) * a.k_mul * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23), 1.17549435e-38f), 3.402823466e+38f);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f[j][e] = __shfl_sync(0xffffffffu, back, 8 * t + 4 * e);
      l[j][e] = __shfl_sync(0xffffffffu, lse, 8 * t + 4 * e);
    }
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) q[j][4 * i + k] = f16x2_pack(__uint_as_float(x[k] << 16) * mul, __uint_as_float(x[k] & 0xffff0000u) * mul);
    }
  }
}

// the block's sums over a chunk of rows; the lane gets that of its token.  fresh: the
// position of the block's first token behind the old ones; see: it has such tokens
template <int D, int NR>
__device__ __forceinline__ float wg_block(const WgRaw<D>& r, const uint32_t (&q)[NR][D / 8], const float (&f)[NR][2], const float (&l)[NR][2],
                                          bool see, int fresh, int row0, int G) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float sum[4];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float d[NR][4];
#pragma unroll
    for (int j = 0; j < NR; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
    uint32_t s0 = e4m3x2_to_f16(r.scale[2 * m]), s1 = e4m3x2_to_f16(r.scale[2 * m + 1]);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {   // eight codes of each of two tokens: two steps of 16
      uint32_t lo[4], hi[4];
      e2m1x8_to_f16(r.code[2 * m][i], lo);
      e2m1x8_to_f16(r.code[2 * m + 1][i], hi);
      const uint32_t sel = i < 2 ? 0x1010u : 0x3232u, x0 = __byte_perm(s0, 0u, sel), x1 = __byte_perm(s1, 0u, sel);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo[k] = f16x2_mul(lo[k], x0);
        hi[k] = f16x2_mul(hi[k], x1);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 A = make_uint4(lo[2 * k], hi[2 * k], lo[2 * k + 1], hi[2 * k + 1]);
#pragma unroll
        for (int j = 0; j < NR; ++j) mma_f16(d[j], A, q[j][4 * i + 2 * k], q[j][4 * i + 2 * k + 1]);
      }
    }
    // a score that is no number weighs nothing
    float x[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float z = fmaxf(__fmaf_rn(d[j][e + 2 * u], f[j][e], -l[j][e]), kNegInf);
          if (see && (fresh + 16 * m + 8 * u + g) * G > row0 + 8 * j + 2 * t + e) z = kNegInf;
          x[u] += ex2_approx(z);
        }
    sum[2 * m] = x[0];
    sum[2 * m + 1] = x[1];
  }
  // over the four lanes of a token, each of which keeps one of the four tokens
  const bool up = t & 2, odd = t & 1;
  const float a0 = up ? sum[2] : sum[0], a1 = up ? sum[3] : sum[1], b0 = up ? sum[0] : sum[2], b1 = up ? sum[1] : sum[3];
  const float y0 = a0 + __shfl_xor_sync(0xffffffffu, b0, 2), y1 = a1 + __shfl_xor_sync(0xffffffffu, b1, 2);
  return (odd ? y1 : y0) + __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
}

__host__ __device__ constexpr int wg_ctas(int NR) { return NR <= 2 ? 5 : NR == 3 ? 4 : 3; }

template <int D, int NR>
__global__ void __launch_bounds__(WG_THREADS, wg_ctas(NR)) weigh_q4_kernel(const WeighArgs a) {
  extern __shared__ long long wg_dynamic[];
  __shared__ long long scratch[WG_THREADS / 32];
  long long* prefix = wg_dynamic;                             // [B + 1]
  int* all_rows = reinterpret_cast<int*>(prefix + a.B + 1);   // [B]
  wg_prefix<WG_THREADS>(a, Q4_BLOCK, prefix, all_rows, scratch);
  const long long units = prefix[a.B] * a.Hkv;
  const long long warps = static_cast<long long>(gridDim.x) * (WG_THREADS / 32);
  const long long w = static_cast<long long>(threadIdx.x >> 5) * gridDim.x + blockIdx.x;   // (short lists spread over the SMs)
  const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  const int tok = (t >> 1) * 16 + (t & 1) * 8 + g;
  long long u = units * w / warps;
  const long long u1 = units * (w + 1) / warps;
  while (u < u1) {
    int lo = 0, hi = a.B - 1;   // last b with prefix[b] * Hkv <= u that has blocks
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] * a.Hkv <= u) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, blocks = static_cast<int>(prefix[b + 1] - prefix[b]);
    const long long rem = u - prefix[b] * a.Hkv;
    const int h = static_cast<int>(rem / blocks), k0 = static_cast<int>(rem - static_cast<long long>(h) * blocks);
    const int k1 = static_cast<int>(min(static_cast<long long>(blocks), k0 + (u1 - u)));
    u += k1 - k0;
    const int n = all_rows[b], old = a.lengths[b], end = old + n, rows = n * a.G;
    const int32_t* table = a.table + static_cast<long long>(b) * a.W;
    for (int row0 = 0; row0 == 0 || row0 < rows; row0 += 8 * NR) {
      uint32_t q[NR][D / 8];
      float f[NR][2], l[NR][2];
      wg_load_q<D, NR>(a, b, h, row0, rows, q, f, l);
      const float* from = row0 == 0 ? a.weights : a.new_weights;
      const int begun = row0 == 0 ? old : end;   // tokens that have a weight
      const float decay = row0 == 0 ? a.decay : 1.f;
      WgRaw<D> next;
      int page = table[k0 * Q4_BLOCK / a.P];
      wg_fetch<D>(a, h, page, k0 * Q4_BLOCK % a.P, k0 * Q4_BLOCK, end, begun, from, next);
      page = k0 + 1 < k1 ? table[(k0 + 1) * Q4_BLOCK / a.P] : -1;
      for (int k = k0; k < k1; ++k) {
        const WgRaw<D> now = next;
        const int t0 = k * Q4_BLOCK;
        if (k + 1 < k1) wg_fetch<D>(a, h, page, (t0 + Q4_BLOCK) % a.P, t0 + Q4_BLOCK, end, begun, from, next);
        page = k + 2 < k1 ? table[(t0 + 2 * Q4_BLOCK) / a.P] : -1;
        const float x = wg_block<D, NR>(now, q, f, l, t0 + Q4_BLOCK > old, t0 - old, row0, a.G);
        if (now.at >= 0) {
          a.new_weights[now.at] = t0 + tok < begun ? __fmaf_rn(decay, now.weight, x) : x;
          if (row0 == 0 && a.positions && t0 + tok >= old) a.positions[now.at] = (a.first ? a.first[b] : old) + (t0 + tok - old);
        }
      }
    }
  }
}

}  // namespace sv
