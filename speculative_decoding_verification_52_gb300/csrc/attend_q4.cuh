// attend_q4.cuh -- verification attention over a paged cache held in 4 bits.
//
// N query nodes per sequence (the last token and its drafts: a chain or a tree)
// attend to the sequence's cached tokens and, under the nodes' mask, to the
// fresh bf16 keys and values of the nodes themselves:
//   z = scale * q.k,  out = softmax(z) v,  lse = log(sum exp z).
// The rows of one kv head are its N * G (node, query head) pairs.
//
// Few rows (this kernel).  The cache is read once and each element takes part in
// 2 * rows multiply-adds, so up to a few tens of rows the 9/16 byte an element has
// to cross the HBM bus is the bound; next to it stands the work of unpacking the
// codes, a conversion and a multiplication for two elements.
//
// * The unit of work is a tile of 64 tokens: two blocks, each one contiguous run
//   of 36 * D bytes and one bulk copy.  All tiles of all (sequence, head, row
//   tile) triples form one list, a triple's fresh tiles before its cached ones;
//   every pair of warps takes an equal, contiguous share of it, whatever the
//   lengths, and fetches it through a ring of its own.  A triple that lies in one
//   pair's share is finished there.  A fresh tile counts as three: it waits for
//   its loads, where a cached tile's have arrived (256 sequences of 4 nodes at
//   2,048 tokens, 16 rows: 210 us when it counts as one, 206 as three).  The pairs
//   of a CTA have neighbouring shares and join what they share at the end; what
//   CTAs share goes through the workspace (reference, sum, sum of v) and a second
//   kernel.  All joins are in the list's order.
// * In a pair, each warp scores one block; the weights are exchanged, and each
//   warp adds up one half of v's columns over both blocks.  So every code is
//   unpacked once for all rows, and the sums of a warp fit its registers beside
//   the operands (a warp that kept all columns of 24 rows moved 137 registers a
//   block through local memory and took a seventh longer).  One barrier of the
//   two warps a tile: the weights are 2^(z - ref) for a reference that both know,
//   and only a score above ref + 15 makes them agree on a new one.
// * Everything is unpacked in f16, exactly: a code times its scale has 6
//   significant bits.  q enters as f16 too, scaled by a power of two per row so
//   that its largest element lies in [128, 256): what f16 then cannot hold is
//   below 2^-32 of that element.
// * No unpacked element crosses shared memory.  The products are
//   mma.m16n8k16 with the rows as N, eight at a time: k q^T (tokens as M), then
//   v^T p^T (columns as M).  A thread's part of a key operand is D / 4
//   consecutive elements of one token (the contraction index is permuted alike
//   in q), of a value operand D / 16 consecutive elements of four tokens (the
//   output columns are permuted), with the nibbles of two tokens interleaved
//   before they are widened.  The weights pass from the first product's result
//   to the second's operand by an 8 x 8 transpose across the warp.  The tokens
//   of a group of 8 are taken in the order 0 1 3 2 4 5 7 6, which spreads both
//   kinds of reads over the banks as well as 64-byte rows allow.
// * Measured rates of an SM: mma.m16n8k16 1 per 2 clocks, packed f16
//   multiplications and conversions from e2m1 2 warps a clock each.  A block
//   (D = 128) crosses the bus in about 196 clocks; it takes 128 conversions, 128
//   multiplications (64 clocks each) and 32 products per eight rows (64 clocks).
//   With the rows as M, 16 at a time, eight rows cost 128 clocks of products.
// * The weights of v are f16 of at most 2^15: a weight has 11 significant bits
//   down to 2^-21 of the largest and a step of 2^-31 below.  Sums are fp32.
// * The fresh entries are bf16 with bf16's range, so their blocks use bf16
//   products, with each weight as the sum of two bf16.
#pragma once

#include "common.cuh"
#include "kv_q4.cuh"
#include "q4_ops.cuh"

namespace sv {

constexpr int AT_PAIRS = 2;                 // pairs of warps of a CTA
constexpr int AT_THREADS = 64 * AT_PAIRS;
constexpr int AT_TILE = 2 * Q4_BLOCK;       // tokens of a tile
constexpr int AT_FRESH = 3;                 // what a fresh tile counts in the list, in cached tiles
constexpr int AT_QUEUE = 32;                // places of a pair's list of fetches
constexpr int AT_MAX_B = 4096;
// Weights are 2^(score - reference).  A reference is set so that the largest
// score then known gets the weight 2^7, and serves up to 2^15.
constexpr float AT_PSHIFT = 7.f;
constexpr float AT_ABOVE = 8.f;
constexpr float AT_UNSET = -3.402823466e+38f;   // a reference before any score

struct AttendArgs {
  const uint16_t* q;         // [B, N, Hkv * G, D] bf16
  const uint16_t* k_new;     // [B, N, Hkv, D] bf16 or null
  const uint16_t* v_new;
  const uint32_t* masks;     // [B, N, NW] or null (a chain)
  const unsigned char* cache;
  const int32_t* table;      // [B, W]
  const int32_t* lengths;    // [B]
  int B, N, G, Hkv, P, pages, W, NW;
  int row_tiles;             // row tiles of a (sequence, head)
  uint32_t by_g;             // ceil(2^32 / G), 0 for G = 1: a row r < 65536 is of node r * by_g / 2^32
  int tile;                  // tokens of a tile
  int fresh, fresh_more;     // what a triple's first tile of fresh entries counts in the list, and another one
  float scale_log2;          // scale * log2(e)
  float k_mul, v_mul;        // 2^shift
  uint16_t* out;             // [B, N, Hkv * G, D] bf16
  float* lse;                // [B, N, Hkv * G] or null
  float* ws;
  unsigned long long timeout_ns;
  int stall;                 // test hook: 1 + the CTA whose first stage waits for one arrival too many (0: none)
};

// ---------------------------------------------------------------------------
// the list of work
// ---------------------------------------------------------------------------
// Units of sequence b for one (head, row tile): those of the fresh tiles, then the
// cached tiles; at least one, so that every output is written.
__device__ __forceinline__ bool at_len_ok(const AttendArgs& a, int len) {
  return len >= 0 && static_cast<long long>(len) <= static_cast<long long>(a.W) * a.P;
}
__device__ __forceinline__ int at_fresh_units(const AttendArgs& a) {
  return a.k_new ? a.fresh + a.fresh_more * ((a.N + a.tile - 1) / a.tile - 1) : 0;
}
__device__ __forceinline__ int at_units(const AttendArgs& a, int len) {
  if (!at_len_ok(a, len)) return 1;
  const int n = (len + a.tile - 1) / a.tile + at_fresh_units(a);
  return n > 0 ? n : 1;
}

// prefix[b] = units of sequences 0..b-1 (one head and row tile), prefix[B] the sum
template <int THREADS>
__device__ void at_prefix(const AttendArgs& a, long long* prefix, long long* scratch) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    long long v = b < a.B ? at_units(a, a.lengths[b]) : 0;
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

// position in the list
struct AtCursor {
  int b, pair, i, units;   // sequence, (head, row tile) of it, unit of it, its units
  int len;
};
__device__ __forceinline__ void at_seek(const AttendArgs& a, const long long* prefix, int HR, long long u, AtCursor& c) {
  int lo = 0, hi = a.B - 1;   // last b with prefix[b] * HR <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] * HR <= u) lo = mid;
    else hi = mid - 1;
  }
  c.b = lo;
  c.len = a.lengths[lo];
  c.units = static_cast<int>(prefix[lo + 1] - prefix[lo]);
  const long long rem = u - prefix[lo] * HR;
  c.pair = static_cast<int>(rem / c.units);
  c.i = static_cast<int>(rem - static_cast<long long>(c.pair) * c.units);
}
__device__ __forceinline__ void at_next(const AttendArgs& a, const long long* prefix, int HR, AtCursor& c) {
  if (++c.i < c.units) return;
  c.i = 0;
  if (++c.pair < HR) return;
  c.pair = 0;
  if (++c.b >= a.B) return;
  c.len = a.lengths[c.b];
  c.units = static_cast<int>(prefix[c.b + 1] - prefix[c.b]);
}

// CTAs that get work: the list is cut in `shares` parts a CTA, none of the CTAs empty
__device__ __forceinline__ int at_active(long long units, int ctas, int shares) {
  return static_cast<int>(min((units + shares - 1) / shares, static_cast<long long>(ctas)));
}
// share w of n of a list of `units`: [at_start(w), at_start(w + 1)), and the share that unit u falls in
__device__ __forceinline__ long long at_start(long long units, int n, long long w) { return units * w / n; }
__device__ __forceinline__ int at_owner(long long units, int n, long long u) {
  return static_cast<int>(((u + 1) * n - 1) / units);
}

// ---------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------
// factor that takes sums from an old maximum to a new one; never zero, so that
// an infinite sum stays one
__device__ __forceinline__ float at_corr(float d) { return fmaxf(ex2_approx(d), 1.17549435e-38f); }
// token of a group of 8 that column j of a product stands for
__device__ __forceinline__ int at_token(int j) { return j ^ ((j >> 1) & 1); }

// 8 x 8 matrix of 16-bit elements, transposed across the warp's fragments
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__host__ __device__ constexpr int at_stage_bytes(int D) { return 2 * q4_block_bytes(D); }
// of a pair: the queries' operand; in exchange, two buffers each, the weights
// (each warp's operands), the maxima or sums, and the flags; a flag a stage (at
// most 8); the list of fetches
__host__ __device__ constexpr int at_q_bytes(int D, int NR) { return NR * (D / 32) * 512; }
__host__ __device__ constexpr int at_p_bytes(int NR) { return 2 * 2 * 2 * NR * 256; }
__host__ __device__ constexpr int at_m_bytes(int NR) { return 2 * 2 * 8 * NR * 4; }
__host__ __device__ constexpr int at_pair_bytes(int D, int NR) { return at_q_bytes(D, NR) + at_p_bytes(NR) + at_m_bytes(NR) + 64 + 8 * AT_QUEUE; }
// The workspace.  A CTA has two partials, of the triple that it shares with the
// CTAs before it and of the one that it shares with those behind:
//   [8 NR rows x D] sums of v, then m[8 NR], l[8 NR] of the first and the second
//   half of the columns' warps;
// a warp has a state in its lanes' order, which its CTA's other pairs join.
__host__ __device__ constexpr size_t at_partial_floats(int D, int NR) { return static_cast<size_t>(8 * NR) * (D + 4); }
__host__ __device__ constexpr size_t at_state_floats(int D, int NR) { return static_cast<size_t>(32 * NR) * (D / 8 + 4); }
__host__ __device__ constexpr size_t at_cta_floats(int D, int NR) {
  return 2 * at_partial_floats(D, NR) + 2 * AT_PAIRS * at_state_floats(D, NR);
}

__device__ __forceinline__ int at_node(const AttendArgs& a, int r) { return a.by_g ? static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.by_g)) : r; }
__device__ __forceinline__ long long at_row(const AttendArgs& a, int b, int h, int r) {
  const int n = at_node(a, r);
  return (static_cast<long long>(b) * a.N + n) * (a.Hkv * a.G) + (h * a.G + r - n * a.G);
}

// ---------------------------------------------------------------------------
// the state of one (sequence, head, row tile) in a warp's registers: warp x of
// the pair, lane (g, t) holds rows 8 j + 2 t + e and the D / 16 columns from
// x * D / 2 + g * D / 16
// ---------------------------------------------------------------------------
template <int D, int NR>
struct AtState {
  static constexpr int MT = D / 32;   // products that cover the warp's columns
  float o[NR][MT][4];                 // [.][i][e + 2 f]: column 2 i + f of the lane's
  float ref[NR][2];                   // the references (log2 domain; the pair's)
  float l[NR][2];                     // this lane's part of the sum of weights

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NR; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][i][k] = 0.f;
      ref[j][0] = ref[j][1] = AT_UNSET;
      l[j][0] = l[j][1] = 0.f;
    }
  }
  __device__ __forceinline__ void poison() {
#pragma unroll
    for (int j = 0; j < NR; ++j) l[j][0] = l[j][1] = __int_as_float(0x7fc00000);
  }
  // to a reference of `to` (not below the present one)
  __device__ __forceinline__ void raise(int j, int e, float to) {
    const float corr = at_corr(ref[j][e] - to);
    l[j][e] *= corr;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      o[j][i][e] *= corr;
      o[j][i][e + 2] *= corr;
    }
    ref[j][e] = to;
  }

  // the state in the order of its lanes: only the lane that wrote a value reads it
  // (or the same lane of the same half in another pair)
  __device__ __forceinline__ void save(float* p) const {
    float4* q = reinterpret_cast<float4*>(p) + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) q[32 * (j * (MT + 1) + i)] = make_float4(o[j][i][0], o[j][i][1], o[j][i][2], o[j][i][3]);
      q[32 * (j * (MT + 1) + MT)] = make_float4(ref[j][0], ref[j][1], l[j][0], l[j][1]);
    }
  }
  // joins a saved state of the same rows
  __device__ __forceinline__ void join(const float* p) {
    const float4* q = reinterpret_cast<const float4*>(p) + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const float4 x = q[32 * (j * (MT + 1) + MT)];
      const float pm[2] = {x.x, x.y}, pl[2] = {x.z, x.w};
      float c1[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float to = fmaxf(ref[j][e], pm[e]);
        raise(j, e, to);
        c1[e] = at_corr(pm[e] - to);
        l[j][e] += pl[e] * c1[e];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const float4 y = q[32 * (j * (MT + 1) + i)];
        o[j][i][0] += y.x * c1[0];
        o[j][i][1] += y.y * c1[1];
        o[j][i][2] += y.z * c1[0];
        o[j][i][3] += y.w * c1[1];
      }
    }
  }
};

constexpr int AT_STUCK = 1 << 8;

// What the two warps of a pair share.
template <int D, int NR>
struct AtPair {
  unsigned char* base;   // of the pair's exchange area
  int x, id;             // the warp's half; the pair's named barrier
  __device__ __forceinline__ uint4* q() const { return reinterpret_cast<uint4*>(base); }
  // a warp's operands of one buffer: [2 steps][NR][32 lanes]
  __device__ __forceinline__ uint2* p(int buf, int warp) const {
    return reinterpret_cast<uint2*>(base + at_q_bytes(D, NR)) + (buf * 2 + warp) * 2 * NR * 32;
  }
  __device__ __forceinline__ float* top(int buf, int warp) const {
    return reinterpret_cast<float*>(base + at_q_bytes(D, NR) + at_p_bytes(NR)) + (buf * 2 + warp) * 8 * NR;
  }
  __device__ __forceinline__ int* flag(int buf, int warp) const {
    return reinterpret_cast<int*>(base + at_q_bytes(D, NR) + at_p_bytes(NR) + at_m_bytes(NR)) + buf * 2 + warp;
  }
  __device__ __forceinline__ int* arrived(int stage) const { return flag(2, 0) + stage; }
  __device__ __forceinline__ uint2* queue() const {
    return reinterpret_cast<uint2*>(base + at_q_bytes(D, NR) + at_p_bytes(NR) + at_m_bytes(NR) + 64);
  }
  __device__ __forceinline__ void sync() const { named_bar_sync(id, 64); }
};

// Queries of a row tile: the f16 operand into `qf` (the same lanes of both warps
// read what one of them wrote), the rows' factors from f16 products to the log2
// domain into c.
template <int D, int NR>
__device__ __forceinline__ void at_load_q(const AttendArgs& a, int b, int h, int row0, int rows, const AtPair<D, NR>& pr, float (&c)[NR][2]) {
  constexpr int CH = D / 4, WK = D / 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int r = row0 + 8 * j + g;
    uint4 w[CH / 8];
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const uint4* p = reinterpret_cast<const uint4*>(a.q + at_row(a, b, h, r) * D + t * CH);
#pragma unroll
      for (int i = 0; i < CH / 8; ++i) w[i] = __ldg(p + i);
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
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int sh = top > 0.f ? min(7 - ex, 100) : 0;
    // (the factor is above zero, so that products compare as scores do: the
    // scale's sign goes into the operand, and no scale at all becomes a tiny one)
    const float mul = copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), a.scale_log2);
    // A row with a NaN has no other scores, and the factor says so.  (An infinity makes
    // infinite ones of either sign, whatever the finite elements have become.)  A finite
    // factor leaves a score of 0 what it is.
    const float f = top <= __builtin_huge_valf()
                        ? fminf(fmaxf(fabsf(a.scale_log2) * a.k_mul * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23), 1.17549435e-38f),
                                3.402823466e+38f)
                        : __int_as_float(0x7fc00000);
    c[j][0] = __shfl_sync(0xffffffffu, f, 8 * t);
    c[j][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = f16x2_pack(__uint_as_float(x[k] << 16) * mul, __uint_as_float(x[k] & 0xffff0000u) * mul);
      if (pr.x == 0) pr.q()[(j * WK + i) * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  pr.sync();
}

// The codes of one product step of v (16 tokens), widened and scaled: w[k] the
// lane's codes of tokens 2t, 2t+1 of the two groups of eight, BYTES bytes of them
// from byte `from`; s01, s23 their scales.
template <int BYTES, int NR, int MT>
__device__ __forceinline__ void at_add_v(const uint32_t (&w)[4], int from, uint32_t s01, uint32_t s23, const uint2 (&p)[NR],
                                         float (&o)[NR][MT][4]) {
  uint32_t e01[4], o01[4], e23[4], o23[4];
  e2m1x8_to_f16((w[0] & 0x0f0f0f0fu) | ((w[1] << 4) & 0xf0f0f0f0u), e01);
  e2m1x8_to_f16(((w[0] >> 4) & 0x0f0f0f0fu) | (w[1] & 0xf0f0f0f0u), o01);
  e2m1x8_to_f16((w[2] & 0x0f0f0f0fu) | ((w[3] << 4) & 0xf0f0f0f0u), e23);
  e2m1x8_to_f16(((w[2] >> 4) & 0x0f0f0f0fu) | (w[3] & 0xf0f0f0f0u), o23);
#pragma unroll
  for (int i = 0; i < BYTES; ++i) {
    const int y = from + i;
    const uint4 v = make_uint4(f16x2_mul(e01[y], s01), f16x2_mul(o01[y], s01), f16x2_mul(e23[y], s23), f16x2_mul(o23[y], s23));
#pragma unroll
    for (int j = 0; j < NR; ++j) mma_f16(o[j][i], v, p[j].x, p[j].y);
  }
}

// The products of 16 tokens of a block (16 mt ...; own: the sequence's tokens of it)
// with the rows: z[.][e + 2 f], row 2 t + e, token g of the f-th eight.
template <int D, int NR>
__device__ __forceinline__ void at_scores(const unsigned char* sb, const uint4* qf, int mt, int own, float (&z)[NR][4]) {
  constexpr int WK = D / 32;   // words of a key chunk
  const int lane = threadIdx.x & 31, t = lane & 3, tr = at_token(lane >> 2);
  uint32_t kw[2][WK];
  uint32_t ks2[2][D / 64];   // the chunk's scales, each twice
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int tok = 16 * mt + 8 * f + tr;
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(sb + tok * 64 + t * 16);
      kw[f][0] = x.x; kw[f][1] = x.y; kw[f][2] = x.z; kw[f][3] = x.w;
      const uint32_t two = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(sb + 32 * D + tok * 8 + t * 2));
      ks2[f][0] = __byte_perm(two, two, 0x1010);
      ks2[f][1] = __byte_perm(two, two, 0x3232);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(sb + tok * 32 + t * 8);
      kw[f][0] = x.x; kw[f][1] = x.y;
      const uint32_t one = sb[32 * D + tok * 4 + t];
      ks2[f][0] = e4m3x2_to_f16(one * 0x101u);
    }
  }
#pragma unroll
  for (int w = 0; w < WK; ++w) {
    uint32_t r0[4], r1[4];   // tokens g and g + 8
    e2m1x8_to_f16(kw[0][w], r0);
    e2m1x8_to_f16(kw[1][w], r1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r0[i] = f16x2_mul(r0[i], ks2[0][w / 2]);
      r1[i] = f16x2_mul(r1[i], ks2[1][w / 2]);
    }
    const uint4 k0 = make_uint4(r0[0], r1[0], r0[1], r1[1]), k1 = make_uint4(r0[2], r1[2], r0[3], r1[3]);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const uint4 qb = qf[(j * WK + w) * 32];
      if (w == 0) mma_f16_zero(z[j], k0, qb.x, qb.y);
      else mma_f16(z[j], k0, qb.x, qb.y);
      mma_f16(z[j], k1, qb.z, qb.w);
    }
  }
  if (own < 16 * mt + 16) {   // the sequence ends here (what the stage holds behind it may be anything)
#pragma unroll
    for (int f = 0; f < 2; ++f)
      if (16 * mt + 8 * f + tr >= own) {
#pragma unroll
        for (int j = 0; j < NR; ++j) z[j][2 * f] = z[j][2 * f + 1] = kNegInf;
      }
  }
}

// New references for the pair, of a tile with a score too far above an old one.
// mx: the lane's largest products of the warp's block.  (Arrays are copies, so that
// the state stays in registers.)
template <int D, int NR>
__device__ __noinline__ void at_agree(const AtPair<D, NR>& pr, int buf, const float* mx, const float* c, const float* ref, float* to) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2 * NR; ++i) {
    float m = mx[i];
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if (g == 0) pr.top(buf, pr.x)[8 * (i >> 1) + 2 * t + (i & 1)] = m * c[i];
  }
  pr.sync();
#pragma unroll
  for (int i = 0; i < 2 * NR; ++i) {
    const int r = 8 * (i >> 1) + 2 * t + (i & 1);
    to[i] = fmaxf(ref[i], fmaxf(pr.top(buf, 0)[r], pr.top(buf, 1)[r]) - AT_PSHIFT);
  }
  pr.sync();   // the maxima have been read, and what follows is written anew
}

// A cached tile: `left` tokens of it (1..64) belong to the sequence.  `after` runs
// once both warps are done with the tile before.
//
// Both halves of the work are loops over 16 tokens, unrolled where the registers hold
// what that interleaves and the code of a tile stays small: up to 8 KB a warp gets
// through it at about the rate of its scheduler, at 16 KB it takes 2.7 clocks an
// instruction to fetch.  256 sequences at 2,048 tokens, D = 128: 32 rows unrolled 347
// us, rolled 360; 24 rows two steps at a time 281, rolled 277; 16 rows unrolled 206, two
// steps 214; 8 rows unrolled 155, rolled 169.  D = 64: 32 rows rolled 244, two steps 257;
// 24 rows two steps 197, rolled 207; 8 rows unrolled 119, rolled 128.  So that they can be
// loops, the weights are taken at once against the references as they are, and
// only then the warps look whether a score was too far above one; if so, they agree on
// new references and score the tile again.
//
// (The exchange area has two buffers, taken in turn: with one barrier a tile, what a
// warp writes for a tile was last read two barriers before.)
__host__ __device__ constexpr int at_unroll(int D, int NR) { return NR == 1 ? 4 : D == 64 ? (NR < 4 ? 2 : 1) : NR == 3 ? 1 : 4; }
template <int D, int NR, class F>
__device__ __forceinline__ void at_cached_tile(const unsigned char* tile, int left, int buf, const float (&c)[NR][2],
                                               const AtPair<D, NR>& pr, AtState<D, NR>& st, F&& after) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int own = left - pr.x * Q4_BLOCK;   // tokens of the warp's block
  const unsigned char* sb = tile + pr.x * q4_block_bytes(D);
  uint2* out = pr.p(buf, pr.x) + lane;
  float lt[NR][2];
  for (;;) {
    float mx[NR][2];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        lt[j][e] = 0.f;
        mx[j][e] = kNegInf;
      }
#pragma unroll at_unroll(D, NR)
    for (int mt = 0; mt < 2; ++mt) {
      float z[NR][4];
      at_scores<D, NR>(sb, pr.q() + lane, mt, own, z);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[j][e] = fmaxf(mx[j][e], fmaxf(z[j][e], z[j][e + 2]));
          // (the product is rounded as the reference was: a fused one would leave half a
          // step of a score, which is beyond any weight for scores above 2^28)
          z[j][e] = ex2_approx(__fsub_rn(__fmul_rn(z[j][e], c[j][e]), st.ref[j][e]));
          z[j][e + 2] = ex2_approx(__fsub_rn(__fmul_rn(z[j][e + 2], c[j][e]), st.ref[j][e]));
          lt[j][e] += z[j][e] + z[j][e + 2];
        }
        out[(mt * NR + j) * 32] = make_uint2(transpose8(f16x2_pack(z[j][0], z[j][1])), transpose8(f16x2_pack(z[j][2], z[j][3])));
      }
    }
    bool above = false;
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) above |= __fmul_rn(mx[j][e], c[j][e]) - AT_PSHIFT > st.ref[j][e] + AT_ABOVE;
    above = __any_sync(0xffffffffu, above);
    if (lane == 0) *pr.flag(buf, pr.x) = above;
    pr.sync();
    if (__builtin_expect(!above && !*pr.flag(buf, pr.x ^ 1), 1)) break;
    float m2[2 * NR], c2[2 * NR], ref[2 * NR], to[2 * NR];
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i) {
      m2[i] = mx[i >> 1][i & 1];
      c2[i] = c[i >> 1][i & 1];
      ref[i] = st.ref[i >> 1][i & 1];
    }
    at_agree<D, NR>(pr, buf, m2, c2, ref, to);
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i) st.raise(i >> 1, i & 1, to[i]);
  }
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) st.l[j][e] += lt[j][e];
  after();

  // v: steps of 16 tokens (D = 128), or of 32 (D = 64, whose codes of two steps make a word)
  constexpr int STEPS = D == 128 ? 4 : 2, S = 4 / STEPS;
#pragma unroll at_unroll(D, NR)
  for (int y = 0; y < STEPS; ++y) {
    const int blk = y / (STEPS / 2), s0 = D == 128 ? y & 1 : 0;
    const int have = left - blk * Q4_BLOCK;   // tokens of that block
    if (have <= 16 * s0) break;
    const unsigned char* vb = tile + blk * q4_block_bytes(D);
    const uint2* in = pr.p(buf, blk) + lane;
    uint2 p[S][NR];
    uint32_t w[S][4], sc[S][4];
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < NR; ++j) p[s][j] = in[((s0 + s) * NR + j) * 32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = 16 * (s0 + s) + 8 * (k >> 1) + at_token(2 * t + (k & 1));
        if constexpr (D == 128) {
          w[s][k] = *reinterpret_cast<const uint32_t*>(vb + 16 * D + tok * 64 + pr.x * 32 + g * 4);
          sc[s][k] = vb[34 * D + tok * 8 + pr.x * 4 + (g >> 1)];
        } else {
          w[s][k] = *reinterpret_cast<const uint16_t*>(vb + 16 * D + tok * 32 + pr.x * 16 + g * 2);
          sc[s][k] = vb[34 * D + tok * 4 + pr.x * 2 + (g >> 2)];
        }
      }
      if (have < 16 * (s0 + s) + 16) {   // what lies behind the last token may be a NaN
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (16 * (s0 + s) + 8 * (k >> 1) + at_token(2 * t + (k & 1)) >= have) sc[s][k] = 0u;
      }
    }
    if constexpr (D == 128) {
      at_add_v<4, NR>(w[0], 0, e4m3x2_to_f16(sc[0][0] + sc[0][1] * 256u), e4m3x2_to_f16(sc[0][2] + sc[0][3] * 256u), p[0], st.o);
    } else {
      uint32_t both[4];   // the codes of both steps, widened at once
#pragma unroll
      for (int k = 0; k < 4; ++k) both[k] = w[0][k] + w[S - 1][k] * 65536u;
#pragma unroll
      for (int s = 0; s < S; ++s)
        at_add_v<2, NR>(both, 2 * s, e4m3x2_to_f16(sc[s][0] + sc[s][1] * 256u), e4m3x2_to_f16(sc[s][2] + sc[s][3] * 256u), p[s], st.o);
    }
  }
}

__device__ __forceinline__ bool bf16x2_unbounded(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// A tile of fresh entries: nodes j0 .. j0 + 63.  Unlike in a cached tile, the
// references follow the maxima.
template <int D, int NR>
__device__ __forceinline__ void at_fresh_tile(const AttendArgs& a, int b, int h, int row0, int rows, int j0,
                                              const AtPair<D, NR>& pr, AtState<D, NR>& st) {
  constexpr int CH = D / 4, KS = D / 16, CV = D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tr = at_token(g);
  const long long rstride = static_cast<long long>(a.Hkv) * D;
  const long long base = (static_cast<long long>(b) * a.N * a.Hkv + h) * D;   // node 0's entry
  float z[2][NR][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[mt][j][k] = 0.f;
  long long qat[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) qat[j] = row0 + 8 * j + g < rows ? at_row(a, b, h, row0 + 8 * j + g) * D + t * CH : -1;
  const int jx = j0 + pr.x * Q4_BLOCK;   // the warp's nodes
  // (most tiles have few nodes and wait for their loads: what can be asked for
  // early is)
  uint32_t sees[NR][2][2];   // nodes of the tile that the lane's rows attend to
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = at_node(a, row0 + 8 * j + 2 * t + e);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int at = j0 + y * Q4_BLOCK;
        uint32_t see = 0u;
        if (n < a.N && at < a.N) {
          if (a.masks) see = __ldg(a.masks + (static_cast<long long>(b) * a.N + n) * a.NW + at / 32);
          else see = n - at >= 31 ? ~0u : n < at ? 0u : (2u << (n - at)) - 1u;
        }
        sees[j][e][y] = see;
      }
    }
  if (j0 + lane < a.N) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.v_new + base + (j0 + lane) * rstride + pr.x * (D / 2)));
  if (jx < a.N) {
#pragma unroll 2
    for (int ks = 0; ks < KS; ++ks) {
      uint2 qb[NR];
#pragma unroll
      for (int j = 0; j < NR; ++j)
        qb[j] = qat[j] >= 0 ? __ldg(reinterpret_cast<const uint2*>(a.q + qat[j] + 4 * ks)) : make_uint2(0u, 0u);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        if (mt == 1 && jx + 16 >= a.N) break;
        uint2 kx[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int n = jx + 16 * mt + 8 * f + tr;
          kx[f] = n < a.N ? __ldg(reinterpret_cast<const uint2*>(a.k_new + base + n * rstride + t * CH + 4 * ks)) : make_uint2(0u, 0u);
        }
        const uint4 k = make_uint4(kx[0].x, kx[1].x, kx[0].y, kx[1].y);
#pragma unroll
        for (int j = 0; j < NR; ++j) mma_bf16(z[mt][j], k, qb[j].x, qb[j].y);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {   // (no node behind the last)
        const int behind = a.N - j0 - y * Q4_BLOCK;
        if (behind < 32) sees[j][e][y] &= behind > 0 ? (1u << behind) - 1u : 0u;
      }
      const uint32_t see = pr.x ? sees[j][e][1] : sees[j][e][0];
      float m = kNegInf;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float& x = z[mt][j][e + 2 * f];
          x = (see >> (16 * mt + 8 * f + tr)) & 1u ? x * a.scale_log2 : kNegInf;
          m = fmaxf(m, x);
        }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if (g == 0) pr.top(0, pr.x)[8 * j + 2 * t + e] = m;
    }
  pr.sync();
  // the sums of v are kept in units of 2^v_shift
  const float unit = __fdiv_rn(1.f, a.v_mul);
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * j + 2 * t + e;
      st.raise(j, e, fmaxf(st.ref[j][e], fmaxf(pr.top(0, 0)[r], pr.top(0, 1)[r]) - AT_PSHIFT));
      const float ref = st.ref[j][e];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int f = 0; f < 2; ++f) z[mt][j][e + 2 * f] = ex2_approx(z[mt][j][e + 2 * f] - ref);
      st.l[j][e] += (z[0][j][e] + z[0][j][e + 2]) + (z[1][j][e] + z[1][j][e + 2]);
    }
  // weights as the sum of two bf16: buffer 0 the larger parts, buffer 1 the rest
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const float x = z[s][j][2 * f] * unit, y = z[s][j][2 * f + 1] * unit;
        hi[f] = bf16x2_pack(x, y);
        lo[f] = transpose8(bf16x2_pack(x - __uint_as_float(hi[f] << 16), y - __uint_as_float(hi[f] & 0xffff0000u)));
        hi[f] = transpose8(hi[f]);
      }
      pr.p(0, pr.x)[(s * NR + j) * 32 + lane] = make_uint2(hi[0], hi[1]);
      pr.p(1, pr.x)[(s * NR + j) * 32 + lane] = make_uint2(lo[0], lo[1]);
    }
  pr.sync();
#pragma unroll 1
  for (int y = 0; y < 4; ++y) {   // 16 nodes at a time
    const int blk = y >> 1, s = y & 1, n0 = j0 + 16 * y;
    if (n0 >= a.N) break;
    uint2 hi[NR], lo[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      hi[j] = pr.p(0, blk)[(s * NR + j) * 32 + lane];
      lo[j] = pr.p(1, blk)[(s * NR + j) * 32 + lane];
    }
    uint32_t most = 0u, vw[4][CV / 2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + 8 * (k >> 1) + at_token(2 * t + (k & 1));
      const uint16_t* from = a.v_new + base + n * rstride + pr.x * (D / 2) + g * CV;
      if constexpr (D == 128) {
        const uint4 x = n < a.N ? __ldg(reinterpret_cast<const uint4*>(from)) : make_uint4(0u, 0u, 0u, 0u);
        vw[k][0] = x.x; vw[k][1] = x.y; vw[k][2] = x.z; vw[k][3] = x.w;
      } else {
        const uint2 x = n < a.N ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0u, 0u);
        vw[k][0] = x.x; vw[k][1] = x.y;
      }
#pragma unroll
      for (int i = 0; i < CV / 2; ++i) most = bf16x2_max_nan(most, vw[k][i] & 0x7fff7fffu);
    }
    const bool odd = bf16x2_unbounded(most);   // this lane saw a NaN or an infinity
    if (__builtin_expect(odd, 0)) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < CV / 2; ++i) {
          if ((vw[k][i] & 0x7f80u) == 0x7f80u) vw[k][i] &= 0xffff0000u;
          if ((vw[k][i] & 0x7f800000u) == 0x7f800000u) vw[k][i] &= 0xffffu;
        }
    }
#pragma unroll
    for (int i = 0; i < CV / 2; ++i) {
      const uint4 v = make_uint4(__byte_perm(vw[0][i], vw[1][i], 0x5410), __byte_perm(vw[0][i], vw[1][i], 0x7632),
                                 __byte_perm(vw[2][i], vw[3][i], 0x5410), __byte_perm(vw[2][i], vw[3][i], 0x7632));
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        mma_bf16(st.o[j][i], v, hi[j].x, hi[j].y);
        mma_bf16(st.o[j][i], v, lo[j].x, lo[j].y);
      }
    }
    // A product takes 0 * inf for NaN, so such elements were left out above and
    // reach only the rows that see their node (with a weight above zero, however
    // small: a weight that underflowed counts as the smallest one).
    if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
      for (int k = 0; k < 16; ++k) {
        const int n = n0 + (k & 8) + at_token(k & 7);
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // row 2 t + e of the operand is in lanes of that row, column k in their lane (k & 7) / 2
            const uint32_t w = __shfl_sync(0xffffffffu, k & 8 ? hi[j].y : hi[j].x, 4 * (2 * t + e) + ((k & 7) >> 1));
            const float p = __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
            const uint32_t see = blk ? sees[j][e][1] : sees[j][e][0];
            if (n >= a.N || !((see >> (n - j0 - blk * Q4_BLOCK)) & 1u)) continue;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const uint32_t v = a.v_new[base + n * rstride + pr.x * (D / 2) + g * CV + 2 * i + f];
                if ((v & 0x7f80u) == 0x7f80u) st.o[j][i][e + 2 * f] += (p == 0.f ? 1.17549435e-38f : p) * __uint_as_float(v << 16);
              }
          }
      }
    }
  }
  pr.sync();   // the exchange area is free again
}

__device__ __forceinline__ float at_lse(float ref, float l) {
  return l == 0.f ? kNegInf : (ref + log2f(l)) * 0.69314718055994530942f;   // l: the sum of weights, relative to 2^ref
}

// CTAs an SM, of four warps: what the registers of a row tile leave room for.  256
// sequences at 2,048 tokens, D = 128: 32 rows 347 us with two, 437 with three (part of
// the sums in local memory, for which the shared memory in use leaves little cache); 24
// rows 277 with three, 305 with two; 16 rows 206 with three, 212 with four.  D = 64, half
// the sums: 32 rows 244 us with three, 258 with two; 24 rows 197 and 209.
__host__ __device__ constexpr int at_ctas(int D, int NR) { return NR == 1 ? 4 : D == 64 ? (NR == 2 ? 4 : 3) : NR < 4 ? 3 : 2; }

// the warp's part of a row's sum of weights
__device__ __forceinline__ float at_sum(float l) {
  l += __shfl_xor_sync(0xffffffffu, l, 4);
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  return l;
}
// the lane's rows and columns of a finished state (both warps of the pair call this)
template <int D, int NR>
__device__ __forceinline__ void at_write(const AttendArgs& a, int b, int h, int row0, int rows, const AtPair<D, NR>& pr,
                                         const AtState<D, NR>& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float l[NR][2];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[j][e] = at_sum(st.l[j][e]);
      if (g == 0) pr.top(0, pr.x)[8 * j + 2 * t + e] = l[j][e];
    }
  pr.sync();
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + 8 * j + 2 * t + e;
      if (r >= rows) continue;
      const float sum = pr.top(0, 0)[8 * j + 2 * t + e] + pr.top(0, 1)[8 * j + 2 * t + e];
      const long long at = at_row(a, b, h, r);
      const float inv = sum == 0.f ? 0.f : a.v_mul / sum;
      uint32_t w[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[i] = bf16x2_pack(st.o[j][i][e] * inv, st.o[j][i][e + 2] * inv);
      uint16_t* to = a.out + at * D + pr.x * (D / 2) + g * (D / 16);
      if constexpr (D == 128) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      if (a.lse && pr.x == 0 && g == 0) a.lse[at] = at_lse(st.ref[j][e], sum);
    }
  pr.sync();   // the exchange area is free again
}
// the same as a partial
template <int D, int NR>
__device__ __forceinline__ void at_write_partial(float* part, const AtPair<D, NR>& pr, const AtState<D, NR>& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float l = at_sum(st.l[j][e]);
      const int lr = 8 * j + 2 * t + e;
      float* to = part + static_cast<size_t>(lr) * D + pr.x * (D / 2) + g * (D / 16);
#pragma unroll
      for (int i = 0; i < D / 32; i += 2)
        *reinterpret_cast<float4*>(to + 2 * i) = make_float4(st.o[j][i][e], st.o[j][i][e + 2], st.o[j][i + 1][e], st.o[j][i + 1][e + 2]);
      if (g == 0) {
        if (pr.x == 0) part[8 * NR * D + lr] = st.ref[j][e];
        part[8 * NR * D + 8 * NR * (1 + pr.x) + lr] = l;
      }
    }
}

// A place of a pair's list of fetches: the blocks of a cached tile in the cache,
// the second AT_NONE where it lies behind the sequence's last token; AT_NONE for
// a unit without a cached tile, AT_BAD for a page id out of range.
constexpr uint32_t AT_NONE = 0xffffffffu, AT_BAD = 0xfffffffeu;
__device__ __forceinline__ uint2 at_source(const AttendArgs& a, const long long* prefix, int HR, int nfresh, long long u) {
  AtCursor c;
  at_seek(a, prefix, HR, u, c);
  uint2 r = make_uint2(AT_NONE, AT_NONE);
  const int blk = 2 * (c.i - AT_FRESH * nfresh), bpp = a.P / Q4_BLOCK;
  if (!at_len_ok(a, c.len) || blk < 0 || blk * Q4_BLOCK >= c.len) return r;
  const int head = c.pair / a.row_tiles;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int x = blk + k;
    if (x * Q4_BLOCK >= c.len) break;
    const int page = __ldg(a.table + static_cast<long long>(c.b) * a.W + x / bpp);
    const uint32_t at = page >= 0 && page < a.pages ? (static_cast<uint32_t>(page) * a.Hkv + head) * bpp + x % bpp : AT_BAD;
    if (at == AT_BAD) r.x = AT_BAD;
    else if (k == 0) r.x = at;
    else r.y = at;
  }
  return r;
}

// Once one of the pair's waits has failed: waits until no copy is on its way to the
// stages, or, where some never came or none was started, for the limit once more.  (What
// was started and not waited for is the next phase of its stage.)
__device__ __noinline__ void at_drain(uint64_t* bars, int stages, uint32_t phase, unsigned long long limit) {
  const uint64_t t0 = global_ns();
  uint32_t open = (1u << stages) - 1u;
  for (int i = 0; i < (1 << 24) && open; ++i) {
    for (int s = 0; s < stages; ++s)
      if (((open >> s) & 1u) && mbar_try_wait(&bars[s], (phase >> s) & 1u)) open ^= 1u << s;
    if (global_ns() - t0 > limit) return;
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(AT_THREADS, at_ctas(D, NR)) attend_q4_kernel(const __grid_constant__ AttendArgs a, int stages) {
  extern __shared__ __align__(128) unsigned char at_smem[];
  __shared__ long long scratch[AT_THREADS / 32];
  __shared__ int stuck[AT_PAIRS];   // AT_STUCK and the stages' phases at the time, once a wait of the first warp has failed
  constexpr int SB = at_stage_bytes(D), BB = q4_block_bytes(D);
  const int pair = threadIdx.x >> 6;
  unsigned char* ring = at_smem + static_cast<size_t>(pair) * stages * SB;
  AtPair<D, NR> pr;
  pr.base = at_smem + static_cast<size_t>(AT_PAIRS) * stages * SB + pair * at_pair_bytes(D, NR);
  pr.x = (threadIdx.x >> 5) & 1;
  pr.id = 1 + pair;
  uint64_t* bars = reinterpret_cast<uint64_t*>(at_smem + static_cast<size_t>(AT_PAIRS) * (stages * SB + at_pair_bytes(D, NR))) + pair * stages;
  long long* prefix = reinterpret_cast<long long*>(at_smem + static_cast<size_t>(AT_PAIRS) * (stages * SB + at_pair_bytes(D, NR))) + AT_PAIRS * stages;

  if ((threadIdx.x & 63) == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
    if (a.stall == static_cast<int>(blockIdx.x) + 1 && pair == 0) mbar_init(&bars[0], 2);   // (test hook)
    stuck[pair] = 0;
    mbar_fence_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the join kernel may start; it waits for this grid's end)
  at_prefix<AT_THREADS>(a, prefix, scratch);   // (synchronises the CTA)

  const int HR = a.Hkv * a.row_tiles;
  const long long units = prefix[a.B] * HR;
  const int ctas = at_active(units, gridDim.x, AT_PAIRS);
  if (blockIdx.x >= ctas) return;
  const int shares = ctas * AT_PAIRS, share = blockIdx.x * AT_PAIRS + pair;
  const long long u0 = at_start(units, shares, share), u1 = at_start(units, shares, share + 1);
  float* cta_ws = a.ws + static_cast<size_t>(blockIdx.x) * at_cta_floats(D, NR);
  float* states = cta_ws + 2 * at_partial_floats(D, NR);   // [pair][x]

  const int rows = a.N * a.G;
  const int nfresh = a.k_new ? (a.N + AT_TILE - 1) / AT_TILE : 0;
  AtState<D, NR> st;
  AtCursor cur;
  // the piece in registers at the end
  int first = 0, last = 0, h = 0, row0 = 0;
  long long upiece = u0;

  if (u0 < u1) {
    at_seek(a, prefix, HR, u0, cur);
    // The first warp of a pair fetches for both.  A list of the next 32 units'
    // blocks, a unit a lane, keeps the way from a unit to its place in the cache
    // out of the loop over the tiles.
    long long next = u0;                   // unit of the next fetch
    uint32_t phase = 0u;                   // a bit per stage
    bool failed = false;
    auto fetch = [&](int s) {              // the next cached tile of the share into stage s
      uint2 e = make_uint2(AT_NONE, AT_NONE);
      while (next < u1 && e.x == AT_NONE) {
        const int at = static_cast<int>(next - u0) % AT_QUEUE;
        if (at == 0) {
          __syncwarp();
          if (next + (threadIdx.x & 31) < u1) pr.queue()[threadIdx.x & 31] = at_source(a, prefix, HR, nfresh, next + (threadIdx.x & 31));
          __syncwarp();
        }
        e = pr.queue()[at];
        ++next;
      }
      if (e.x == AT_NONE || (threadIdx.x & 31) != 0 || failed) return;
      *pr.arrived(s) = e.x != AT_BAD;
      if (e.x == AT_BAD) {
        mbar_arrive(&bars[s]);
      } else if (e.y == e.x + 1) {         // neighbours in one page
        mbar_arrive_expect_tx(&bars[s], 2 * BB);
        bulk_g2s(ring + s * SB, a.cache + static_cast<unsigned long long>(e.x) * BB, 2 * BB, &bars[s]);
      } else {
        mbar_arrive_expect_tx(&bars[s], e.y == AT_NONE ? BB : 2 * BB);
        bulk_g2s(ring + s * SB, a.cache + static_cast<unsigned long long>(e.x) * BB, BB, &bars[s]);
        if (e.y != AT_NONE) bulk_g2s(ring + s * SB + BB, a.cache + static_cast<unsigned long long>(e.y) * BB, BB, &bars[s]);
      }
    };
    if (pr.x == 0)
      for (int s = 0; s < stages; ++s) fetch(s);

    // A stage is free once both warps have passed the barrier of the next tile,
    // and is filled again from there: all stages but one are on their way.
    int stage = 0, buf = 0, done = -1;
    auto refill = [&] {
      if (done >= 0 && pr.x == 0) fetch(done);
      done = -1;
    };
    for (long long u = u0;;) {
      // one triple, or the part of it that lies in the share
      h = cur.pair / a.row_tiles;
      row0 = (cur.pair - h * a.row_tiles) * 8 * NR;
      first = cur.i;
      last = static_cast<int>(min(static_cast<long long>(cur.units), first + (u1 - u)));
      upiece = u;
      bool poison = !at_len_ok(a, cur.len);
      const int nf = poison ? 0 : AT_FRESH * nfresh, ncached = poison ? 0 : (cur.len + AT_TILE - 1) / AT_TILE;
      // (a fresh tile is worked on by the share that has its first unit)
      const int f0 = (first + AT_FRESH - 1) / AT_FRESH, f1 = (min(last, nf) + AT_FRESH - 1) / AT_FRESH;
      // (In line: in a function of their own these tiles leave the cached ones' loop
      // more registers, but the state and the arguments then pass through memory: 24
      // rows of 256 sequences at 2,048 tokens took 4 % longer, of 32 at 16,384 3 % less.)
      st.clear();
#pragma unroll 1
      for (int i = f0; i < f1; ++i) at_fresh_tile<D, NR>(a, cur.b, h, row0, rows, i * AT_TILE, pr, st);
      const int c1 = min(last - nf, ncached);
      int c = max(first - nf, 0);
      float factor[NR][2];
      if (c < c1) {
        at_load_q<D, NR>(a, cur.b, h, row0, rows, pr, factor);
        refill();
      }
      for (; c < c1; ++c) {
        // (a warp whose wait gave up goes on in step with the other one, over what
        // the stage holds, and its result is void)
        if (!failed && !mbar_wait(&bars[stage], (phase >> stage) & 1u, a.timeout_ns)) {
          failed = true;   // no more copies are started
          if ((threadIdx.x & 63) == 0) stuck[pair] = static_cast<int>(phase) | AT_STUCK;
        }
        phase ^= 1u << stage;
        poison |= !*pr.arrived(stage);
        at_cached_tile<D, NR>(ring + stage * SB, min(cur.len - c * AT_TILE, AT_TILE), buf, factor, pr, st, refill);
        buf ^= 1;
        done = stage;
        stage = stage + 1 == stages ? 0 : stage + 1;
      }
      if (poison || failed) st.poison();
      u += last - first;
      if (first == 0 && last == cur.units) at_write<D, NR>(a, cur.b, h, row0, rows, pr, st);
      else if (first != 0) st.save(states + (threadIdx.x >> 5) * at_state_floats(D, NR));
      if (u >= u1) break;
      cur.i = last - 1;
      at_next(a, prefix, HR, cur);
    }
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0 && __builtin_expect(stuck[pair], 0)) at_drain(bars, stages, stuck[pair], a.timeout_ns);

  // Joins within the CTA.  A triple that begins in a pair's share and goes on is
  // joined by that pair, whose registers hold its first part; the other parts
  // were saved.
  if (u0 < u1 && first == 0 && last != cur.units) {
    const long long tri_end = upiece + cur.units;
    for (int w = pair + 1; w < AT_PAIRS; ++w) {
      const long long s0 = at_start(units, shares, share + w - pair), s1 = at_start(units, shares, share + w - pair + 1);
      if (s0 >= tri_end) break;
      if (s0 < s1) st.join(states + (2 * w + pr.x) * at_state_floats(D, NR));
    }
    if (tri_end <= at_start(units, shares, (blockIdx.x + 1) * AT_PAIRS)) at_write<D, NR>(a, cur.b, h, row0, rows, pr, st);
    else at_write_partial<D, NR>(cta_ws + at_partial_floats(D, NR), pr, st);
  }
  // A triple that came from the CTA before is joined by the first pair.
  if (pair == 0) {
    AtCursor c;
    at_seek(a, prefix, HR, u0, c);
    if (c.i != 0) {
      const long long tri_end = u0 + (c.units - c.i);
      st.clear();
      for (int w = 0; w < AT_PAIRS; ++w) {
        const long long s0 = at_start(units, shares, share + w), s1 = at_start(units, shares, share + w + 1);
        if (s0 >= tri_end) break;
        if (s0 < s1) st.join(states + (2 * w + pr.x) * at_state_floats(D, NR));
      }
      at_write_partial<D, NR>(cta_ws, pr, st);
    }
  }
}

// Joins the partials of triples that several CTAs worked on: a warp takes eight
// rows of a triple (a lane D / 32 columns).  Where a triple is spread over many
// CTAs, a CTA's warps take its partials in turn and their results are joined.
// R8: rows of a tile, in units of 8; a CTA's two partials are at the start of its
// part of the workspace, `stride` floats apart from the next CTA's.
constexpr int ATJ_WARPS = 8, ATJ_THREADS = 32 * ATJ_WARPS;
template <int D, bool SPREAD>
__global__ void __launch_bounds__(ATJ_THREADS) attend_q4_join_kernel(const __grid_constant__ AttendArgs a, int grid, int shares,
                                                                     int R8, size_t stride) {
  extern __shared__ __align__(128) unsigned char at_smem[];
  __shared__ long long scratch[ATJ_WARPS];
  constexpr int C = D / 32, PL = SPREAD ? ATJ_WARPS : 1;
  __shared__ float sml[PL][2][8], so[PL][8][SPREAD ? D : 1];
  long long* prefix = reinterpret_cast<long long*>(at_smem);
  at_prefix<ATJ_THREADS>(a, prefix, scratch);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // every CTA, before it reads a partial or ends
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HR = a.Hkv * a.row_tiles, rows = a.N * a.G;
  const long long units = prefix[a.B] * HR;
  const int ctas = at_active(units, grid, shares);
  const size_t partial = static_cast<size_t>(8 * R8) * (D + 4);
  const int items = a.B * HR * R8;
  const int step = gridDim.x * (SPREAD ? 1 : ATJ_WARPS);
  for (int x = SPREAD ? blockIdx.x : blockIdx.x * ATJ_WARPS + warp; x < items; x += step) {
    const int y = x / R8, j = x - y * R8, b = y / HR, pair = y - b * HR;
    const long long n = prefix[b + 1] - prefix[b], u = prefix[b] * HR + pair * n;
    const int wa = at_owner(units, ctas, u), wb = at_owner(units, ctas, u + n - 1);
    if (wa == wb) continue;
    const int h = pair / a.row_tiles, r0 = ((pair - h * a.row_tiles) * R8 + j) * 8;
    if (r0 >= rows) continue;
    float m[8], l[8], o[8][C];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      m[r] = kNegInf;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) o[r][i] = 0.f;
    }
    for (int w = wa + (SPREAD ? warp : 0); w <= wb; w += PL) {
      const float* part = a.ws + static_cast<size_t>(w) * stride + (w == wa ? partial : 0);
      const float* ml = part + static_cast<size_t>(8 * R8) * D + 8 * j;
      float pm[8], pl[8], po[8][C];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        pm[r] = ml[r];
        pl[r] = ml[8 * R8 + r] + ml[16 * R8 + r];
#pragma unroll
        for (int i = 0; i < C; ++i) po[r][i] = part[(8 * j + r) * D + i * 32 + lane];
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float mn = fmaxf(m[r], pm[r]), ref = mn == kNegInf ? 0.f : mn;
        const float c0 = at_corr(m[r] - ref), c1 = at_corr(pm[r] - ref);
        l[r] = l[r] * c0 + pl[r] * c1;
#pragma unroll
        for (int i = 0; i < C; ++i) o[r][i] = o[r][i] * c0 + po[r][i] * c1;
        m[r] = mn;
      }
    }
    if constexpr (SPREAD) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (lane == 0) {
          sml[warp][0][r] = m[r];
          sml[warp][1][r] = l[r];
        }
#pragma unroll
        for (int i = 0; i < C; ++i) so[warp][r][i * 32 + lane] = o[r][i];
      }
      __syncthreads();
      // warp r joins row r
      const int r = r0 + warp;
      if (r < rows) {
        float mx = kNegInf, sum = 0.f, acc[C];
        for (int w = 0; w < PL; ++w) mx = fmaxf(mx, sml[w][0][warp]);
        const float ref = mx == kNegInf ? 0.f : mx;
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = 0.f;
        for (int w = 0; w < PL; ++w) {
          const float c = at_corr(sml[w][0][warp] - ref);
          sum += sml[w][1][warp] * c;
#pragma unroll
          for (int i = 0; i < C; ++i) acc[i] += so[w][warp][i * 32 + lane] * c;
        }
        const long long at = at_row(a, b, h, r);
        const float inv = sum == 0.f ? 0.f : a.v_mul / sum;
#pragma unroll
        for (int i = 0; i < C; ++i) a.out[at * D + i * 32 + lane] = static_cast<uint16_t>(bf16x2_pack(acc[i] * inv, 0.f));
        if (a.lse && lane == 0) a.lse[at] = at_lse(mx, sum);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r0 + r >= rows) continue;
        const long long at = at_row(a, b, h, r0 + r);
        const float inv = l[r] == 0.f ? 0.f : a.v_mul / l[r];
#pragma unroll
        for (int i = 0; i < C; ++i) a.out[at * D + i * 32 + lane] = static_cast<uint16_t>(bf16x2_pack(o[r][i] * inv, 0.f));
        if (a.lse && lane == 0) a.lse[at] = at_lse(m[r], l[r]);
      }
    }
  }
}

}  // namespace sv
