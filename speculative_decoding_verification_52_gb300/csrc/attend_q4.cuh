// attend_q4.cuh -- verification attention over a paged cache held in 4 bits.
//
// N query nodes per sequence (the last token and its drafts: a chain or a tree)
// attend to the sequence's cached tokens and, under the nodes' mask, to the
// fresh bf16 keys and values of the nodes themselves:
//   z = scale * q.k,  out = softmax(z) v,  lse = log(sum exp z).
// The rows of one kv head are its N * G (node, query head) pairs.
//
// Few rows (this kernel).  The cache is read once and each element takes part
// in 2 * rows multiply-adds, so up to a few tens of rows the 9/16 byte an
// element has to cross the HBM bus is the bound, and the work next to it is to
// unpack the codes: the budget is about three instructions an element.
//
// * The unit of work is a block of 32 tokens (one contiguous run of 36 * D
//   bytes, one bulk copy).  All blocks of all (sequence, head, row tile) triples
//   form one list, a triple's fresh blocks before its cached ones; every warp
//   takes an equal, contiguous share of it, whatever the lengths, and fetches it
//   through a ring of its own.  A triple that lies in one warp's share is
//   finished there.  The warps of a CTA have neighbouring shares and join what
//   they share at the end; what CTAs share goes through the workspace (maximum,
//   sum, sum of v) and a second kernel.  All joins are in the list's order.
// * Everything is unpacked in f16, exactly: a code times its scale has 6
//   significant bits.  q enters as f16 too, scaled by a power of two per row so
//   that its largest element lies in [128, 256): what f16 then cannot hold is
//   below 2^-32 of that element.
// * No unpacked element crosses shared memory.  The products are
//   mma.m16n8k16 with the rows as N, eight at a time: k q^T (tokens as M), then
//   v^T p^T (columns as M).  A thread's part of a key operand is D / 4
//   consecutive elements of one token (the contraction index is permuted alike
//   in q), of a value operand D / 8 consecutive elements of four tokens (the
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
// * The weights of v are 2^(z - max + 15) in f16: the largest is 2^15, so a
//   weight has 11 significant bits down to 2^-29 of it.  Sums are fp32.
// * The fresh entries are bf16 with bf16's range, so their blocks use bf16
//   products, with each weight as the sum of two bf16.
#pragma once

#include "common.cuh"
#include "kv_q4.cuh"

namespace sv {

constexpr int AT_WARPS = 4;                 // warps of a CTA
constexpr int AT_THREADS = 32 * AT_WARPS;
constexpr int AT_MAX_B = 4096;
constexpr float AT_PSHIFT = 15.f;           // log2 of the largest weight

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
  float scale_log2;          // scale * log2(e)
  float k_mul, v_mul;        // 2^shift
  uint16_t* out;             // [B, N, Hkv * G, D] bf16
  float* lse;                // [B, N, Hkv * G] or null
  float* ws;
  unsigned long long timeout_ns;
};

// ---------------------------------------------------------------------------
// the list of work
// ---------------------------------------------------------------------------
// Blocks of sequence b for one (head, row tile): its cached blocks, then the
// blocks of fresh entries; at least one, so that every output is written.
__device__ __forceinline__ bool at_len_ok(const AttendArgs& a, int len) {
  return len >= 0 && static_cast<long long>(len) <= static_cast<long long>(a.W) * a.P;
}
__device__ __forceinline__ int at_units(const AttendArgs& a, int len) {
  if (!at_len_ok(a, len)) return 1;
  const int n = (len + Q4_BLOCK - 1) / Q4_BLOCK + (a.k_new ? (a.N + Q4_BLOCK - 1) / Q4_BLOCK : 0);
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
  int b, pair, i, units;   // sequence, (head, row tile) of it, block of it, its blocks
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

// CTAs that get work: the list is cut in AT_WARPS shares a CTA, none of the CTAs empty
__device__ __forceinline__ int at_active(long long units, int ctas) {
  return static_cast<int>(min((units + AT_WARPS - 1) / AT_WARPS, static_cast<long long>(ctas)));
}
// share w of n of a list of `units`: [at_start(w), at_start(w + 1)), and the share that unit u falls in
__device__ __forceinline__ long long at_start(long long units, int n, long long w) { return units * w / n; }
__device__ __forceinline__ int at_owner(long long units, int n, long long u) {
  return static_cast<int>(((u + 1) * n - 1) / units);
}

// ---------------------------------------------------------------------------
// products and conversions
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_f16(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* d, const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// eight codes to four f16 pairs (of one byte each), unscaled
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
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

__host__ __device__ constexpr int at_stage_bytes(int D) { return q4_block_bytes(D); }
__host__ __device__ constexpr int at_q_bytes(int D, int NR) { return NR * (D / 32) * 512; }
// The workspace.  A CTA has two partials, of the triple that it shares with the
// CTAs before it and of the one that it shares with those behind:
//   [8 NR rows x D] sums of v, then m[8 NR], l[8 NR];
// a warp has two copies of a state in its lanes' order: what its CTA's other
// warps join, and the result of a triple's fresh blocks.
__host__ __device__ constexpr size_t at_partial_floats(int D, int NR) { return static_cast<size_t>(8 * NR) * (D + 2); }
__host__ __device__ constexpr size_t at_state_floats(int D, int NR) { return static_cast<size_t>(32 * NR) * (D / 4 + 4); }
__host__ __device__ constexpr size_t at_cta_floats(int D, int NR) {
  return 2 * at_partial_floats(D, NR) + 2 * AT_WARPS * at_state_floats(D, NR);
}

// ---------------------------------------------------------------------------
// the state of one (sequence, head, row tile) in a warp's registers: lane
// (g, t) holds rows 8 j + 2 t + e and the D / 8 columns from g * D / 8
// ---------------------------------------------------------------------------
template <int D, int NR>
struct AtState {
  static constexpr int MT = D / 16;   // products that cover the output's columns
  float o[NR][MT][4];                 // [.][i][e + 2 f]: column g * D / 8 + 2 i + f of row e
  float m[NR][2], l[NR][2];           // running maximum (log2 domain) and this lane's part of the sum
  float c[NR][2];                     // factor from a row's f16 products to the log2 domain

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NR; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][i][k] = 0.f;
      m[j][0] = m[j][1] = kNegInf;
      l[j][0] = l[j][1] = 0.f;
    }
  }

  // the state in the order of its lanes: only the lane that wrote a value reads it
  __device__ __forceinline__ void save(float* p) const {
    float4* q = reinterpret_cast<float4*>(p) + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) q[32 * (j * (MT + 1) + i)] = make_float4(o[j][i][0], o[j][i][1], o[j][i][2], o[j][i][3]);
      q[32 * (j * (MT + 1) + MT)] = make_float4(m[j][0], m[j][1], l[j][0], l[j][1]);
    }
  }
  __device__ __forceinline__ void load(const float* p) {
    const float4* q = reinterpret_cast<const float4*>(p) + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const float4 x = q[32 * (j * (MT + 1) + i)];
        o[j][i][0] = x.x; o[j][i][1] = x.y; o[j][i][2] = x.z; o[j][i][3] = x.w;
      }
      const float4 x = q[32 * (j * (MT + 1) + MT)];
      m[j][0] = x.x; m[j][1] = x.y; l[j][0] = x.z; l[j][1] = x.w;
    }
  }
  // joins a saved state of the same rows
  __device__ __forceinline__ void join(const float* p) {
    const float4* q = reinterpret_cast<const float4*>(p) + (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const float4 x = q[32 * (j * (MT + 1) + MT)];
      const float pm[2] = {x.x, x.y}, pl[2] = {x.z, x.w};
      float c0[2], c1[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[j][e], pm[e]), ref = mn == kNegInf ? 0.f : mn;
        c0[e] = at_corr(m[j][e] - ref);
        c1[e] = at_corr(pm[e] - ref);
        l[j][e] = l[j][e] * c0[e] + pl[e] * c1[e];
        m[j][e] = mn;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const float4 y = q[32 * (j * (MT + 1) + i)];
        o[j][i][0] = o[j][i][0] * c0[0] + y.x * c1[0];
        o[j][i][1] = o[j][i][1] * c0[1] + y.y * c1[1];
        o[j][i][2] = o[j][i][2] * c0[0] + y.z * c1[0];
        o[j][i][3] = o[j][i][3] * c0[1] + y.w * c1[1];
      }
    }
  }

  // z (log2 domain, -inf where masked; [.][.][e + 2 f]: token g + 8 f of row e)
  // becomes the weights 2^(z - max + 15)
  __device__ __forceinline__ void weigh(float (&z)[2][NR][4]) {
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      float mn[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(fmaxf(z[0][j][e], z[0][j][e + 2]), fmaxf(z[1][j][e], z[1][j][e + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        mn[e] = fmaxf(m[j][e], mx);
      }
      if (__any_sync(0xffffffffu, mn[0] > m[j][0] || mn[1] > m[j][1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float corr = mn[e] == kNegInf ? 1.f : at_corr(m[j][e] - mn[e]);
          l[j][e] *= corr;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[j][i][e] *= corr;
            o[j][i][e + 2] *= corr;
          }
          m[j][e] = mn[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = (mn[e] == kNegInf ? 0.f : mn[e]) - AT_PSHIFT;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int f = 0; f < 2; ++f) z[mt][j][e + 2 * f] = ex2_approx(z[mt][j][e + 2 * f] - ref);
        l[j][e] += (z[0][j][e] + z[0][j][e + 2]) + (z[1][j][e] + z[1][j][e + 2]);
      }
    }
  }
};

__device__ __forceinline__ long long at_row(const AttendArgs& a, int b, int h, int r) {
  const int n = r / a.G;
  return ((static_cast<long long>(b) * a.N + n) * a.Hkv + h) * a.G + (r - n * a.G);
}

// Queries of a row tile: the f16 operand into the lane's own part of `qf`
// (nothing is shared between lanes), the rows' factors into st.c.
template <int D, int NR>
__device__ __forceinline__ void at_load_q(const AttendArgs& a, int b, int h, int row0, int rows, uint4* qf, AtState<D, NR>& st) {
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
    const float mul = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
    // a row with a NaN or an infinity has no finite scores: the factor says so
    const float c = top < __builtin_huge_valf()
                        ? a.scale_log2 * a.k_mul * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23)
                        : __int_as_float(0x7fc00000);
    st.c[j][0] = __shfl_sync(0xffffffffu, c, 8 * t);
    st.c[j][1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < CH / 8; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = f16x2_pack(__uint_as_float(x[k] << 16) * mul, __uint_as_float(x[k] & 0xffff0000u) * mul);
      qf[(j * WK + i) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
    }
  }
}

// A cached block: `left` tokens of it (1..32) belong to the sequence.
template <int D, int NR>
__device__ __forceinline__ void at_cached_block(const unsigned char* sb, int left, const uint4* qf, AtState<D, NR>& st) {
  constexpr int WK = D / 32;   // words of a key chunk
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tr = at_token(g);
  float z[2][NR][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[mt][j][k] = 0.f;

  uint32_t kw[4][WK];
  uint32_t ks2[4][D / 64];   // the chunk's scales, each twice
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    const int tok = 8 * nt + tr;
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(sb + tok * 64 + t * 16);
      kw[nt][0] = x.x; kw[nt][1] = x.y; kw[nt][2] = x.z; kw[nt][3] = x.w;
      const uint32_t two = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(sb + 32 * D + tok * 8 + t * 2));
      ks2[nt][0] = __byte_perm(two, two, 0x1010);
      ks2[nt][1] = __byte_perm(two, two, 0x3232);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(sb + tok * 32 + t * 8);
      kw[nt][0] = x.x; kw[nt][1] = x.y;
      const uint32_t one = sb[32 * D + tok * 4 + t];
      ks2[nt][0] = e4m3x2_to_f16(one | (one << 8));
    }
  }
#pragma unroll
  for (int w = 0; w < WK; ++w) {
    uint4 qb[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) qb[j] = qf[(j * WK + w) * 32 + lane];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t r0[4], r1[4];   // tokens g and g + 8
      e2m1x8_to_f16(kw[2 * mt][w], r0);
      e2m1x8_to_f16(kw[2 * mt + 1][w], r1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r0[i] = f16x2_mul(r0[i], ks2[2 * mt][w / 2]);
        r1[i] = f16x2_mul(r1[i], ks2[2 * mt + 1][w / 2]);
      }
      const uint4 k0 = make_uint4(r0[0], r1[0], r0[1], r1[1]), k1 = make_uint4(r0[2], r1[2], r0[3], r1[3]);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        mma_f16(z[mt][j], k0, qb[j].x, qb[j].y);
        mma_f16(z[mt][j], k1, qb[j].z, qb[j].w);
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[mt][j][k] *= st.c[j][k & 1];
  if (left < Q4_BLOCK) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int f = 0; f < 2; ++f)
        if (16 * mt + 8 * f + tr >= left) {
#pragma unroll
          for (int j = 0; j < NR; ++j) z[mt][j][2 * f] = z[mt][j][2 * f + 1] = kNegInf;
        }
  }
  st.weigh(z);

#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t p[NR][2];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int f = 0; f < 2; ++f) p[j][f] = transpose8(f16x2_pack(z[s][j][2 * f], z[s][j][2 * f + 1]));
    uint32_t vw[4][D / 64];   // tokens 2t, 2t+1 of the two groups of 8
    uint32_t sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int tok = 16 * s + 8 * (k >> 1) + at_token(2 * t + (k & 1));
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(sb + 16 * D + tok * 64 + g * 8);
        vw[k][0] = x.x; vw[k][1] = x.y;
        sc[k] = sb[34 * D + tok * 8 + g];
      } else {
        vw[k][0] = *reinterpret_cast<const uint32_t*>(sb + 16 * D + tok * 32 + g * 4);
        sc[k] = sb[34 * D + tok * 4 + (g >> 1)];
      }
      if (tok >= left) sc[k] = 0u;   // what lies behind the last token may be a NaN
    }
    const uint32_t s01 = e4m3x2_to_f16(sc[0] | (sc[1] << 8)), s23 = e4m3x2_to_f16(sc[2] | (sc[3] << 8));
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      uint32_t e01[4], o01[4], e23[4], o23[4];
      e2m1x8_to_f16((vw[0][w] & 0x0f0f0f0fu) | ((vw[1][w] << 4) & 0xf0f0f0f0u), e01);
      e2m1x8_to_f16(((vw[0][w] >> 4) & 0x0f0f0f0fu) | (vw[1][w] & 0xf0f0f0f0u), o01);
      e2m1x8_to_f16((vw[2][w] & 0x0f0f0f0fu) | ((vw[3][w] << 4) & 0xf0f0f0f0u), e23);
      e2m1x8_to_f16(((vw[2][w] >> 4) & 0x0f0f0f0fu) | (vw[3][w] & 0xf0f0f0f0u), o23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = make_uint4(f16x2_mul(e01[i], s01), f16x2_mul(o01[i], s01), f16x2_mul(e23[i], s23), f16x2_mul(o23[i], s23));
#pragma unroll
        for (int j = 0; j < NR; ++j) mma_f16(st.o[j][4 * w + i], v, p[j][0], p[j][1]);
      }
    }
  }
}

__device__ __forceinline__ bool bf16x2_unbounded(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// A block of fresh entries: nodes j0 .. j0 + 31.
template <int D, int NR>
__device__ __forceinline__ void at_fresh_block(const AttendArgs& a, int b, int h, int row0, int rows, int j0, AtState<D, NR>& st) {
  constexpr int CH = D / 4, KS = D / 16, CV = D / 8;
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
#pragma unroll 2
  for (int ks = 0; ks < KS; ++ks) {
    uint2 qb[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j)
      qb[j] = qat[j] >= 0 ? __ldg(reinterpret_cast<const uint2*>(a.q + qat[j] + 4 * ks)) : make_uint2(0u, 0u);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint2 kx[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int n = j0 + 16 * mt + 8 * f + tr;
        kx[f] = n < a.N ? __ldg(reinterpret_cast<const uint2*>(a.k_new + base + n * rstride + t * CH + 4 * ks)) : make_uint2(0u, 0u);
      }
      const uint4 k = make_uint4(kx[0].x, kx[1].x, kx[0].y, kx[1].y);
#pragma unroll
      for (int j = 0; j < NR; ++j) mma_bf16(z[mt][j], k, qb[j].x, qb[j].y);
    }
  }
  uint32_t sees[NR][2];   // nodes of the block that the lane's rows attend to
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = (row0 + 8 * j + 2 * t + e) / a.G;
      uint32_t see = 0u;
      if (n < a.N) {
        if (a.masks) see = __ldg(a.masks + (static_cast<long long>(b) * a.N + n) * a.NW + j0 / 32);
        else see = n - j0 >= 31 ? ~0u : n < j0 ? 0u : (2u << (n - j0)) - 1u;
        if (a.N - j0 < 32) see &= (1u << (a.N - j0)) - 1u;
      }
      sees[j][e] = see;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float& x = z[mt][j][e + 2 * f];
          x = (see >> (16 * mt + 8 * f + tr)) & 1u ? x * a.scale_log2 : kNegInf;
        }
    }
  st.weigh(z);

  // the sums of v are kept in units of 2^v_shift
  const float unit = __fdiv_rn(1.f, a.v_mul);
  bool odd = false;   // this lane saw a NaN or an infinity
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t hi[NR][2], lo[NR][2];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const float x = z[s][j][2 * f] * unit, y = z[s][j][2 * f + 1] * unit;
        const uint32_t ph = bf16x2_pack(x, y);
        lo[j][f] = transpose8(bf16x2_pack(x - __uint_as_float(ph << 16), y - __uint_as_float(ph & 0xffff0000u)));
        hi[j][f] = transpose8(ph);
      }
#pragma unroll
    for (int w = 0; w < CV / 8; ++w) {   // eight columns of the chunk at a time
      uint32_t vw[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int n = j0 + 16 * s + 8 * (k >> 1) + at_token(2 * t + (k & 1));
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (n < a.N) x = __ldg(reinterpret_cast<const uint4*>(a.v_new + base + n * rstride + g * CV) + w);
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vw[k][i] = y[i];
          if (bf16x2_unbounded(y[i])) {
            odd = true;
            if ((y[i] & 0x7f80u) == 0x7f80u) vw[k][i] &= 0xffff0000u;
            if ((y[i] & 0x7f800000u) == 0x7f800000u) vw[k][i] &= 0xffffu;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = make_uint4(__byte_perm(vw[0][i], vw[1][i], 0x5410), __byte_perm(vw[0][i], vw[1][i], 0x7632),
                                   __byte_perm(vw[2][i], vw[3][i], 0x5410), __byte_perm(vw[2][i], vw[3][i], 0x7632));
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          mma_bf16(st.o[j][4 * w + i], v, hi[j][0], hi[j][1]);
          mma_bf16(st.o[j][4 * w + i], v, lo[j][0], lo[j][1]);
        }
      }
    }
  }
  // A product takes 0 * inf for NaN, so such elements were left out above and
  // reach only the rows that see their node (with a weight above zero, however
  // small: a weight that underflowed counts as the smallest one).
  if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
    for (int x = 0; x < 8; ++x) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int n = 16 * mt + 8 * f + at_token(x);
#pragma unroll
          for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = __shfl_sync(0xffffffffu, z[mt][j][e + 2 * f], 4 * x + t);
              if (!((sees[j][e] >> n) & 1u)) continue;
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint32_t v = a.v_new[base + (j0 + n) * rstride + g * CV + 2 * i + k];
                  if ((v & 0x7f80u) == 0x7f80u) st.o[j][i][e + 2 * k] += (p == 0.f ? 1.17549435e-38f : p) * __uint_as_float(v << 16);
                }
            }
        }
    }
  }
}

// The state after fresh blocks first .. last - 1 of a triple, saved at `p`.  A
// function of its own: these blocks are few, and their registers would push the
// cached blocks' loop into local memory.
template <int D, int NR>
__device__ __noinline__ void at_fresh(const AttendArgs& a, int b, int h, int row0, int rows, int first, int last, float* p) {
  AtState<D, NR> st;
  st.clear();
  for (int i = first; i < last; ++i) at_fresh_block<D, NR>(a, b, h, row0, rows, i * Q4_BLOCK, st);
  st.save(p);
}

__device__ __forceinline__ float at_lse(float m, float l) {
  // m in the log2 domain, l relative to 2^(m - 15)
  return l == 0.f ? kNegInf : (m - AT_PSHIFT + log2f(l)) * 0.69314718055994530942f;
}

// CTAs an SM: what the registers of a row tile leave room for
__host__ __device__ constexpr int at_ctas(int NR) { return NR == 1 ? 4 : NR == 4 ? 2 : 3; }

// this lane's rows of a finished state
template <int D, int NR>
__device__ __forceinline__ void at_write(const AttendArgs& a, int b, int h, int row0, int rows, const AtState<D, NR>& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = st.l[j][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int r = row0 + 8 * j + 2 * t + e;
      if (r >= rows) continue;
      const long long at = at_row(a, b, h, r);
      const float inv = l == 0.f ? 0.f : a.v_mul / l;
      uint4* p = reinterpret_cast<uint4*>(a.out + at * D + g * (D / 8));
#pragma unroll
      for (int i = 0; i < D / 16; i += 4)
        p[i / 4] = make_uint4(bf16x2_pack(st.o[j][i][e] * inv, st.o[j][i][e + 2] * inv),
                              bf16x2_pack(st.o[j][i + 1][e] * inv, st.o[j][i + 1][e + 2] * inv),
                              bf16x2_pack(st.o[j][i + 2][e] * inv, st.o[j][i + 2][e + 2] * inv),
                              bf16x2_pack(st.o[j][i + 3][e] * inv, st.o[j][i + 3][e + 2] * inv));
      if (a.lse && g == 0) a.lse[at] = at_lse(st.m[j][e], l);
    }
}
// the same as a partial
template <int D, int NR>
__device__ __forceinline__ void at_write_partial(float* part, const AtState<D, NR>& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = st.l[j][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int lr = 8 * j + 2 * t + e;
      float4* p = reinterpret_cast<float4*>(part + static_cast<size_t>(lr) * D + g * (D / 8));
#pragma unroll
      for (int i = 0; i < D / 16; i += 2)
        p[i / 2] = make_float4(st.o[j][i][e], st.o[j][i][e + 2], st.o[j][i + 1][e], st.o[j][i + 1][e + 2]);
      if (g == 0) {
        part[8 * NR * D + lr] = st.m[j][e];
        part[8 * NR * D + 8 * NR + lr] = l;
      }
    }
}

template <int D, int NR>
__global__ void __launch_bounds__(AT_THREADS, at_ctas(NR)) attend_q4_kernel(const __grid_constant__ AttendArgs a, int stages) {
  extern __shared__ __align__(128) unsigned char at_smem[];
  __shared__ long long scratch[AT_WARPS];
  constexpr int SB = at_stage_bytes(D), QB = at_q_bytes(D, NR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = at_smem + static_cast<size_t>(warp) * stages * SB;
  uint4* qf = reinterpret_cast<uint4*>(at_smem + static_cast<size_t>(AT_WARPS) * stages * SB + warp * QB);
  uint64_t* bars = reinterpret_cast<uint64_t*>(at_smem + static_cast<size_t>(AT_WARPS) * (stages * SB + QB)) + warp * stages;
  long long* prefix = reinterpret_cast<long long*>(at_smem + static_cast<size_t>(AT_WARPS) * (stages * SB + QB)) + AT_WARPS * stages;

  if (lane == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
    mbar_fence_init();
  }
  at_prefix<AT_THREADS>(a, prefix, scratch);   // (synchronises the CTA)

  const int HR = a.Hkv * a.row_tiles;
  const long long units = prefix[a.B] * HR;
  const int ctas = at_active(units, gridDim.x);
  if (blockIdx.x >= ctas) return;
  const int shares = ctas * AT_WARPS, share = blockIdx.x * AT_WARPS + warp;
  const long long u0 = at_start(units, shares, share), u1 = at_start(units, shares, share + 1);
  float* cta_ws = a.ws + static_cast<size_t>(blockIdx.x) * at_cta_floats(D, NR);
  float* states = cta_ws + 2 * at_partial_floats(D, NR);
  float* mine = states + warp * at_state_floats(D, NR);
  float* fresh_at = states + (AT_WARPS + warp) * at_state_floats(D, NR);

  const int rows = a.N * a.G, bpp = a.P / Q4_BLOCK;
  const int nfresh = a.k_new ? (a.N + Q4_BLOCK - 1) / Q4_BLOCK : 0;
  AtState<D, NR> st;
  AtCursor pre, cur;
  uint32_t phase = 0u, have = 0u;        // a bit per stage
  int stage = 0;
  bool failed = false;
  // the piece in registers at the end
  int first = 0, last = 0, h = 0, row0 = 0;
  long long upiece = u0;

  if (u0 < u1) {
    // The cursor of what is fetched runs ahead of what is worked on.  The page
    // id of a fetch was loaded one fetch earlier, so that nothing waits for it.
    at_seek(a, prefix, HR, u0, pre);
    cur = pre;
    int left = static_cast<int>(u1 - u0);            // blocks that the cursor has still to pass
    int pblk = 0, phead = 0, page = -1;
    const int32_t* prow = nullptr;
    auto enter = [&] {                               // the cursor moved into a triple: past its fresh blocks
      if (!at_len_ok(a, pre.len)) return;
      if (pre.i < nfresh) {
        const int skip = min(nfresh - pre.i, left);
        pre.i += skip;
        left -= skip;
      }
      if (left <= 0 || pre.i >= pre.units) return;
      const int c = pre.i - nfresh;
      prow = a.table + static_cast<long long>(pre.b) * a.W + c / bpp;
      pblk = c % bpp;
      phead = pre.pair / a.row_tiles;
      if (c * Q4_BLOCK < pre.len) page = __ldg(prow);
    };
    enter();
    auto fetch = [&](int s) {                        // the next cached block of the share into stage s
      have &= ~(1u << s);
      // triples without a block to fetch are passed over
      while (left > 0 && (pre.i >= pre.units || !at_len_ok(a, pre.len) || (pre.i - nfresh) * Q4_BLOCK >= pre.len)) {
        if (pre.i < pre.units) {                     // its one empty block
          pre.i = pre.units;
          --left;
          continue;
        }
        pre.i = pre.units - 1;
        at_next(a, prefix, HR, pre);
        enter();
      }
      if (left <= 0) return;
      --left;
      if (page >= 0 && page < a.pages) {
        have |= 1u << s;
        if (lane == 0) {
          const unsigned long long blk = (static_cast<unsigned long long>(page) * a.Hkv + phead) * bpp + pblk;
          mbar_arrive_expect_tx(&bars[s], SB);
          bulk_g2s(ring + s * SB, a.cache + blk * SB, SB, &bars[s]);
        }
      }
      ++pre.i;
      if (++pblk == bpp) {
        pblk = 0;
        ++prow;
        if (pre.i < pre.units) page = __ldg(prow);
      }
    };
    for (int s = 0; s < stages; ++s) fetch(s);

    for (long long u = u0;;) {
      // one triple, or the part of it that lies in the share
      h = cur.pair / a.row_tiles;
      row0 = (cur.pair - h * a.row_tiles) * 8 * NR;
      first = cur.i;
      last = static_cast<int>(min(static_cast<long long>(cur.units), first + (u1 - u)));
      upiece = u;
      bool poison = !at_len_ok(a, cur.len);
      const int nf = poison ? 0 : nfresh, ncached = poison ? 0 : (cur.len + Q4_BLOCK - 1) / Q4_BLOCK;
      if (first < nf) {
        at_fresh<D, NR>(a, cur.b, h, row0, rows, first, min(last, nf), fresh_at);
        st.load(fresh_at);
      } else {
        st.clear();
      }
      const int c1 = min(last - nf, ncached);
      int c = max(first - nf, 0);
      if (c < c1) at_load_q<D, NR>(a, cur.b, h, row0, rows, qf, st);
      for (; c < c1; ++c) {
        if (have & (1u << stage)) {
          if (!mbar_wait(&bars[stage], (phase >> stage) & 1u, a.timeout_ns)) {
            failed = true;
            break;   // no copy is started after one that did not arrive
          }
          phase ^= 1u << stage;
          at_cached_block<D, NR>(ring + stage * SB, min(cur.len - c * Q4_BLOCK, Q4_BLOCK), qf, st);
        } else {
          poison = true;
        }
        __syncwarp();
        fetch(stage);
        stage = stage + 1 == stages ? 0 : stage + 1;
      }
      if (failed) break;
      if (poison) {
#pragma unroll
        for (int j = 0; j < NR; ++j) st.l[j][0] = st.l[j][1] = __int_as_float(0x7fc00000);
      }
      u += last - first;
      if (first == 0 && last == cur.units) at_write<D, NR>(a, cur.b, h, row0, rows, st);
      else if (first != 0) st.save(mine);
      if (u >= u1) break;
      cur.i = last - 1;
      at_next(a, prefix, HR, cur);
    }
    if (failed) {
      // copies still on their way land before the warp goes on (or the wait gives up)
      for (int s = 0; s < stages; ++s)
        if (s != stage && (have & (1u << s))) mbar_wait(&bars[s], (phase >> s) & 1u, a.timeout_ns);
      // every triple of the share from here on is void
      bool again = true;
      for (long long u = upiece; again;) {
        st.clear();
#pragma unroll
        for (int j = 0; j < NR; ++j) st.l[j][0] = st.l[j][1] = __int_as_float(0x7fc00000);
        h = cur.pair / a.row_tiles;
        row0 = (cur.pair - h * a.row_tiles) * 8 * NR;
        first = cur.i;
        last = static_cast<int>(min(static_cast<long long>(cur.units), first + (u1 - u)));
        upiece = u;
        u += last - first;
        if (first == 0 && last == cur.units) at_write<D, NR>(a, cur.b, h, row0, rows, st);
        else if (first != 0) st.save(mine);
        again = u < u1;
        if (again) {
          cur.i = last - 1;
          at_next(a, prefix, HR, cur);
        }
      }
    }
  }
  __syncthreads();

  // Joins within the CTA.  A triple that begins in a warp's share and goes on is
  // joined by that warp, whose registers hold its first part; the other parts
  // were saved.
  if (u0 < u1 && first == 0 && last != cur.units) {
    const long long tri_end = upiece + cur.units;
    for (int w = warp + 1; w < AT_WARPS; ++w) {
      const long long s0 = at_start(units, shares, share + w - warp), s1 = at_start(units, shares, share + w - warp + 1);
      if (s0 >= tri_end) break;
      if (s0 < s1) st.join(states + w * at_state_floats(D, NR));
    }
    if (tri_end <= at_start(units, shares, (blockIdx.x + 1) * AT_WARPS)) at_write<D, NR>(a, cur.b, h, row0, rows, st);
    else at_write_partial<D, NR>(cta_ws + at_partial_floats(D, NR), st);
  }
  // A triple that came from the CTA before is joined by warp 0.
  if (warp == 0) {
    AtCursor c;
    at_seek(a, prefix, HR, u0, c);
    if (c.i != 0) {
      const long long tri_end = u0 + (c.units - c.i);
      st.clear();
      for (int w = 0; w < AT_WARPS; ++w) {
        const long long s0 = at_start(units, shares, share + w), s1 = at_start(units, shares, share + w + 1);
        if (s0 >= tri_end) break;
        if (s0 < s1) st.join(states + w * at_state_floats(D, NR));
      }
      at_write_partial<D, NR>(cta_ws, st);
    }
  }
}

// Joins the partials of triples that several CTAs worked on: a warp takes eight
// rows of a triple (a lane D / 32 columns).  Where a triple is spread over many
// CTAs, a CTA's warps take its partials in turn and their results are joined.
constexpr int ATJ_WARPS = 8, ATJ_THREADS = 32 * ATJ_WARPS;
template <int D, int NR, bool SPREAD>
__global__ void __launch_bounds__(ATJ_THREADS) attend_q4_join_kernel(const __grid_constant__ AttendArgs a, int grid) {
  extern __shared__ __align__(128) unsigned char at_smem[];
  __shared__ long long scratch[ATJ_WARPS];
  constexpr int C = D / 32, PL = SPREAD ? ATJ_WARPS : 1;
  __shared__ float sml[PL][2][8], so[PL][8][SPREAD ? D : 1];
  long long* prefix = reinterpret_cast<long long*>(at_smem);
  at_prefix<ATJ_THREADS>(a, prefix, scratch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HR = a.Hkv * a.row_tiles, rows = a.N * a.G;
  const long long units = prefix[a.B] * HR;
  const int ctas = at_active(units, grid);
  const int items = a.B * HR * NR;
  const int step = gridDim.x * (SPREAD ? 1 : ATJ_WARPS);
  for (int x = SPREAD ? blockIdx.x : blockIdx.x * ATJ_WARPS + warp; x < items; x += step) {
    const int y = x / NR, j = x - y * NR, b = y / HR, pair = y - b * HR;
    const long long n = prefix[b + 1] - prefix[b], u = prefix[b] * HR + pair * n;
    const int wa = at_owner(units, ctas, u), wb = at_owner(units, ctas, u + n - 1);
    if (wa == wb) continue;
    const int h = pair / a.row_tiles, r0 = ((pair - h * a.row_tiles) * NR + j) * 8;
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
      const float* part = a.ws + static_cast<size_t>(w) * at_cta_floats(D, NR) + (w == wa ? at_partial_floats(D, NR) : 0);
      float pm[8], pl[8], po[8][C];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        pm[r] = part[8 * NR * D + 8 * j + r];
        pl[r] = part[8 * NR * D + 8 * NR + 8 * j + r];
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
