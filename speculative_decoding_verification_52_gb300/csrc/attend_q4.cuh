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
//   form one list; every warp takes an equal, contiguous share of it, whatever
//   the lengths, and fetches it through a ring of its own.  A triple that lies in
//   one warp's share is finished there; the others leave partial (max, sum, sum
//   of v) in the workspace and a second kernel joins them in a fixed order.
// * Everything is unpacked in f16, exactly: a code times its scale has 6
//   significant bits.  q enters as f16 too, scaled by a power of two per row so
//   that its largest element lies in [128, 256): what f16 then cannot hold is
//   below 2^-32 of that element.
// * No unpacked element crosses shared memory.  The products are
//   mma.m16n8k16 with the rows as M; for q.k a thread's share of the B operand
//   is D / 4 consecutive elements of one token (the contraction index is
//   permuted alike in q), for p.v it is D / 8 consecutive elements of four
//   tokens (the output columns are permuted), with the nibbles of two tokens
//   interleaved before they are widened.  The tokens of a group of 8 are taken
//   in the order 0 1 3 2 4 5 7 6, which spreads both kinds of reads over the
//   banks as well as 64-byte rows allow.
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

// as many shares as there are warps, none of them empty
__device__ __forceinline__ int at_shares(long long units, int warps) {
  return static_cast<int>(min(units, static_cast<long long>(warps)));
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

__host__ __device__ constexpr int at_stage_bytes(int D) { return q4_block_bytes(D); }
__host__ __device__ constexpr int at_q_bytes(int D, int RT) { return RT * (D / 16) * 512; }
// partial: [16 RT rows x D] sums of v, then m[16 RT], l[16 RT]
__host__ __device__ constexpr size_t at_partial_floats(int D, int RT) { return static_cast<size_t>(16 * RT) * (D + 2); }

// ---------------------------------------------------------------------------
// the state of one (sequence, head, row tile) in a warp's registers
// ---------------------------------------------------------------------------
template <int D, int RT>
struct AtState {
  static constexpr int CH = D / 4;    // elements of a row that a thread loads and writes
  static constexpr int NT = D / 8;    // column groups of the output
  float o[RT][NT][4];
  float m[RT][2], l[RT][2];           // running maximum (log2 domain) and this lane's part of the sum
  float c[RT][2];                     // factor from a row's f16 products to the log2 domain

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[rt][i][k] = 0.f;
      m[rt][0] = m[rt][1] = kNegInf;
      l[rt][0] = l[rt][1] = 0.f;
    }
  }

  // z (log2 domain, -inf where masked) becomes the weights 2^(z - max + 15)
  __device__ __forceinline__ void weigh(float (&z)[RT][4][4]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float mx = kNegInf;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(z[rt][nt][2 * hf], z[rt][nt][2 * hf + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[rt][hf], mx);
        if (__any_sync(0xffffffffu, mn > m[rt][hf])) {
          const float corr = mn == kNegInf ? 1.f : at_corr(m[rt][hf] - mn);
          l[rt][hf] *= corr;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[rt][i][2 * hf] *= corr;
            o[rt][i][2 * hf + 1] *= corr;
          }
          m[rt][hf] = mn;
        }
        const float ref = (mn == kNegInf ? 0.f : mn) - AT_PSHIFT;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int k = 2 * hf; k < 2 * hf + 2; ++k) {
            z[rt][nt][k] = ex2_approx(z[rt][nt][k] - ref);
            sum += z[rt][nt][k];
          }
        l[rt][hf] += sum;
      }
  }
};

// Queries of a row tile: the f16 operand into the lane's own part of `qf`
// (nothing is shared between lanes), the rows' factors into st.c.
template <int D, int RT>
__device__ __forceinline__ void at_load_q(const AttendArgs& a, int b, int h, int row0, int rows, uint4* qf, AtState<D, RT>& st) {
  constexpr int CH = D / 4, KS = D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    uint32_t f[2][CH / 2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = row0 + 16 * rt + 8 * hf + g;
      uint4 w[CH / 8];
#pragma unroll
      for (int i = 0; i < CH / 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const int n = r / a.G;
        const long long at = ((static_cast<long long>(b) * a.N + n) * a.Hkv + h) * a.G + (r - n * a.G);
        const uint4* p = reinterpret_cast<const uint4*>(a.q + at * D + t * CH);
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
      const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      const int sh = top > 0.f ? min(7 - e, 100) : 0;
      const float mul = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      // a row with a NaN or an infinity has no finite scores: the factor says so
      st.c[rt][hf] = top < __builtin_huge_valf()
                         ? a.scale_log2 * a.k_mul * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23)
                         : __int_as_float(0x7fc00000);
#pragma unroll
      for (int i = 0; i < CH / 8; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[hf][4 * i + j] = f16x2_pack(__uint_as_float(x[j] << 16) * mul, __uint_as_float(x[j] & 0xffff0000u) * mul);
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      qf[(rt * KS + ks) * 32 + lane] = make_uint4(f[0][2 * ks], f[1][2 * ks], f[0][2 * ks + 1], f[1][2 * ks + 1]);
  }
}

// A cached block: `left` tokens of it (1..32) belong to the sequence.
template <int D, int RT>
__device__ __forceinline__ void at_cached_block(const unsigned char* sb, int left, const uint4* qf, AtState<D, RT>& st) {
  constexpr int KS = D / 16, WK = D / 32;   // words of a key chunk
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tr = at_token(g);
  float z[RT][4][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[rt][nt][k] = 0.f;

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
    uint4 qa[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      qa[rt][0] = qf[(rt * KS + 2 * w) * 32 + lane];
      qa[rt][1] = qf[(rt * KS + 2 * w + 1) * 32 + lane];
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      uint32_t r[4];
      e2m1x8_to_f16(kw[nt][w], r);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = f16x2_mul(r[i], ks2[nt][w / 2]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        mma_f16(z[rt][nt], qa[rt][0], r[0], r[1]);
        mma_f16(z[rt][nt], qa[rt][1], r[2], r[3]);
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[rt][nt][k] *= st.c[rt][k >> 1];
  if (left < Q4_BLOCK) {
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (8 * nt + at_token(2 * t + k) >= left) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) z[rt][nt][k] = z[rt][nt][k + 2] = kNegInf;
        }
  }
  st.weigh(z);

#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint4 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      p[rt] = make_uint4(f16x2_pack(z[rt][2 * s][0], z[rt][2 * s][1]), f16x2_pack(z[rt][2 * s][2], z[rt][2 * s][3]),
                         f16x2_pack(z[rt][2 * s + 1][0], z[rt][2 * s + 1][1]),
                         f16x2_pack(z[rt][2 * s + 1][2], z[rt][2 * s + 1][3]));
    uint32_t vw[4][D / 64];   // tokens of columns 2t, 2t+1 of the two groups
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
      for (int j = 0; j < 4; ++j) {
        const uint32_t b0 = f16x2_mul(e01[j], s01), b1 = f16x2_mul(e23[j], s23);
        const uint32_t d0 = f16x2_mul(o01[j], s01), d1 = f16x2_mul(o23[j], s23);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          mma_f16(st.o[rt][8 * w + 2 * j], p[rt], b0, b1);
          mma_f16(st.o[rt][8 * w + 2 * j + 1], p[rt], d0, d1);
        }
      }
    }
  }
}

__device__ __forceinline__ bool bf16x2_unbounded(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// A block of fresh entries: nodes j0 .. j0 + 31.
template <int D, int RT>
__device__ __forceinline__ void at_fresh_block(const AttendArgs& a, int b, int h, int row0, int rows, int j0, AtState<D, RT>& st) {
  constexpr int CH = D / 4, KS = D / 16, CV = D / 8;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long rstride = static_cast<long long>(a.Hkv) * D;
  const long long base = (static_cast<long long>(b) * a.N * a.Hkv + h) * D;   // node 0's entry
  float z[RT][4][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[rt][nt][k] = 0.f;
  const uint16_t* qrow[RT][2];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = row0 + 16 * rt + 8 * hf + g;
      const int n = r / a.G;
      qrow[rt][hf] = r < rows ? a.q + (((static_cast<long long>(b) * a.N + n) * a.Hkv + h) * a.G + (r - n * a.G)) * D + t * CH : nullptr;
    }
#pragma unroll 1
  for (int ks = 0; ks < KS; ++ks) {
    uint4 qa[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      uint2 x[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        x[hf] = qrow[rt][hf] ? __ldg(reinterpret_cast<const uint2*>(qrow[rt][hf] + 4 * ks)) : make_uint2(0u, 0u);
      qa[rt] = make_uint4(x[0].x, x[1].x, x[0].y, x[1].y);
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int j = j0 + 8 * nt + at_token(g);
      const uint2 kx = j < a.N ? __ldg(reinterpret_cast<const uint2*>(a.k_new + base + j * rstride + t * CH + 4 * ks)) : make_uint2(0u, 0u);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) mma_bf16(z[rt][nt], qa[rt], kx.x, kx.y);
    }
  }
  uint32_t sees[RT][2];   // nodes of the block that the lane's rows attend to
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int n = (row0 + 16 * rt + 8 * hf + g) / a.G;
      uint32_t see = 0u;
      if (n < a.N) {
        if (a.masks) see = __ldg(a.masks + (static_cast<long long>(b) * a.N + n) * a.NW + j0 / 32);
        else see = n - j0 >= 31 ? ~0u : n < j0 ? 0u : (2u << (n - j0)) - 1u;
        if (a.N - j0 < 32) see &= (1u << (a.N - j0)) - 1u;
      }
      sees[rt][hf] = see;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float& x = z[rt][nt][2 * hf + k];
          x = (see >> (8 * nt + at_token(2 * t + k))) & 1u ? x * a.scale_log2 : kNegInf;
        }
    }
  st.weigh(z);

  // the sums of v are kept in units of 2^v_shift
  const float unit = __fdiv_rn(1.f, a.v_mul);
  bool odd = false;   // this lane saw a NaN or an infinity
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint4 hi[RT], lo[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = z[rt][2 * s + (k >> 1)][2 * (k & 1)] * unit, y = z[rt][2 * s + (k >> 1)][2 * (k & 1) + 1] * unit;
        ph[k] = bf16x2_pack(x, y);
        pl[k] = bf16x2_pack(x - __uint_as_float(ph[k] << 16), y - __uint_as_float(ph[k] & 0xffff0000u));
      }
      hi[rt] = make_uint4(ph[0], ph[1], ph[2], ph[3]);
      lo[rt] = make_uint4(pl[0], pl[1], pl[2], pl[3]);
    }
#pragma unroll
    for (int w = 0; w < CV / 8; ++w) {   // eight columns of the chunk at a time
      uint32_t vw[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + 16 * s + 8 * (k >> 1) + at_token(2 * t + (k & 1));
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (j < a.N) x = __ldg(reinterpret_cast<const uint4*>(a.v_new + base + j * rstride + g * CV) + w);
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
        const uint32_t b0 = __byte_perm(vw[0][i], vw[1][i], 0x5410), b1 = __byte_perm(vw[2][i], vw[3][i], 0x5410);
        const uint32_t d0 = __byte_perm(vw[0][i], vw[1][i], 0x7632), d1 = __byte_perm(vw[2][i], vw[3][i], 0x7632);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          mma_bf16(st.o[rt][8 * w + 2 * i], hi[rt], b0, b1);
          mma_bf16(st.o[rt][8 * w + 2 * i], lo[rt], b0, b1);
          mma_bf16(st.o[rt][8 * w + 2 * i + 1], hi[rt], d0, d1);
          mma_bf16(st.o[rt][8 * w + 2 * i + 1], lo[rt], d0, d1);
        }
      }
    }
  }
  // A product takes 0 * inf for NaN, so such elements were left out above and
  // reach only the rows that see their node (with a weight above zero, however
  // small: a weight that underflowed counts as the smallest one).
  if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
    for (int col = 0; col < 8; ++col) {
      const int src = (lane & ~3) | (col >> 1);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const int j = j0 + 8 * nt + at_token(col);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float p = __shfl_sync(0xffffffffu, col & 1 ? z[rt][nt][2 * hf + 1] : z[rt][nt][2 * hf], src);
            if (!((sees[rt][hf] >> (j - j0)) & 1u)) continue;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t v = a.v_new[base + j * rstride + t * CH + e * (D / 8) + i];
                if ((v & 0x7f80u) == 0x7f80u) st.o[rt][i][2 * hf + e] += (p == 0.f ? 1.17549435e-38f : p) * __uint_as_float(v << 16);
              }
          }
      }
    }
  }
}

// out row of this lane's chunk from a sum, 1 / l and the row's place
template <int D>
__device__ __forceinline__ void at_write_row(const AttendArgs& a, int b, int h, int r, const float* x, float inv, int t) {
  constexpr int CH = D / 4;
  const int n = r / a.G;
  const long long at = ((static_cast<long long>(b) * a.N + n) * a.Hkv + h) * a.G + (r - n * a.G);
  uint4* p = reinterpret_cast<uint4*>(a.out + at * D + t * CH);
#pragma unroll
  for (int i = 0; i < CH / 8; ++i)
    p[i] = make_uint4(bf16x2_pack(x[8 * i] * inv, x[8 * i + 1] * inv), bf16x2_pack(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                      bf16x2_pack(x[8 * i + 4] * inv, x[8 * i + 5] * inv), bf16x2_pack(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
}
__device__ __forceinline__ float at_lse(float m, float l) {
  // m in the log2 domain, l relative to 2^(m - 15)
  return l == 0.f ? kNegInf : (m - AT_PSHIFT + log2f(l)) * 0.69314718055994530942f;
}

template <int D, int RT>
__global__ void __launch_bounds__(AT_THREADS, RT == 1 ? 3 : 2) attend_q4_kernel(const AttendArgs a, int stages) {
  extern __shared__ __align__(128) unsigned char at_smem[];
  __shared__ long long scratch[AT_WARPS];
  constexpr int SB = at_stage_bytes(D), QB = at_q_bytes(D, RT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
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
  const int shares = at_shares(units, gridDim.x * AT_WARPS);
  const int share = warp * gridDim.x + blockIdx.x;   // few shares: one an SM
  if (share >= shares) return;
  const long long u0 = at_start(units, shares, share), u1 = at_start(units, shares, share + 1);

  const int rows = a.N * a.G, bpp = a.P / Q4_BLOCK;
  AtState<D, RT> st;
  AtCursor cur, pre;   // the block at hand; the next one to fetch
  at_seek(a, prefix, HR, u0, cur);
  pre = cur;
  long long pu = u0;
  uint32_t phase = 0u;      // a bit per stage
  bool failed = false;

  // Fetches the next block of the share into stage s (if it is a cached one
  // with a page in range); bit s of `have` says so.
  uint32_t have = 0u, bad = 0u;
  auto fetch = [&](int s) {
    have &= ~(1u << s);
    bad &= ~(1u << s);
    if (pu >= u1) return;
    if (at_len_ok(a, pre.len) && pre.i * Q4_BLOCK < pre.len) {
      const int page = __ldg(a.table + static_cast<long long>(pre.b) * a.W + pre.i / bpp);
      if (page >= 0 && page < a.pages) {
        have |= 1u << s;
        if (lane == 0) {
          const unsigned long long blk = (static_cast<unsigned long long>(page) * a.Hkv + pre.pair / a.row_tiles) * bpp + pre.i % bpp;
          mbar_arrive_expect_tx(&bars[s], SB);
          bulk_g2s(ring + s * SB, a.cache + blk * SB, SB, &bars[s]);
        }
      } else {
        bad |= 1u << s;
      }
    }
    at_next(a, prefix, HR, pre);
    ++pu;
  };
  for (int s = 0; s < stages; ++s) fetch(s);

  bool start = true, poison = false;   // a new triple begins; its result is void
  int first_i = 0, stage = 0;
  for (long long u = u0; u < u1; ++u) {
    const int h = cur.pair / a.row_tiles, row0 = (cur.pair - h * a.row_tiles) * 16 * RT;
    if (start) {
      st.clear();
      at_load_q<D, RT>(a, cur.b, h, row0, rows, qf, st);
      first_i = cur.i;
      start = poison = false;
    }
    if (!at_len_ok(a, cur.len)) {
      poison = true;
    } else if (cur.i * Q4_BLOCK < cur.len) {
      if (have & (1u << stage)) {
        if (!mbar_wait(&bars[stage], (phase >> stage) & 1u, a.timeout_ns)) failed = true;
        phase ^= 1u << stage;
        if (failed) poison = true;
        else at_cached_block<D, RT>(ring + stage * SB, min(cur.len - cur.i * Q4_BLOCK, Q4_BLOCK), qf, st);
      }
      if (bad & (1u << stage)) poison = true;
    } else if (a.k_new) {
      const int cached = (cur.len + Q4_BLOCK - 1) / Q4_BLOCK;
      at_fresh_block<D, RT>(a, cur.b, h, row0, rows, (cur.i - cached) * Q4_BLOCK, st);
    }
    __syncwarp();
    if (failed) break;   // no copy is started after one that did not arrive
    fetch(stage);
    stage = stage + 1 == stages ? 0 : stage + 1;

    if (cur.i + 1 == cur.units || u + 1 == u1) {
      const bool whole = first_i == 0 && cur.i + 1 == cur.units;
      float* part = a.ws + (static_cast<size_t>(share) * 2 + (first_i == 0 ? 1 : 0)) * at_partial_floats(D, RT);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float l = st.l[rt][hf];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          if (poison) l = __int_as_float(0x7fc00000);
          float x[D / 4];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            x[i] = st.o[rt][i][2 * hf];
            x[D / 8 + i] = st.o[rt][i][2 * hf + 1];
          }
          const int lr = 16 * rt + 8 * hf + g, r = row0 + lr;
          if (whole) {
            if (r < rows) {
              at_write_row<D>(a, cur.b, h, r, x, l == 0.f ? 0.f : a.v_mul / l, t);
              if (a.lse && t == 0) {
                const int n = r / a.G;
                a.lse[((static_cast<long long>(cur.b) * a.N + n) * a.Hkv + h) * a.G + (r - n * a.G)] = at_lse(st.m[rt][hf], l);
              }
            }
          } else {
            float4* p = reinterpret_cast<float4*>(part + static_cast<size_t>(lr) * D + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            if (t == 0) {
              part[16 * RT * D + lr] = st.m[rt][hf];
              part[16 * RT * D + 16 * RT + lr] = l;
            }
          }
        }
      start = true;
    }
    at_next(a, prefix, HR, cur);
  }
  if (failed) {
    // copies still on their way land before the warp leaves (or the wait gives up)
    for (int s = 0; s < stages; ++s)
      if (s != stage && (have & (1u << s))) mbar_wait(&bars[s], (phase >> s) & 1u, a.timeout_ns);
    // what this share did not finish is void: every triple of it
    AtCursor c;
    at_seek(a, prefix, HR, u0, c);
    for (long long u = u0; u < u1;) {
      const long long end = min(u1, u + c.units - c.i);
      const bool whole = c.i == 0 && end - u == c.units;
      const int h = c.pair / a.row_tiles, row0 = (c.pair - h * a.row_tiles) * 16 * RT;
      float* part = a.ws + (static_cast<size_t>(share) * 2 + (c.i == 0 ? 1 : 0)) * at_partial_floats(D, RT);
      for (int lr = lane; lr < 16 * RT; lr += 32) {
        const int r = row0 + lr, n = r / a.G;
        if (!whole) {
          for (int d = 0; d < D; ++d) part[lr * D + d] = 0.f;
          part[16 * RT * D + lr] = 0.f;
          part[16 * RT * D + 16 * RT + lr] = __int_as_float(0x7fc00000);
        } else if (r < rows) {
          const long long at = ((static_cast<long long>(c.b) * a.N + n) * a.Hkv + h) * a.G + (r - n * a.G);
          for (int d = 0; d < D; ++d) a.out[at * D + d] = 0x7fc0u;
          if (a.lse) a.lse[at] = __int_as_float(0x7fc00000);
        }
      }
      for (; u < end; ++u) at_next(a, prefix, HR, c);
    }
  }
}

// Joins the partials of triples that several shares worked on: a CTA a triple,
// a thread four columns of a row, the shares in their order.
constexpr int AJN_THREADS = 128;
template <int D, int RT>
__global__ void __launch_bounds__(AJN_THREADS) attend_q4_join_kernel(const AttendArgs a, int warps) {
  extern __shared__ __align__(128) unsigned char at_smem[];
  __shared__ long long scratch[AJN_THREADS / 32];
  long long* prefix = reinterpret_cast<long long*>(at_smem);
  at_prefix<AJN_THREADS>(a, prefix, scratch);
  const int HR = a.Hkv * a.row_tiles, rows = a.N * a.G;
  const long long units = prefix[a.B] * HR;
  const int shares = at_shares(units, warps);
  for (long long x = blockIdx.x; x < static_cast<long long>(a.B) * HR; x += gridDim.x) {
    const int b = static_cast<int>(x / HR), pair = static_cast<int>(x % HR);
    const long long n = prefix[b + 1] - prefix[b], u = prefix[b] * HR + pair * n;
    const int wa = at_owner(units, shares, u), wb = at_owner(units, shares, u + n - 1);
    if (wa == wb) continue;
    const int h = pair / a.row_tiles, row0 = (pair - h * a.row_tiles) * 16 * RT;
    for (int e = threadIdx.x; e < 16 * RT * (D / 4); e += AJN_THREADS) {
      const int lr = e / (D / 4), d4 = e % (D / 4), r = row0 + lr;
      if (r >= rows) continue;
      float m = kNegInf, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = wa; w <= wb; ++w) {
        const float* part = a.ws + (static_cast<size_t>(w) * 2 + (w == wa ? 1 : 0)) * at_partial_floats(D, RT);
        const float pm = part[16 * RT * D + lr], pl = part[16 * RT * D + 16 * RT + lr];
        const float4 po = *reinterpret_cast<const float4*>(part + static_cast<size_t>(lr) * D + d4 * 4);
        const float mn = fmaxf(m, pm), ref = mn == kNegInf ? 0.f : mn;
        const float c0 = at_corr(m - ref), c1 = at_corr(pm - ref);
        l = l * c0 + pl * c1;
        o.x = o.x * c0 + po.x * c1;
        o.y = o.y * c0 + po.y * c1;
        o.z = o.z * c0 + po.z * c1;
        o.w = o.w * c0 + po.w * c1;
        m = mn;
      }
      const float inv = l == 0.f ? 0.f : a.v_mul / l;
      const int node = r / a.G;
      const long long at = ((static_cast<long long>(b) * a.N + node) * a.Hkv + h) * a.G + (r - node * a.G);
      *reinterpret_cast<uint2*>(a.out + at * D + d4 * 4) = make_uint2(bf16x2_pack(o.x * inv, o.y * inv), bf16x2_pack(o.z * inv, o.w * inv));
      if (a.lse && d4 == 0) a.lse[at] = at_lse(m, l);
    }
  }
}

}  // namespace sv
