// kv_q4.cuh -- the cache held in 4 bits: its format, and the two kernels that
// quantise bf16 keys and values into its pages.
//
// Format.  The cache is [pages, Hkv, P / 32, 36 * D] bytes: a page keeps each
// kv head's tokens in blocks of 32.  A block is one contiguous run that a
// reader fetches with a single bulk copy:
//   [32 x D/2 key codes | 32 x D/2 value codes | 32 x D/16 key scales | 32 x D/16 value scales]
// and element d of a token stands for
//   e2m1(code) * e4m3(scale of the 16 elements d / 16) * 2^shift
// (codes two to a byte, the even element in the low half).  e2m1 has 2 and e4m3
// has 4 significant bits, so code * scale has at most 6 and lies in
// [2^-10, 2688]: it is exact in f16 and in bf16, and so is everything a reader
// dequantises.  The shift is a power of two for the same reason.
//
// Quantising a group of 16 x: s = e4m3(max|x| 2^-shift / 6), rounded to nearest
// even and saturated at 448; code = e2m1(x 2^-shift / s), rounded to nearest
// even and saturated at 6.  s = 0 gives codes 0; a group with a NaN or an
// infinity gets the scale NaN and codes 0, so that a reader sees the NaN.
#pragma once

#include "common.cuh"

namespace sv {

constexpr int Q4_BLOCK = 32;     // tokens of a block
constexpr int Q4_THREADS = 256;

__host__ __device__ constexpr int q4_block_bytes(int D) { return 36 * D; }

struct KvQ4Args {
  const uint16_t* k;           // [rows, Hkv, D] bf16
  const uint16_t* v;
  unsigned char* cache;
  const int32_t* slots;        // store: [T]
  const int32_t* table;        // commit: [B, W]
  const int32_t* lengths;      // commit: [B]
  const int32_t* path;         // commit: [B, PW] or null
  const int32_t* count;        // commit: [B]
  int32_t* new_lengths;        // commit: [B]
  int T, Hkv, P, pages;
  int B, N, W, PW;
  float k_mul, v_mul;          // 2^-shift
};

__device__ __forceinline__ uint32_t bf16x2_abs(uint32_t x) { return x & 0x7fff7fffu; }

// x / 6 for an x of 8 significant bits, as close as rounding it to e4m3 needs: x / 6
// either is a border between two e4m3 values (6 times one has 7 bits), or at least
// 2^-8 of its size away from it.  So the product with 1 / 6, off by 2^-23, is rounded
// to 12 bits, which restores a border and passes none.  (What lies below 2^-9 of
// e4m3's smallest value becomes 0 in any case.)
__device__ __forceinline__ float q4_sixth(float x) {
  const float y = x * (1.f / 6.f), c = __fmul_rn(fminf(y, 1e30f), 4097.f);
  return __fsub_rn(c, __fsub_rn(c, y));
}

// One group of 16 elements: 8 code bytes and the scale byte.
//
// x / s is formed as x * (1 / s), a few f32 units off, and then rounded to
// multiples of 2^-10 by adding and subtracting 1.5 * 2^13.  That gives the same
// code as the exact quotient: x has 8 significant bits and t * s at most 7 for
// each border t between two codes, so x / s either is t, and the rounding
// restores it, or differs from t by at least t * 2^-8 >= 2^-10, twice the
// rounding.  (Divisions cost about ten instructions each: 32,001 tokens of 8 heads of
// 128 take 30.7 us, 5.5 TB/s, issue slots 78 % used, and took an eighth longer with two
// divisions a group.)  The sign of a zero that the rounding loses is put back.
__device__ __forceinline__ void q4_group(const uint4& lo, const uint4& hi, float mul, uint2& codes, uint32_t& scale) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t m = bf16x2_abs(w[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = bf16x2_max_nan(m, bf16x2_abs(w[i]));
  const float top = fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  codes = make_uint2(0u, 0u);
  if (!(top < __builtin_huge_valf())) {
    scale = 0x7fu;
    return;
  }
  // (a finite element times 2^-shift may pass fp32's range: the scale is 448 then)
  uint16_t e;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e) : "f"(0.f), "f"(q4_sixth(fminf(top * mul, 3.402823466e+38f))));
  scale = e & 0xffu;
  if (scale == 0u) return;
  uint32_t s2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(e));
  float s;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(s) : "r"(s2));
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
  r *= mul;
  const float kRound = 12288.f;   // 1.5 * 2^13: f32 keeps multiples of 2^-10 there
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xffff0000u);
    const float y0 = copysignf(__fsub_rn(__fadd_rn(__fmul_rn(x0, r), kRound), kRound), x0);
    const float y1 = copysignf(__fsub_rn(__fadd_rn(__fmul_rn(x1, r), kRound), kRound), x1);
    uint32_t q;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}" : "=r"(q) : "f"(y0), "f"(y1));
    out[i] = q;
  }
  codes.x = out[0] | (out[1] << 8) | (out[2] << 16) | (out[3] << 24);
  codes.y = out[4] | (out[5] << 8) | (out[6] << 16) | (out[7] << 24);
}

// where token t of head h starts, in blocks
__device__ __forceinline__ unsigned char* q4_block(unsigned char* cache, int page, int h, int in_page, int Hkv, int P, int D) {
  const unsigned long long blk = (static_cast<unsigned long long>(page) * Hkv + h) * (P / Q4_BLOCK) + in_page / Q4_BLOCK;
  return cache + blk * q4_block_bytes(D);
}

// the group's 8 code bytes and its scale into the block
template <int D>
__device__ __forceinline__ void q4_put(unsigned char* blk, int row, int g, bool value, const uint2& codes, uint32_t scale) {
  *reinterpret_cast<uint2*>(blk + (value ? Q4_BLOCK * D / 2 : 0) + row * (D / 2) + g * 8) = codes;
  blk[Q4_BLOCK * D + (value ? Q4_BLOCK * D / 16 : 0) + row * (D / 16) + g] = static_cast<unsigned char>(scale);
}

// One group a thread, key and value: consecutive threads take a token's D / 16
// groups, then the next token of the same head, so that a warp's loads cover
// whole rows and its code and scale stores fill whole 32-byte sectors of a
// block wherever the tokens are neighbours in the cache.
template <int D>
__global__ void __launch_bounds__(Q4_THREADS) kv_store_q4_kernel(const KvQ4Args a) {
  constexpr int GR = D / 16, TOK = Q4_THREADS / GR;   // groups of a row, tokens of a CTA
  const int h = blockIdx.y;
  const int g = threadIdx.x % GR;
  const long long t = static_cast<long long>(blockIdx.x) * TOK + threadIdx.x / GR;
  if (t >= a.T) return;
  const int slot = a.slots[t];
  if (slot < 0) return;
  const int page = slot / a.P, in_page = slot - page * a.P;
  if (page >= a.pages) return;
  const long long at = (t * a.Hkv + h) * D + g * 16;
  const uint4* kp = reinterpret_cast<const uint4*>(a.k + at);
  const uint4* vp = reinterpret_cast<const uint4*>(a.v + at);
  const uint4 k0 = __ldcs(kp), k1 = __ldcs(kp + 1), v0 = __ldcs(vp), v1 = __ldcs(vp + 1);
  unsigned char* blk = q4_block(a.cache, page, h, in_page, a.Hkv, a.P, D);
  uint2 codes;
  uint32_t scale;
  q4_group(k0, k1, a.k_mul, codes, scale);
  q4_put<D>(blk, in_page % Q4_BLOCK, g, false, codes, scale);
  q4_group(v0, v1, a.v_mul, codes, scale);
  q4_put<D>(blk, in_page % Q4_BLOCK, g, true, codes, scale);
}

// Accepted drafts into the pages behind lengths[b].  One CTA or more a sequence, whose
// threads take a group each, key and value; every CTA checks the request first, as a
// whole, so that a refused one changes nothing.
template <int D>
__global__ void __launch_bounds__(Q4_THREADS) kv_commit_q4_kernel(const KvQ4Args a) {
  constexpr int GR = D / 16;
  const int b = blockIdx.x;
  const int n = a.count[b], L = a.lengths[b];
  if (n < 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) a.new_lengths[b] = L;
    return;
  }
  bool ok = L >= 0 && static_cast<long long>(L) + n <= static_cast<long long>(a.W) * a.P && n <= (a.path ? a.PW : a.N);
  const int32_t* table = a.table + static_cast<long long>(b) * a.W;
  const int32_t* path = a.path ? a.path + static_cast<long long>(b) * a.PW : nullptr;
  for (int j = threadIdx.x; ok && j < n; j += Q4_THREADS) {
    const int page = table[(L + j) / a.P];
    const int src = path ? path[j] : j;
    ok = page >= 0 && page < a.pages && src >= 0 && src < a.N;
  }
  ok = __syncthreads_and(ok);
  if (blockIdx.y == 0 && threadIdx.x == 0) a.new_lengths[b] = ok ? L + n : -1;
  if (!ok) return;
  const long long items = static_cast<long long>(n) * a.Hkv * GR;
  for (long long i = static_cast<long long>(blockIdx.y) * Q4_THREADS + threadIdx.x; i < items;
       i += static_cast<long long>(gridDim.y) * Q4_THREADS) {
    const int g = static_cast<int>(i % GR);
    const int h = static_cast<int>((i / GR) % a.Hkv), j = static_cast<int>(i / GR / a.Hkv);
    const int src = path ? path[j] : j;
    const int pos = L + j, page = table[pos / a.P], in_page = pos % a.P;
    const long long at = ((static_cast<long long>(b) * a.N + src) * a.Hkv + h) * D + g * 16;
    const uint4* kp = reinterpret_cast<const uint4*>(a.k + at);
    const uint4* vp = reinterpret_cast<const uint4*>(a.v + at);
    const uint4 k0 = __ldcs(kp), k1 = __ldcs(kp + 1), v0 = __ldcs(vp), v1 = __ldcs(vp + 1);
    unsigned char* blk = q4_block(a.cache, page, h, in_page, a.Hkv, a.P, D);
    uint2 codes;
    uint32_t scale;
    q4_group(k0, k1, a.k_mul, codes, scale);
    q4_put<D>(blk, in_page % Q4_BLOCK, g, false, codes, scale);
    q4_group(v0, v1, a.v_mul, codes, scale);
    q4_put<D>(blk, in_page % Q4_BLOCK, g, true, codes, scale);
  }
}

}  // namespace sv
