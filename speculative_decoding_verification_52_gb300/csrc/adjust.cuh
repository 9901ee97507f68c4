// adjust.cuh -- what changes the logits between the model and the verification:
// penalties for tokens that were seen, biases, and grammar masks.
//
// For row r of sequence b and token v, in fp32, rounded once at the end:
//   n    = times v was generated (history[prompt..]) or proposed before the row
//          (chain: node_tokens[0..r-1]; tree: the row's node and its ancestors)
//   l    = logit;  if v was in the prompt or n > 0:  l = l > 0 ? l / rep : l * rep
//   l   -= freq * n + (n > 0 ? pres : 0);  l += sum of v's biases
//   l    = -inf where the row's mask has no bit for v
//
// What bounds it: one read and one write of every logit (and no read where a mask
// rules out a whole vector).  A CTA takes a chunk of one sequence's vocabulary and
// all its rows (or a share of them):
//   1. the history is counted into shared memory, one word a token: seen flag, patch
//      flag (proposed or biased), count;
//   2. the rows stream through, 16 bytes at a time (rows whose start is not aligned
//      are cut at the first 16-byte border).  A lane has one place in all rows, whose
//      words it reads once; seen tokens are changed on the way, element by element of
//      the vector where some lane of the warp has one;
//   3. proposed and biased tokens, which differ from row to row and are few, are
//      computed one by one from the input, a warp to a token and a lane to a row.
//      Step 2 leaves them as they are (or masked), so the output may be the input.
// Measured at 256 x 6 rows of 128,256 bf16, 2,048 tokens of history each: the copy
// alone 130 us (6.1 TB/s), 154 us with the history's penalties, 176 us with 64
// biases and a mask a row too (a step's mask words and then its logits are two loads
// that wait for each other; ALU 54 %).  Seen tokens done in step 3 as well, 3 million single
// updates, cost 52 us more than the copy; penalties on all vectors alike, with one
// test a vector, 296 us in all.
#pragma once

#include "common.cuh"

namespace sv {

constexpr int AJ_THREADS = 256;
constexpr int AJ_MAX_CHUNK = 4096;

struct AdjustArgs {
  const unsigned char* logits;   // [B, R, V]
  unsigned char* out;            // [B, R, V], may be logits
  const int32_t* history;        // [B, H] or null
  const int32_t* prompt_len;     // [B] or null (nothing of the history is prompt)
  const int32_t* hist_len;       // [B]
  const float* repetition;       // [B] or null
  const float* frequency;        // [B] or null
  const float* presence;         // [B] or null
  const int32_t* nodes;          // [B, Nt] or null
  const uint32_t* masks;         // [B, R, NW] or null (a chain)
  const int32_t* bias_tokens;    // [B, M] or null
  const float* bias_values;      // [B, M]
  const uint32_t* allowed;       // [B, R, VW] or null
  int B, R, V, H, Nt, NW, M, VW;
  int chunk, chunks;             // tokens of a chunk (a multiple of 32), chunks of the vocabulary
  int row_splits;                // CTAs that share a chunk's rows
};

constexpr uint32_t AJ_SEEN = 1u, AJ_PATCH = 2u, AJ_ONE = 4u;   // flag, flag, one generated token

struct AdjustScalars {
  // inv = 1 / rep, rounded: a quotient is its product with the logit, off by 2^-23 at most
  // where one rounding would be 2^-24.  (Divisions take 197 us where this takes 176: 256 x 6
  // rows of 128,256 bf16, everything on.)
  float rep, inv, freq, pres;
};

__device__ __forceinline__ float adjust_one(float l, uint32_t word, int more, const AdjustScalars& s) {
  const int n = static_cast<int>(word >> 2) + more;
  if ((word & AJ_SEEN) || n > 0) l *= l > 0.f ? s.inv : s.rep;
  if (n > 0) l = __fsub_rn(l, __fadd_rn(__fmul_rn(s.freq, static_cast<float>(n)), s.pres));
  return l;
}

__device__ __forceinline__ uint16_t bf16_bits(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

template <class T>
__device__ __forceinline__ void adjust_store(unsigned char* base, long long i, float x) {
  if constexpr (T::esz == 4) reinterpret_cast<float*>(base)[i] = x;
  else reinterpret_cast<uint16_t*>(base)[i] = bf16_bits(x);
}

// bytes of ones for the set ones of four bits
__device__ __forceinline__ uint32_t adjust_bytes(uint32_t four) { return ((four * 0x00204081u) & 0x01010101u) * 0xffu; }
// a 16-byte vector of logits with -inf where its mask has no bit
template <class T>
__device__ __forceinline__ uint4 adjust_mask(uint4 r, uint32_t bits) {
  const uint32_t lo = adjust_bytes(bits & 15u);
  if constexpr (T::esz == 4) {
    const uint32_t k[4] = {__byte_perm(lo, 0u, 0x0000), __byte_perm(lo, 0u, 0x1111), __byte_perm(lo, 0u, 0x2222), __byte_perm(lo, 0u, 0x3333)};
    r.x = (r.x & k[0]) | (0xff800000u & ~k[0]);
    r.y = (r.y & k[1]) | (0xff800000u & ~k[1]);
    r.z = (r.z & k[2]) | (0xff800000u & ~k[2]);
    r.w = (r.w & k[3]) | (0xff800000u & ~k[3]);
  } else {
    const uint32_t hi = adjust_bytes(bits >> 4);
    const uint32_t k[4] = {__byte_perm(lo, 0u, 0x1100), __byte_perm(lo, 0u, 0x3322), __byte_perm(hi, 0u, 0x1100), __byte_perm(hi, 0u, 0x3322)};
    r.x = (r.x & k[0]) | (0xff80ff80u & ~k[0]);
    r.y = (r.y & k[1]) | (0xff80ff80u & ~k[1]);
    r.z = (r.z & k[2]) | (0xff80ff80u & ~k[2]);
    r.w = (r.w & k[3]) | (0xff80ff80u & ~k[3]);
  }
  return r;
}

// Seen tokens of U rows' vectors: word[e] belongs to element e of each; `here`
// the elements that this lane changes, `some` those that any lane of the warp does.
template <class T, int U>
__device__ __forceinline__ void adjust_seen(uint4 (&q)[U], const uint32_t* word, uint32_t here, uint32_t some, const AdjustScalars& s) {
#pragma unroll
  for (int e = 0; e < T::vpe; ++e) {
    if (!((some >> e) & 1u)) continue;
    const bool mine = (here >> e) & 1u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t& w = (&q[u].x)[T::esz == 4 ? e : e / 2];
      if constexpr (T::esz == 4) {
        const float y = adjust_one(__uint_as_float(w), word[e], 0, s);
        if (mine) w = __float_as_uint(y);
      } else {
        const float y = adjust_one(__uint_as_float(e & 1 ? w & 0xffff0000u : w << 16), word[e], 0, s);
        const uint32_t z = __byte_perm(w, bf16_bits(y), e & 1 ? 0x5410 : 0x3254);
        if (mine) w = z;
      }
    }
  }
}

// The sum of a token's biases, in the list's order (the warp together).
__device__ __forceinline__ float adjust_bias(const AdjustArgs& a, int b, int tok) {
  const int lane = threadIdx.x & 31;
  float bias = 0.f;
  if (a.bias_tokens) {
    const int32_t* bt = a.bias_tokens + static_cast<long long>(b) * a.M;
    for (int m0 = 0; m0 < a.M; m0 += 32) {
      uint32_t hit = __ballot_sync(0xffffffffu, m0 + lane < a.M && bt[m0 + lane] == tok);
      for (; hit; hit &= hit - 1)
        bias = __fadd_rn(bias, a.bias_values[static_cast<long long>(b) * a.M + m0 + __ffs(hit) - 1]);
    }
  }
  return bias;
}
// A proposed or biased token in the lane's row r (the warp together); false where
// there is no such row.
template <class T>
__device__ __forceinline__ bool adjust_patch(const AdjustArgs& a, int b, int r, int r1, int tok, uint32_t word, float bias,
                                             const AdjustScalars& s, float& x) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(b) * a.R + r;
  int more = 0;
  if (a.nodes) {
    const int32_t* nb = a.nodes + static_cast<long long>(b) * a.Nt;
    for (int j0 = 0; j0 < a.Nt; j0 += 32) {
      const uint32_t hit = __ballot_sync(0xffffffffu, j0 + lane < a.Nt && nb[j0 + lane] == tok);
      if (!hit || r >= r1) continue;
      uint32_t before;
      if (a.masks) before = a.masks[row * a.NW + j0 / 32] & (j0 == 0 ? ~1u : ~0u);
      else before = r <= j0 ? 0u : r - j0 >= 32 ? ~0u : (1u << (r - j0)) - 1u;
      more += __popc(hit & before);
    }
  }
  if (r >= r1) return false;
  x = kNegInf;
  if (a.allowed && !((a.allowed[row * a.VW + (tok >> 5)] >> (tok & 31)) & 1u)) return true;
  x = adjust_one(T::load(a.logits, row * a.V + tok), word, more, s);
  if (a.bias_tokens) x = __fadd_rn(x, bias);
  return true;
}

// VEC: input and output have the same offset from 16-byte borders.
template <class T, bool VEC>
__global__ void __launch_bounds__(AJ_THREADS, 6) adjust_logits_kernel(const AdjustArgs a) {
  extern __shared__ __align__(16) unsigned char aj_smem[];
  __shared__ int n_patch, n_taken;
  uint32_t* word = reinterpret_cast<uint32_t*>(aj_smem);                      // [chunk]
  uint16_t* patch = reinterpret_cast<uint16_t*>(word + a.chunk);              // [min(chunk, Nt + M)]

  const int split = blockIdx.x % a.row_splits;
  const int bc = blockIdx.x / a.row_splits;
  const int b = bc / a.chunks, c = bc - b * a.chunks;
  const int v0 = c * a.chunk, n = min(a.chunk, a.V - v0);
  const int r0 = static_cast<int>(static_cast<long long>(a.R) * split / a.row_splits);
  const int r1 = static_cast<int>(static_cast<long long>(a.R) * (split + 1) / a.row_splits);

  if (threadIdx.x == 0) n_patch = n_taken = 0;
  for (int i = threadIdx.x; i < a.chunk / 4; i += AJ_THREADS) reinterpret_cast<uint4*>(word)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  if (a.history) {
    const int hl = min(max(a.hist_len[b], 0), a.H), pl = a.prompt_len ? a.prompt_len[b] : 0;
    const int32_t* hb = a.history + static_cast<long long>(b) * a.H;
    for (int i0 = threadIdx.x; i0 < hl; i0 += 4 * AJ_THREADS) {
      uint32_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = i0 + u * AJ_THREADS < hl ? static_cast<uint32_t>(__ldg(hb + i0 + u * AJ_THREADS)) - static_cast<uint32_t>(v0) : ~0u;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (v[u] >= static_cast<uint32_t>(n)) continue;
        if (i0 + u * AJ_THREADS < pl) atomicOr(&word[v[u]], AJ_SEEN);
        else atomicAdd(&word[v[u]], AJ_ONE);
      }
    }
  }
  const int nn = a.nodes ? a.Nt : 0, extra = nn + (a.bias_tokens ? a.M : 0);
  for (int i = threadIdx.x; i < extra; i += AJ_THREADS) {
    const int tok = i < nn ? a.nodes[static_cast<long long>(b) * a.Nt + i] : a.bias_tokens[static_cast<long long>(b) * a.M + i - nn];
    const uint32_t v = static_cast<uint32_t>(tok) - static_cast<uint32_t>(v0);
    if (v >= static_cast<uint32_t>(n)) continue;
    if (!(atomicOr(&word[v], AJ_PATCH) & AJ_PATCH)) patch[atomicAdd(&n_patch, 1)] = static_cast<uint16_t>(v);
  }
  __syncthreads();

  AdjustScalars s;
  s.rep = a.repetition ? a.repetition[b] : 1.f;
  s.inv = __fdiv_rn(1.f, s.rep);
  s.freq = a.frequency ? a.frequency[b] : 0.f;
  s.pres = a.presence ? a.presence[b] : 0.f;
  const int lane = threadIdx.x & 31;
  const long long row0 = static_cast<long long>(b) * a.R;
  const long long at0 = (row0 + r0) * a.V + v0;   // first element of the first row
  const int nr = r1 - r0;
  auto changes = [](uint32_t w) { return w != 0u && !(w & AJ_PATCH); };
  // Each warp's first proposed or biased token, before the stream, which the other
  // warps have begun by then: its loads wait one for the other.
  const bool early = (threadIdx.x >> 5) < n_patch;
  bool ready = false;
  float early_x = 0.f;
  if (early) {
    const int v = patch[threadIdx.x >> 5];
    ready = adjust_patch<T>(a, b, r0 + lane, r1, v0 + v, word[v], adjust_bias(a, b, v0 + v), s, early_x);
  }
  if constexpr (VEC) {
    // a piece: 32 vectors, one a lane, three rows at a time
    constexpr int E = T::vpe, U = 3;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(a.logits) & 15u) / T::esz);
    const bool even = a.V % E == 0 && off == 0;   // every row starts at a border
    const int blocks = (n / E + 31) / 32;
    for (;;) {
      int blk = 0;
      if (lane == 0) blk = atomicAdd(&n_taken, 1);
      blk = __shfl_sync(0xffffffffu, blk, 0);
      if (blk >= blocks) break;
      const int i0 = (blk * 32 + lane) * E;
      uint32_t w[E];
      uint32_t here = 0u, some = 0u;
      if (even) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const uint4 x = i0 + E <= n ? reinterpret_cast<const uint4*>(word)[(i0 + e) / 4] : make_uint4(0u, 0u, 0u, 0u);
          w[e] = x.x; w[e + 1] = x.y; w[e + 2] = x.z; w[e + 3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) here |= static_cast<uint32_t>(changes(w[e])) << e;
        some = __reduce_or_sync(0xffffffffu, here);
        const uint32_t* mw = a.allowed ? a.allowed + (row0 + r0) * a.VW + ((v0 + i0) >> 5) : nullptr;
        const bool in = i0 + E <= n;
        for (int r = 0; r < nr; r += U) {
          uint4 q[U];
          uint32_t bits[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            bits[u] = in && r + u < nr ? (1u << E) - 1u : 0u;
            if (mw && bits[u]) bits[u] &= __ldg(mw + static_cast<long long>(r + u) * a.VW) >> ((v0 + i0) & 31);
          }
          const long long at = (at0 + static_cast<long long>(r) * a.V + i0) * T::esz;
          const long long rb = static_cast<long long>(a.V) * T::esz;
#pragma unroll
          for (int u = 0; u < U; ++u)
            q[u] = bits[u] ? __ldcs(reinterpret_cast<const uint4*>(a.logits + at + u * rb)) : make_uint4(0u, 0u, 0u, 0u);
          if (some) adjust_seen<T, U>(q, w, here, some, s);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (in && r + u < nr) __stcs(reinterpret_cast<uint4*>(a.out + at + u * rb), mw ? adjust_mask<T>(q[u], bits[u]) : q[u]);
        }
      } else {
        for (int r = 0; r < nr; ++r) {
          const long long row = at0 + static_cast<long long>(r) * a.V;
          // elements before the row's first border
          const int e0 = i0 + ((E - static_cast<int>((row + off) & (E - 1))) & (E - 1));
          const bool in = e0 + E <= n;
          uint32_t bits = in ? (1u << E) - 1u : 0u;
          if (a.allowed && in) {
            const int v = v0 + e0;
            const uint32_t* mw = a.allowed + (row0 + r0 + r) * a.VW + (v >> 5);
            bits &= __funnelshift_r(__ldg(mw), (v & 31) + E > 32 ? __ldg(mw + 1) : 0u, v & 31);
          }
          uint4 q[1] = {bits ? __ldcs(reinterpret_cast<const uint4*>(a.logits + (row + e0) * T::esz)) : make_uint4(0u, 0u, 0u, 0u)};
          here = 0u;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            w[e] = in ? word[e0 + e] : 0u;
            here |= static_cast<uint32_t>(changes(w[e])) << e;
          }
          some = __reduce_or_sync(0xffffffffu, here);
          if (some) adjust_seen<T, 1>(q, w, here, some, s);
          if (in) __stcs(reinterpret_cast<uint4*>(a.out + (row + e0) * T::esz), a.allowed ? adjust_mask<T>(q[0], bits) : q[0]);
        }
      }
    }
    // what the borders cut off at the rows' starts and ends
    if (!even || n % E != 0) {
      for (int k = threadIdx.x; k < nr * 2 * E; k += AJ_THREADS) {
        const int rr = k / (2 * E), j = k % (2 * E);
        const long long row = at0 + static_cast<long long>(rr) * a.V;
        const int head = min(n, (E - static_cast<int>((row + off) & (E - 1))) & (E - 1));
        const int e = j < E ? j : head + (n - head) / E * E + j - E;
        if (j < E ? e >= head : e >= n) continue;
        const int v = v0 + e;
        const bool ok = !a.allowed || ((a.allowed[(row0 + r0 + rr) * a.VW + (v >> 5)] >> (v & 31)) & 1u);
        float x = ok ? T::load(a.logits, row + e) : kNegInf;
        if (ok && changes(word[e])) x = adjust_one(x, word[e], 0, s);
        adjust_store<T>(a.out, row + e, x);
      }
    }
  } else {
    for (int k = threadIdx.x; k < n; k += AJ_THREADS)
#pragma unroll 4
      for (int r = 0; r < nr; ++r) {
        const int v = v0 + k;
        const bool ok = !a.allowed || ((a.allowed[(row0 + r0 + r) * a.VW + (v >> 5)] >> (v & 31)) & 1u);
        const long long at = at0 + static_cast<long long>(r) * a.V + k;
        float x = ok ? T::load(a.logits, at) : kNegInf;
        if (ok && changes(word[k])) x = adjust_one(x, word[k], 0, s);
        adjust_store<T>(a.out, at, x);
      }
  }
  __syncthreads();   // what was streamed comes before what follows

  // The first token of each warp is known already; its place was left alone.
  if (early && ready) adjust_store<T>(a.out, at0 + static_cast<long long>(lane) * a.V + patch[threadIdx.x >> 5], early_x);
  for (int i = threadIdx.x >> 5; i < n_patch; i += AJ_THREADS / 32) {
    const int v = patch[i];
    const bool first = i < AJ_THREADS / 32;
    if (first && nr <= 32) continue;
    const float bias = adjust_bias(a, b, v0 + v);
    for (int rb = first ? 32 : 0; rb < nr; rb += 32) {
      float x;
      if (adjust_patch<T>(a, b, r0 + rb + lane, r1, v0 + v, word[v], bias, s, x))
        adjust_store<T>(a.out, at0 + static_cast<long long>(rb + lane) * a.V + v, x);
    }
  }
}

}  // namespace sv
