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
// What bounds it: one read and one write of every logit (and no read where a
// mask rules out a whole vector).  So a CTA takes a chunk of one sequence's
// vocabulary and all its rows (or a share of them): the history is counted once
// into shared memory (one word a token: seen flag, patch flag, count), the rows
// stream past it with 16-byte vectors, and each thread keeps the words of its
// vectors in registers while it goes through the rows.  Tokens that differ from
// row to row (proposed ones) or carry a bias are few: they are flagged, skipped
// by the stream and done one by one afterwards, a warp to a token and a lane to
// a row.  Nothing is written before it has been read by the same CTA, so the
// output may be the input.
#pragma once

#include "common.cuh"

namespace sv {

constexpr int AJ_THREADS = 256;
constexpr int AJ_MAX_CHUNK = 8192;

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
  float rep, freq, pres;
};

__device__ __forceinline__ float adjust_one(float l, uint32_t word, int more, const AdjustScalars& s) {
  const int n = static_cast<int>(word >> 2) + more;
  if ((word & AJ_SEEN) || n > 0) l = l > 0.f ? __fdiv_rn(l, s.rep) : __fmul_rn(l, s.rep);
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

// one 16-byte vector of logits under its words and mask bits
template <class T>
__device__ __forceinline__ uint4 adjust_vec(const uint4& q, const uint32_t* word, uint32_t any, uint32_t bits,
                                            const AdjustScalars& s) {
  constexpr int E = T::vpe;
  uint4 r = q;
  if (any) {
    float x[E];
    T::unpack(q, x);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (word[e]) x[e] = adjust_one(x[e], word[e], 0, s);
    if constexpr (T::esz == 4) {
      r = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
      r = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  constexpr uint32_t kAll = (1u << E) - 1u;
  if (bits != kAll) {
    uint32_t* w = &r.x;
    if constexpr (T::esz == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!((bits >> e) & 1u)) w[e] = 0xff800000u;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!((bits >> (2 * e)) & 1u)) w[e] = (w[e] & 0xffff0000u) | 0xff80u;
        if (!((bits >> (2 * e + 1)) & 1u)) w[e] = (w[e] & 0xffffu) | 0xff800000u;
      }
    }
  }
  return r;
}

template <class T, bool VEC>
__global__ void __launch_bounds__(AJ_THREADS) adjust_logits_kernel(const AdjustArgs a) {
  extern __shared__ __align__(16) unsigned char aj_smem[];
  __shared__ int n_patch;
  uint32_t* word = reinterpret_cast<uint32_t*>(aj_smem);                      // [chunk]
  uint16_t* patch = reinterpret_cast<uint16_t*>(word + a.chunk);              // [min(chunk, Nt + M)]

  const int split = blockIdx.x % a.row_splits;
  const long long bc = blockIdx.x / a.row_splits;
  const int b = static_cast<int>(bc / a.chunks), c = static_cast<int>(bc % a.chunks);
  const int v0 = c * a.chunk, n = min(a.chunk, a.V - v0);
  const int r0 = static_cast<int>(static_cast<long long>(a.R) * split / a.row_splits);
  const int r1 = static_cast<int>(static_cast<long long>(a.R) * (split + 1) / a.row_splits);

  for (int i = threadIdx.x; i < a.chunk / 4; i += AJ_THREADS) reinterpret_cast<uint4*>(word)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (threadIdx.x == 0) n_patch = 0;
  __syncthreads();
  if (a.history) {
    const int hl = min(max(a.hist_len[b], 0), a.H), pl = a.prompt_len ? a.prompt_len[b] : 0;
    const int32_t* hb = a.history + static_cast<long long>(b) * a.H;
    for (int i = threadIdx.x; i < hl; i += AJ_THREADS) {
      const uint32_t v = static_cast<uint32_t>(hb[i]) - static_cast<uint32_t>(v0);
      if (v >= static_cast<uint32_t>(n)) continue;
      if (i < pl) atomicOr(&word[v], AJ_SEEN);
      else atomicAdd(&word[v], AJ_ONE);
    }
  }
  const int extra = (a.nodes ? a.Nt : 0) + (a.bias_tokens ? a.M : 0);
  for (int i = threadIdx.x; i < extra; i += AJ_THREADS) {
    const int nn = a.nodes ? a.Nt : 0;
    const int tok = i < nn ? a.nodes[static_cast<long long>(b) * a.Nt + i] : a.bias_tokens[static_cast<long long>(b) * a.M + i - nn];
    const uint32_t v = static_cast<uint32_t>(tok) - static_cast<uint32_t>(v0);
    if (v >= static_cast<uint32_t>(n)) continue;
    if (!(atomicOr(&word[v], AJ_PATCH) & AJ_PATCH)) patch[atomicAdd(&n_patch, 1)] = static_cast<uint16_t>(v);
  }
  __syncthreads();

  AdjustScalars s;
  s.rep = a.repetition ? a.repetition[b] : 1.f;
  s.freq = a.frequency ? a.frequency[b] : 0.f;
  s.pres = a.presence ? a.presence[b] : 0.f;
  const long long row0 = static_cast<long long>(b) * a.R;

  if constexpr (VEC) {
    constexpr int E = T::vpe, U = 4;
    const int nv = n / E;
    for (int i = threadIdx.x; i < nv; i += AJ_THREADS) {
      uint32_t w[E];
      uint32_t any = 0u;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const uint4 x = reinterpret_cast<const uint4*>(word)[(i * E + e) / 4];
        w[e] = x.x; w[e + 1] = x.y; w[e + 2] = x.z; w[e + 3] = x.w;
        any |= x.x | x.y | x.z | x.w;
      }
      const bool patched = any & AJ_PATCH;
      for (int r = r0; r < r1; r += U) {
        uint4 q[U];
        uint32_t bits[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          bits[u] = 0u;
          if (r + u >= r1) continue;
          bits[u] = (1u << E) - 1u;
          if (a.allowed) {
            const unsigned char* mb = reinterpret_cast<const unsigned char*>(a.allowed + (row0 + r + u) * a.VW);
            const int v = v0 + i * E;
            bits[u] = (mb[v >> 3] >> (v & 7)) & ((1u << E) - 1u);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (bits[u]) q[u] = __ldcs(reinterpret_cast<const uint4*>(a.logits + ((row0 + r + u) * a.V + v0) * T::esz) + i);
          else q[u] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (r + u >= r1) continue;
          const uint4 y = adjust_vec<T>(q[u], w, any, bits[u], s);
          unsigned char* ob = a.out + ((row0 + r + u) * a.V + v0) * T::esz;
          if (!patched) {
            __stcs(reinterpret_cast<uint4*>(ob) + i, y);
          } else {
            const uint32_t* yw = &y.x;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              if (w[e] & AJ_PATCH) continue;
              if constexpr (T::esz == 4) reinterpret_cast<uint32_t*>(ob)[i * E + e] = yw[e];
              else reinterpret_cast<uint16_t*>(ob)[i * E + e] = static_cast<uint16_t>(yw[e / 2] >> (16 * (e & 1)));
            }
          }
        }
      }
    }
  } else {
    constexpr int U = 4;
    for (int i = threadIdx.x; i < n; i += AJ_THREADS) {
      const uint32_t w = word[i];
      if (w & AJ_PATCH) continue;
      for (int r = r0; r < r1; r += U) {
        float x[U];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          ok[u] = r + u < r1;
          if (ok[u] && a.allowed) ok[u] = (a.allowed[(row0 + r + u) * a.VW + ((v0 + i) >> 5)] >> ((v0 + i) & 31)) & 1u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = ok[u] ? T::load(a.logits, (row0 + r + u) * a.V + v0 + i) : kNegInf;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (r + u >= r1) continue;
          if (ok[u] && w) x[u] = adjust_one(x[u], w, 0, s);
          adjust_store<T>(a.out, (row0 + r + u) * a.V + v0 + i, x[u]);
        }
      }
    }
  }

  // proposed and biased tokens: a warp to a token, a lane to a row
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n_patch; i += AJ_THREADS / 32) {
    const int v = patch[i], tok = v0 + v;
    const uint32_t w = word[v];
    float bias = 0.f;
    if (a.bias_tokens) {
      const int32_t* bt = a.bias_tokens + static_cast<long long>(b) * a.M;
      for (int m0 = 0; m0 < a.M; m0 += 32) {
        uint32_t hit = __ballot_sync(0xffffffffu, m0 + lane < a.M && bt[m0 + lane] == tok);
        for (; hit; hit &= hit - 1)   // in the order of the list
          bias = __fadd_rn(bias, a.bias_values[static_cast<long long>(b) * a.M + m0 + __ffs(hit) - 1]);
      }
    }
    for (int rb = r0; rb < r1; rb += 32) {
      const int r = rb + lane;
      int more = 0;
      if (a.nodes) {
        const int32_t* nb = a.nodes + static_cast<long long>(b) * a.Nt;
        for (int j0 = 0; j0 < a.Nt; j0 += 32) {
          const uint32_t hit = __ballot_sync(0xffffffffu, j0 + lane < a.Nt && nb[j0 + lane] == tok);
          if (!hit || r >= r1) continue;
          uint32_t before;
          if (a.masks) before = a.masks[(row0 + r) * a.NW + j0 / 32] & (j0 == 0 ? ~1u : ~0u);
          else before = r <= j0 ? 0u : r - j0 >= 32 ? ~0u : (1u << (r - j0)) - 1u;
          more += __popc(hit & before);
        }
      }
      if (r >= r1) continue;
      const bool ok = !a.allowed || ((a.allowed[(row0 + r) * a.VW + (tok >> 5)] >> (tok & 31)) & 1u);
      float x = kNegInf;
      if (ok) {
        x = adjust_one(T::load(a.logits, (row0 + r) * a.V + tok), w, more, s);
        if (a.bias_tokens) x = __fadd_rn(x, bias);
      }
      adjust_store<T>(a.out, (row0 + r) * a.V + tok, x);
    }
  }
}

}  // namespace sv
