// attend_q4_tc.cuh -- verification attention over the 4-bit cache for more rows
// than the bus alone bounds (chains of grouped heads, trees, chunks of prompts),
// on the tcgen05 tensor cores.
//
// The products keep the tokens, not the rows, as M, so that any number of rows
// fits without padding M:
//   S^T[128 tokens x NC rows] = K[128 x D] Q^T      (A = K in tensor memory, B = Q)
//   O^T[128 >= D x NC rows] += V^T[D x 128] P^T     (A = V, B = P in shared memory)
// NC, the rows of a tile, is 64 or 128.  What this buys beside that:
// * a thread of the unpacking warps has one token: it reads the token's codes,
//   widens them (exactly, in f16, as attend_q4.cuh does) and stores its row of K
//   straight into its lane of tensor memory; V goes to shared memory in the plain
//   core-matrix order (8 x 16 bytes), which a warp of tokens writes without
//   conflicts.  The codes come by tensor-map copies whose 64- or 32-byte swizzle
//   spreads a warp's reads, one row a lane, over the banks.
// * a thread of the softmax warps has one token and 32 of the tile's rows; the
//   weights go to shared memory the way V does.
// A row's maximum over the tokens would be a reduction across threads in every
// tile.  Instead the weights are 2^(z - ref + 7) against a reference per row that
// all threads know; only when some score exceeds its row's reference by 8 (always
// in a triple's first tile, rarely later) the four warps that have the row agree on
// new references and rescale their rows of O^T and of the sums.
//
// Roles of a CTA (one an SM): four softmax warps for each 32 rows, which also write
// the results; four or eight warps for the queries and the unpacking; one that issues
// the products, and one for the copies.  K, S^T, V and P have two buffers each,
// queries and O^T two where tensor and shared memory hold them (NC = 64).  Each CTA
// has one contiguous share of the list of tiles (attend_q4.cuh), with at most two
// triples cut off at its ends, whose parts the join kernel puts together.  Fresh tiles
// count for several cached ones in the list: their keys and values come by loads that
// somebody waits for, and with the first come the queries, the first references and the
// triple's end.
//
// Bounds, per tile of 128 tokens and D = 128: 784 clocks of the bus; products
// 1,024 clocks at NC = 128; unpacking 256 conversions, 256 multiplications and 16
// stores of 16 bytes a thread.  A cached tile takes 1.75 us, 3,600 clocks (32 trees of
// 64 nodes without fresh entries, 8,192 tokens against 4,096: 473 and 285 us, 108 tiles
// of a CTA apart): the softmax of its 16,384 scores, about 240 instructions a warp for
// 32 rows and 32 tokens, is what takes them, by latency rather than by any unit's rate.
// (With 64 rows a thread, in eight warps, it was a quarter more: half as many warps to
// wait with, and 13 KB of code.)  That is 189 of the 285 us; the other 96 are the 3.4
// triples of a CTA, whose queries, first references and ends pass through it one after
// the other, and the call.  The trees' own entries add 50.  64 sequences of 128 rows at
// 2,048 tokens take 189 us without fresh entries and 236 with them, where the products
// at the rate of a large library product would take 37.
//
// The fresh entries are bf16 with bf16's range, and so are their products: the queries
// stay as they are until a triple's first cached tile, keys and values go to their
// buffers unchanged, and each weight is the sum of two bf16, in the two buffers of P.
// A value that is a NaN or an infinity (rare) is left out of the product, which takes
// 0 * inf for NaN, and added to O^T afterwards for the rows that see it.
#pragma once

#include <cuda.h>

#include "attend_q4.cuh"
#include "tcgen05.cuh"

namespace sv {

constexpr int TC_TILE = 128;                 // tokens of a tile
// What a triple's first fresh tile counts in the list, in cached tiles, and another one.
// 2 chunks of 1,024 tokens behind about 8,192 (D = 64): 9 and 1 378 us, 9 and 2 348, 9
// and 4 312, 12 and 4 322; 32 trees of 64 nodes behind about 4,096, where only the first
// matters: 6 357 us, 9 342, 12 335; behind 4,096 each: 338, 340, 344.
constexpr int TC_FRESH_UNITS = 9, TC_FRESH_MORE = 4;
constexpr int TC_PART = 32;                  // rows of a softmax thread
// 7 - reference before any score.  Finite, so that a score of -inf weighs nothing
// against it; every other score is far above the reference and sets a new one.
constexpr float TC_UNSET = -AT_UNSET;
constexpr uint32_t TC_VBUF = 128 * 128 * 2;  // bytes of a V buffer (16 groups of 8 columns, also for D = 64)

template <int D, int NC>
struct TcLayout {
  static constexpr int SOFT = NC / 8;                          // softmax warps: four for each part of 32 rows
  // Unpacking: four warps for keys and four for values; at NC = 128, where the
  // softmax needs the registers, four for both.
  static constexpr int UNPACK = NC == 128 ? 4 : 8;
  static constexpr int WARPS = SOFT + UNPACK + 2, THREADS = 32 * WARPS;
  static constexpr int QB = NC <= 64 ? 2 : 1;                  // buffers of queries and of O^T
  static constexpr int STAGES = NC == 128 ? 2 : 4;
  static constexpr uint32_t stage_bytes = 4 * q4_block_bytes(D);
  static constexpr uint32_t q_bytes = NC * D * 2, p_bytes = 128 * NC * 2;
  // offsets (each a multiple of 1024 where a swizzled copy lands, of 128 elsewhere)
  static constexpr uint32_t ring = 0;
  static constexpr uint32_t v = ring + ((STAGES * stage_bytes + 1023) / 1024) * 1024;
  static constexpr uint32_t p = v + 2 * TC_VBUF;
  static constexpr uint32_t q = p + 2 * p_bytes;
  static constexpr uint32_t factor = q + QB * q_bytes;         // [2][NC]: from products to the log2 domain
  static constexpr uint32_t shift = factor + 2 * NC * 4;      // [NC]: 7 - reference (TC_UNSET: none yet)
  static constexpr uint32_t corr = shift + NC * 4;             // [NC]
  static constexpr uint32_t top = corr + NC * 4;               // [4][NC]: maxima or sums of the four warps
  static constexpr uint32_t fresh = top + 4 * NC * 4;          // [4][NC]: sums of the fresh tiles' weights, of the four warps
  static constexpr uint32_t rows = fresh + 4 * NC * 4;         // [NC] 8 bytes: the rows' places in the output
  static constexpr uint32_t bars = rows + NC * 8;
  static constexpr uint32_t bytes = bars + 384;
  // tensor memory columns
  static constexpr uint32_t t_s = 0, t_o = 2 * NC, t_k = t_o + QB * NC;
  static constexpr uint32_t t_need = t_k + 2 * (D / 2);
  static constexpr uint32_t t_cols = t_need <= 256 ? 256 : 512;
};
// A CTA's part of the workspace: two partials as in attend_q4.cuh, then the
// weights of one tile (for fresh values that are no numbers)
__host__ __device__ constexpr size_t tc_cta_floats(int D, int NC) {
  return 2 * static_cast<size_t>(NC) * (D + 4) + static_cast<size_t>(128) * NC;
}

struct TcBars {
  uint64_t full[4], empty[4], kready[2], vready[2], qready[2], qfree[2], sready[2], sfree[2], pready[2],
      pvdone[2], ofree[2], drain;
  uint32_t tmem;
  int dead;       // a wait ran out of time
  float common[2]; // the factor of all rows of a triple, 0: they differ
  float qmax[4], qmin[4];
  int wide[2];    // 1 + the last tile of the buffer that has fresh values that are no numbers
  int arrived[4]; // the stage's tile came (its page ids are in range)
  int copied;     // tiles whose copies were started, once the copying warp has ended
  // arguments that functions out of line read
  const uint32_t* masks;
  unsigned long long limit;
  uint16_t* out;
  float* lse;
  int N, G, Hq, NW, rows;
  uint32_t by_g;
  float scale_log2, k_mul, v_mul;
};
static_assert(sizeof(TcBars) <= 384, "barriers");

// whether any of the N threads at a named barrier says so
template <int N>
__device__ __forceinline__ bool tc_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "n"(N)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bounded wait.  False when time is up here or was up elsewhere in the CTA.  The
// roles hand over to each other several times a tile, so a wait polls without a
// hint how long it may sleep (with one of a millisecond, a hand-over took about 500
// clocks), and looks at the time once in 64 polls.
__device__ __noinline__ bool tc_wait_long(uint64_t* bar, uint32_t parity, TcBars* b, unsigned long long limit) {
  if (*reinterpret_cast<volatile int*>(&b->dead)) return false;   // (at once: the others go on in step)
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1; i < (1u << 28); ++i) {
    if (tc_poll(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*reinterpret_cast<volatile int*>(&b->dead)) return false;
      if (global_ns() - t0 > limit) break;
    }
  }
  *reinterpret_cast<volatile int*>(&b->dead) = 1;
  return false;
}
__device__ __forceinline__ bool tc_wait_one(uint64_t* bar, uint32_t parity, TcBars* b, unsigned long long limit) {
  if (__builtin_expect(tc_poll(bar, parity), 1)) return true;
  return tc_wait_long(bar, parity, b, limit);
}

// the same for a whole warp, whose lanes go on alike
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, TcBars* b, unsigned long long limit) {
  return __all_sync(0xffffffffu, tc_wait_one(bar, parity, b, limit));
}

// byte `o` of a block of rows of 64 (D = 128) or 32 bytes, as the swizzled copy leaves it
template <int D>
__device__ __forceinline__ uint32_t tc_swz(uint32_t o) {
  return D == 128 ? o ^ (((o >> 7) & 3u) << 4) : o ^ (((o >> 7) & 1u) << 4);
}

// (Functions that are not inlined and that run for every triple take values, not the
// kernel's arguments by reference: those are read like global memory, at a few
// hundred clocks a time.  Chunks of 1,024 tokens took a fifth longer with the reference.)

// ---------------------------------------------------------------------------
// the list of tiles of a CTA, walked alike by all roles
// ---------------------------------------------------------------------------
struct TcTile {
  AtCursor c;
  int h, row0;           // kv head, first row
  int kind, at, left;    // what the tile is; its first token or node; tokens of it (0..128)
  int step;              // units of the list that it stands for
  bool first, last;      // of the triple's part in the share
  bool ends;             // the triple's end, in the share
};
enum { TC_CACHED = 0, TC_FRESH = 1, TC_VOID = 2 };   // void: a length out of range (left = 1), or nothing at all (left = 0)

// A triple's first fresh tile stands for TC_FRESH_UNITS units, another one for
// TC_FRESH_MORE, a cached tile for one (nfresh: units of the fresh tiles).  A share that
// begins within a fresh tile's units has a tile of nothing first.
template <int NC>
__device__ __noinline__ void tc_open_slow(int row_tiles, int N, bool len_ok, int nfresh, TcTile& t) {
  t.h = t.c.pair / row_tiles;
  t.row0 = (t.c.pair - t.h * row_tiles) * NC;
  t.at = 0;
  t.step = 1;
  if (!len_ok) {
    t.kind = TC_VOID;
    t.left = 1;
  } else if (t.c.i < nfresh) {
    const int j = t.c.i < TC_FRESH_UNITS ? 0 : (t.c.i - TC_FRESH_UNITS) / TC_FRESH_MORE + 1;
    const int from = j ? TC_FRESH_UNITS + (j - 1) * TC_FRESH_MORE : 0;
    t.at = j * TC_TILE;
    t.left = min(N - t.at, TC_TILE);
    t.kind = TC_FRESH;
    t.step = (j ? from + TC_FRESH_MORE : TC_FRESH_UNITS) - t.c.i;
    if (t.c.i > from) {
      t.kind = TC_VOID;
      t.left = 0;
    }
  } else {
    t.at = (t.c.i - nfresh) * TC_TILE;
    t.left = min(t.c.len - t.at, TC_TILE);
    t.kind = t.left > 0 ? TC_CACHED : TC_VOID;
    if (t.left < 0) t.left = 0;
  }
}
template <int NC>
__device__ __forceinline__ void tc_open(const AttendArgs& a, int nfresh, TcTile& t) {
  TcTile x = t;   // (by a copy: the tile itself stays in registers)
  tc_open_slow<NC>(a.row_tiles, a.N, at_len_ok(a, t.c.len), nfresh, x);
  t = x;
}
template <int NC>
__device__ __forceinline__ void tc_begin(const AttendArgs& a, const long long* prefix, int HR, int nfresh, long long u, int n, TcTile& t) {
  at_seek(a, prefix, HR, u, t.c);
  tc_open<NC>(a, nfresh, t);
  t.first = true;
  t.ends = t.c.i + t.step == t.c.units && t.step <= n;
  t.last = t.ends || t.step >= n;
}
// to the next tile; `left`: units of the share from there on
template <int NC>
__device__ __forceinline__ void tc_step(const AttendArgs& a, const long long* prefix, int HR, int nfresh, int left, TcTile& t) {
  t.c.i += t.step;
  if (TC_RARE(t.c.i == t.c.units || t.c.i == nfresh || t.kind == TC_VOID)) {   // another triple, or its first cached tile
    t.first = t.c.i == t.c.units;
    --t.c.i;
    at_next(a, prefix, HR, t.c);
    tc_open<NC>(a, nfresh, t);
  } else {
    t.first = false;
    t.step = t.kind == TC_FRESH ? TC_FRESH_MORE : 1;
    t.at += TC_TILE;
    t.left = min((t.kind == TC_FRESH ? a.N : t.c.len) - t.at, TC_TILE);
  }
  t.ends = t.c.i + t.step == t.c.units && t.step <= left;
  t.last = t.ends || t.step >= left;
}

// ---------------------------------------------------------------------------
// unpacking
// ---------------------------------------------------------------------------
// the largest of |m| and the elements (above infinity if there is a NaN)
__device__ __forceinline__ uint32_t tc_most(uint32_t m, const uint4& x) {
  return bf16x2_max_nan(m, bf16x2_max_nan(bf16x2_max_nan(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), bf16x2_max_nan(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
}
// 0 for the elements that are no numbers
__device__ __forceinline__ uint32_t tc_numbers(uint32_t two) {
  if ((two & 0x7f80u) == 0x7f80u) two &= 0xffff0000u;
  if ((two & 0x7f800000u) == 0x7f800000u) two &= 0xffffu;
  return two;
}

// a row of D elements to the L2 cache
template <int D>
__device__ __forceinline__ void tc_prefetch(const uint16_t* p) {
#pragma unroll
  for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
}

// Rows of fresh nodes (128 threads, `left` nodes of 128, zeros for the others; from:
// the first one's, `stride` elements from node to node) by
// asynchronous copies to where a value buffer has them, as they are: chunk j of 8
// elements of node n at j * 2048 + n * 16.  Eight lanes take eight nodes, which lie
// in different banks; a thread afterwards has a node's chunks to itself.
template <int D>
__device__ __forceinline__ void tc_fresh_copy(const uint16_t* from, int stride, int left, unsigned char* to, int id) {
  const int tid = threadIdx.x & 127, n0 = 8 * (tid >> 5) + (tid & 7), part = (tid >> 3) & 3;
#pragma unroll 1
  for (int n = n0; n < TC_TILE; n += 32) {
    const bool there = n < left;
    const uint16_t* p = from + static_cast<long long>(there ? n : 0) * stride + part * (D / 4);
    const uint32_t at = smem_addr(to + part * (D / 32) * 2048 + n * 16);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + i * 2048), "l"(p + 8 * i), "r"(there ? 16 : 0) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  named_bar_sync(id, 128);
}

// A fresh tile's keys into tensor memory, a thread a node, its lane; they pass
// through the values' buffer.
template <int D>
__device__ __noinline__ void tc_fresh_key(const uint16_t* from, int stride, int left, uint32_t k_at, unsigned char* vbuf) {
  const unsigned char* mine = vbuf + (threadIdx.x & 127) * 16;
  tc_fresh_copy<D>(from, stride, left, vbuf, 6);
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(mine + (4 * c + i) * 2048);
      r[4 * i] = x.x;
      r[4 * i + 1] = x.y;
      r[4 * i + 2] = x.z;
      r[4 * i + 3] = x.w;
    }
    __syncwarp();
    tc_st16(k_at + c * 16, r);
  }
}
// Its values, in place; 0 for what is no number, and true if there is any.  id: the
// threads' barrier.
template <int D>
__device__ __noinline__ bool tc_fresh_value(const uint16_t* from, int stride, int left, unsigned char* vbuf, int id) {
  unsigned char* mine = vbuf + (threadIdx.x & 127) * 16;
  tc_fresh_copy<D>(from, stride, left, vbuf, id);
  uint32_t most = 0u;
#pragma unroll 4
  for (int j = 0; j < D / 8; ++j) most = tc_most(most, *reinterpret_cast<const uint4*>(mine + j * 2048));
  if (!bf16x2_unbounded(most)) return false;
#pragma unroll 1
  for (int j = 0; j < D / 8; ++j) {
    uint4* at = reinterpret_cast<uint4*>(mine + j * 2048);
    const uint4 x = *at;
    *at = make_uint4(tc_numbers(x.x), tc_numbers(x.y), tc_numbers(x.z), tc_numbers(x.w));
  }
  return true;
}

// Queries of a row tile (128 threads; from: the first row's of the kv head), as they
// are, by asynchronous copies.
template <int D, int NC>
__device__ __noinline__ void tc_copy_q(const uint16_t* from, int row0, int qb, unsigned char* smem) {
  using L = TcLayout<D, NC>;
  const TcBars* bar = reinterpret_cast<const TcBars*>(smem + L::bars);
  const int G = bar->G, Hq = bar->Hq, rows = bar->rows;
  const uint32_t by_g = bar->by_g;
  // Four threads of a warp have a row, eight lanes eight rows (so that they access
  // different banks); a thread has W columns of core matrices.
  constexpr int W = D / 32;
  const int tid = threadIdx.x - 32 * L::SOFT, part = (tid >> 3) & 3, r0 = 8 * (tid >> 5) + (tid & 7);
  unsigned char* to = smem + L::q + qb * L::q_bytes + W * part * (NC * 16);
#pragma unroll 1
  for (int r = r0; r < NC; r += 32) {
    const bool there = row0 + r < rows;
    const int x = there ? row0 + r : row0, node = by_g ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), by_g)) : x;
    const uint16_t* p = from + (static_cast<long long>(node) * Hq + (x - node * G)) * D + part * (D / 4);
    const uint32_t at = smem_addr(to + r * 16);
#pragma unroll
    for (int i = 0; i < W; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + i * (NC * 16)), "l"(p + 8 * i), "r"(there ? 16 : 0) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The same, made f16 in place (each thread what it copied).  Usually one power of two
// scales all rows, so that the largest element lies in [128, 256); where the rows'
// largest elements lie more than 2^8 apart, each row gets its own (an element is off by 2^-25 at
// most: 2^-24 of its row's largest with one power of two, 2^-32 with its own).
// (What runs once a triple is short loops: its code has left the instruction
// caches by then, and a line of it takes as long to fetch as ten hot instructions
// an instruction.  Unrolled, this function took 15,000 clocks.)
template <int D, int NC>
__device__ __noinline__ void tc_scale_q(int qb, int fb, unsigned char* smem) {
  using L = TcLayout<D, NC>;
  TcBars* bar = reinterpret_cast<TcBars*>(smem + L::bars);
  const float scale_log2 = bar->scale_log2, k_mul = bar->k_mul;
  constexpr int W = D / 32;
  const int tid = threadIdx.x - 32 * L::SOFT, part = (tid >> 3) & 3, quad = tid >> 5, r0 = 8 * quad + (tid & 7);
  unsigned char* to = smem + L::q + qb * L::q_bytes + W * part * (NC * 16);
  float* factor = reinterpret_cast<float*>(smem + L::factor) + fb * NC;
  // the rows' largest elements, in the factors' place
  float hi = 0.f, lo = __builtin_huge_valf();
  bool odd = false;
#pragma unroll 1
  for (int r = r0; r < NC; r += 32) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(to + r * 16 + i * (NC * 16));
      m = bf16x2_max_nan(m, bf16x2_max_nan(bf16x2_max_nan(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), bf16x2_max_nan(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) m = bf16x2_max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float top = fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    odd |= !(top < __builtin_huge_valf());
    hi = fmaxf(hi, top);
    if (top > 0.f) lo = fminf(lo, top);
    if (part == 0) factor[r] = top;
  }
  // over the four warps
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  odd = __any_sync(0xffffffffu, odd);
  if ((tid & 31) == 0) {
    bar->qmax[quad] = odd ? __builtin_huge_valf() : hi;
    bar->qmin[quad] = lo;
  }
  named_bar_sync(6, 128);
  hi = fmaxf(fmaxf(bar->qmax[0], bar->qmax[1]), fmaxf(bar->qmax[2], bar->qmax[3]));
  lo = fminf(fminf(bar->qmin[0], bar->qmin[1]), fminf(bar->qmin[2], bar->qmin[3]));
  const float common = hi < __builtin_huge_valf() && hi > 0.f && hi <= lo * 256.f ? hi : 0.f;
  // in place, times the power of two that takes the largest to [128, 256); the
  // factor is what takes the products back, with the scale (finite, so that a score of 0
  // stays one)
  auto power = [](float top) { return top > 0.f ? min(7 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 100) : 0; };
  auto mult = [&](int e) { return copysignf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23), scale_log2); };
  auto back = [&](int e) {
    return fminf(fmaxf(fabsf(scale_log2) * k_mul * __uint_as_float(static_cast<uint32_t>(127 - e) << 23), 1.17549435e-38f), 3.402823466e+38f);
  };
  float mul = mult(power(common)), f = back(power(common));
  if (tid == 0) bar->common[fb] = common > 0.f ? f : 0.f;
#pragma unroll 1
  for (int r = r0; r < NC; r += 32) {
    if (TC_RARE(common == 0.f)) {
      const float top = factor[r];
      __syncwarp();   // (the threads of a row are in one warp)
      mul = mult(power(top));
      f = top <= __builtin_huge_valf() ? back(power(top)) : __int_as_float(0x7fc00000);   // (a NaN has no other scores, an infinity has)
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      uint4* at = reinterpret_cast<uint4*>(to + r * 16 + i * (NC * 16));
      const uint4 w = *at;
      *at = make_uint4(f16x2_pack(__uint_as_float(w.x << 16) * mul, __uint_as_float(w.x & 0xffff0000u) * mul),
                       f16x2_pack(__uint_as_float(w.y << 16) * mul, __uint_as_float(w.y & 0xffff0000u) * mul),
                       f16x2_pack(__uint_as_float(w.z << 16) * mul, __uint_as_float(w.z & 0xffff0000u) * mul),
                       f16x2_pack(__uint_as_float(w.w << 16) * mul, __uint_as_float(w.w & 0xffff0000u) * mul));
    }
    if (part == 0) factor[r] = f;
  }
  named_bar_sync(6, 128);   // qmax and qmin are free again
}

// Adds the fresh values that are no numbers to O^T: this thread's column d, the rows from
// col0; weights (negative: the row does not see the node) at w[node][NC].
template <int D, int NC>
__device__ __noinline__ void tc_wide_values(const AttendArgs& args, int b, int h, int node0, int left, int d, int col0, int cols,
                                            const float* w, uint32_t addr) {
  const AttendArgs a = args;
  for (int j = 0; j < left; ++j) {
    float v = 0.f;
    if (d < D)
      v = __uint_as_float(static_cast<uint32_t>(a.v_new[((static_cast<long long>(b) * a.N + node0 + j) * a.Hkv + h) * D + d]) << 16);
    const bool odd = !(fabsf(v) < __builtin_huge_valf());
    if (!__any_sync(0xffffffffu, odd)) continue;
    for (int c = 0; c < cols; ++c) {
      const float p = __ldcg(w + j * NC + col0 + c);
      float o = tc_ld1(addr + c);
      __syncwarp();
      if (odd && !(p < 0.f)) o += (p == 0.f ? 1.17549435e-38f : p) * v;
      __syncwarp();
      tc_st1(addr + c, o);
      tc_wait_st();
    }
  }
}

// the largest of column i of 32 over the lanes of a warp, in lane i
__device__ __forceinline__ float tc_top(float (&x)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    // lanes with bit o keep the upper half of what is left
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
      x[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return x[0];
}

// New references for a part's rows: the 128 threads of a part call this together.
// s_at: the tile's products (hide: bits of rows that do not see this thread's
// token), o_at: the rows' sums of v so far, if there are any.  factor: of each row, or
// null: the scale is.
template <int D, int NC>
__device__ __noinline__ void tc_raise(unsigned char* smem, uint32_t s_at, uint32_t o_at, const float* factor, uint32_t hide, bool sums) {
  using L = TcLayout<D, NC>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, col0 = (threadIdx.x >> 7) * TC_PART, id = 1 + (threadIdx.x >> 7);
  float* shift = reinterpret_cast<float*>(smem + L::shift) + col0;
  float* corr = reinterpret_cast<float*>(smem + L::corr) + col0;
  float* top = reinterpret_cast<float*>(smem + L::top) + col0;
  float* fresh = reinterpret_cast<float*>(smem + L::fresh) + col0;
  const float all = reinterpret_cast<const TcBars*>(smem + L::bars)->scale_log2;
  float z[TC_PART];
  tc_ld<TC_PART>(s_at, z);
#pragma unroll
  for (int i = 0; i < TC_PART; i += 4) {
    const float4 x = factor ? *reinterpret_cast<const float4*>(factor + i) : make_float4(all, all, all, all);
    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) z[i + k] = (hide >> (i + k)) & 1u ? kNegInf : fmaxf(z[i + k] * f[k], kNegInf);   // (no NaN)
  }
  const float mx = tc_top(z);
  top[quad * NC + lane] = mx;
  named_bar_sync(id, 128);
  if (quad == 0) {
    const float m = fmaxf(fmaxf(top[lane], top[NC + lane]), fmaxf(top[2 * NC + lane], top[3 * NC + lane]));
    const float old = shift[lane];                                // 7 - ref
    const float now = m == kNegInf ? old : fminf(old, AT_PSHIFT - m);
    shift[lane] = now;
    corr[lane] = at_corr(now - old);
  }
  named_bar_sync(id, 128);
  if (sums) {
    fresh[quad * NC + lane] *= corr[lane];
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < TC_PART; i += 8) {
      float o[8];
      tc_ld<8>(o_at + i, o);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= corr[i + k];
      tc_st8(o_at + i, o);
    }
    tc_wait_st();
  }
}

// The sum of column lane / 4 of 8 over the lanes of a warp.
__device__ __forceinline__ float tc_total(const float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    y[i] = (up ? x[i + 4] : x[i]) + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + 4], 16);
  }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & (4 * o);
      const float give = up ? y[i] : y[i + o];
      y[i] = (up ? y[i + o] : y[i]) + __shfl_xor_sync(0xffffffffu, give, 4 * o);
    }
  y[0] += __shfl_xor_sync(0xffffffffu, y[0], 2);
  return y[0] + __shfl_xor_sync(0xffffffffu, y[0], 1);
}

// The softmax of a tile without cached tokens: of fresh entries of sequence b, or of
// nothing (n: the tile's number).  Called by the 128 threads of a part together.  True
// (for all of them alike) when the tile has values that are no numbers, whose weights
// then are in wide_w.  (It takes few arguments and keeps no array that is addressed:
// local memory, for which the shared memory in use leaves next to no cache, made a tile
// 10,000 clocks longer.)
template <int D, int NC>
__device__ __noinline__ bool tc_fresh_softmax(unsigned char* smem, bool of_fresh, int b, int row0, int at, int left, bool first, int n, uint32_t s_at,
                                              uint32_t o_at, float* wide_w) {
  using L = TcLayout<D, NC>;
  TcBars* bar = reinterpret_cast<TcBars*>(smem + L::bars);
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, part = threadIdx.x >> 7, col0 = part * TC_PART, id = 1 + part;
  const int tok = 32 * quad + lane, x = n & 1;
  float* shift = reinterpret_cast<float*>(smem + L::shift) + col0;
  float* fresh = reinterpret_cast<float*>(smem + L::fresh) + col0;
  // which of the part's rows do not see this thread's node
  uint32_t hide = 0u;
  if (of_fresh) {
    const int open = (at + tok) * bar->G - row0 - col0;   // a chain: the node's first row
    hide = open <= 0 ? 0u : open >= 32 ? ~0u : (1u << open) - 1u;
    if (bar->masks) {   // a tree: the warp's 32 nodes are one word of each row's mask, a row a lane
      const int r = row0 + col0 + lane, N = bar->N;
      uint32_t w = 0u;
      if (r < bar->rows && at + 32 * quad < N) w = __ldg(bar->masks + (static_cast<long long>(b) * N + r / bar->G) * bar->NW + at / 32 + quad);
      hide = 0u;
#pragma unroll 4
      for (int i = 0; i < TC_PART; ++i) hide |= (~(__shfl_sync(0xffffffffu, w, i) >> lane) & 1u) << i;
    }
  }
  if (tok >= left) hide = ~0u;
  const unsigned long long limit = bar->limit;
  const float scale = bar->scale_log2;
  tc_wait(&bar->sready[x], (n >> 1) & 1, bar, limit);
  tc_fence_after();
  // Eight rows' scores against their references (the products are rounded as those were).
  auto scores = [&](int i, float (&y)[8]) {
    __syncwarp();
    tc_ld<8>(s_at + i, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = (hide >> (i + k)) & 1u ? kNegInf : __fadd_rn(__fmul_rn(y[k], scale), shift[i + k]);
  };
  float m = 0.f;
#pragma unroll 1
  for (int i = 0; i < TC_PART; i += 8) {
    float y[8];
    scores(i, y);
#pragma unroll
    for (int k = 0; k < 8; k += 2) m = fmax3_nan(m, y[k], y[k + 1]);
  }
  if (tc_any<128>(id, !(m <= AT_PSHIFT + AT_ABOVE))) {
    if (!first) tc_wait(&bar->pvdone[x ^ 1], ((n - 1) >> 1) & 1, bar, limit);
    tc_raise<D, NC>(smem, s_at, o_at, nullptr, hide, !first);
  }
  // (one answer for the part, whatever the flag does once a wait has failed)
  tc_wait(&bar->vready[x], (n >> 1) & 1, bar, limit);
  const bool wide = tc_any<128>(id, *reinterpret_cast<volatile int*>(&bar->wide[x]) == n + 1);
  // Each weight as the sum of two bf16, in the two buffers, in units of the sums of v; for
  // values that are no numbers as it is, or -1 where the row does not see the node.
  if (n >= 2) tc_wait(&bar->pvdone[x], ((n >> 1) & 1) ^ 1, bar, limit);
  if (n >= 1) tc_wait(&bar->pvdone[x ^ 1], ((n - 1) >> 1) & 1, bar, limit);
  unsigned char* hi = smem + L::p + x * L::p_bytes + tok * 16 + col0 / 8 * 2048;
  unsigned char* lo = smem + L::p + (x ^ 1) * L::p_bytes + tok * 16 + col0 / 8 * 2048;
  const float unit = __fdiv_rn(1.f, bar->v_mul);
#pragma unroll 1
  for (int i = 0; i < TC_PART; i += 8) {
    float y[8];
    scores(i, y);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[k] = ex2_approx(y[k]);
      if (wide) __stcg(wide_w + static_cast<size_t>(tok) * NC + col0 + i + k, (hide >> (i + k)) & 1u ? -1.f : y[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float p0 = y[2 * k] * unit, p1 = y[2 * k + 1] * unit;
      h[k] = bf16x2_pack(p0, p1);
      l[k] = bf16x2_pack(p0 - __uint_as_float(h[k] << 16), p1 - __uint_as_float(h[k] & 0xffff0000u));
    }
    *reinterpret_cast<uint4*>(hi + i / 8 * 2048) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(lo + i / 8 * 2048) = make_uint4(l[0], l[1], l[2], l[3]);
    const float total = tc_total(y);
    float* at = fresh + quad * NC + i + (lane >> 2);
    if ((lane & 3) == 0) *at = (first ? 0.f : *at) + total;
  }
  tc_fence_before();
  tc_proxy_fence();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(&bar->sfree[x]);   // the scores have been read
    mbar_arrive(&bar->pready[x]);
  }
  return wide;
}

// Where the 128 threads of a part of the rows leave their sums of weights of row c,
// a token each: in the weights' buffers (p: the part's share of the first), which
// nothing reads by then.
template <int D, int NC>
__device__ __forceinline__ float* tc_sums(const unsigned char* p, int c) {
  using L = TcLayout<D, NC>;
  return reinterpret_cast<float*>(const_cast<unsigned char*>(p) + c / (TC_PART / 2) * L::p_bytes) + c % (TC_PART / 2) * 128;
}

// The end of a triple, or of its part in the share: the sums of weights over the
// tokens' threads, then O^T row by row, as the result or (not
// whole) as a partial.
template <int D, int NC>
__device__ __noinline__ void tc_finish(unsigned char* smem, long long base, int row0, bool whole, float* partial, uint32_t o_at) {
  using L = TcLayout<D, NC>;
  const TcBars* bar = reinterpret_cast<const TcBars*>(smem + L::bars);
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, part = threadIdx.x >> 7, col0 = part * TC_PART, id = 1 + part, d = 32 * quad + lane;
  const int rows = bar->rows;
  uint16_t* out = bar->out;
  const unsigned char* p = smem + L::p + col0 / 8 * 2048;
  const float* shift = reinterpret_cast<const float*>(smem + L::shift) + col0;
  const float* fresh = reinterpret_cast<const float*>(smem + L::fresh) + col0;
  float* corr = reinterpret_cast<float*>(smem + L::corr) + col0;
  float* top = reinterpret_cast<float*>(smem + L::top) + col0;
  long long* place = reinterpret_cast<long long*>(smem + L::rows) + col0;
  tc_fence_after();
  named_bar_sync(id, 128);
  // a warp adds up its 32 tokens of the part's rows, a row a lane, rotated so that
  // the lanes read different banks
  {
    const float* from = tc_sums<D, NC>(p, lane) + 32 * quad;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int t = 0; t < 32; t += 4)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] += from[(t + k + lane) & 31];
    top[quad * NC + lane] = ((x[0] + x[1]) + (x[2] + x[3])) + fresh[quad * NC + lane];
  }
  named_bar_sync(id, 128);
  if (quad == 0) {
    const int i = lane, G = bar->G;
    const uint32_t by_g = bar->by_g;
    const int x = min(row0 + col0 + i, rows - 1), node = by_g ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), by_g)) : x;
    place[i] = (base + static_cast<long long>(node) * bar->Hq + (x - node * G)) * D;
    const float sum = (top[i] + top[NC + i]) + (top[2 * NC + i] + top[3 * NC + i]);
    const int r = row0 + col0 + i;
    const float ref = -shift[i];
    corr[i] = sum == 0.f ? 0.f : bar->v_mul / sum;
    if (whole) {
      if (r < rows && bar->lse) bar->lse[place[i] / D] = at_lse(ref, sum);
    } else {
      float* ml = partial + static_cast<size_t>(NC) * D + col0 + i;
      ml[0] = ref;
      ml[NC] = sum;
      ml[2 * NC] = 0.f;
    }
  }
  named_bar_sync(id, 128);
  const int real = rows - row0 - col0;   // rows of the part that there are
#pragma unroll 1
  for (int c0 = 0; c0 < TC_PART; c0 += 8) {
    float o[8];
    __syncwarp();
    tc_ld<8>(o_at + c0, o);
    if (d >= D) continue;
    if (whole) {
      const float4 f0 = *reinterpret_cast<const float4*>(corr + c0), f1 = *reinterpret_cast<const float4*>(corr + c0 + 4);
      const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const longlong2 at = *reinterpret_cast<const longlong2*>(place + c0 + i);
        const uint32_t two = bf16x2_pack(o[i] * f[i], o[i + 1] * f[i + 1]);
        if (c0 + i < real) out[at.x + d] = static_cast<uint16_t>(two);
        if (c0 + i + 1 < real) out[at.y + d] = static_cast<uint16_t>(two >> 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) partial[static_cast<size_t>(col0 + c0 + i) * D + d] = o[i];
    }
  }
}

template <int D, int NC>
__global__ void __launch_bounds__(TcLayout<D, NC>::THREADS, 1) attend_q4_tc_kernel(const __grid_constant__ AttendArgs a,
                                                                     const __grid_constant__ CUtensorMap map) {
  using L = TcLayout<D, NC>;
  extern __shared__ unsigned char tc_raw[];
  __shared__ long long scratch[L::WARPS];
  unsigned char* tc_smem = tc_raw + ((1024u - (smem_addr(tc_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TcBars* bar = reinterpret_cast<TcBars*>(tc_smem + L::bars);
  long long* prefix = reinterpret_cast<long long*>(tc_smem + L::bytes);
  const uint32_t sbase = smem_addr(tc_smem);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar->full[i], i == 0 && a.stall == static_cast<int>(blockIdx.x) + 1 ? 2 : 1);   // (2: test hook)
      mbar_init(&bar->empty[i], L::UNPACK);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->kready[i], 4);
      mbar_init(&bar->vready[i], 4);
      mbar_init(&bar->qready[i], 4);
      mbar_init(&bar->qfree[i], 1);
      mbar_init(&bar->sready[i], 1);
      mbar_init(&bar->sfree[i], L::SOFT);
      mbar_init(&bar->pready[i], L::SOFT);
      mbar_init(&bar->pvdone[i], 1);
      mbar_init(&bar->ofree[i], L::SOFT);
      bar->wide[i] = 0;
    }
    mbar_init(&bar->drain, 1);
    bar->dead = bar->copied = 0;
    bar->masks = a.masks;
    bar->limit = a.timeout_ns;
    bar->N = a.N;
    bar->G = a.G;
    bar->NW = a.NW;
    bar->rows = a.N * a.G;
    bar->scale_log2 = a.scale_log2;
    bar->v_mul = a.v_mul;
    bar->k_mul = a.k_mul;
    bar->by_g = a.by_g;
    bar->Hq = a.Hkv * a.G;
    bar->out = a.out;
    bar->lse = a.lse;
    mbar_fence_init();
  }
  at_prefix<L::THREADS>(a, prefix, scratch);   // (synchronises the CTA)
  const int HR = a.Hkv * a.row_tiles;
  const long long units = prefix[a.B] * HR;
  const int ctas = at_active(units, gridDim.x, 1);
  if (blockIdx.x >= ctas) return;
  const long long u0 = at_start(units, ctas, blockIdx.x);
  const int ntiles = static_cast<int>(at_start(units, ctas, blockIdx.x + 1) - u0);
  const int rows = a.N * a.G, nfresh = at_fresh_units(a);
  if (warp == L::SOFT + L::UNPACK) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bar->tmem)), "r"(L::t_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  float* cta_ws = a.ws + static_cast<size_t>(blockIdx.x) * tc_cta_floats(D, NC);

  if (warp == L::SOFT + L::UNPACK + 1) {
    // ---- copies: up to four blocks a tile, a lane each --------------------------------
    TcTile t;
    tc_begin<NC>(a, prefix, HR, nfresh, u0, ntiles, t);
    int n = 0;                        // cached tiles so far
    int page = -1, page_at = -1;      // a lane's entry of the 32 blocks from page_at on (of this triple)
    const int bpp = a.P / Q4_BLOCK;
    for (int u = 0;;) {
      if (t.kind == TC_CACHED) {
        const int blk = t.at / Q4_BLOCK, nblk = (t.left + Q4_BLOCK - 1) / Q4_BLOCK;
        if (t.first || page_at < 0 || blk >= page_at + 32) {
          page_at = blk;
          const int x = blk + lane;
          page = x * Q4_BLOCK < t.c.len ? __ldg(a.table + static_cast<long long>(t.c.b) * a.W + x / bpp) : -1;
        }
        const int mine = __shfl_sync(0xffffffffu, page, blk - page_at + (lane & 3));
        const bool ok = lane >= nblk || (mine >= 0 && mine < a.pages);
        const int s = n % L::STAGES;
        // (Warps whose wait has failed go on in step and release stages whose copies may
        // still be on their way; the flag was set before they did.)
        bool go = true;
        if (n >= L::STAGES)
          go = tc_wait(&bar->empty[s], ((n / L::STAGES) & 1) ^ 1, bar, a.timeout_ns) && !__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&bar->dead));
        if (!go) break;
        const bool all = __all_sync(0xffffffffu, ok);
        if (lane == 0) bar->arrived[s] = all;
        if (all) {
          if (lane == 0) mbar_arrive_expect_tx(&bar->full[s], nblk * q4_block_bytes(D));
          __syncwarp();
          if (lane < nblk) {
            const int x = blk + lane;
            const int z = static_cast<int>((static_cast<long long>(mine) * a.Hkv + t.h) * bpp + x % bpp);
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                    sbase + L::ring + s * L::stage_bytes + lane * q4_block_bytes(D)),
                "l"(&map), "r"(0), "r"(0), "r"(z), "r"(smem_addr(&bar->full[s]))
                : "memory");
          }
        } else if (lane == 0) {
          mbar_arrive(&bar->full[s]);
        }
        ++n;
      } else {
        page_at = -1;
      }
      // what the other warps load themselves is asked for as the copies come to it
      if (t.first)
        for (int r = lane; r < NC && t.row0 + r < rows; r += 32) tc_prefetch<D>(a.q + at_row(a, t.c.b, t.h, t.row0 + r) * D);
      if (t.kind == TC_FRESH)
        for (int j = lane; j < t.left; j += 32) {
          const long long at = ((static_cast<long long>(t.c.b) * a.N + t.at + j) * a.Hkv + t.h) * D;
          tc_prefetch<D>(a.k_new + at);
          tc_prefetch<D>(a.v_new + at);
        }
      if ((u += t.step) >= ntiles) break;
      tc_step<NC>(a, prefix, HR, nfresh, ntiles - u, t);
    }
    if (lane == 0) bar->copied = n;
  } else if (warp == L::SOFT + L::UNPACK) {
    // ---- products: one thread ------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t id_s = tc_idesc(NC, false, false, false), id_o = tc_idesc(NC, false, true, true);
      constexpr uint32_t id_sb = tc_idesc(NC, true, false, false), id_ob = tc_idesc(NC, true, true, true);
      TcTile t;
      tc_begin<NC>(a, prefix, HR, nfresh, u0, ntiles, t);
      bool pfirst = false, pfresh = false;   // the tile before: was it a triple's first, one of fresh entries
      int n = 0, tri = 0, ptri = 0;     // tiles, triples so far; the tile before's triple
      uint32_t qphase = 0u;             // a bit per buffer of the queries
      auto add_v = [&](int m, bool first, bool fresh, int tr) {   // O^T += V^T P^T of tile m
        const int x = m & 1;
        if (!tc_wait_one(&bar->pready[x], (m >> 1) & 1, bar, a.timeout_ns) || !tc_wait_one(&bar->vready[x], (m >> 1) & 1, bar, a.timeout_ns)) return false;
        const int ob = tr % L::QB;
        if (first && tr >= L::QB && !tc_wait_one(&bar->ofree[(tr - L::QB) & 1], ((tr - L::QB) >> 1) & 1, bar, a.timeout_ns)) return false;
        tc_fence_after();
        const uint64_t vd = tc_desc(sbase + L::v + x * TC_VBUF, 128, 2048), pd = tc_desc(sbase + L::p + x * L::p_bytes, 128, 2048);
        const uint32_t id = fresh ? id_ob : id_o;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)   // (16 tokens: 256 bytes on)
          tc_mma_ss(tmem + L::t_o + ob * NC, vd + ks * 16, pd + ks * 16, id, !(first && ks == 0));
        if (TC_RARE(fresh)) {   // the rest of the weights
          const uint64_t rd = tc_desc(sbase + L::p + (x ^ 1) * L::p_bytes, 128, 2048);
#pragma unroll 1
          for (int ks = 0; ks < 8; ++ks) tc_mma_ss(tmem + L::t_o + ob * NC, vd + ks * 16, rd + ks * 16, id, true);
        }
        tc_commit(&bar->pvdone[x]);
        return true;
      };
      bool ok = true;
      for (int u = 0;;) {
        const int x = n & 1, qb = tri % L::QB;
        if (t.first && n > 0) ok = add_v(n - 1, pfirst, pfresh, ptri);   // (the triple before is finished beside the load of the queries)
        if (t.first || (t.kind == TC_CACHED && t.at == 0)) {   // the queries, or the queries made f16
          ok = ok && tc_wait_one(&bar->qready[qb], (qphase >> qb) & 1u, bar, a.timeout_ns);
          qphase ^= 1u << qb;
        }
        ok = ok && tc_wait_one(&bar->kready[x], (n >> 1) & 1, bar, a.timeout_ns);
        if (ok && n >= 2) ok = tc_wait_one(&bar->sfree[x], ((n >> 1) & 1) ^ 1, bar, a.timeout_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = tc_desc(sbase + L::q + qb * L::q_bytes, NC * 16, 128);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)   // (16 elements: two core-matrix columns on)
          tc_mma_ts(tmem + L::t_s + x * NC, tmem + L::t_k + x * (D / 2) + ks * 8, qd + ks * (2 * NC), t.kind == TC_CACHED ? id_s : id_sb, ks > 0);
        tc_commit(&bar->sready[x]);   // (and K's buffer is free)
        if (t.last) tc_commit(&bar->qfree[qb]);
        if (n > 0 && !t.first) ok = add_v(n - 1, pfirst, pfresh, ptri);
        if (!ok) break;
        pfirst = t.first;
        pfresh = t.kind == TC_FRESH;
        ptri = tri;
        if (t.last) ++tri;
        ++n;
        if ((u += t.step) >= ntiles) {
          add_v(n - 1, pfirst, pfresh, ptri);
          break;
        }
        tc_step<NC>(a, prefix, HR, nfresh, ntiles - u, t);
      }
      tc_commit(&bar->drain);
      mbar_wait(&bar->drain, 0, a.timeout_ns);   // nothing is in flight when tensor memory is given back
    }
    __syncwarp();
  } else if (warp >= L::SOFT) {
    // ---- queries and unpacking: a thread a token ----------------------------------------------
    const int quad = warp & 3, tok = 32 * quad + lane;
    const uint32_t lane_at = static_cast<uint32_t>(32 * quad) << 16;
    const bool keys = warp < L::SOFT + 4, values = L::UNPACK == 4 || !keys;
    TcTile t;
    tc_begin<NC>(a, prefix, HR, nfresh, u0, ntiles, t);
    int n = 0, tri = 0, copies = 0;
    // (A warp whose wait fails goes on in step with the others, as the softmax warps
    // do: over what the buffers hold, for results that are void.)
    for (int u = 0;;) {
      const int x = n & 1;
      if (TC_RARE(t.first || t.at == 0) && keys) {
        // A triple's queries are bf16 for its fresh tiles and f16 from its first cached one.
        const bool cached = t.kind == TC_CACHED;
        if (t.first) {
          // (the factors have two buffers, which the softmax warps read to the triple's end)
          if (tri >= L::QB) tc_wait(&bar->qfree[tri % L::QB], ((tri / L::QB) & 1) ^ 1, bar, a.timeout_ns);
          if (tri >= 2) tc_wait(&bar->ofree[tri & 1], ((tri >> 1) & 1) ^ 1, bar, a.timeout_ns);
          tc_copy_q<D, NC>(a.q + at_row(a, t.c.b, t.h, 0) * D, t.row0, tri % L::QB, tc_smem);
          ++tri;
        } else if (cached) {   // the products of the tile before have read them
          tc_wait(&bar->sready[x ^ 1], ((n - 1) >> 1) & 1, bar, a.timeout_ns);
        }
        const int qb = (tri - 1) % L::QB;
        if (cached) tc_scale_q<D, NC>(qb, (tri - 1) & 1, tc_smem);
        if (cached || t.first) {
          tc_proxy_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->qready[qb]);
        }
      }
      const int stage = copies % L::STAGES;
      if (t.kind == TC_CACHED) tc_wait(&bar->full[stage], (copies / L::STAGES) & 1, bar, a.timeout_ns);
      const unsigned char* blk = tc_smem + L::ring + stage * L::stage_bytes + quad * q4_block_bytes(D);
      // A token that counts has its scales; others get 0, and one of a tile that did
      // not come, or of a length out of range, NaN for its key.
      const bool mine = tok < t.left;
      const bool good = t.kind == TC_CACHED && *reinterpret_cast<volatile int*>(&bar->arrived[stage]);
      auto fresh_at = [&] { return ((static_cast<long long>(t.c.b) * a.N + t.at) * a.Hkv + t.h) * D; };
      auto scales = [&](int from) -> uint64_t {
        if constexpr (D == 128) return *reinterpret_cast<const uint64_t*>(blk + tc_swz<D>(from + lane * 8));
        else return *reinterpret_cast<const uint32_t*>(blk + tc_swz<D>(from + lane * 4));
      };
      // Where the same warps do both, the key goes first: its buffer is free long
      // before the value's, and the scores of this tile can then be taken beside the
      // weights of the last one.  (Rolled loops: a warp that is alone on its
      // scheduler waits for its instructions otherwise.)
      if (keys) {
        if (n >= 2) tc_wait(&bar->sready[x], ((n >> 1) & 1) ^ 1, bar, a.timeout_ns);
        tc_fence_after();
        const uint32_t k_at = tmem + lane_at + L::t_k + x * (D / 2);
        if (TC_RARE(t.kind == TC_FRESH)) {
          if (n >= 2) tc_wait(&bar->pvdone[x], ((n >> 1) & 1) ^ 1, bar, a.timeout_ns);
          tc_fresh_key<D>(a.k_new + fresh_at(), a.Hkv * D, t.left, k_at, tc_smem + L::v + x * TC_VBUF);
        } else {
          uint64_t sc = !mine ? 0ull : good ? scales(32 * D) : 0x7f7f7f7f7f7f7f7full;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(blk + tc_swz<D>(lane * (D / 2) + c * 16));
            uint32_t r[16];
            tc_widen(w.x, w.y, tc_scale(static_cast<uint32_t>(sc), 0), r);
            tc_widen(w.z, w.w, tc_scale(static_cast<uint32_t>(sc), 1), r + 8);
            tc_st16(k_at + c * 16, r);
            sc >>= 16;
          }
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->kready[x]);
      }
      // In a fresh tile the keys' and the values' warps meet once the keys have left
      // the values' buffer.  (Both wait: an arrival for one tile would otherwise count
      // for the tile before.)
      if (TC_RARE(t.kind == TC_FRESH)) named_bar_sync(L::UNPACK == 4 ? 6 : 8, 32 * L::UNPACK);
      if (values) {
        if (n >= 2) tc_wait(&bar->pvdone[x], ((n >> 1) & 1) ^ 1, bar, a.timeout_ns);
        unsigned char* vb = tc_smem + L::v + x * TC_VBUF + tok * 16;
        if (TC_RARE(t.kind == TC_FRESH)) {
          if (tc_fresh_value<D>(a.v_new + fresh_at(), a.Hkv * D, t.left, tc_smem + L::v + x * TC_VBUF, L::UNPACK == 4 ? 6 : 7))
            *reinterpret_cast<volatile int*>(&bar->wide[x]) = n + 1;
        } else {
          uint64_t sc = mine && good ? scales(34 * D) : 0ull;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(blk + tc_swz<D>(16 * D + lane * (D / 2) + c * 16));
            uint32_t r[16];
            tc_widen(w.x, w.y, tc_scale(static_cast<uint32_t>(sc), 0), r);
            tc_widen(w.z, w.w, tc_scale(static_cast<uint32_t>(sc), 1), r + 8);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(vb + (4 * c + i) * 2048) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            sc >>= 16;
          }
        }
        tc_proxy_fence();
      }
      __syncwarp();
      if (lane == 0) {
        if (values) mbar_arrive(&bar->vready[x]);
        if (t.kind == TC_CACHED) mbar_arrive(&bar->empty[stage]);
      }
      if (t.kind == TC_CACHED) ++copies;
      ++n;
      if ((u += t.step) >= ntiles) break;
      tc_step<NC>(a, prefix, HR, nfresh, ntiles - u, t);
    }
  } else {
    // ---- softmax: a thread a token and a part of the rows ---------------------------------------
    constexpr int HC = TC_PART;
    const int part = warp >> 2, quad = warp & 3, tok = 32 * quad + lane, id = 1 + part, col0 = part * HC;
    const uint32_t lane_at = static_cast<uint32_t>(32 * quad) << 16;
    float* shift = reinterpret_cast<float*>(tc_smem + L::shift) + col0;
    float* corr = reinterpret_cast<float*>(tc_smem + L::corr) + col0;
    // Sums of weights of two neighbouring tokens: an even lane has the first half of
    // the rows, an odd one the second (a sum a row and thread beside the 32 scores
    // would not fit the registers).
    float l[HC / 2];
    const bool odd = lane & 1;
    TcTile t;
    tc_begin<NC>(a, prefix, HR, nfresh, u0, ntiles, t);
    int n = 0, u = 0;
    for (int tri = 0;; ++tri) {
      // The part of a triple in the share: first the tiles without cached tokens, then, in a
      // loop of their own, the cached ones.
      // (A warp whose wait fails goes on in step with the others, which it meets at
      // barriers; every wait then returns at once.)
      const int itri = t.c.i;
      const uint32_t o_at = tmem + lane_at + L::t_o + tri % L::QB * NC + col0;
      for (int i = threadIdx.x & 127; i < HC; i += 128) shift[i] = TC_UNSET;
      named_bar_sync(id, 128);
      bool first = true, ends = false;
      if (t.kind == TC_CACHED) {
        reinterpret_cast<float*>(tc_smem + L::fresh)[quad * NC + col0 + lane] = 0.f;
      } else {
        for (;;) {
          float* w = cta_ws + 2 * static_cast<size_t>(NC) * (D + 4);
          if (tc_fresh_softmax<D, NC>(tc_smem, t.kind == TC_FRESH, t.c.b, t.row0, t.at, t.left, first, n, tmem + lane_at + L::t_s + (n & 1) * NC + col0, o_at, w)) {
            named_bar_sync(id, 128);   // the weights are written
            tc_wait(&bar->pvdone[n & 1], (n >> 1) & 1, bar, a.timeout_ns);
            tc_fence_after();
            tc_wide_values<D, NC>(a, t.c.b, t.h, t.at, t.left, tok, col0, HC, w, o_at);
            tc_fence_before();
          }
          first = false;
          ends = t.ends;
          ++n;
          u += t.step;
          if (t.last) break;
          tc_step<NC>(a, prefix, HR, nfresh, ntiles - u, t);
          if (t.kind == TC_CACHED) break;
        }
      }
#pragma unroll
      for (int i = 0; i < HC / 2; ++i) l[i] = 0.f;
      if (t.kind == TC_CACHED) {
        const float* factor = reinterpret_cast<const float*>(tc_smem + L::factor) + (tri & 1) * NC + col0;
        tc_wait(&bar->sready[n & 1], (n >> 1) & 1, bar, a.timeout_ns);   // (and so the queries have their factors)
        const float common = bar->common[tri & 1];   // the rows' factor, 0: each its own
        const unsigned long long common2 = common == 0.f ? f2_pack(1.f, 1.f) : f2_pack(common, common);
        const int tiles = min(t.c.units - t.c.i, ntiles - u), n0 = n;
        int left = t.c.len - t.at;                   // tokens of the sequence from the tile on
        for (const int end = n + tiles; n < end; ++n, left -= TC_TILE) {
          const int x = n & 1;
          tc_wait(&bar->sready[x], (n >> 1) & 1, bar, a.timeout_ns);
          tc_fence_after();
          const uint32_t s_at = tmem + lane_at + L::t_s + x * NC + col0;
          const bool some = left < TC_TILE, hides = tok >= left;   // no token of the sequence
          float y[HC];
          for (bool again = false;; again = true) {
            tc_ld<HC>(s_at, y);
            float m = 0.f;
            // (After new references the products are rounded as those were: of scores above
            // 2^28 a fused product would leave half a step, which is beyond any weight.)
            const unsigned long long by = again ? f2_pack(1.f, 1.f) : common2;
            if (TC_RARE(again || common == 0.f)) {
#pragma unroll
              for (int i = 0; i < HC; ++i) y[i] *= factor[i];
            }
            // (one factor for all rows: a value for each row and tile less to read, where
            // the bandwidth of shared memory is what bounds a tile of many rows)
#pragma unroll
            for (int i = 0; i < HC; i += 4) {
              const float4 s = *reinterpret_cast<const float4*>(shift + i);
              f2_unpack(f2_fma(f2_pack(y[i], y[i + 1]), by, f2_pack(s.x, s.y)), y[i], y[i + 1]);
              f2_unpack(f2_fma(f2_pack(y[i + 2], y[i + 3]), by, f2_pack(s.z, s.w)), y[i + 2], y[i + 3]);
            }
            if (TC_RARE(some)) {
#pragma unroll
              for (int i = 0; i < HC; ++i)
                if (hides) y[i] = kNegInf;
            }
#pragma unroll
            for (int i = 0; i < HC; i += 2) m = fmax3_nan(m, y[i], y[i + 1]);
            // (in a row without a reference every score but -inf is far above it)
            if (__builtin_expect(again || !tc_any<128>(id, !(m <= AT_PSHIFT + AT_ABOVE)), 1)) break;
            const bool sums = !(first && n == n0);
            if (sums) tc_wait(&bar->pvdone[x ^ 1], ((n - 1) >> 1) & 1, bar, a.timeout_ns);
            tc_raise<D, NC>(tc_smem, s_at, o_at, factor, hides ? ~0u : 0u, sums);
#pragma unroll
            for (int i = 0; i < HC / 2; ++i) l[i] *= corr[(odd ? HC / 2 : 0) + i];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->sfree[x]);   // the scores have been read
#pragma unroll
          for (int i = 0; i < HC; ++i) y[i] = ex2_approx(y[i]);
#pragma unroll
          for (int i = 0; i < HC / 2; ++i) {
            const float keep = odd ? y[i + HC / 2] : y[i], give = odd ? y[i] : y[i + HC / 2];
            l[i] += keep + __shfl_xor_sync(0xffffffffu, give, 1);
          }
          if (n >= 2) tc_wait(&bar->pvdone[x], ((n >> 1) & 1) ^ 1, bar, a.timeout_ns);
          // (a fresh tile's weights are in both buffers)
          if (TC_RARE(n == n0 && n >= 1)) tc_wait(&bar->pvdone[x ^ 1], ((n - 1) >> 1) & 1, bar, a.timeout_ns);
          unsigned char* pb = tc_smem + L::p + x * L::p_bytes + tok * 16 + col0 / 8 * 2048;
#pragma unroll
          for (int i = 0; i < HC; i += 8)
            *reinterpret_cast<uint4*>(pb + i / 8 * 2048) = make_uint4(f16x2_pack(y[i], y[i + 1]), f16x2_pack(y[i + 2], y[i + 3]),
                                                                      f16x2_pack(y[i + 4], y[i + 5]), f16x2_pack(y[i + 6], y[i + 7]));
          tc_fence_before();
          tc_proxy_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->pready[x]);
        }
        u += tiles;
        ends = t.c.i + tiles == t.c.units;
      }
      // the part's end
      tc_wait(&bar->pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, bar, a.timeout_ns);
      unsigned char* sums = tc_smem + L::p + col0 / 8 * 2048;
#pragma unroll
      for (int i = 0; i < HC / 2; ++i) {
        tc_sums<D, NC>(sums, i)[tok] = odd ? 0.f : l[i];
        tc_sums<D, NC>(sums, i + HC / 2)[tok] = odd ? l[i] : 0.f;
      }
      tc_finish<D, NC>(tc_smem, at_row(a, t.c.b, t.h, 0), t.row0, itri == 0 && ends, cta_ws + (itri == 0 ? static_cast<size_t>(NC) * (D + 4) : 0), o_at);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->ofree[tri & 1]);
      named_bar_sync(id, 128);   // top, corr and shift are free again
      if (u >= ntiles) break;
      t.c.i = t.c.units - 1;   // the next triple
      t.step = 1;
      tc_step<NC>(a, prefix, HR, nfresh, ntiles - u, t);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the join kernel may start; it waits for this grid's end)
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&bar->dead)) {
    // A wait ran out of time (every role has ended, so this is settled).  Copies still on
    // their way land before the CTA ends, or a wait for them gives up.
    if (warp == L::SOFT + L::UNPACK + 1) {
      const int n = *reinterpret_cast<volatile int*>(&bar->copied);
      for (int i = max(0, n - L::STAGES); i < n; ++i) mbar_wait(&bar->full[i % L::STAGES], (i / L::STAGES) & 1, a.timeout_ns);
    }
    // Every triple of the share is void.
    TcTile t;
    tc_begin<NC>(a, prefix, HR, nfresh, u0, ntiles, t);
    int i0 = t.c.i;
    for (int u = 0;;) {
      if (t.first) i0 = t.c.i;
      if (t.last) {
        const bool whole = i0 == 0 && t.ends;
        float* part = cta_ws + (i0 == 0 ? static_cast<size_t>(NC) * (D + 4) : 0);
        for (int e = threadIdx.x; e < NC * D; e += L::THREADS) {
          const int r = e / D, d = e - r * D;
          if (!whole) {
            part[e] = 0.f;
            if (d < 3) part[static_cast<size_t>(NC) * D + d * NC + r] = d == 0 ? 0.f : __int_as_float(0x7fc00000);
          } else if (t.row0 + r < rows) {
            const long long at = at_row(a, t.c.b, t.h, t.row0 + r);
            a.out[at * D + d] = 0x7fc0u;
            if (a.lse && d == 0) a.lse[at] = __int_as_float(0x7fc00000);
          }
        }
      }
      if ((u += t.step) >= ntiles) break;
      tc_step<NC>(a, prefix, HR, nfresh, ntiles - u, t);
    }
  }
  if (warp == L::SOFT + L::UNPACK)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::t_cols) : "memory");
}

}  // namespace sv
