// after_verify.cu -- host side of the steps after a verification declared in
// include/spec_verify.h: log probabilities of the emitted tokens, weights of the cached
// tokens, eviction by them (plan, moves).  Argument checks, launch shapes, dispatch;
// one launch a call on the caller's stream, no sync.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "evict.cuh"
#include "host.cuh"
#include "spec_verify.h"
#include "token_logprobs.cuh"
#include "weigh_q4.cuh"
#include "weigh_q4_tc.cuh"

namespace {

using namespace sv;
using namespace svh;

constexpr int kMaxShift = 32;
constexpr int kSmemPerSm = 227 * 1024;   // shared memory that the CTAs of an SM can use together

bool q4_dim(int D) { return D == 64 || D == 128; }
bool below_2g(long long a, long long b) { return a * b < (1LL << 31); }

// what all calls over the cache's slots ask of its sizes
spec_status_t check_pool(int B, int Hkv, int P, int pages, int max_pages) {
  if (B < 0 || Hkv < 1 || P < 1 || pages < 1 || max_pages < 1)
    return fail(SPEC_ERR_INVALID_ARG, "bad sizes B=%d Hkv=%d page_tokens=%d num_pages=%d max_pages=%d", B, Hkv, P, pages, max_pages);
  if (P % Q4_BLOCK != 0) return fail(SPEC_ERR_INVALID_ARG, "page_tokens=%d is not a multiple of %d", P, Q4_BLOCK);
  if (!below_2g(P, pages) || !below_2g(max_pages, P))
    return fail(SPEC_ERR_UNSUPPORTED, "num_pages and max_pages times page_tokens must stay below 2^31");
  if (static_cast<long long>(pages) * (P / Q4_BLOCK) * Hkv >= 0xffffffffLL)   // (blocks are numbered in 32 bits)
    return fail(SPEC_ERR_UNSUPPORTED, "num_pages * page_tokens * Hkv must stay below 2^37");
  return SPEC_OK;
}

template <class K, class A>
spec_status_t launch_cluster(K kern, dim3 grid, int threads, size_t smem, int C, cudaStream_t st, const A& a, const char* what) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e == cudaSuccess ? SPEC_OK : cuda_fail(e, what);
}

// ---------------------------------------------------------------------------
// log probabilities
// ---------------------------------------------------------------------------
template <class T, int WARPS, bool TOP>
spec_status_t launch_logprobs(int dev, const LogprobArgs& a, cudaStream_t st) {
  auto kern = token_logprobs_kernel<T, WARPS, TOP>;
  constexpr int TEAMS = lp_threads(WARPS) / (32 * WARPS);
  constexpr size_t smem = sizeof(LpShared<WARPS>) * TEAMS;
  if (smem > 48 * 1024 && !once_per_device(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) == cudaSuccess;
      }))
    return fail(SPEC_ERR_CUDA, "log probabilities setup failed: %s", cudaGetErrorString(cudaGetLastError()));
  const long long places = static_cast<long long>(a.B) * a.M, grid = (places + TEAMS - 1) / TEAMS * a.C;
  if (grid > 0x7fffffffLL) return fail(SPEC_ERR_UNSUPPORTED, "batch too large for one call");
  return launch_cluster(kern, dim3(static_cast<unsigned>(grid)), lp_threads(WARPS), smem, a.C, st, a, "log probabilities launch");
}
template <class T>
spec_status_t launch_logprobs(int dev, bool warp, const LogprobArgs& a, cudaStream_t st) {
  if (warp) return a.top ? launch_logprobs<T, 1, true>(dev, a, st) : launch_logprobs<T, 1, false>(dev, a, st);
  return a.top ? launch_logprobs<T, LP_WARPS, true>(dev, a, st) : launch_logprobs<T, LP_WARPS, false>(dev, a, st);
}

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------
template <int D, int NR>
spec_status_t launch_weigh(const DevInfo& di, int dev, const WeighArgs& a, cudaStream_t st) {
  auto kern = weigh_q4_kernel<D, NR>;
  constexpr int WARPS = WG_THREADS / 32;
  // as many CTAs an SM as the registers allow, with two to eight stages; fewer CTAs
  // where the largest batches leave no room for that (2.25 KB a CTA: the system's and the static part)
  const size_t fixed = 8 * (static_cast<size_t>(a.B) + 1) + 4 * static_cast<size_t>(a.B), stage = WARPS * (wg_stage_bytes(D) + 8);
  int ctas = wg_ctas(NR);
  auto room = [&](int n) { return static_cast<long long>(kSmemPerSm / n) - 2304 - static_cast<long long>(fixed); };
  while (ctas > 1 && room(ctas) < static_cast<long long>(3 * stage)) --ctas;
  const int stages = static_cast<int>(std::min<long long>(8, room(ctas) / static_cast<long long>(stage)));
  if (!once_per_device(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm - 4096) == cudaSuccess;
      }))
    return fail(SPEC_ERR_CUDA, "weighing setup failed: %s", cudaGetErrorString(cudaGetLastError()));
  kern<<<static_cast<unsigned>(di.sms * ctas), WG_THREADS, fixed + stages * stage, st>>>(a, stages);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : cuda_fail(e, "weighing launch");
}
template <int D>
spec_status_t launch_weigh(int NR, const DevInfo& di, int dev, const WeighArgs& a, cudaStream_t st) {
  switch (NR) {
    case 1: return launch_weigh<D, 1>(di, dev, a, st);
    case 2: return launch_weigh<D, 2>(di, dev, a, st);
    case 3: return launch_weigh<D, 3>(di, dev, a, st);
    default: return launch_weigh<D, 4>(di, dev, a, st);
  }
}

template <int D>
spec_status_t launch_weigh_tc(const DevInfo& di, int dev, const WeighArgs& a, cudaStream_t st) {
  auto kern = weigh_q4_tc_kernel<D>;
  TensorMapEncode encode = tensor_map_encode();
  if (!encode) return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  // the queries as [B][N][Hq][D], in boxes of the nodes and the kv head's query heads of a tile
  CUtensorMap map;
  const cuuint64_t heads = static_cast<cuuint64_t>(a.Hkv) * a.G, row = 2 * D;
  const cuuint64_t dims[4] = {D, heads, static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.B)};
  const cuuint64_t strides[3] = {row, row * heads, row * heads * a.N};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(WT_ROWS / a.G), 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(a.q), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled: %d", static_cast<int>(r));
  const size_t fixed = (sizeof(WtShared<D>) + 15) / 16 * 16 + 1024 + 8;
  if (!once_per_device(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(fixed + 12 * WG_MAX_B)) == cudaSuccess;
      }))
    return fail(SPEC_ERR_CUDA, "weighing setup failed: %s", cudaGetErrorString(cudaGetLastError()));
  kern<<<static_cast<unsigned>(2 * di.sms), WT_THREADS, fixed + 12 * static_cast<size_t>(a.B), st>>>(a, map);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : cuda_fail(e, "weighing launch");
}

// Which kernel, by the rows that a sequence may commit and D: few rows, whose kernel's time
// grows with the rows, or tiles of 64 of them on the tensor cores.  256 sequences at 2,048
// tokens and 8 at 16,384, 8 kv heads of 4 query heads, in us:
//   D = 128   36 rows 227 and 61 (few), 308 and 68 (many);   52: 308 and 67 (many)
//   D = 64    68 rows 246 and 67 (few), 302 and 66 (many);   100: 336 and 90 (few), 304 and 66 (many)
// so few rows up to what two and three turns of 32 hold.  A path's nodes do not lie side by
// side: few rows.
constexpr int kWeighFewRows128 = 48, kWeighFewRows64 = 96;

}  // namespace

extern "C" {

spec_status_t spec_token_logprobs(const void* logits, spec_dtype_t dtype, const int32_t* tokens, const int32_t* path,
                                  float temperature, int B, int R, int V, int M, int W, int top_n, float* logprobs,
                                  float* entropy, int32_t* ranks, int32_t* top_tokens, float* top_logprobs, void* stream) {
  try {
    if (B < 0 || R < 1 || V < 1 || M < 1 || top_n < 0)
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes B=%d R=%d V=%d M=%d top_n=%d", B, R, V, M, top_n);
    if (V > (1 << 30)) return fail(SPEC_ERR_UNSUPPORTED, "V=%d beyond 2^30", V);
    if (top_n > LP_MAX_TOP) return fail(SPEC_ERR_UNSUPPORTED, "top_n=%d beyond %d", top_n, LP_MAX_TOP);
    if (!dtype_ok(dtype)) return fail(SPEC_ERR_INVALID_ARG, "bad dtype");
    if (!(temperature > 0.f) || !std::isfinite(temperature)) return fail(SPEC_ERR_INVALID_ARG, "temperature must be positive and finite");
    if (temperature < 1e-4f) return fail(SPEC_ERR_UNSUPPORTED, "temperature %g below 1e-4", static_cast<double>(temperature));
    if (path ? W < M - 1 : R < M) return fail(SPEC_ERR_INVALID_ARG, "M=%d tokens for %s of %d", M, path ? "a path" : "rows", path ? W : R);
    if (static_cast<long long>(B) * M > 0x7fffffffLL) return fail(SPEC_ERR_UNSUPPORTED, "batch too large for one call");
    if (B == 0) return SPEC_OK;
    if (!logits || !tokens || !logprobs) return fail(SPEC_ERR_INVALID_ARG, "NULL logits/tokens/logprobs");
    if (top_n > 0 && (!top_tokens || !top_logprobs)) return fail(SPEC_ERR_INVALID_ARG, "NULL top_tokens/top_logprobs");
    if (reinterpret_cast<uintptr_t>(logits) % esz_of(dtype)) return fail(SPEC_ERR_INVALID_ARG, "logits must be aligned to their elements");
    int dev;
    DevInfo di;
    spec_status_t s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    LogprobArgs a{};
    a.logits = static_cast<const unsigned char*>(logits);
    a.tokens = tokens;
    a.path = path;
    a.B = B;
    a.R = R;
    a.V = V;
    a.M = M;
    a.W = W;
    a.top = top_n;
    a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.ranks = ranks;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    // A warp a row where the rows are short or many enough, else a CTA, and a cluster of
    // CTAs where the rows alone do not fill the device.  In us, five alternatives, a CTA
    // against a warp a row: rows of 1 KB, 16 of them 14.8 and 5.5; of 4 KB, 304 of them 6.2
    // and 7.2, 608 8.5 and 7.2, 2,432 28 and 8.6; of 16 KB, 608 9.1 and 15.3, 2,432 28 and
    // 18; of 32 KB, 5,000 73 and 67; of 64 KB, 5,000 103 and 121.  CTAs a row, 128,256 bf16
    // and 20 alternatives: one row, 1 15.5, 2 12.6, 4 9.9, 8 9.9; 64 rows, 1 16.9, 4 12.2, 8
    // 17.1; 152 rows, 1 17.4, 2 15.9, 4 22.1; 320 rows, 1 26.0, 2 30.6.
    const long long places = static_cast<long long>(B) * M, bytes = static_cast<long long>(V) * esz_of(dtype);
    const bool warp = bytes <= 2048 || (bytes <= 32768 && 1024 * places >= di.sms * bytes);
    a.C = 1;
    if (!warp)
      while (a.C < 8 && places * 2 * a.C <= 2LL * di.sms && bytes / (2 * a.C) >= 8192) a.C *= 2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    s = dtype == SPEC_BF16 ? launch_logprobs<BF16T>(dev, warp, a, st) : launch_logprobs<F32T>(dev, warp, a, st);
    if (s != SPEC_OK) return s;
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

spec_status_t spec_kv_weigh_q4(const void* q, const float* lse, const int32_t* path, const int32_t* count, const void* cache,
                               const int32_t* block_table, const int32_t* lengths, const int32_t* first_positions, int B,
                               int N, int W, int Hq, int Hkv, int D, int page_tokens, int num_pages, int max_pages,
                               int k_shift, float scale, float decay, const float* weights, float* new_weights,
                               int32_t* positions, void* stream) {
  try {
    if (!q4_dim(D)) return fail(SPEC_ERR_UNSUPPORTED, "D=%d: the 4-bit cache takes 64 or 128", D);
    spec_status_t s = check_pool(B, Hkv, page_tokens, num_pages, max_pages);
    if (s != SPEC_OK) return s;
    if (N < 1 || N > SPEC_MAX_TREE_NODES || (path && W < 1))
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes N=%d W=%d (N in [1, %d])", N, W, SPEC_MAX_TREE_NODES);
    if (Hq < 1 || Hq % Hkv != 0) return fail(SPEC_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
    if (Hq / Hkv > 64) return fail(SPEC_ERR_UNSUPPORTED, "%d query heads to a kv head: at most 64", Hq / Hkv);
    if (B > WG_MAX_B) return fail(SPEC_ERR_UNSUPPORTED, "B=%d beyond %d", B, WG_MAX_B);
    if (path && W > SPEC_MAX_TREE_NODES) return fail(SPEC_ERR_UNSUPPORTED, "W=%d beyond %d", W, SPEC_MAX_TREE_NODES);
    if (std::abs(k_shift) > kMaxShift) return fail(SPEC_ERR_INVALID_ARG, "k_shift %d outside [-%d, %d]", k_shift, kMaxShift, kMaxShift);
    if (!std::isfinite(scale) || !std::isfinite(decay)) return fail(SPEC_ERR_INVALID_ARG, "scale and decay must be finite");
    if (B == 0) return SPEC_OK;
    if (!q || !lse || !cache || !block_table || !lengths || !weights || !new_weights)
      return fail(SPEC_ERR_INVALID_ARG, "NULL q/lse/cache/block_table/lengths/weights/new_weights");
    if (!aligned16(q) || !aligned16(cache)) return fail(SPEC_ERR_INVALID_ARG, "q and cache must be 16-byte aligned");
    int dev;
    DevInfo di;
    s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    WeighArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.lse = lse;
    a.path = path;
    a.count = count;
    a.cache = static_cast<const unsigned char*>(cache);
    a.table = block_table;
    a.lengths = lengths;
    a.first = first_positions;
    a.weights = weights;
    a.new_weights = new_weights;
    a.positions = positions;
    a.B = B;
    a.N = N;
    a.PW = path ? W : 0;
    a.most = path ? W : N;
    a.G = Hq / Hkv;
    a.Hkv = Hkv;
    a.P = page_tokens;
    a.pages = num_pages;
    a.W = max_pages;
    a.scale_log2 = static_cast<float>(1.4426950408889634 * static_cast<double>(scale));
    a.k_mul = std::ldexp(1.f, k_shift);
    a.decay = decay;
    a.timeout_ns = kWaitNs;
    const int rows = a.most * a.G, tiles = ceil_div(rows, 32), NR = ceil_div(ceil_div(rows, 8), tiles);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    if (!path && rows > (D == 128 ? kWeighFewRows128 : kWeighFewRows64)) s = D == 128 ? launch_weigh_tc<128>(di, dev, a, st) : launch_weigh_tc<64>(di, dev, a, st);
    else s = D == 128 ? launch_weigh<128>(NR, di, dev, a, st) : launch_weigh<64>(NR, di, dev, a, st);
    if (s != SPEC_OK) return s;
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

spec_status_t spec_kv_evict_plan(const float* weights, const int32_t* positions, const int32_t* block_table,
                                 const int32_t* lengths, const int32_t* budgets, const int32_t* next_positions, int B,
                                 int Hkv, int page_tokens, int num_pages, int max_pages, int sinks, int recent,
                                 int max_moves, int32_t* moves, int32_t* move_counts, int32_t* new_lengths, void* stream) {
  try {
    spec_status_t s = check_pool(B, Hkv, page_tokens, num_pages, max_pages);
    if (s != SPEC_OK) return s;
    if (sinks < 0 || recent < 0 || max_moves < 1)
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes sinks=%d recent=%d max_moves=%d", sinks, recent, max_moves);
    if (B == 0) return SPEC_OK;
    if (!weights || !positions || !block_table || !lengths || !budgets || !next_positions || !moves || !move_counts || !new_lengths)
      return fail(SPEC_ERR_INVALID_ARG, "NULL pointer argument");
    if (new_lengths == lengths) return fail(SPEC_ERR_INVALID_ARG, "new_lengths must not be lengths");
    if (reinterpret_cast<uintptr_t>(moves) & 7u) return fail(SPEC_ERR_INVALID_ARG, "moves must be 8-byte aligned");
    int dev;
    DevInfo di;
    s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    PlanArgs a{};
    a.weights = weights;
    a.positions = positions;
    a.table = block_table;
    a.lengths = lengths;
    a.budgets = budgets;
    a.next = next_positions;
    a.B = B;
    a.Hkv = Hkv;
    a.P = page_tokens;
    a.pages = num_pages;
    a.W = max_pages;
    a.max_moves = max_moves;
    a.sinks = sinks;
    a.recent = recent;
    a.moves = moves;
    a.counts = move_counts;
    a.new_lengths = new_lengths;
    // A cluster where the heads alone do not fill the device and the table has room for long
    // sequences (64 heads of 32,768 tokens, in us: 1 CTA a head 366, 2 144, 4 29, 8 27; 16 of
    // 65,536: 736, 362, 140, 29).
    const long long pairs = static_cast<long long>(B) * Hkv, most = static_cast<long long>(max_pages) * page_tokens;
    a.C = 1;
    while (a.C < EV_CLUSTER && pairs * a.C < 2LL * di.sms && most / a.C > 4096) a.C *= 2;
    if (pairs * a.C > 0x7fffffffLL) return fail(SPEC_ERR_UNSUPPORTED, "batch too large for one call");
    a.cap = static_cast<int>(std::min<long long>(EV_CAP, (most + a.C * 128 - 1) / (a.C * 128) * 128 + (a.C > 1 ? 128 : 0)));
    // Several heads a CTA, whose warps look for few tokens to drop, where that leaves two
    // CTAs an SM, with 48 KB of keys at most (2,048 heads, in us: 1 a CTA 43, 2 24, 4 15;
    // that drop half of 4,096 tokens, CTA by CTA: 64, 65, 65).
    a.rows = 1;
    while (a.C == 1 && a.rows < EV_ROWS && pairs / (2 * a.rows) >= 2LL * di.sms && 2 * a.rows * a.cap <= 12288) a.rows *= 2;
    const size_t smem = 4 * (static_cast<size_t>(EV_HISTS) * EV_BINS + static_cast<size_t>(a.rows) * a.cap);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    auto kern = a.C > 1 ? evict_plan_kernel<true> : evict_plan_kernel<false>;
    if (!once_per_device(dev, [&] {
          const int all = 4 * (EV_HISTS * EV_BINS + std::max(EV_CAP, 12288));
          return cudaFuncSetAttribute(evict_plan_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, all) == cudaSuccess &&
                 cudaFuncSetAttribute(evict_plan_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, all) == cudaSuccess;
        }))
      return fail(SPEC_ERR_CUDA, "eviction plan setup failed: %s", cudaGetErrorString(cudaGetLastError()));
    s = launch_cluster(kern, dim3(static_cast<unsigned>((pairs + a.rows - 1) / a.rows * a.C)), EV_THREADS, smem, a.C, st, a, "eviction plan launch");
    if (s != SPEC_OK) return s;
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

spec_status_t spec_kv_move_q4(void* cache, float* weights, int32_t* positions, const int32_t* moves, const int32_t* move_counts,
                              int B, int Hkv, int D, int page_tokens, int num_pages, int max_moves, void* stream) {
  try {
    if (!q4_dim(D)) return fail(SPEC_ERR_UNSUPPORTED, "D=%d: the 4-bit cache takes 64 or 128", D);
    spec_status_t s = check_pool(B, Hkv, page_tokens, num_pages, 1);
    if (s != SPEC_OK) return s;
    if (max_moves < 1) return fail(SPEC_ERR_INVALID_ARG, "max_moves=%d must be positive", max_moves);
    const long long pairs = static_cast<long long>(B) * Hkv;
    if (pairs > 0x7fffffffLL) return fail(SPEC_ERR_UNSUPPORTED, "batch too large for one call");
    if (B == 0) return SPEC_OK;
    if (!cache || !moves || !move_counts) return fail(SPEC_ERR_INVALID_ARG, "NULL cache/moves/move_counts");
    if (!aligned16(cache)) return fail(SPEC_ERR_INVALID_ARG, "cache must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(moves) & 7u) return fail(SPEC_ERR_INVALID_ARG, "moves must be 8-byte aligned");
    int dev;
    DevInfo di;
    s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    MoveArgs a{};
    a.cache = static_cast<unsigned char*>(cache);
    a.weights = weights;
    a.positions = positions;
    a.moves = moves;
    a.counts = move_counts;
    a.Hkv = Hkv;
    a.P = page_tokens;
    a.pages = num_pages;
    a.max_moves = max_moves;
    // enough CTAs a head for its longest list, no more than fill the device
    const long long want = ceil_div(max_moves, MV_THREADS), room = std::max<long long>(1, di.sms * 16 / pairs);
    const dim3 grid(static_cast<unsigned>(pairs), static_cast<unsigned>(std::min(std::min(want, room), 65535LL)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    if (D == 128) kv_move_q4_kernel<128><<<grid, MV_THREADS, 0, st>>>(a);
    else kv_move_q4_kernel<64><<<grid, MV_THREADS, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "kv move launch");
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

}  // extern "C"
