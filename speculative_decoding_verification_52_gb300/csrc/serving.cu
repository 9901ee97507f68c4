// serving.cu -- host side of the serving steps around verification declared in
// include/spec_verify.h: the paged 4-bit cache (page map, store, commit,
// attention) and the logit adjustments.  Argument checks, launch shapes,
// dispatch; one or two launches a call on the caller's stream, no sync.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "adjust.cuh"
#include "attend_q4.cuh"
#include "attend_q4_tc.cuh"
#include "common.cuh"
#include "host.cuh"
#include "kv_q4.cuh"
#include "page_map.cuh"
#include "spec_verify.h"

namespace {

using namespace sv;
using namespace svh;

constexpr int kMaxShift = 32;
constexpr int kSmemPerSm = 227 * 1024;   // shared memory that the CTAs of an SM can use together
constexpr int kMaxDynSmem = kSmemPerSm - 1024;   // dynamic part of a CTA that is alone on an SM, beside its static part

bool q4_dim(int D) { return D == 64 || D == 128; }
bool below_2g(long long a, long long b) { return a * b < (1LL << 31); }

spec_status_t check_q4(int Hkv, int D, int P, int pages, int k_shift, int v_shift) {
  if (!q4_dim(D)) return fail(SPEC_ERR_UNSUPPORTED, "D=%d: the 4-bit cache takes 64 or 128", D);
  if (Hkv < 1 || P < 1 || pages < 1) return fail(SPEC_ERR_INVALID_ARG, "bad sizes Hkv=%d page_tokens=%d num_pages=%d", Hkv, P, pages);
  if (P % Q4_BLOCK != 0) return fail(SPEC_ERR_INVALID_ARG, "page_tokens=%d is not a multiple of %d", P, Q4_BLOCK);
  if (!below_2g(P, pages)) return fail(SPEC_ERR_UNSUPPORTED, "num_pages * page_tokens must stay below 2^31");
  if (std::abs(k_shift) > kMaxShift || std::abs(v_shift) > kMaxShift)
    return fail(SPEC_ERR_INVALID_ARG, "shifts (%d, %d) outside [-%d, %d]", k_shift, v_shift, kMaxShift, kMaxShift);
  return SPEC_OK;
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// Rows of a warp's tile, in units of 8: as few tiles of at most 32 rows as hold
// them all, since a block is fetched and unpacked once for each tile, and no
// wider than that needs.
void attend_tiles(int rows, int& tiles, int& NR) {
  tiles = ceil_div(rows, 32);
  NR = ceil_div(ceil_div(rows, 8), tiles);
}
constexpr int kMaxSms = 160;   // bound of the workspace size; the grid never exceeds it

// Joins what the CTAs' shares cut.  Few triples: each is spread over many CTAs,
// and a CTA joins eight rows of one; else a warp does.
template <int D>
spec_status_t launch_join(const DevInfo& di, const AttendArgs& a, int grid, int shares, int R8, size_t stride, cudaStream_t st) {
  const long long triples = static_cast<long long>(a.B) * a.Hkv * a.row_tiles, items = triples * R8;
  const size_t smem = 8 * (static_cast<size_t>(a.B) + 1);
  if (items > 0x7fffffffLL) return fail(SPEC_ERR_UNSUPPORTED, "batch too large for one call");
  const bool spread = triples * 4 <= grid;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(spread ? items : std::min<long long>((items + ATJ_WARPS - 1) / ATJ_WARPS, static_cast<long long>(di.sms) * 4)));
  cfg.blockDim = dim3(ATJ_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];   // starts beside the attention's last CTAs and waits for them (a tenth less for one token)
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, spread ? attend_q4_join_kernel<D, true> : attend_q4_join_kernel<D, false>, a, grid, shares, R8, stride);
  return e == cudaSuccess ? SPEC_OK : cuda_fail(e, "attention join launch");
}

template <int D, int NR>
spec_status_t launch_attend(const DevInfo& di, int dev, const AttendArgs& a, cudaStream_t st) {
  auto kern = attend_q4_kernel<D, NR>;
  const size_t fixed = static_cast<size_t>(AT_PAIRS) * at_pair_bytes(D, NR) + 8 * (static_cast<size_t>(a.B) + 1);
  const size_t stage = static_cast<size_t>(AT_PAIRS) * (at_stage_bytes(D) + 8);
  // As many CTAs an SM as the registers allow, with as many stages (2 to 6) as
  // leave room for them; fewer CTAs where two stages do not.  (1.25 KB a CTA: the
  // system's and the static part.)
  int ctas = at_ctas(D, NR);
  auto room = [&](int n) { return static_cast<long long>(kSmemPerSm / n) - 1280 - static_cast<long long>(fixed); };
  while (ctas > 1 && room(ctas) < static_cast<long long>(2 * stage)) --ctas;
  const int stages = static_cast<int>(std::min<long long>(6, room(ctas) / static_cast<long long>(stage)));
  if (stages < 2) return fail(SPEC_ERR_UNSUPPORTED, "batch too large for one call");
  const size_t smem = fixed + stages * stage;
  if (!once_per_device(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynSmem) == cudaSuccess;
      }))
    return fail(SPEC_ERR_CUDA, "attention kernel setup failed: %s", cudaGetErrorString(cudaGetLastError()));
  const int grid = std::min(di.sms, kMaxSms) * ctas;
  kern<<<grid, AT_THREADS, smem, st>>>(a, stages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return launch_join<D>(di, a, grid, AT_PAIRS, NR, at_cta_floats(D, NR), st);
}

template <int D>
spec_status_t launch_attend(int NR, const DevInfo& di, int dev, const AttendArgs& a, cudaStream_t st) {
  switch (NR) {
    case 1: return launch_attend<D, 1>(di, dev, a, st);
    case 2: return launch_attend<D, 2>(di, dev, a, st);
    case 3: return launch_attend<D, 3>(di, dev, a, st);
    default: return launch_attend<D, 4>(di, dev, a, st);
  }
}

// ---------------------------------------------------------------------------
// attention on the tcgen05 tensor cores
// ---------------------------------------------------------------------------
using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TensorMapEncode tensor_map_encode() {
  static TensorMapEncode fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    cudaGetLastError();
    return reinterpret_cast<TensorMapEncode>(p);
  }();
  return fn;
}

// dynamic shared memory: the layout, its alignment, the batch's prefix sums
size_t tc_smem_bytes(uint32_t layout, int B) { return layout + 1024 + 8 * (static_cast<size_t>(B) + 1); }
size_t tc_smem_bytes(int D, int NC, int B) {
  return tc_smem_bytes(D == 64 ? TcLayout<64, 128>::bytes : NC == 64 ? TcLayout<128, 64>::bytes : TcLayout<128, 128>::bytes, B);
}

template <int D, int NC>
spec_status_t launch_attend_tc(const DevInfo& di, int dev, const AttendArgs& a, cudaStream_t st) {
  auto kern = attend_q4_tc_kernel<D, NC>;
  TensorMapEncode encode = tensor_map_encode();
  if (!encode) return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  // the cache as blocks of 72 rows of D / 2 bytes (32 of keys, 32 of values, 8 of scales)
  CUtensorMap map;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D / 2), 72,
                              static_cast<cuuint64_t>(a.pages) * a.Hkv * (a.P / Q4_BLOCK)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D / 2), static_cast<cuuint64_t>(q4_block_bytes(D))};
  const cuuint32_t box[3] = {D / 2, 72, 1}, step[3] = {1, 1, 1};
  const CUresult r = encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<unsigned char*>(a.cache), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled: %d", static_cast<int>(r));
  if (!once_per_device(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynSmem) == cudaSuccess;
      }))
    return fail(SPEC_ERR_CUDA, "attention kernel setup failed: %s", cudaGetErrorString(cudaGetLastError()));
  const int grid = std::min(di.sms, kMaxSms);
  kern<<<grid, TcLayout<D, NC>::THREADS, tc_smem_bytes(TcLayout<D, NC>::bytes, a.B), st>>>(a, map);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return launch_join<D>(di, a, grid, 1, NC / 8, tc_cta_floats(D, NC), st);
}

spec_status_t launch_attend_tc(int D, int NC, const DevInfo& di, int dev, const AttendArgs& a, cudaStream_t st) {
  if (D == 64) return launch_attend_tc<64, 128>(di, dev, a, st);
  return NC == 64 ? launch_attend_tc<128, 64>(di, dev, a, st) : launch_attend_tc<128, 128>(di, dev, a, st);
}

// Which kernel, and its row tile.
struct AttendPlan {
  bool tc;
  int tiles;      // row tiles of a (sequence, head)
  int size;       // NR of attend_q4_kernel (rows / 8 of a tile), NC of attend_q4_tc_kernel
  size_t floats;  // of the workspace
};
// Up to how many rows attend_q4_kernel is taken, against the tensor cores' kernel, whose
// time hardly depends on the rows of a tile.  256 sequences at 2,048 tokens, and 32 at
// 8,192, with fresh entries: D = 128, 48 rows (two tiles of 24) 508 us against 735, and
// 244 against 225; 56 rows (two of 32) 640 against 730, and 298 against 224; 64 rows 648
// against 732, and 304 against 226.  D = 64, 72 rows (three of 24) 523 against 746, and
// 237 against 249; 80 rows (three of 32) 661 against 742, and 299 against 250.  So up to
// the rows that tiles of 24 hold: beyond them one loses more with long contexts than it
// gains with many short ones.
constexpr int kFewRows128 = 48, kFewRows64 = 72;
AttendPlan attend_plan(int B, int rows, int D) {
  AttendPlan p{};
  const int NC = D == 128 && rows <= 64 ? 64 : 128;   // (what there are kernels for)
  // (the largest batches leave no room for the tensor cores' kernel)
  p.tc = rows > (D == 128 ? kFewRows128 : kFewRows64) && tc_smem_bytes(D, NC, B) <= static_cast<size_t>(kMaxDynSmem);
  if (p.tc) {
    p.size = NC;
    p.tiles = ceil_div(rows, NC);
    p.floats = static_cast<size_t>(kMaxSms) * tc_cta_floats(D, NC);
  } else {
    attend_tiles(rows, p.tiles, p.size);
    p.floats = static_cast<size_t>(kMaxSms) * at_ctas(D, p.size) * at_cta_floats(D, p.size);
  }
  return p;
}

// spec_attend_q4, and with stall_cta >= 0 its test hook
spec_status_t attend_entry(const void* q, const void* k_new, const void* v_new, const uint32_t* masks,
                           const void* cache, const int32_t* block_table, const int32_t* lengths, int B, int N,
                           int Hq, int Hkv, int D, int page_tokens, int num_pages, int max_pages, int k_shift,
                           int v_shift, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                           void* stream, int stall_cta = -1, unsigned long long timeout_ns = kWaitNs) {
  try {
    spec_status_t s = check_q4(Hkv, D, page_tokens, num_pages, k_shift, v_shift);
    if (s != SPEC_OK) return s;
    if (B < 0 || N < 1 || N > SPEC_MAX_TREE_NODES || max_pages < 1)
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes B=%d N=%d max_pages=%d (N in [1, %d])", B, N, max_pages, SPEC_MAX_TREE_NODES);
    if (Hq < 1 || Hq % Hkv != 0) return fail(SPEC_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
    if (Hq / Hkv > 64) return fail(SPEC_ERR_UNSUPPORTED, "%d query heads to a kv head: at most 64", Hq / Hkv);
    if (B > AT_MAX_B) return fail(SPEC_ERR_UNSUPPORTED, "B=%d beyond %d", B, AT_MAX_B);
    if (!below_2g(max_pages, page_tokens)) return fail(SPEC_ERR_UNSUPPORTED, "max_pages * page_tokens must stay below 2^31");
    if (!std::isfinite(scale)) return fail(SPEC_ERR_INVALID_ARG, "scale must be finite");
    if ((k_new == nullptr) != (v_new == nullptr)) return fail(SPEC_ERR_INVALID_ARG, "k_new and v_new come together");
    if (masks && !k_new) return fail(SPEC_ERR_INVALID_ARG, "masks without k_new and v_new");
    if (B == 0) return SPEC_OK;
    if (!q || !cache || !block_table || !lengths || !out) return fail(SPEC_ERR_INVALID_ARG, "NULL q/cache/block_table/lengths/out");
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(k_new) || !aligned16(v_new))
      return fail(SPEC_ERR_INVALID_ARG, "q, k_new, v_new, cache and out must be 16-byte aligned");
    s = check_ws(workspace, workspace_bytes, spec_attend_workspace_bytes(B, N, Hq, Hkv, D));
    if (s != SPEC_OK) return s;
    int dev;
    DevInfo di;
    s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    AttendArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k_new = static_cast<const uint16_t*>(k_new);
    a.v_new = static_cast<const uint16_t*>(v_new);
    a.masks = masks;
    a.cache = static_cast<const unsigned char*>(cache);
    a.table = block_table;
    a.lengths = lengths;
    a.B = B;
    a.N = N;
    a.G = Hq / Hkv;
    a.Hkv = Hkv;
    a.P = page_tokens;
    a.pages = num_pages;
    a.W = max_pages;
    a.NW = (N + 31) / 32;
    const AttendPlan plan = attend_plan(B, N * a.G, D);
    a.row_tiles = plan.tiles;
    a.by_g = a.G > 1 ? static_cast<uint32_t>((0x100000000ull + a.G - 1) / a.G) : 0u;
    a.tile = plan.tc ? TC_TILE : AT_TILE;
    a.fresh = plan.tc ? TC_FRESH_UNITS : AT_FRESH;
    a.fresh_more = plan.tc ? TC_FRESH_MORE : AT_FRESH;
    a.scale_log2 = static_cast<float>(1.4426950408889634 * static_cast<double>(scale));
    a.k_mul = std::ldexp(1.f, k_shift);
    a.v_mul = std::ldexp(1.f, v_shift);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.ws = static_cast<float*>(workspace);
    a.timeout_ns = timeout_ns;
    a.stall = stall_cta + 1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    if (plan.tc) s = launch_attend_tc(D, plan.size, di, dev, a, st);
    else s = D == 128 ? launch_attend<128>(plan.size, di, dev, a, st) : launch_attend<64>(plan.size, di, dev, a, st);
    if (s != SPEC_OK) return s;
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

// ---------------------------------------------------------------------------
// logit adjustments
// ---------------------------------------------------------------------------
template <class T, bool VEC>
spec_status_t launch_adjust(int dev, unsigned grid, const AdjustArgs& a, cudaStream_t st) {
  auto kern = adjust_logits_kernel<T, VEC>;
  if (!once_per_device(dev, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 6 * AJ_MAX_CHUNK) == cudaSuccess;
      }))
    return fail(SPEC_ERR_CUDA, "logit adjustment setup failed: %s", cudaGetErrorString(cudaGetLastError()));
  const long long marks = (a.nodes ? a.Nt : 0) + static_cast<long long>(a.bias_tokens ? a.M : 0);
  const size_t smem = 4 * static_cast<size_t>(a.chunk) + 2 * static_cast<size_t>(std::min<long long>(a.chunk, marks));
  kern<<<grid, AJ_THREADS, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "logit adjustment launch");
  return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_q4_block_bytes(int D) { return q4_dim(D) ? static_cast<size_t>(q4_block_bytes(D)) : 0; }

spec_status_t spec_page_map(const int32_t* lengths, const int32_t* count, const int32_t* held, int32_t* ring,
                            const int32_t* ring_state, int32_t* block_table, int B, int ring_size, int page_tokens,
                            int max_pages, int max_tokens, int32_t* offsets, int32_t* slots, int32_t* positions,
                            int32_t* new_held, int32_t* new_ring_state, int32_t* status, void* stream) {
  try {
    if (B < 0 || ring_size < 1 || page_tokens < 1 || max_pages < 1 || max_tokens < 0)
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes B=%d ring_size=%d page_tokens=%d max_pages=%d max_tokens=%d", B,
                  ring_size, page_tokens, max_pages, max_tokens);
    if (!below_2g(ring_size, page_tokens) || !below_2g(max_pages, page_tokens))
      return fail(SPEC_ERR_UNSUPPORTED, "ring_size and max_pages times page_tokens must stay below 2^31");
    if (!ring || !ring_state || !offsets || !new_ring_state || (max_tokens > 0 && (!slots || !positions)) ||
        (B > 0 && (!lengths || !count || !held || !block_table || !new_held || !status)))
      return fail(SPEC_ERR_INVALID_ARG, "NULL pointer argument");
    if ((B > 0 && new_held == held) || new_ring_state == ring_state)
      return fail(SPEC_ERR_INVALID_ARG, "new_held / new_ring_state must not be held / ring_state");
    int dev;
    DevInfo di;
    spec_status_t s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    PageMapArgs a{};
    a.lengths = lengths;
    a.count = count;
    a.held = held;
    a.ring = ring;
    a.ring_state = ring_state;
    a.table = block_table;
    a.B = B;
    a.F = ring_size;
    a.P = page_tokens;
    a.W = max_pages;
    a.T = max_tokens;
    a.offsets = offsets;
    a.slots = slots;
    a.positions = positions;
    a.new_held = new_held;
    a.new_ring_state = new_ring_state;
    a.status = status;
    a.vec = aligned16(slots) && aligned16(positions);
    const int grid = std::max(1, ceil_div(max_tokens, PM_TILE));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    page_map_kernel<<<grid, PM_THREADS, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "page map launch");
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

spec_status_t spec_kv_store_q4(const void* k, const void* v, const int32_t* slots, int T, int Hkv, int D,
                               int page_tokens, int num_pages, int k_shift, int v_shift, void* cache, void* stream) {
  try {
    spec_status_t s = check_q4(Hkv, D, page_tokens, num_pages, k_shift, v_shift);
    if (s != SPEC_OK) return s;
    if (T < 0) return fail(SPEC_ERR_INVALID_ARG, "T=%d must be >= 0", T);
    if (Hkv > 65535) return fail(SPEC_ERR_UNSUPPORTED, "Hkv=%d beyond 65535", Hkv);
    if (T == 0) return SPEC_OK;
    if (!k || !v || !slots || !cache) return fail(SPEC_ERR_INVALID_ARG, "NULL k/v/slots/cache");
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache))
      return fail(SPEC_ERR_INVALID_ARG, "k, v and cache must be 16-byte aligned");
    int dev;
    DevInfo di;
    s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    KvQ4Args a{};
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.cache = static_cast<unsigned char*>(cache);
    a.slots = slots;
    a.T = T;
    a.Hkv = Hkv;
    a.P = page_tokens;
    a.pages = num_pages;
    a.k_mul = std::ldexp(1.f, -k_shift);
    a.v_mul = std::ldexp(1.f, -v_shift);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(ceil_div(T, Q4_THREADS / (D / 16))), static_cast<unsigned>(Hkv));
    prof_mark(0, st);
    if (D == 128) kv_store_q4_kernel<128><<<grid, Q4_THREADS, 0, st>>>(a);
    else kv_store_q4_kernel<64><<<grid, Q4_THREADS, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "kv store launch");
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

spec_status_t spec_kv_commit_q4(void* cache, const int32_t* block_table, const int32_t* lengths, const void* k,
                                const void* v, const int32_t* path, const int32_t* count, int B, int N, int W, int Hkv,
                                int D, int page_tokens, int num_pages, int max_pages, int k_shift, int v_shift,
                                int32_t* new_lengths, void* stream) {
  try {
    spec_status_t s = check_q4(Hkv, D, page_tokens, num_pages, k_shift, v_shift);
    if (s != SPEC_OK) return s;
    if (B < 0 || N < 1 || max_pages < 1 || (path && W < 1))
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes B=%d N=%d W=%d max_pages=%d", B, N, W, max_pages);
    if (!below_2g(max_pages, page_tokens)) return fail(SPEC_ERR_UNSUPPORTED, "max_pages * page_tokens must stay below 2^31");
    if (B == 0) return SPEC_OK;
    if (!cache || !block_table || !lengths || !k || !v || !count || !new_lengths)
      return fail(SPEC_ERR_INVALID_ARG, "NULL cache/block_table/lengths/k/v/count/new_lengths");
    if (new_lengths == lengths) return fail(SPEC_ERR_INVALID_ARG, "new_lengths must not be lengths");
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache))
      return fail(SPEC_ERR_INVALID_ARG, "k, v and cache must be 16-byte aligned");
    int dev;
    DevInfo di;
    s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    KvQ4Args a{};
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.cache = static_cast<unsigned char*>(cache);
    a.table = block_table;
    a.lengths = lengths;
    a.path = path;
    a.count = count;
    a.new_lengths = new_lengths;
    a.B = B;
    a.N = N;
    a.W = max_pages;
    a.PW = path ? W : 0;
    a.Hkv = Hkv;
    a.P = page_tokens;
    a.pages = num_pages;
    a.k_mul = std::ldexp(1.f, -k_shift);
    a.v_mul = std::ldexp(1.f, -v_shift);
    // enough CTAs a sequence for its largest request, no more than fill the device
    const long long items = static_cast<long long>(path ? W : N) * Hkv * (D / 16);
    const long long want = (items + Q4_THREADS - 1) / Q4_THREADS;
    const long long cap = std::max(1, di.sms * 16 / B);
    const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>(std::min(std::min(want, cap), 65535LL)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    if (D == 128) kv_commit_q4_kernel<128><<<grid, Q4_THREADS, 0, st>>>(a);
    else kv_commit_q4_kernel<64><<<grid, Q4_THREADS, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "kv commit launch");
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

size_t spec_attend_workspace_bytes(int B, int N, int Hq, int Hkv, int D) {
  if (B < 0 || B > AT_MAX_B || N < 1 || N > SPEC_MAX_TREE_NODES || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 ||
      Hq / Hkv > 64 || !q4_dim(D))
    return 0;
  return align_up(attend_plan(B, N * (Hq / Hkv), D).floats * sizeof(float), 256);
}

spec_status_t spec_attend_q4(const void* q, const void* k_new, const void* v_new, const uint32_t* masks,
                             const void* cache, const int32_t* block_table, const int32_t* lengths, int B, int N,
                             int Hq, int Hkv, int D, int page_tokens, int num_pages, int max_pages, int k_shift,
                             int v_shift, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return attend_entry(q, k_new, v_new, masks, cache, block_table, lengths, B, N, Hq, Hkv, D, page_tokens, num_pages,
                      max_pages, k_shift, v_shift, scale, out, lse, workspace, workspace_bytes, stream);
}

spec_status_t spec_debug_attend_stall(const void* q, const void* k_new, const void* v_new, const uint32_t* masks,
                                      const void* cache, const int32_t* block_table, const int32_t* lengths, int B,
                                      int N, int Hq, int Hkv, int D, int page_tokens, int num_pages, int max_pages,
                                      int k_shift, int v_shift, float scale, int stall_cta, unsigned timeout_us,
                                      void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (stall_cta < 0 || timeout_us < 100 || timeout_us > 1000000)
    return fail(SPEC_ERR_INVALID_ARG, "stall_cta=%d timeout_us=%u (at least 0; 100..1000000)", stall_cta, timeout_us);
  return attend_entry(q, k_new, v_new, masks, cache, block_table, lengths, B, N, Hq, Hkv, D, page_tokens, num_pages,
                      max_pages, k_shift, v_shift, scale, out, lse, workspace, workspace_bytes, stream, stall_cta,
                      1000ull * timeout_us);
}

spec_status_t spec_adjust_logits(const void* logits, spec_dtype_t dtype, const int32_t* history,
                                 const int32_t* prompt_lengths, const int32_t* history_lengths,
                                 const float* repetition, const float* frequency, const float* presence,
                                 const int32_t* node_tokens, const uint32_t* masks, const int32_t* bias_tokens,
                                 const float* bias_values, const uint32_t* allowed, int B, int R, int V, int H, int Nt,
                                 int M, void* out, void* stream) {
  try {
    if (B < 0 || R < 1 || R > SPEC_MAX_TREE_NODES || V < 1 || H < 0 || Nt < 0 || Nt > SPEC_MAX_TREE_NODES || M < 0)
      return fail(SPEC_ERR_INVALID_ARG, "bad sizes B=%d R=%d V=%d H=%d Nt=%d M=%d (R, Nt at most %d)", B, R, V, H, Nt, M,
                  SPEC_MAX_TREE_NODES);
    if (V > (1 << 30)) return fail(SPEC_ERR_UNSUPPORTED, "V=%d beyond 2^30", V);
    if (!dtype_ok(dtype)) return fail(SPEC_ERR_INVALID_ARG, "bad dtype");
    if (history && H > 0 && !history_lengths) return fail(SPEC_ERR_INVALID_ARG, "history without history_lengths");
    if (masks && (!node_tokens || Nt != R)) return fail(SPEC_ERR_INVALID_ARG, "masks need node_tokens of R columns (Nt=%d, R=%d)", Nt, R);
    if (node_tokens && !masks && Nt < R - 1) return fail(SPEC_ERR_INVALID_ARG, "node_tokens has %d columns for %d rows", Nt, R);
    if ((bias_tokens == nullptr) != (bias_values == nullptr)) return fail(SPEC_ERR_INVALID_ARG, "bias_tokens and bias_values come together");
    if (B == 0) return SPEC_OK;
    if (!logits || !out) return fail(SPEC_ERR_INVALID_ARG, "NULL logits/out");
    const int esz = esz_of(dtype);
    if (reinterpret_cast<uintptr_t>(logits) % esz || reinterpret_cast<uintptr_t>(out) % esz)
      return fail(SPEC_ERR_INVALID_ARG, "logits and out must be aligned to their elements");
    int dev;
    DevInfo di;
    spec_status_t s = device_info(di, dev);
    if (s != SPEC_OK) return s;
    AdjustArgs a{};
    a.logits = static_cast<const unsigned char*>(logits);
    a.out = static_cast<unsigned char*>(out);
    a.history = H > 0 ? history : nullptr;
    a.prompt_len = prompt_lengths;
    a.hist_len = history_lengths;
    a.repetition = repetition;
    a.frequency = frequency;
    a.presence = presence;
    a.nodes = Nt > 0 ? node_tokens : nullptr;
    a.masks = masks;
    a.bias_tokens = M > 0 ? bias_tokens : nullptr;
    a.bias_values = bias_values;
    a.allowed = allowed;
    a.B = B;
    a.R = R;
    a.V = V;
    a.H = a.history ? H : 0;
    a.Nt = Nt;
    a.NW = (R + 31) / 32;
    a.M = M;
    a.VW = (V + 31) / 32;
    const bool vec = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    // Chunks as large as shared memory likes (a CTA counts the whole history),
    // smaller ones where the batch alone does not give every SM two CTAs; and the
    // rows shared out, four a CTA at least, to eight CTAs an SM.
    const long long want = 2LL * di.sms;
    a.chunk = AJ_MAX_CHUNK;
    while (a.chunk > 1024 && static_cast<long long>(B) * ceil_div(V, a.chunk) < want) a.chunk /= 2;
    while (a.chunk > 32 && a.chunk / 2 >= V) a.chunk /= 2;
    a.chunks = ceil_div(V, a.chunk);
    const long long ctas = static_cast<long long>(B) * a.chunks;
    a.row_splits = static_cast<int>(std::max<long long>(
        1, std::min<long long>(ceil_div(R, 4), (4 * want + ctas - 1) / std::max<long long>(1, ctas))));
    if (ctas * a.row_splits > 0x7fffffffLL) return fail(SPEC_ERR_UNSUPPORTED, "grid too large");
    const unsigned grid = static_cast<unsigned>(ctas * a.row_splits);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    prof_mark(0, st);
    if (dtype == SPEC_BF16) s = vec ? launch_adjust<BF16T, true>(dev, grid, a, st) : launch_adjust<BF16T, false>(dev, grid, a, st);
    else s = vec ? launch_adjust<F32T, true>(dev, grid, a, st) : launch_adjust<F32T, false>(dev, grid, a, st);
    if (s != SPEC_OK) return s;
    prof_mark(1, st);
    prof_mark(2, st);
    return SPEC_OK;
  } catch (...) {
    return fail(SPEC_ERR_CUDA, "unexpected host exception");
  }
}

}  // extern "C"
