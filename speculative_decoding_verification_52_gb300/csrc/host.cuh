// host.cuh -- host-side helpers shared by the C ABI's translation units: the
// calling thread's last error, per-device facts and one-time kernel setup, the
// timing hooks of spec_profile_begin / spec_profile_end, argument predicates.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <vector>

#include "spec_verify.h"

namespace svh {

inline thread_local char g_err[512] = "";

inline spec_status_t fail(spec_status_t s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

inline spec_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(SPEC_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;
constexpr unsigned long long kWaitNs = 1000000000ull;   // bounded waits: 1 s

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

struct DevInfo {
  bool ready = false;
  int sms = 0;
  int max_cluster = 8;
};
inline std::mutex g_mu;
inline DevInfo g_dev[kMaxDevices];

// Unique id of the calling thread's current CUDA context, plus one (0: no
// context yet, or the driver entry points are unavailable).  A device reset or
// a re-created primary context gets a new id, so per-device caches keyed on it
// are set up again instead of reusing state of a context that is gone.
inline unsigned long long current_ctx_id() {
  using GetCurrent = int (*)(void**);
  using GetId = int (*)(void*, unsigned long long*);
  static GetCurrent get_current = nullptr;
  static GetId get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<GetCurrent>(fn);
    fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<GetId>(fn);
    cudaGetLastError();
  });
  if (!get_current || !get_id) return 0;
  void* ctx = nullptr;
  if (get_current(&ctx) != 0 || !ctx) return 0;
  unsigned long long id = 0;
  if (get_id(ctx, &id) != 0) return 0;
  return id + 1;
}

// per-kernel one-time attribute setup, per device and context (attributes do
// not survive a device reset); without a context id it runs every time
template <class F>
inline bool once_per_device(int dev, F&& f) {
  static unsigned long long done[kMaxDevices] = {};   // context id the setup ran in
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 0 || dev >= kMaxDevices) return false;
  const unsigned long long id = current_ctx_id();
  if (id == 0 || done[dev] != id) {
    if (!f()) return false;
    done[dev] = current_ctx_id();   // (the setup may have created the context)
  }
  return true;
}

inline spec_status_t device_info(DevInfo& out, int& dev) {
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(SPEC_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& d = g_dev[dev];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    int major = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (major < 10) return fail(SPEC_ERR_UNSUPPORTED, "compute capability %d.x: this library is built for sm_103a", major);
    d.ready = true;
  }
  out = d;
  return SPEC_OK;
}

// ---------------------------------------------------------------------------
// profiling events
// ---------------------------------------------------------------------------
struct Prof {
  bool on = false;
  int max_calls = 0;
  int calls = 0;
  std::vector<cudaEvent_t> ev;
};
inline Prof g_prof;

inline void prof_mark(int slot, cudaStream_t st) {
  if (!g_prof.on || g_prof.calls >= g_prof.max_calls) return;
  cudaEventRecord(g_prof.ev[3 * g_prof.calls + slot], st);
  if (slot == 2) ++g_prof.calls;
}

// cuTensorMapEncodeTiled, null where the driver has none
using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline TensorMapEncode tensor_map_encode() {
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

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int esz_of(spec_dtype_t d) { return d == SPEC_BF16 ? 2 : 4; }
inline bool dtype_ok(spec_dtype_t d) { return d == SPEC_F32 || d == SPEC_BF16; }

inline spec_status_t check_ws(void* ws, size_t have, size_t need) {
  if (need == 0) return SPEC_OK;
  if (!ws) return fail(SPEC_ERR_WORKSPACE, "NULL workspace (need %zu bytes)", need);
  if (!aligned16(ws)) return fail(SPEC_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  if (have < need) return fail(SPEC_ERR_WORKSPACE, "workspace %zu bytes < required %zu", have, need);
  return SPEC_OK;
}

}  // namespace svh
