// What the host side of the operators shares: workspace laid out over a call,
// launches with their errors, and the guard at the C boundary.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "dmuon.h"
#include "errors.h"
#include "timing.h"

namespace dmuon {
namespace {

#define HIP_TRY(expr)                                                              \
  do {                                                                             \
    hipError_t e_ = (expr);                                                        \
    if (e_ != hipSuccess)                                                          \
      return fail(DMUON_EHIP, "%s failed: %s", #expr, hipGetErrorString(e_));      \
  } while (0)
#define TRY(expr)                  \
  do {                             \
    const int rc_ = (expr);        \
    if (rc_ != DMUON_OK) return rc_; \
  } while (0)

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int esize_of(int dtype) { return dtype == DMUON_BF16 ? 2 : 4; }
inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// Workspace laid out front to back.  Without a base it only counts, which is
// how the *_workspace functions size a call: they run it without launches.
// Nothing in a call's layout or choices may depend on more than its sizes,
// its type and `unaligned`, so that both runs agree; a launch behind memory
// that was not counted is refused.
struct Arena {
  char* base = nullptr;
  int64_t cap = 0;
  int64_t used = 0, peak = 0;
  bool dry = true;
  bool unaligned = false;  // some pointer of the call is not 16-byte aligned
  hipStream_t st = nullptr;
  void* take(int64_t bytes) {
    void* p = base ? base + used : nullptr;
    used += round_up(bytes, 256);
    peak = std::max(peak, used);
    return p;
  }
};

template <class F>
int launch(const Arena& ar, const char* name, double flops, double bytes, F&& f) {
  if (ar.dry) return DMUON_OK;
  if (ar.peak > ar.cap) return fail(DMUON_EINVAL, "%s: workspace overrun", name);
  const hipError_t e = timed_launch(name, flops, bytes, ar.st, f);
  if (e != hipSuccess) return fail(DMUON_EHIP, "%s: %s", name, hipGetErrorString(e));
  return DMUON_OK;
}

// No C++ exception crosses the C boundary.
template <class F>
auto guard(F&& f) -> decltype(f()) {
  try {
    return f();
  } catch (...) {
    return fail(DMUON_ENOMEM, "host allocation failed");
  }
}
// run `f` dry, then, when the workspace holds it, for real
template <class F>
int sized(void* ws, int64_t bytes, bool unaligned, void* stream, F&& f) {
  Arena dry;
  dry.unaligned = unaligned;
  TRY(f(dry));
  if (dry.peak > bytes)
    return fail(DMUON_EINVAL, "workspace of %lld bytes, %lld needed", (long long)bytes, (long long)dry.peak);
  if (dry.peak > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)))
    return fail(DMUON_EINVAL, "workspace is NULL or not 256-byte aligned");
  Arena ar;
  ar.base = (char*)ws;
  ar.cap = bytes;
  ar.dry = false;
  ar.unaligned = unaligned;
  ar.st = static_cast<hipStream_t>(stream);
  return guard([&] { return f(ar); });
}

}  // namespace
}  // namespace dmuon
