// Pieces shared by the files that implement the C-ABI: argument checks,
// workspace carving and the per-launch trace.
#pragma once

#include <hip/hip_runtime.h>
#include <climits>
#include <cstdint>
#include <vector>

#include "moe.h"

namespace moe {

constexpr int64_t kMaxInt = 2147483647;
// Operand matrices (h, grouped rows, hidden activations, one expert's weight
// matrix) hold at most 2^31 - 2^22 elements and d, width are at most 2^20, so that
// 32-bit element offsets, and the byte offsets of the GEMMs' buffer loads (row
// offset + k offset), never wrap.
constexpr int64_t kMaxElems = (int64_t{1} << 31) - (int64_t{1} << 22);
constexpr int64_t kMaxDim = int64_t{1} << 20;

inline size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// A tensor pointer: NULL only when the tensor has no elements; 16-byte aligned.
inline int check_ptr(const void* p, bool has_elements) {
  if (p == nullptr) return has_elements ? MOE_ERR_NULL : MOE_OK;
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

inline int check_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (need > 0 && ws == nullptr) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

#define MOE_CHECK(expr)              \
  do {                               \
    const int _s = (expr);           \
    if (_s != MOE_OK) return _s;     \
  } while (0)

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

struct TraceState {
  bool on = false;
  int cap = 0;
  int n = 0;
  std::vector<hipEvent_t> ev;
  std::vector<int32_t> kid;
};
extern TraceState g_trace;  // api.hip

template <typename F>
hipError_t traced(int kid, hipStream_t st, F&& launch) {
  if (!g_trace.on || g_trace.n >= g_trace.cap) return launch();
  const int i = g_trace.n++;
  g_trace.kid[i] = kid;
  (void)hipEventRecord(g_trace.ev[2 * i], st);
  const hipError_t err = launch();
  (void)hipEventRecord(g_trace.ev[2 * i + 1], st);
  return err;
}

#define MOE_LAUNCH(kid, st, call)                                      \
  do {                                                                 \
    const hipError_t _e = moe::traced((kid), (st), [&] { return call; }); \
    if (_e != hipSuccess) return MOE_ERR_HIP;                          \
  } while (0)

}  // namespace moe
