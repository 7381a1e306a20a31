// api_checks.h - argument checks, status macros and workspace header of the C ABI's entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.h"

namespace moe {

// Workspace: the count/scan state (ScanWorkspace: [0] status word, [64, 160) the count/scan
// ticket, done counter and failure flag, [256 ...) look-back flags, expert totals and per-block
// rows), whose bytes [160 + 16 s, 176 + 16 s) hold the GEMM tile schedule of call site s
// (s < 6); then the gating partials.
constexpr size_t kWsHeader = 256;
enum SchedSlot : int { kSchedGating = 0, kSchedGateUp, kSchedDown, kSchedDense, kSchedSharedGateUp, kSchedSharedDown };

inline int* ws_status(void* ws) { return reinterpret_cast<int*>(ws); }
inline int* ws_sched(void* ws, SchedSlot s) { return reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(ws) + 160 + 16 * s); }

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

#define MOE_TRY(expr)                      \
  do {                                     \
    const moe_status _s = (expr);          \
    if (_s != MOE_OK) return _s;           \
  } while (0)

#define MOE_CUDA(expr)                                        \
  do {                                                        \
    if ((expr) != cudaSuccess) return MOE_ERR_CUDA;           \
  } while (0)

inline moe_status common_checks(const moe_dims* d) {
  MOE_TRY(check_dims(d));
  if (!device_ok()) return MOE_ERR_NO_DEVICE;
  return MOE_OK;
}

// The grouped GEMMs use only the workspace header (status word and tile-schedule counters).
inline moe_status check_ws_header(const void* ws, size_t ws_bytes) {
  if (!ws || ws_bytes < kWsHeader || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace moe
