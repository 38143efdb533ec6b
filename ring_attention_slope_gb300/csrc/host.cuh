// What the C entry points share: the last error's text, pointer checks and the
// NVTX range of a public call.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

#include "slope.h"

namespace slope {

// Records the text of a failing CUDA call (slope_last_error) and returns SLOPE_ERR_CUDA.
slope_status cuda_fail(const char* where, cudaError_t e);
slope_status cuda_fail(const char* where);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// fp32 [H, S], any positive strides.
slope_status check_lse(const slope_tensor* t, int64_t H, int64_t S);
// [S, H, dv] output, fp32 (or bf16 when allowed); 16-byte vector stores.
slope_status check_out(const slope_tensor* t, int64_t S, int64_t H, int64_t dv, bool allow_bf16);

uint64_t wait_limit_ns();
float resolve_scale(float scale, int64_t dqk);

// One NVTX range around each public call that queues GPU work, named after the call, so that
// Nsight tools group its launches (ncu --nvtx).  With no tool attached a push or pop is a check
// of a function pointer.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

}  // namespace slope
