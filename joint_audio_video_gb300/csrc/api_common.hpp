// What the C entry points share: the per-device context, argument checks, the
// NVTX range and the H3_DEBUG_SYNC epilogue.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>

#include "../../include/h3attn.h"
#include "kernels.hpp"

namespace h3 {

// The current device's status word, SM count and wait limit.
h3_status dev_ctx(DevCtx* ctx);

// What an entry point returns after its last launch: `s`, or with H3_DEBUG_SYNC
// the device status once the stream is done.
h3_status finish(h3_status s, h3_stream_t stream);

inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline bool valid_d(int32_t d) { return d >= 128 && d <= 16384 && d % 128 == 0; }
// head counts of 128-wide heads that give a valid d (checked before any
// multiplication, so a huge count cannot wrap around to a valid width)
inline bool valid_heads(int32_t n_heads) { return n_heads >= 1 && n_heads <= 16384 / 128; }

inline h3_status launched(cudaError_t e) { return e == cudaSuccess ? H3_OK : H3_ERR_CUDA; }

// An NVTX range named after the entry point around its host-side work, so a
// timeline tool shows which call enqueued which kernels.
struct Trace {
  explicit Trace(const char* name) { nvtxRangePushA(name); }
  ~Trace() { nvtxRangePop(); }
  Trace(const Trace&) = delete;
  Trace& operator=(const Trace&) = delete;
};

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace h3
