// Host helpers of the C ABI's entry points.
#pragma once

#include <cmath>

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

namespace kvq {

// test hook: the tile the next split decode of this host thread withholds
inline thread_local int g_withheld_tile = -1;
inline int take_withheld_tile() {
  const int t = g_withheld_tile;
  g_withheld_tile = -1;
  return t;
}

namespace {

// One NVTX range per enqueueing ABI call (named after it), so that a
// timeline profiler shows which call enqueued which kernels.  NVTX is
// header-only and costs a branch when no tool is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr size_t kAlign = 256;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t dtype_size(kvq_dtype t) { return t == KVQ_F32 ? 4 : 2; }
inline bool dtype_ok(int t) { return t == KVQ_F32 || t == KVQ_BF16 || t == KVQ_F16; }

inline kvq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }
inline double inv_sqrt_d() { return 1.0 / std::sqrt((double)kHeadDim); }

}  // namespace
}  // namespace kvq
