// entry.cuh -- what the entry points of attention share: results, checks of arguments,
// and the frame around a call. Host code.
#pragma once

#include "attend_internal.cuh"

#include <nvtx3/nvToolsExt.h>

#include <string>

namespace kvx {

inline int invalid(const char* msg) {
  set_last_error(msg);
  return KVEVICT_ERR_INVALID_ARG;
}

inline int cuda_result(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return KVEVICT_OK;
  set_last_error(std::string(what) + ": " + cudaGetErrorString(e));
  return e == cudaErrorMemoryAllocation ? KVEVICT_ERR_OOM : KVEVICT_ERR_CUDA;
}

inline bool aligned(const void* p, unsigned to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Whole 16-byte pieces between the entries of every dimension that has several.
template <int K>
bool strides16(const int64_t (&s)[K], const int32_t (&extent)[K], int elem) {
  for (int i = 0; i < K; ++i)
    if (extent[i] > 1 && ((s[i] * elem) & 15)) return false;
  return true;
}

// Rows of D elements that cannot lie apart (written by several threads at once).
template <int K>
bool rows_overlap(const int64_t (&s)[K], const int32_t (&extent)[K], int D) {
  for (int i = 0; i < K; ++i)
    if (extent[i] > 1 && s[i] < D && s[i] > -D) return true;
  return false;
}

inline bool is16(int dtype) { return dtype == kFp16 || dtype == kBf16; }

// An NVTX range named after the entry point, and no C++ exception past it (an
// error message is the only thing that allocates).
template <typename F>
int entry(const char* name, F&& body) {
  nvtxRangePushA(name);
  int rc;
  try {
    rc = body();
  } catch (...) {
    rc = KVEVICT_ERR_OOM;
  }
  nvtxRangePop();
  return rc;
}

}  // namespace kvx
