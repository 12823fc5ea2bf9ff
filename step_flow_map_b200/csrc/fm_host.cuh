// Host-side error reporting shared by the library's translation units.
#pragma once
#include <cuda_runtime.h>

#include "flashmap.h"

// Records the text fm_last_error() returns on this thread; returns `st`.
fm_status set_err(fm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)))
__attribute__((visibility("hidden")));

#define FM_CUDA(call)                                                               \
  do {                                                                              \
    cudaError_t e_ = (call);                                                        \
    if (e_ != cudaSuccess)                                                          \
      return set_err(FM_ERR_CUDA, "%s failed: %s (%s:%d)", #call,                   \
                     cudaGetErrorString(e_), __FILE__, __LINE__);                   \
  } while (0)
#define FM_LAUNCHED() FM_CUDA(cudaGetLastError())
#define FM_TRY(expr)                  \
  do {                                \
    fm_status s_ = (expr);            \
    if (s_ != FM_OK) return s_;       \
  } while (0)
