// What the C entry points share: statuses with a message, checks of pointers, and returns on the first failure.
#pragma once

#include <cuda_runtime.h>

#include <cstdio>
#include <initializer_list>

#include "../../include/tpmlp.h"
#include "tpmlp_internal.h"

namespace tpmlp {

inline tpmlp_status err(tpmlp_status st, const char* msg) { return static_cast<tpmlp_status>(report_error(st, msg)); }

inline tpmlp_status cuda_err(cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return err(TPMLP_ERR_CUDA, msg);
}

// a: a power of two. A null pointer is aligned.
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline tpmlp_status check_ptrs(std::initializer_list<const void*> ptrs, size_t a, const char* what) {
  for (const void* p : ptrs) {
    if (!p) return err(TPMLP_ERR_INVALID, "null pointer");
    if (!aligned(p, a)) return err(TPMLP_ERR_ALIGN, what);
  }
  return TPMLP_OK;
}

}  // namespace tpmlp

#define TPMLP_PASS(expr)                       \
  do {                                         \
    const tpmlp_status _s = (expr);            \
    if (_s != TPMLP_OK) return _s;             \
  } while (0)
#define TPMLP_PASS_CUDA(expr, what)                      \
  do {                                                   \
    const cudaError_t _e = (expr);                       \
    if (_e != cudaSuccess) return cuda_err(_e, what);    \
  } while (0)
