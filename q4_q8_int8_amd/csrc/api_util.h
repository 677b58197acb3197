// Argument checks shared by the entry-point sources beside api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "mmq.h"
#include "mmq_internal.h"

namespace mmq {

inline int fail(int status, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return api_fail(status, msg);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_pointers(std::initializer_list<const void*> needed,
                          const void* optional = nullptr) {
  for (const void* p : needed) {
    if (!p) return fail(MMQ_E_ARG, "null device pointer");
    if (!aligned16(p)) return fail(MMQ_E_ARG, "device pointers must be 16-byte aligned");
  }
  if (!aligned16(optional)) return fail(MMQ_E_ARG, "device pointers must be 16-byte aligned");
  return MMQ_OK;
}

inline int hip_status(const char* what, hipError_t e) {
  return e == hipSuccess ? api_ok() : fail(MMQ_E_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

}  // namespace mmq
