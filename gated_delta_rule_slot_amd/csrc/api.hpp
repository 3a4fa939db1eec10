// api.hpp -- what the C entry points of the GPU library share: export, messages, argument
// checks and the status of a launch.  Internal; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "errors.hpp"

#define GDN_API extern "C" __attribute__((visibility("default")))
#define fail(...) gdn::set_error(__VA_ARGS__)

namespace gdn {

inline gdn_status ok() { return clear_error(); }

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline gdn_status launched(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(GDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace gdn
