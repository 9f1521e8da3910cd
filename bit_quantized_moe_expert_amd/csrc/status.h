// Status plumbing shared by the C ABI files: the thread-local message of the
// last failure, and argument checks.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/nf4moe.h"

namespace nf4moe {

// Sets this thread's nf4moe_last_error() message and returns st.
nf4moe_status_t fail(nf4moe_status_t st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
nf4moe_status_t hip_status(hipError_t e, const char *what);

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace nf4moe
