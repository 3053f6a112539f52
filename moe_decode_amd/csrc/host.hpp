// host.hpp -- what the C entry points share: the error return with its
// thread-local message, and the argument checks more than one file makes.
// Internal to libmoe_decode; defined in abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_decode.h"

namespace md {

md_status fail(md_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
md_status ok();
md_status hip_fail(hipError_t e, const char* what);
md_status check_qmatrix(const char* what, const md_qmatrix* W);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace md
