// check.h -- argument checks shared by the entry points of the norm, the
// experts' products and the few-token layer.
#pragma once

#include <cstdint>

#include "moeroute.h"

namespace moe {

// A device pointer of a buffer of `bytes` bytes: 16-byte aligned, null only
// where the buffer is empty.
inline bool ok_buffer(const void *p, int64_t bytes) {
    if (bytes == 0) return true;
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The same for an output or input that may be left out.
inline bool ok_optional(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A width of weights or rows: whole blocks of 128, at most 65536.
inline int check_width(int64_t n) {
    if (n <= 0 || n % 128 != 0) return MOE_EINVAL;
    return n > 65536 ? MOE_ENOTSUP : MOE_OK;
}

}  // namespace moe
