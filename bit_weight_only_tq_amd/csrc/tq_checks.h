// Argument checks that the files of C entry points share.
#pragma once

#include "tq.h"

#include <stdint.h>

namespace {

constexpr int64_t kInt32Max = 0x7FFFFFFF;

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline tq_status from_hip(hipError_t e) { return e == hipSuccess ? TQ_OK : TQ_ERR_HIP; }

// `bytes` bytes of a caller's buffer; empty ones overlap nothing.
struct Span {
    const void* p;
    int64_t bytes;
    bool overlaps(const Span& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return bytes > 0 && o.bytes > 0 && a < b + (uintptr_t)o.bytes && b < a + (uintptr_t)bytes;
    }
};

}  // namespace
