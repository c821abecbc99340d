// spans.h -- host checks of pointers that the entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "skinny_gemm.h"

namespace skg {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A tensor's memory, for the overlap checks (null: none).
struct Span {
    const void *p;
    size_t bytes;
};
inline bool overlap(Span a, Span b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
template <size_t N, size_t L>
bool any_overlap(const Span (&outs)[N], const Span (&ins)[L]) {
    for (size_t i = 0; i < N; ++i) {
        for (size_t j = i + 1; j < N; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (const Span &s : ins)
            if (overlap(outs[i], s)) return true;
    }
    return false;
}

inline int hip_status(int hip) { return hip == (int)hipSuccess ? SKG_OK : SKG_ERR_HIP; }

}  // namespace skg
