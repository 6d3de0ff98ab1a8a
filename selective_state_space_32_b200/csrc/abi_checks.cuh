// abi_checks.cuh -- host-side argument checks shared by the C entry points of the
// recurrent block's operators (glr.cu, norm.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include "sscan.h"

namespace sscan {

struct Span {  // a caller's buffer: p may be null (absent)
    const void *p;
    size_t bytes;
};

inline bool spans_overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// 16-byte alignment of every buffer, outputs disjoint from the inputs and from each
// other, the workspace disjoint from all of them.
template <int NI, int NO>
inline int check_buffers(const Span (&ins)[NI], const Span (&outs)[NO], const Span &ws) {
    for (const Span &s : ins)
        if (reinterpret_cast<uintptr_t>(s.p) & 15u) return SSCAN_ERR_ALIGN;
    for (const Span &s : outs)
        if (reinterpret_cast<uintptr_t>(s.p) & 15u) return SSCAN_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(ws.p) & 15u) return SSCAN_ERR_ALIGN;
    for (int i = 0; i < NO; ++i) {
        for (const Span &s : ins)
            if (spans_overlap(outs[i], s)) return SSCAN_ERR_INVALID;
        for (int k = i + 1; k < NO; ++k)
            if (spans_overlap(outs[i], outs[k])) return SSCAN_ERR_INVALID;
        if (spans_overlap(outs[i], ws)) return SSCAN_ERR_WORKSPACE;
    }
    for (const Span &s : ins)
        if (spans_overlap(s, ws)) return SSCAN_ERR_WORKSPACE;
    return SSCAN_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round_up_256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace sscan
