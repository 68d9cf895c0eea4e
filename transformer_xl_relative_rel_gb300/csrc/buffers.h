// buffers.h -- host-side checks of the buffers a call is given.
#pragma once

#include <initializer_list>
#include <stddef.h>
#include <stdint.h>

#include "txl.h"

namespace txl {

struct CallBuffer {
    const void *p;
    size_t bytes, align;
    bool need;           // NULL is an error (unless it holds nothing)
};

inline bool at_boundary(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline bool buffers_overlap(const CallBuffer &a, const CallBuffer &b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}

// TXL_ERR_INVALID for a missing or misaligned buffer, or an output that
// overlaps an input or another output.
inline txl_status check_buffers(std::initializer_list<CallBuffer> ins, std::initializer_list<CallBuffer> outs)
{
    for (const auto *list : {&ins, &outs})
        for (const CallBuffer &b : *list)
            if ((b.need && b.bytes && !b.p) || !at_boundary(b.p, b.align)) return TXL_ERR_INVALID;
    for (const CallBuffer &o : outs) {
        for (const CallBuffer &i : ins)
            if (buffers_overlap(o, i)) return TXL_ERR_INVALID;
        for (const CallBuffer &p : outs)
            if (&p != &o && buffers_overlap(o, p)) return TXL_ERR_INVALID;
    }
    return TXL_OK;
}

}  // namespace txl
