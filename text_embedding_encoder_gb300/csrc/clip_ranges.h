// Memory ranges of the tensors that are clipped together (host code).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

// Whether an output overlaps another one or a gradient that is not its own: 1 or 0, and -1
// where there is no memory to find out.  outs NULL: all in place.
inline int clip_overlaps(const void* const* grads, const int64_t* counts, const int32_t* types, int32_t bf16_type,
                         void* const* outs, int n) {
    struct Range {
        uintptr_t begin, end;
        bool out;
    };
    // (an exception must not leave the library's entry points)
    const std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * (size_t)n + 1]);
    if (!r) return -1;
    Range* end = r.get();
    for (int i = 0; i < n; ++i) {
        if (counts[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)counts[i] * (types[i] == bf16_type ? 2 : 4);
        const uintptr_t g = (uintptr_t)grads[i], o = (uintptr_t)(outs ? outs[i] : grads[i]);
        *end++ = Range{o, o + bytes, true};
        if (g != o) *end++ = Range{g, g + bytes, false};
    }
    std::sort(r.get(), end, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    uintptr_t any = 0, out = 0;   // ends of what lies before
    for (const Range* x = r.get(); x < end; ++x) {
        if (x->begin < (x->out ? any : out)) return 1;
        any = std::max(any, x->end);
        if (x->out) out = std::max(out, x->end);
    }
    return 0;
}
