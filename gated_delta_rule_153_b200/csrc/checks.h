// checks.h -- host-side argument checks shared by entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace gdn {

struct Range {
    const void* p;
    size_t bytes;
};

inline bool aligned_to(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}

// True when some output shares bytes with an input or with another output.
inline bool outputs_overlap(std::initializer_list<Range> in, std::initializer_list<Range> out) {
    for (const Range& o : out) {
        for (const Range& i : in)
            if (overlap(o, i)) return true;
        for (const Range& o2 : out)
            if (&o2 != &o && overlap(o, o2)) return true;
    }
    return false;
}

inline bool all_aligned_to(unsigned a, std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned_to(p, a)) return false;
    return true;
}

}  // namespace gdn
