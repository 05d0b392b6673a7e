// Host-side argument checks shared by the C ABI entry points.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace xlstm {

inline bool aligned16(const void *p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
    const char *lo;
    size_t bytes;
};

inline bool overlap(Range a, Range b) {
    if (!a.lo || !b.lo || a.bytes == 0 || b.bytes == 0) return false;
    return a.lo < b.lo + b.bytes && b.lo < a.lo + a.bytes;
}

inline Range rg(const void *p, size_t bytes) { return Range{static_cast<const char *>(p), bytes}; }

// No output range meets an input range or another output range.
template <int NI, int NO>
inline bool outputs_disjoint(const Range (&ins)[NI], const Range (&outs)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(outs[o], ins[i])) return false;
        for (int o2 = 0; o2 < o; ++o2)
            if (overlap(outs[o], outs[o2])) return false;
    }
    return true;
}

}  // namespace xlstm
