// Host checks shared by the entry points of the operators around the expert FFN.
#pragma once

#include "status.h"

namespace moe {

// bytes [lo, hi) that a matrix of `rows` rows touches
struct Span {
    uintptr_t lo, hi;
};
inline Span span(const void* p, int64_t rows, int64_t ld, int64_t cols, int es) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (!p || rows < 1) return {0, 0};
    return {b, b + static_cast<uintptr_t>(((rows - 1) * ld + cols) * es)};
}
inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
inline int esize(int32_t dt) { return dt == MOE_F32 ? 4 : 2; }

// Rows of ld elements that no address space holds (2^48 bytes and more): refused, so
// that the byte counts of a span stay inside 64 bits.
inline bool beyond(int64_t rows, int64_t ld) { return rows > 1 && ld > (1ll << 46) / rows; }

// no two outputs meet, and no output meets an input
inline moe_status check_apart(const char* fn, const Span* in, int n_in, const Span* out, int n_out) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return fail(MOE_E_ARG, fn, "two outputs overlap");
        for (int j = 0; j < n_in; ++j)
            if (meet(out[i], in[j])) return fail(MOE_E_ARG, fn, "an output overlaps an input");
    }
    return MOE_OK;
}

}  // namespace moe
