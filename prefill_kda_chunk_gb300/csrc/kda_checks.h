// Checks of arguments that the C entry points around KDA share: alignment,
// and whether blocks of strided rows share a byte.
#pragma once

#include <stdint.h>

namespace kda {

constexpr int64_t kMaxElems = int64_t(1) << 40;

// A block of rows: `row` bytes each, `step` bytes apart.
struct Rows {
    const void *p;
    int64_t rows, row, step;
};

inline bool misaligned(const void *p, uintptr_t a) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

inline Rows flat(const void *p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Whether two blocks share a byte. Two slices of one fused buffer (equal
// steps) overlap as ranges without sharing any: their rows are compared modulo
// the step.
inline bool share(const Rows &a, const Rows &b) {
    if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.row <= 0 || b.row <= 0)
        return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t ea = pa + (a.rows - 1) * a.step + a.row, eb = pb + (b.rows - 1) * b.step + b.row;
    if (pa >= eb || pb >= ea) return false;
    if (a.step == b.step && a.rows > 1 && b.rows > 1) {
        const int64_t step = a.step;
        const int64_t off = pb >= pa ? static_cast<int64_t>((pb - pa) % step)
                                     : (step - static_cast<int64_t>((pa - pb) % step)) % step;
        return off < a.row || off + b.row > step;   // b's rows start `off` bytes after a's
    }
    return true;
}

inline bool any_shared(const Rows *outs, int n_out, const Rows *ins, int n_in) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (share(outs[o], ins[i])) return true;
        for (int i = o + 1; i < n_out; ++i)
            if (share(outs[o], outs[i])) return true;
    }
    return false;
}

inline bool rows_fit(int64_t rows, int64_t stride, int64_t width) {
    return stride >= width && stride <= kMaxElems && rows <= kMaxElems / stride;
}

}  // namespace kda
