// Whether two strided tensors share an element (host code).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace matopt {

struct Axis {
    int64_t n, stride;   // stride >= 0, in elements
};
// Rows of `dim` consecutive elements from `at` (in elements) on, along three axes of one element at least.
struct Place {
    int64_t at;
    Axis axes[3];
    int64_t dim;
};

// A difference of addresses is a sum of terms c stride: one for an axis whose
// stride both have (c the difference of the indexes), else one for each tensor's.
struct Terms {
    struct { __int128 lo, hi, stride; } t[6];
    __int128 lo[7], hi[7];   // what the terms from one on, and the place in a row, add up to
    int n, left;
};

// Does `want` lie among the sums of the terms from k on? A term takes only
// the values that those after it can make up for: one or two where strides step over
// what lies within them, as those of views of one buffer do. Taken for true
// where it would take more than `left` tries.
inline bool reaches(Terms& x, int k, __int128 want) {
    if (want < x.lo[k] || want > x.hi[k]) return false;
    if (k == x.n || --x.left < 0) return true;
    const auto floor_div = [](__int128 a, __int128 b) { return a / b - (a % b < 0); };
    const auto& t = x.t[k];
    const __int128 from = std::max(t.lo, -floor_div(x.hi[k + 1] - want, t.stride));
    const __int128 to = std::min(t.hi, floor_div(want - x.lo[k + 1], t.stride));
    for (__int128 c = from; c <= to; ++c)
        if (reaches(x, k + 1, want - c * t.stride)) return true;
    return false;
}

inline bool shares(const Place& a, const Place& b) {
    const auto end = [](const Place& p) {
        __int128 e = (__int128)p.at + p.dim;
        for (const Axis& x : p.axes) e += (__int128)(x.n - 1) * x.stride;
        return e;
    };
    if (end(a) <= b.at || end(b) <= a.at) return false;
    Terms x;
    x.n = 0, x.left = 1 << 14;
    const auto term = [&](int64_t lo, int64_t hi, int64_t stride) {
        if (stride && lo < hi) x.t[x.n++] = {lo, hi, stride};
    };
    for (int i = 0; i < 3; ++i) {
        const Axis &p = a.axes[i], &q = b.axes[i];
        if (p.stride == q.stride) {
            term(1 - q.n, p.n - 1, p.stride);
        } else {
            term(0, p.n - 1, p.stride);
            term(1 - q.n, 0, q.stride);
        }
    }
    std::sort(x.t, x.t + x.n, [](const auto& p, const auto& q) { return p.stride > q.stride; });
    x.lo[x.n] = 1 - b.dim, x.hi[x.n] = a.dim - 1;   // a's place in its row less b's
    for (int k = x.n; k-- > 0;) {
        x.lo[k] = x.lo[k + 1] + x.t[k].lo * x.t[k].stride;
        x.hi[k] = x.hi[k + 1] + x.t[k].hi * x.t[k].stride;
    }
    return reaches(x, 0, (__int128)b.at - a.at);
}

}  // namespace matopt
