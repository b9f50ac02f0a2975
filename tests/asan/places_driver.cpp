// csrc/places.h against a walk over all elements. Test infrastructure: built and
// run by tests/test_places_host.py.
#include "places.h"

#include <chrono>
#include <cstdio>
#include <random>
#include <set>

using namespace matopt;

static void elements(const Place& p, std::set<int64_t>& out) {
    for (int64_t i = 0; i < p.axes[0].n; ++i)
        for (int64_t j = 0; j < p.axes[1].n; ++j)
            for (int64_t k = 0; k < p.axes[2].n; ++k)
                for (int64_t e = 0; e < p.dim; ++e)
                    out.insert(p.at + i * p.axes[0].stride + j * p.axes[1].stride + k * p.axes[2].stride + e);
}

int main() {
    std::mt19937_64 r(1);
    int wrong = 0, shared = 0;
    const int cases = 60000;
    for (int n = 0; n < cases; ++n) {
        Place a, b;
        a.dim = 1 + r() % 4, b.dim = r() % 2 ? a.dim : 1 + r() % 4;
        a.at = r() % 60, b.at = r() % 60;
        for (int i = 0; i < 3; ++i) {
            a.axes[i] = {(int64_t)(1 + r() % 4), (int64_t)(r() % 30)};
            b.axes[i] = {(int64_t)(1 + r() % 4), r() % 2 ? a.axes[i].stride : (int64_t)(r() % 30)};
        }
        std::set<int64_t> x, y;
        elements(a, x), elements(b, y);
        bool want = false;
        for (int64_t e : x) want |= y.count(e) > 0;
        shared += want;
        if (shares(a, b) != want || shares(b, a) != want) ++wrong;
    }
    // queries and keys of one projection, 16384 tokens of 16 / 8 heads of 128; another one's; a row of it; swapped
    const int64_t t = 32 * 128;
    const Place q = {0, {{2, 8192 * t}, {8192, t}, {16, 128}}, 128}, k = {16 * 128, {{2, 8192 * t}, {8192, t}, {8, 128}}, 128};
    const Place far = {1 << 30, {{2, 8192 * t}, {8192, t}, {16, 128}}, 128};
    const Place in = {24 * 128 - 1, {{2, 8192 * t}, {8192, t}, {8, 128}}, 128};
    if (shares(q, k) || shares(k, q) || shares(q, far) || !shares(q, q) || !shares(k, in) || shares(q, in)) ++wrong;
    // huge strides, whose sums pass 64 bits
    const int64_t most = INT64_MAX / 8;
    const Place huge = {0, {{1 << 30, most}, {1 << 30, most}, {65536, most}}, 512};
    if (!shares(huge, huge) || !shares(huge, q)) ++wrong;
    // strides that have nothing in common: the search ends
    const auto start = std::chrono::steady_clock::now();
    const Place odd = {1, {{1, 0}, {1 << 20, 2 * 1009}, {1 << 10, 2 * 1013}}, 1}, even = {0, {{1, 0}, {1 << 20, 2 * 997}, {1 << 10, 2 * 991}}, 1};
    shares(odd, even);
    const double ms = std::chrono::duration<double, std::milli>(std::chrono::steady_clock::now() - start).count();
    if (ms > 1000) ++wrong;
    std::printf("%d wrong, %d of %d shared, %.2f ms\n", wrong, shared, cases, ms);
    return wrong || shared < cases / 20 || shared > cases * 19 / 20;
}
