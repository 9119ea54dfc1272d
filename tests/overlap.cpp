// Compares overlap.h with the sets of bytes: prints the number of pairs that
// share memory and were not told so; of pairs of one buffer's parts (columns,
// rows, matrices, heads) that share nothing and were told otherwise; and of
// tensors whose places share memory and were not told so, or whose axes do not
// and were told otherwise.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "overlap.h"

using namespace muon::ops;

namespace {

std::vector<int64_t> bytes(const Area& a) {
    std::vector<int64_t> got{int64_t(a.p)};
    for (int i = 0; i < a.axes; ++i) {
        std::vector<int64_t> more;
        for (int64_t v : got)
            for (int64_t k = 0; k < a.n[i]; ++k) more.push_back(v + k * a.stride[i]);
        got.swap(more);
    }
    std::vector<int64_t> all;
    for (int64_t v : got)
        for (int64_t k = 0; k < a.run; ++k) all.push_back(v + k);
    std::sort(all.begin(), all.end());
    return all;
}
bool meet(const Area& a, const Area& b) {
    const auto x = bytes(a), y = bytes(b);
    std::vector<int64_t> both;
    std::set_intersection(x.begin(), x.end(), y.begin(), y.end(), std::back_inserter(both));
    return !both.empty();
}
bool twice(const Area& a) {
    const auto x = bytes(a);
    return std::adjacent_find(x.begin(), x.end()) != x.end();
}
const void* at(int64_t v) { return reinterpret_cast<const void*>(v); }

}  // namespace

int main() {
    std::mt19937 rng(1);
    auto pick = [&](int64_t lo, int64_t hi) { return lo + int64_t(rng() % uint64_t(hi - lo + 1)); };
    int missed = 0, refused = 0, folds = 0;
    for (int i = 0; i < 200000; ++i) {
        auto any = [&] {
            Area a(at(pick(100, 160)), pick(1, 6));
            for (int64_t k = pick(0, 3); k > 0; --k) a.axis(pick(1, 4), pick(0, 24));
            return a;
        };
        const Area a = any(), b = any();
        missed += meet(a, b) && !share(a, b);
        folds += twice(a) && !a.folded();
    }
    for (int i = 0; i < 200000; ++i) {
        // two parts of one buffer of matrices x rows x columns
        const int64_t rows = pick(1, 5), cols = pick(1, 8), all = rows * cols + pick(0, 3), count = pick(1, 4);
        auto part = [&] {
            const int64_t r0 = pick(0, rows - 1), c0 = pick(0, cols - 1), m0 = pick(0, count - 1);
            const int64_t r = pick(1, rows - r0), c = pick(1, cols - c0), m = pick(1, count - m0);
            Area a(at(1000 + m0 * all + r0 * cols + c0), c);
            a.axis(r, cols).axis(m, all);
            return a;
        };
        const Area a = part(), b = part();
        const bool really = meet(a, b);
        missed += really && !share(a, b);
        refused += !really && share(a, b);
        folds += a.folded();
        // different matrices of one buffer, each expert's after another's
        const int64_t k = pick(1, 4), n = pick(1, 4);
        Area g(at(5000), k), d(at(5000 + k * n), n);
        g.axis(n, k).axis(count, 2 * k * n);
        d.axis(k, n).axis(count, 2 * k * n);
        refused += share(g, d);
    }
    std::printf("%d %d %d\n", missed, refused, folds);
    return 0;
}
