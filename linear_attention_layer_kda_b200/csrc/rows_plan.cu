// rows_plan.cu -- host-only: the order in which a set of row moves can be made in place.
//
// A destination may be written once every move that reads it has been made.  Making the moves in
// that order leaves only cycles, which are disjoint; each is opened by keeping one row's bytes aside.
// Moves that share no row, directly or through others, form separate chains and run in parallel.
#include <algorithm>
#include <numeric>

#include "rows.h"

namespace kda {
namespace rows {

constexpr size_t kCut = 4;

bool plan(const int *dst, const int *src, int n, bool in_place, Plan *out)
{
    out->steps.clear();
    out->first.assign(1, 0);
    std::vector<int> by_dst(n);  // moves by destination row
    std::iota(by_dst.begin(), by_dst.end(), 0);
    std::sort(by_dst.begin(), by_dst.end(), [&](int a, int b) { return dst[a] < dst[b]; });
    for (int i = 1; i < n; ++i)
        if (dst[by_dst[i]] == dst[by_dst[i - 1]]) return false;
    auto writer = [&](int row) {  // the move that writes `row`, or -1
        auto it = std::lower_bound(by_dst.begin(), by_dst.end(), row, [&](int m, int r) { return dst[m] < r; });
        return it != by_dst.end() && dst[*it] == row ? *it : -1;
    };

    // chains: moves joined by a shared source, or (in place) by a row that one reads and another writes
    std::vector<int> up(n);
    std::iota(up.begin(), up.end(), 0);
    auto root = [&](int m) {
        while (up[m] != m) m = up[m] = up[up[m]];
        return m;
    };
    std::vector<int> by_src(n);
    std::iota(by_src.begin(), by_src.end(), 0);
    std::sort(by_src.begin(), by_src.end(), [&](int a, int b) { return src[a] != src[b] ? src[a] < src[b] : a < b; });
    std::vector<int> readers(n, 0);  // of the row that a move writes: moves still to be made that read it
    std::vector<char> done(n, 0);
    for (int i = 0; i < n; ++i) {
        const int m = by_src[i];
        if (src[m] < 0) continue;
        if (i > 0 && src[by_src[i - 1]] == src[m]) up[root(m)] = root(by_src[i - 1]);
        if (!in_place) continue;
        if (src[m] == dst[m]) {
            done[m] = 1;  // nothing to do, and nobody waits for it
            continue;
        }
        const int w = writer(src[m]);
        if (w >= 0 && src[w] != dst[w]) {
            up[root(m)] = root(w);
            ++readers[w];
        }
    }

    std::vector<int> order, ready;  // order: (move, or ~row to save before the cycle's next step)
    order.reserve(2 * n);
    auto make = [&](int m) {
        done[m] = 1;
        if (!in_place || src[m] < 0) return;
        const int w = writer(src[m]);
        if (w >= 0 && !done[w] && --readers[w] == 0) ready.push_back(w);
    };
    std::vector<std::vector<Step>> chain(n);
    for (int i = n - 1; i >= 0; --i)  // by source, so that the copies of one row follow one another
        if (!done[by_src[i]] && readers[by_src[i]] == 0) ready.push_back(by_src[i]);
    while (!ready.empty()) {
        const int m = ready.back();
        ready.pop_back();
        chain[root(m)].push_back({src[m] < 0 ? kZero : src[m], dst[m]});
        make(m);
    }
    for (int m0 = 0; m0 < n; ++m0) {
        if (done[m0]) continue;
        std::vector<Step> &c = chain[root(m0)];
        c.push_back({dst[m0], kSave});
        for (int m = m0; !done[m];) {
            done[m] = 1;
            const int w = writer(src[m]);
            c.push_back({w == m0 ? kSaved : src[m], dst[m]});
            m = w;
        }
    }
    for (int m = 0; m < n; ++m) {
        const std::vector<Step> &c = chain[m];
        if (c.empty()) continue;
        // copies of one row that nobody writes need no order: cut, so that a wide fork is many blocks'
        // work (the row is read once for every kCut copies, from the L2 after the first time)
        bool fork = c[0].src >= 0 && !(in_place && writer(c[0].src) >= 0);
        for (const Step &s : c) fork = fork && s.src == c[0].src && s.dst >= 0;
        for (size_t i = 0; i < c.size(); ++i) {
            out->steps.push_back(c[i]);
            if (i + 1 == c.size() || (fork && (i + 1) % kCut == 0)) out->first.push_back((int)out->steps.size());
        }
    }
    return true;
}

}  // namespace rows
}  // namespace kda
