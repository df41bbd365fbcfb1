// rows_plan.cu -- host-only: the order in which a set of row moves can be made in place.
//
// A destination may be written once every move that reads it has been made.  Making the moves in
// that order leaves only cycles, which are disjoint; each is opened by keeping one row's bytes aside.
// Moves that share no row, directly or through others, form separate chains and run in parallel.
#include <algorithm>
#include <numeric>
#include <utility>

#include "rows.h"

namespace kda {
namespace rows {

constexpr int kCut = 4;

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

    std::vector<int> ready;
    std::vector<std::pair<int, Step>> all;  // steps with their chains, each chain's in order
    all.reserve(2 * (size_t)n);
    ready.reserve(n);
    auto make = [&](int m) {
        done[m] = 1;
        if (!in_place || src[m] < 0) return;
        const int w = writer(src[m]);
        if (w >= 0 && !done[w] && --readers[w] == 0) ready.push_back(w);
    };
    for (int i = n - 1; i >= 0; --i)  // by source, so that the copies of one row follow one another
        if (!done[by_src[i]] && readers[by_src[i]] == 0) ready.push_back(by_src[i]);
    while (!ready.empty()) {
        const int m = ready.back();
        ready.pop_back();
        all.push_back({root(m), {src[m] < 0 ? kZero : src[m], dst[m]}});
        make(m);
    }
    for (int m0 = 0; m0 < n; ++m0) {
        if (done[m0]) continue;
        const int c = root(m0);
        all.push_back({c, {dst[m0], kSave}});
        for (int m = m0; !done[m];) {
            done[m] = 1;
            const int w = writer(src[m]);
            all.push_back({c, {w == m0 ? kSaved : src[m], dst[m]}});
            m = w;
        }
    }
    std::vector<int> at(n + 1, 0);  // the chains' places, by counting
    for (const auto &x : all) ++at[x.first + 1];
    for (int m = 0; m < n; ++m) at[m + 1] += at[m];
    out->steps.resize(all.size());
    std::vector<int> next(at.begin(), at.end() - 1);
    for (const auto &x : all) out->steps[next[x.first]++] = x.second;
    for (int m = 0; m < n; ++m) {
        const int i0 = at[m], i1 = at[m + 1];
        if (i0 == i1) continue;
        // copies of one row that nobody writes need no order: cut, so that a wide fork is many blocks'
        // work (the row is read once for every kCut copies, from the L2 after the first time)
        const int row = out->steps[i0].src;
        bool fork = row >= 0 && !(in_place && writer(row) >= 0);
        for (int i = i0; i < i1; ++i) fork = fork && out->steps[i].src == row && out->steps[i].dst >= 0;
        for (int i = i0 + 1; i <= i1; ++i)
            if (i == i1 || (fork && (i - i0) % kCut == 0)) out->first.push_back(i);
    }
    return true;
}

}  // namespace rows
}  // namespace kda
