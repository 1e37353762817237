// Random batches: every (sequence, tile, group that sees the tile) is in one share, each tile's sums are written once or left in
// the slots that the joining kernel reads, and the shares are even. With an argument: chunks that may be longer than their keys.
#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "key_weight_plan.cuh"

using namespace kvr;

struct Shapes {
    const std::vector<KwShape>* v;
    KwShape operator()(int n) const { return (*v)[n]; }
};

static int fail(const char* what, int batch) {
    printf("%s (batch %d)\n", what, batch);
    return 1;
}

int main(int argc, char**) {
    const bool chunks = argc > 1;
    std::mt19937 r(1);
    double worst = 0;
    for (int batch = 0; batch < (chunks ? 150 : 3000); ++batch) {
        const int N = 1 + r() % 12, H = 1 + r() % 130, shift = 5 + r() % 4, rows = 1 << shift, pairs = 1 + r() % 76;
        const bool causal = r() % 3;
        std::vector<KwShape> v;
        for (int n = 0; n < N; ++n) {
            if (chunks) {
                const int L = 1 + r() % 6000, K = r() % (r() % 2 ? 40 : (r() % 2 ? 3000 : 9000));
                v.push_back({L, K, H, shift, causal});
                continue;
            }
            const int L = r() % 4 ? 1 + r() % (r() % 2 ? 3 : 200) : 0, K = r() % 7 == 0 ? r() % 5 : r() % (r() % 2 ? 600 : 20000);
            v.push_back({L, K, H, shift, causal});
        }
        int64_t total = 0;
        std::vector<int64_t> base;
        for (auto& s : v) {
            base.push_back(total);
            total += s.cost();
        }
        const int active = kw_active(total, pairs);
        std::vector<KwPos> start;
        for (int p = 0; p <= pairs; ++p) {
            const int64_t u = kw_share(total, p, active);
            KwPos at = {N, 0, 0, 0};
            for (int n = 0; n < N; ++n)
                if (u >= base[n] && u < base[n] + v[n].cost()) at = v[n].locate(n, u - base[n]);
            start.push_back(at);
        }
        std::set<std::tuple<int, int, int>> seen;
        std::map<std::pair<int, int>, std::set<int>> left, read;
        std::map<std::pair<int, int>, int> written;
        double most = 0;
        for (int p = 0; p < pairs; ++p) {
            KwWalk<Shapes> w(Shapes{&v}, start[p], start[p + 1], N);
            double load = 0;
            while (w.next())
                for (int kt = w.kt0; kt < w.kt1; ++kt) {
                    if (w.whole) written[{w.n, kt}]++;
                    else if (!left[{w.n, kt}].insert(p * 2 + (kw_same_tile(start[p], {w.n, kt, 0, 0}) ? 0 : 1)).second) return fail("a slot twice", batch);
                    load += 1 + w.gb - w.ga;
                    for (int g = w.ga; g < w.gb; ++g)
                        if (!seen.insert({w.n, kt, g}).second) return fail("a group twice", batch);
                }
            most = std::max(most, load);
        }
        for (int n = 0; n < N; ++n) {
            const KwShape& s = v[n];
            for (int kt = 0; s.L > 0 && kt < s.tiles(); ++kt) {
                const int g0 = s.first_group(kt);
                if (g0 >= s.groups()) return fail("a tile without a group", batch);
                auto sees = [&](int g) {   // keys of the group's last row
                    const int t = int(std::min<int64_t>(s.L - 1, (int64_t(g) * rows + rows - 1) / H));
                    return causal ? s.K - s.L + t + 1 : s.K;
                };
                if (sees(g0) <= kt * KW_KEYS || (g0 > 0 && sees(g0 - 1) > kt * KW_KEYS)) return fail("not the first group", batch);
                for (int g = g0; g < s.groups(); ++g)
                    if (!seen.count({n, kt, g})) return fail("a group left out", batch);
                if (written.count({n, kt}) + left.count({n, kt}) != 1 || (written.count({n, kt}) && written[{n, kt}] != 1))
                    return fail("a tile not written once", batch);
            }
        }
        for (int b = 1; b < active; ++b) {   // as the joining kernel goes over the begins
            const KwPos x = start[b], before = start[b - 1];
            if (x.n >= N || !x.cut || (kw_same_tile(before, x) && before.cut)) continue;
            std::set<int>& slots = read[{x.n, x.kt}];
            if (!kw_same(before, x)) slots.insert((b - 1) * 2 + (kw_same_tile(before, x) ? 0 : 1));
            for (int q = b; q < active && kw_same_tile(start[q], x); ++q)
                if (!(q + 1 < active && kw_same(start[q], start[q + 1]))) slots.insert(q * 2);
        }
        if (read != left) return fail("the join reads other slots than were written", batch);
        if (total > 40 * active) worst = std::max(worst, most / (double(total) / active));
    }
    printf("%.3f\n", worst);
    return worst > 1.15;
}
