// Host-only check of how the expert layer's work is cut (moe_cut.cuh), the code
// the kernel's roles walk, over sizes, SM counts and numbers of chosen experts:
//   every unit of every chosen expert is run exactly once, in a part that fits
//   the plan; parts and experts agree on which parts an expert meets; no expert
//   meets more parts than Cut::most says;
//   the rows of scratch suffice for the routings that take most of them (the
//   experts with the most parts take every token, the others one each) and for
//   random ones, and are at most a quarter and one round of seams more.
// Prints "ok ..." and exits 0, or prints the first violation and exits 1.
#include <algorithm>
#include <cstdio>
#include <cmath>
#include <functional>
#include <random>
#include <vector>

#include "moe_cut.cuh"

using namespace gbr;
using namespace gbr::moe;

namespace {

struct Bad {};
void need(bool ok, const char* what, const MoeArgs& a, int active) {
    if (ok) return;
    std::printf("FAIL %s (T %d, D %d, F %d, E %d, top_k %d, %d chosen)\n", what, a.T, a.D, a.F, a.E, a.top_k, active);
    throw Bad();
}

// Parts met by each of `active` experts, by walking every CTA.
std::vector<int> walk_all(const MoeArgs& a, const CutSizes& s, int active) {
    const Cut c = make_cut(s, active);
    need(c.parts >= 1 && c.total == active * c.per_expert, "sizes of the cut", a, active);
    std::vector<int> next(active, 0), met(active, 0), last(active, -1), in_part(c.parts, 0);
    int part = -1;
    for (int cta = 0; cta < s.sms; ++cta) {
        Segment g;
        for (Walk w(c, cta, s.sms); w.next(c, s.units, g);) {
            need(g.index >= 0 && g.index < active && g.n >= 1 && g.part >= part && g.part < c.parts, "a segment", a,
                 active);
            need(next[g.index] == g.u0, "units in order, once", a, active);
            next[g.index] += g.n;
            part = g.part;
            in_part[g.part] += g.n;
            if (last[g.index] < 0) need(c.first(g.index) == g.part, "an expert's first part", a, active);
            else need(last[g.index] + 1 == g.part, "an expert's parts in a row", a, active);
            last[g.index] = g.part;
            ++met[g.index];
            need(g.n <= s.max_units, "a segment's units fit", a, active);
        }
    }
    for (int x = 0; x < active; ++x) {
        need(next[x] == s.units, "every unit", a, active);
        need(met[x] == c.count(x), "an expert's number of parts", a, active);
        need(met[x] <= c.most(active), "the most parts of an expert", a, active);
    }
    for (int n : in_part) need(n >= 1 && n <= s.max_units, "a part's units", a, active);
    return met;
}

// Rows that a routing takes which gives the x-th chosen expert tokens[x].
int64_t rows_of(const std::vector<int>& met, const std::vector<int>& tokens) {
    int64_t r = 0;
    for (size_t x = 0; x < met.size(); ++x) r += int64_t(met[x]) * tokens[x];
    return r;
}

}  // namespace

int main() try {
    std::mt19937 rng(7);
    long configs = 0;
    auto check = [&](const MoeArgs& a, int sms, bool all) {
        const ExpertPlan p = plan_experts(a, sms, 232448);
        need(p.stages >= 2 && p.max_units >= 1 && p.smem <= 232448 - 9 * 1024, "the plan", a, 0);
        const CutSizes s = {p.units, p.max_units, sms};
        const int64_t rows = most_part_rows(a, s);
        const int pairs = a.T * a.top_k, most = std::min(pairs, a.E);
        int64_t worst = 0;
        for (int active = a.top_k; active <= most; active += all ? 1 : std::max(1, (most - a.top_k) / 7)) {
            const std::vector<int> met = walk_all(a, s, active);
            // One token each, then as many as there are for those with the most parts.
            std::vector<int> by(met), tokens(active, 1), order(active);
            for (int x = 0; x < active; ++x) order[x] = x;
            std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return met[x] > met[y]; });
            int left = pairs - active;
            for (int x : order) {
                const int more = std::min(left, a.T - 1);
                tokens[x] += more;
                left -= more;
            }
            need(left == 0, "a routing of that many experts", a, active);
            worst = std::max(worst, rows_of(met, tokens));
            ++configs;
            // Random: top_k of the chosen for each token (some may get none).
            for (int r = 0; r < 2; ++r) {
                std::vector<int> t(active, 0), pick(active);
                for (int x = 0; x < active; ++x) pick[x] = x;
                for (int i = 0; i < a.T; ++i) {
                    std::shuffle(pick.begin(), pick.end(), rng);
                    for (int k = 0; k < a.top_k; ++k) ++t[pick[k]];
                }
                if (*std::min_element(t.begin(), t.end()) > 0)
                    need(rows_of(met, t) <= rows, "rows of a random routing", a, active);
            }
        }
        need(worst <= rows, "rows of the routing that takes most", a, most);
        if (all) need(rows <= worst + worst / 4 + 2 * pairs, "rows that nothing can use", a, most);
    };
    auto layer = [](int T, int D, int F, int E, int top_k) {
        MoeArgs a = {};
        a.T = T, a.D = D, a.F = F, a.E = E, a.top_k = top_k;
        return a;
    };
    // Many experts of large models, and the decode batches of the tests.
    for (int sms : {152, 148, 7})
        for (const MoeArgs& a : {layer(64, 4096, 14336, 256, 8), layer(64, 7168, 2048, 256, 8),
                                 layer(1, 4096, 14336, 8, 2), layer(64, 4096, 14336, 8, 2), layer(19, 2048, 1000, 64, 6),
                                 layer(64, 256, 14336, 64, 8), layer(40, 512, 72, 250, 8), layer(64, 128, 64, 256, 8),
                                 layer(64, 8, 8, 1, 1), layer(2, 64, 65536, 3, 2), layer(33, 1672, 320, 64, 1)})
            check(a, sms, true);
    std::uniform_real_distribution<double> unit(0.0, 1.0);
    auto spread = [&](int lo, int hi) {
        return std::max(lo, std::min(hi, int(lo * std::pow(double(hi) / lo, unit(rng)) + 0.5)));
    };
    for (int i = 0; i < 400; ++i) {
        const int E = spread(1, 256);
        check(layer(spread(1, 64), 8 * spread(1, 900), 8 * spread(1, 4000), E, 1 + int(rng() % std::min(E, 8))),
              i % 3 ? 152 : spread(1, 200), false);
    }
    std::printf("ok %ld cuts\n", configs);
    return 0;
} catch (const Bad&) {
    return 1;
}
