// CPU check of how the attention kernel's threads find their block's start
// (tree_schedule.cuh): the kernel's threads in turn, each with a run of the requests,
// against the two lines of work laid out tile by tile.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <tuple>
#include <vector>

#include "tree_schedule.cuh"

using namespace swiglu;

#define CHECK(x)                                                      \
    do {                                                              \
        if (!(x)) {                                                   \
            std::printf("line %d: %s (case %d)\n", __LINE__, #x, it); \
            return 1;                                                 \
        }                                                             \
    } while (0)

int main(int argc, char **argv) {
    const int cases = argc > 1 ? std::atoi(argv[1]) : 100;
    const int threads = 640, sms = 152;
    std::mt19937 rng(11);
    auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
    for (int it = 0; it < cases; ++it) {
        TreeGeom g{};
        const int sizes[] = {1, 2, 5, 60, 639, 640, 641, 700, 1279, 1281, 1500, 4000};
        g.requests = sizes[pick(0, 11)];
        g.kv_heads = pick(1, 8);
        g.group = pick(1, 12);
        g.tpt = 128 / g.group;
        g.recip = tree_recip(g.tpt);
        g.causal = pick(0, 1);
        g.max_rows = 16 * pick(1, 300);
        const int mix = pick(0, 4);   // nothing, single tokens, trees, and runs of each
        std::vector<int> start{0}, ctx;
        for (int r = 0; r < g.requests; ++r) {
            const int kind = mix == 0 ? 1 : mix == 1 ? 2 : mix == 2 ? r / 97 % 3 : pick(0, 2);
            start.push_back(start.back() + (kind == 0 ? 0 : kind == 1 ? 1 : pick(2, 90)));
            ctx.push_back(pick(0, 3) ? pick(0, 400) : pick(0, 5000));
        }
        g.tokens = start.back();
        auto load = [&](int r) { return tree_request(g, start[r], start[r + 1], ctx[r]); };
        CHECK(tree_fits(g));
        // request, head, item and tile of each unit of the lines; the wide units' cost
        std::vector<std::tuple<int, int, int, int>> line[2];
        double cost = 0;
        for (int r = 0; r < g.requests; ++r) {
            const TreeReq q = load(r);
            const bool narrow = q.n * g.group <= kTreeNarrow;
            for (int h = 0; h < g.kv_heads; ++h)
                for (int i = 0; i * 2 * g.tpt < q.n; ++i) {
                    const int sees = g.causal ? tree_min(q.n, (i + 1) * 2 * g.tpt) : q.n;
                    const int len = tree_min(q.ctx + sees, g.max_rows);
                    for (int t = 0; t * kTreeTile < len; ++t) {
                        line[narrow].push_back({r, h, i, t});
                        if (!narrow)
                            cost += q.n - i * 2 * g.tpt <= g.tpt ? kTreeOneCost : kTreePairCost;
                    }
                }
        }
        const int wide = static_cast<int>(line[0].size()), narrow = static_cast<int>(line[1].size());

        // the threads' sums
        const int per = (g.requests + threads - 1) / threads;
        std::vector<TreeUnits> mine(threads);
        std::vector<std::pair<int, int>> run, before;   // requests; units of earlier threads
        TreeUnits all{};
        for (int t = 0; t < threads; ++t) {
            const int r0 = tree_min(t * per, g.requests), r1 = tree_min(r0 + per, g.requests);
            run.push_back({r0, r1});
            for (int r = r0; r < r1; ++r) tree_add_units(g, load(r), &mine[t]);
            before.push_back({all.wide, all.narrow});
            all.wide += mine[t].wide;
            all.narrow += mine[t].narrow;
            all.cost += mine[t].cost;
        }
        CHECK(all.wide == wide && all.narrow == narrow);
        CHECK(all.cost > 0.999 * cost - 1 && all.cost < 1.001 * cost + 1);
        // the lines' blocks, all of them with work
        const int blocks = tree_min(sms, wide + narrow);
        const int nb = tree_min(tree_narrow_blocks(narrow, wide, all.cost, blocks), narrow);
        const int wb = tree_min(blocks - nb, wide);
        CHECK(nb >= 0 && wb >= 0 && nb + wb <= blocks);
        CHECK((nb > 0) == (narrow > 0) && (wb > 0) == (wide > 0));
        for (int form = 0; form < 2; ++form) {
            const int total = form ? narrow : wide, count = form ? nb : wb;
            if (count == 0) continue;
            const TreeCut cut = tree_cut(total, count);
            CHECK(tree_block_begin(cut, 0) == 0 && tree_block_begin(cut, count) == total);
            for (int c = 0; c < count; ++c) {
                const int u0 = tree_block_begin(cut, c);
                int found = 0;
                TreeStart s{};
                for (int t = 0; t < threads; ++t) {
                    const int at = form ? before[t].second : before[t].first;
                    const int own = form ? mine[t].narrow : mine[t].wide;
                    if (u0 < at || u0 >= at + own) continue;
                    CHECK(tree_find(g, load, form == 1, run[t].first, run[t].second, at, u0, &s));
                    ++found;
                }
                CHECK(found == 1);
                CHECK(std::make_tuple(s.r, s.h, s.item, s.tile) == line[form][u0]);
                CHECK(s.q.t0 == start[s.r] && s.q.n == start[s.r + 1] - start[s.r]);
            }
        }
    }
    std::printf("ok\n");
    return 0;
}
