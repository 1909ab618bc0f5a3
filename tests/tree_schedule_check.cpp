// CPU check of the tree-attention work split (tree_schedule.cuh): over random
// batches, every tile of every item is done exactly once, in order, and the
// blocks that share an item are the ones that the partial sums are read from.
#include <cstdio>
#include <cstdlib>
#include <map>
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
    const int cases = argc > 1 ? std::atoi(argv[1]) : 400;
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
    for (int it = 0; it < cases; ++it) {
        TreeGeom g{};
        g.requests = pick(1, it % 5 == 0 ? 300 : 12);
        g.kv_heads = pick(1, 8);
        g.group = it % 7 == 0 ? 128 : pick(1, 12);
        g.tpt = 128 / g.group;
        g.causal = pick(0, 1);
        g.max_rows = 16 * pick(1, it % 3 ? 40 : 2000);
        std::vector<int> start{0}, ctx;
        for (int r = 0; r < g.requests; ++r) {
            start.push_back(start.back() + (pick(0, 3) ? pick(0, it % 4 ? 9 : 300) : 0));
            ctx.push_back(pick(0, it % 2 ? 300 : 20000));
        }
        g.tokens = start.back() - (it % 11 == 0 ? pick(0, 2) : 0);   // sometimes cut short
        if (g.tokens < 0) g.tokens = 0;
        auto load = [&](int r) { return tree_request(g, start[r], start[r + 1], ctx[r]); };
        long long total = 0;
        std::vector<long long> before;
        for (int r = 0; r < g.requests; ++r) {
            before.push_back(total);
            total += g.kv_heads * tree_head_units(g, load(r));
        }
        if (total == 0) continue;
        const int blocks = static_cast<int>(total < 152 ? pick(1, static_cast<int>(total)) : 152);
        std::map<std::tuple<int, int, int>, int> done;   // tiles done so far of an item
        std::map<std::tuple<int, int, int>, std::pair<int, int>> by;   // first and last block
        std::map<std::tuple<int, int, int>, int> says;   // last block as the first one says
        long long units = 0;
        for (int c = 0; c < blocks; ++c) {
            const long long u0 = tree_block_begin(c, total, blocks);
            const long long u1 = tree_block_begin(c + 1, total, blocks);
            CHECK(u1 > u0);
            CHECK(tree_block_of(u0, total, blocks) == c && tree_block_of(u1 - 1, total, blocks) == c);
            int r = 0;
            while (r + 1 < g.requests && before[r + 1] <= u0) ++r;
            while (load(r).n == 0) --r;
            TreeStart s{};
            s.r = r;
            s.units = u1 - u0;
            tree_locate(g, load(r), u0 - before[r], &s);
            TreeWalk w{};
            long long u = u0;
            int seq = 0;
            for (w.begin(g, s, load); w.valid(); ++seq) {
                CHECK(w.seq == seq && w.r < g.requests && w.h < g.kv_heads);
                CHECK(w.q.n > 0 && w.tokens > 0 && w.tokens <= 2 * g.tpt && w.len > 0);
                CHECK(w.item_token0(g) + w.tokens <= w.q.n && w.q.t0 + w.q.n <= g.tokens);
                CHECK(w.tb < w.te && w.te <= w.tiles && w.len <= g.max_rows);
                const auto key = std::make_tuple(w.r, w.h, w.item);
                CHECK(done[key] == w.tb);
                done[key] = w.te;
                u += w.te - w.tb;
                if (w.tb == 0) by[key].first = c;
                by[key].second = c;
                if (w.te < w.tiles && w.tb == 0)
                    says[key] = tree_block_of(u + (w.tiles - w.te) - 1, total, blocks);
                if (w.te < w.tiles) CHECK(u == u1);
                // the steps of both groups cover the item's tiles
                int a = 0, b = 0, steps = 0, last = 0;
                const TreeWalk item = w;
                bool inside = true;
                while (inside) {
                    for (int grp = 0; grp < 2; ++grp) {
                        if (!w.active(grp)) continue;
                        CHECK(w.uses(grp));
                        (grp ? b : a) += 1;
                        CHECK(w.tile(grp) >= item.tb && w.tile(grp) < item.te);
                        last += w.last_of(grp);
                        units += (item.pair ? grp == 0 : true);
                    }
                    ++steps;
                    inside = w.step + 1 < w.steps;
                    w.next_step(g, load);
                }
                CHECK(steps == item.steps);
                CHECK(item.pair ? (a == b && a == item.te - item.tb) : a + b == item.te - item.tb);
                CHECK(last == 1 + (item.uses(1) ? 1 : 0));
            }
            CHECK(u == u1);
        }
        CHECK(units == total);
        for (int r = 0; r < g.requests; ++r)
            for (int h = 0; h < g.kv_heads; ++h)
                for (int i = 0; i < tree_items(g, load(r)); ++i) {
                    const auto key = std::make_tuple(r, h, i);
                    CHECK(done[key] == tree_item_tiles(g, load(r), i));
                    if (by[key].first != by[key].second) CHECK(says[key] == by[key].second);
                    else CHECK(says.find(key) == says.end());
                }
    }
    std::printf("ok\n");
    return 0;
}
