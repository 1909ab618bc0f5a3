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
    for (int tpt = 1, it = 0; tpt <= 128; ++tpt) {   // the division by 2 * tpt
        TreeGeom g{};
        g.tpt = tpt;
        g.recip = tree_recip(tpt);
        for (int n : {0, 1, 2 * tpt - 1, 2 * tpt, 2 * tpt + 1, 999983, (1 << 24) - 1,
                      (1 << 24) / (2 * tpt) * (2 * tpt) - 1, ((1 << 24) - 1) / (2 * tpt) * (2 * tpt)}) {
            const TreeReq q{0, n, 0};
            CHECK(tree_items(g, q) == (n + 2 * tpt - 1) / (2 * tpt));
        }
    }
    for (int it = 0; it < cases; ++it) {
        TreeGeom g{};
        g.requests = pick(1, it % 5 == 0 ? 300 : 12);
        g.kv_heads = pick(1, 8);
        g.group = it % 7 == 0 ? 128 : pick(1, 12);
        g.tpt = 128 / g.group;
        g.recip = tree_recip(g.tpt);
        g.causal = pick(0, 1);
        g.max_rows = 16 * pick(1, it % 3 ? 40 : 2000);
        std::vector<int> start{0}, ctx;
        for (int r = 0; r < g.requests; ++r) {
            start.push_back(start.back() + (pick(0, 3) ? pick(0, it % 4 ? 9 : 300) : 0));
            ctx.push_back(pick(0, it % 2 ? 300 : 20000));
        }
        g.tokens = start.back() - (it % 11 == 0 ? pick(0, 2) : 0);   // sometimes cut short
        if (g.tokens < 0) g.tokens = 0;
        // one of the two lines, as the kernel's loads see it
        const bool narrow = pick(0, 1) != 0;
        auto load = [&](int r) {
            TreeReq q = tree_request(g, start[r], start[r + 1], ctx[r]);
            if (tree_is_narrow(g, q) != narrow) q.n = 0;
            return q;
        };
        CHECK(tree_fits(g));
        int total = 0;
        std::vector<int> before;
        for (int r = 0; r < g.requests; ++r) {
            before.push_back(total);
            total += g.kv_heads * tree_head_units(g, load(r));
        }
        if (total == 0) continue;
        const int blocks = total < 152 ? pick(1, total) : 152;
        std::map<std::tuple<int, int, int>, int> done;   // tiles done so far of an item
        std::map<std::tuple<int, int, int>, std::pair<int, int>> by;   // first and last block
        std::map<std::tuple<int, int, int>, int> says;   // last block as the first one says
        const TreeCut cut = tree_cut(total, blocks);
        int units = 0;
        for (int c = 0; c < blocks; ++c) {
            const int u0 = tree_block_begin(cut, c), u1 = tree_block_begin(cut, c + 1);
            CHECK(u1 > u0 && u1 <= total);
            CHECK(tree_block_of(cut, u0) == c && tree_block_of(cut, u1 - 1) == c);
            int r = 0;
            while (r + 1 < g.requests && before[r + 1] <= u0) ++r;
            while (load(r).n == 0) --r;
            TreeStart s{};
            s.r = r;
            s.units = u1 - u0;
            tree_locate(g, load(r), u0 - before[r], tree_head_units(g, load(r)), &s);
            TreeWalk w{};
            w.begin(g, s);
            int u = u0;
            while (true) {
                const TreeWalk at = w;   // before the entry
                TreeEntry e{};
                w.entry(g, load, &e);
                if (e.steps == 0) break;
                const int items = e.kind == kTreeDuo ? 2 : 1;
                for (int k = 0; k < items; ++k) {
                    const TreePart &p = e.part[k];
                    const int per = 2 * g.tpt, item = p.place / per;
                    const TreeReq q = load(p.r);
                    const auto key = std::make_tuple(p.r, p.h, item);
                    const int tiles = tree_item_tiles(g, q, item);
                    CHECK(p.r < g.requests && p.h < g.kv_heads && item < tree_items(g, q));
                    CHECK(p.place % per == 0 && p.tok == q.t0 + p.place);
                    CHECK(p.len == tree_item_len(g, q, item) && p.len > 0 && p.len <= g.max_rows);
                    CHECK(done[key] == p.first && p.first < p.end && p.end <= tiles);
                    done[key] = p.end;
                    u += p.end - p.first;
                    const bool begins = p.first == 0, whole = begins && p.end == tiles;
                    CHECK(!!(p.flags & kPartBegins) == begins && !!(p.flags & kPartWhole) == whole);
                    if (begins) by[key].first = c;
                    by[key].second = c;
                    if (begins && !whole) says[key] = tree_block_of(cut, u + (tiles - p.end) - 1);
                    if (p.end < tiles) CHECK(u == u1);
                }
                // tokens of the row tiles
                int tokens = 0;
                for (int k = 0; k < 2; ++k) {
                    const TreePart &p = e.part[k];
                    CHECK(p.ntok >= 1 && p.ntok <= g.tpt && p.place + p.ntok <= load(p.r).n);
                    CHECK(p.tok >= 0 && p.tok + p.ntok <= g.tokens);
                    if (k == 0 || e.kind == kTreePair) tokens += p.ntok;
                }
                if (e.kind != kTreeDuo) CHECK(tokens == at.tokens);
                CHECK((e.kind == kTreePair) == at.pair(g));
                // the steps cover each part's tiles, and the parts the entry's
                std::vector<int> seen[2];
                for (int st = 0; st < e.steps; ++st)
                    for (int k = 0; k < 2; ++k)
                        if (e.part[k].active(st)) {
                            seen[k].push_back(e.part[k].tile(st));
                            CHECK(e.part[k].used());
                            CHECK(e.own_kv(st, k) == (k == 0 || e.kind != kTreePair));
                        }
                for (int k = 0; k < 2; ++k) {
                    CHECK(!e.part[k].active(e.steps));
                    CHECK(e.part[k].used() == !seen[k].empty());
                    units += e.kind == kTreePair && k ? 0 : static_cast<int>(seen[k].size());
                }
                // what the MMA issuer goes by
                for (int k = 0; k < 2; ++k) {
                    const TreePart &p = e.part[k];
                    CHECK(e.tiles[k] == static_cast<int>(seen[k].size()));
                    for (int st = 0; st < e.tiles[k]; ++st) {
                        CHECK((st >= e.edge[k]) == p.edge(p.tile(st)));
                        const int rest = p.len - p.tile(st) * kTreeTile;
                        const int count = rest >= kTreeTile ? 8 : (rest + 15) / 16;
                        CHECK((st + 1 == e.tiles[k] ? e.tail[k] : 8) == count);
                    }
                }
                CHECK(e.part[0].used() && (e.kind == kTreeSplit || e.part[1].used()));
                if (e.kind == kTreeSplit)
                    CHECK(static_cast<int>(seen[0].size() + seen[1].size()) == at.te - at.tb);
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
