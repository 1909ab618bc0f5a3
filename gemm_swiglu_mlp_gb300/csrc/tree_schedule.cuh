// How a tree-attention call's work is cut: plain arithmetic shared by every
// role of the kernel (and checked on the CPU).
//
// The 128-row side of the tensor cores' tiles holds (token, head) pairs of one
// request and one kv head: `tpt` = 128 / group tokens of `group` query heads,
// so that all heads that share a kv head share its K and V tiles. An ITEM is
// up to two such row tiles (2 * tpt tokens) of one (request, kv head), against
// the positions its tokens can see, in TILES of 128 positions. Items are
// numbered request by request, then kv head, then token block, and all tiles
// of all items form one line of `total` units; block c of `blocks` takes the
// units [total * c / blocks, total * (c + 1) / blocks), whatever items they
// belong to. So ragged lengths balance to one tile, and an item that crosses
// a block boundary is summed from the blocks' partial results.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SWIGLU_HD __host__ __device__ __forceinline__
#else
#define SWIGLU_HD inline
#endif

namespace swiglu {

constexpr int kTreeTile = 128;   // positions a tile, and rows of a row tile

struct TreeGeom {
    int requests, tokens, kv_heads;
    int group;      // query heads per kv head, 1..128
    int tpt;        // tokens per row tile, 128 / group
    int causal;     // 1: no mask, a token sees the new tokens up to itself
    int max_rows;   // positions a block-table row can hold
};

struct TreeReq {
    int t0;    // first token
    int n;     // new tokens
    int ctx;   // cached tokens
};

SWIGLU_HD int tree_min(int a, int b) { return a < b ? a : b; }
SWIGLU_HD int tree_max(int a, int b) { return a > b ? a : b; }

// A request from its entries in query_start and ctx_lens, kept inside the
// tensors whatever they hold.
SWIGLU_HD TreeReq tree_request(const TreeGeom &g, int start, int end, int ctx) {
    TreeReq q;
    q.t0 = tree_min(tree_max(start, 0), g.tokens);
    q.n = tree_min(tree_max(end, q.t0), g.tokens) - q.t0;
    q.ctx = tree_min(tree_max(ctx, 0), g.max_rows);
    return q;
}

SWIGLU_HD int tree_items(const TreeGeom &g, const TreeReq &q) {
    return (q.n + 2 * g.tpt - 1) / (2 * g.tpt);
}

// Tokens of item `item` of a request.
SWIGLU_HD int tree_item_tokens(const TreeGeom &g, const TreeReq &q, int item) {
    return tree_min(2 * g.tpt, q.n - item * 2 * g.tpt);
}

// Positions that some token of the item may see (>= 1).
SWIGLU_HD int tree_item_len(const TreeGeom &g, const TreeReq &q, int item) {
    const int upto = g.causal ? tree_min(q.n, (item + 1) * 2 * g.tpt) : q.n;
    const long long len = static_cast<long long>(q.ctx) + upto;
    return len < g.max_rows ? static_cast<int>(len) : g.max_rows;
}

SWIGLU_HD int tree_item_tiles(const TreeGeom &g, const TreeReq &q, int item) {
    return (tree_item_len(g, q, item) + kTreeTile - 1) / kTreeTile;
}

// Units of one kv head of a request.
SWIGLU_HD long long tree_head_units(const TreeGeom &g, const TreeReq &q) {
    const int items = tree_items(g, q);
    if (!g.causal) return items ? static_cast<long long>(items) * tree_item_tiles(g, q, 0) : 0;
    long long u = 0;
    for (int i = 0; i < items; ++i) u += tree_item_tiles(g, q, i);
    return u;
}

// Where a block begins: `tile` of item (r, h, item), `units` tiles to do.
struct TreeStart {
    int r, h, item, tile;
    long long units;
};

// The place `rem` units into request r.
SWIGLU_HD void tree_locate(const TreeGeom &g, const TreeReq &q, long long rem, TreeStart *s) {
    const long long per_head = tree_head_units(g, q);
    s->h = static_cast<int>(rem / per_head);
    rem -= s->h * per_head;
    int item = 0;
    while (true) {
        const int tiles = tree_item_tiles(g, q, item);
        if (rem < tiles) break;
        rem -= tiles;
        ++item;
    }
    s->item = item;
    s->tile = static_cast<int>(rem);
}

// Block that does unit u.
SWIGLU_HD int tree_block_of(long long u, long long total, int blocks) {
    return static_cast<int>(((u + 1) * blocks + total - 1) / total) - 1;
}
SWIGLU_HD long long tree_block_begin(int c, long long total, int blocks) {
    return total * c / blocks;
}

// The items of one block in order, and the steps of each. An item of one row
// tile (`pair` false) is worked on by both softmax groups, group s taking the
// tiles tb + s, tb + s + 2, ..: two tiles a step. An item of two row tiles
// gives each group one of them: both see every tile, one a step.
struct TreeWalk {
    TreeReq q;
    int r, h, item;
    int tokens;        // of the item
    int len;           // positions of the item
    int tiles;         // of the item
    int tb, te;        // this block's tiles of it
    long long left;    // units left, this item's included
    int seq;           // items before this one in this block
    int step, steps;
    bool pair;

    SWIGLU_HD bool valid() const { return left > 0; }
    SWIGLU_HD int item_token0(const TreeGeom &g) const { return item * 2 * g.tpt; }
    SWIGLU_HD bool active(int s) const { return pair || tb + 2 * step + s < te; }
    SWIGLU_HD int tile(int s) const { return pair ? tb + step : tb + 2 * step + s; }
    SWIGLU_HD bool last_of(int s) const { return pair ? step + 1 == steps : tb + 2 * step + s + 2 >= te; }
    SWIGLU_HD bool uses(int s) const { return pair || s == 0 || te - tb > 1; }
    // a tile with positions that need a look: new tokens, or past the end
    SWIGLU_HD bool edge(int t) const { return (t + 1) * kTreeTile > q.ctx || (t + 1) * kTreeTile > len; }

    SWIGLU_HD void set_item(const TreeGeom &g, int from) {
        tokens = tree_item_tokens(g, q, item);
        len = tree_item_len(g, q, item);
        tiles = (len + kTreeTile - 1) / kTreeTile;
        tb = from;
        te = static_cast<int>(left < tiles - from ? from + left : tiles);
        pair = tokens > g.tpt;
        step = 0;
        steps = pair ? te - tb : (te - tb + 1) / 2;
    }
    template <typename Load>   // Load(r) -> TreeReq
    SWIGLU_HD void begin(const TreeGeom &g, const TreeStart &s, Load load) {
        r = s.r;
        h = s.h;
        item = s.item;
        left = s.units;
        seq = 0;
        if (left <= 0) return;
        q = load(r);
        set_item(g, s.tile);
    }
    // The next item, or left = 0.
    template <typename Load>
    SWIGLU_HD void next_item(const TreeGeom &g, Load load) {
        left -= te - tb;
        ++seq;
        if (left <= 0) return;
        if (++item == tree_items(g, q)) {
            item = 0;
            if (++h == g.kv_heads) {
                h = 0;
                do q = load(++r);
                while (q.n == 0);
            }
        }
        set_item(g, 0);
    }
    template <typename Load>
    SWIGLU_HD void next_step(const TreeGeom &g, Load load) {
        if (++step == steps) next_item(g, load);
    }
};

}  // namespace swiglu
