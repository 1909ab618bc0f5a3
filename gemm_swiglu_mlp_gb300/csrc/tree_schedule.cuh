// How a tree-attention call's work is cut: plain arithmetic shared by every
// role of the kernel (and checked on the CPU).
//
// The 128-row side of the tensor cores' tiles holds (token, head) pairs of one
// request and one kv head: `tpt` = 128 / group tokens of `group` query heads,
// so that all heads that share a kv head share its K and V tiles. An ITEM is
// up to two such row tiles (2 * tpt tokens) of one (request, kv head), against
// the positions its tokens can see, in TILES of 128 positions. Items are
// numbered request by request, then kv head, then token block, and all tiles
// of all items of one form (tree_is_narrow) are one line of `total` units; each
// of the form's blocks takes as many of them, to one unit, whatever items they
// belong to (tree_cut). So ragged lengths balance to one tile, and an item that
// crosses a block boundary is summed from the blocks' partial results.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SWIGLU_HD __host__ __device__ __forceinline__
#define SWIGLU_HD_CALL __host__ __device__ __noinline__
#else
#define SWIGLU_HD inline
#define SWIGLU_HD_CALL inline
#endif

namespace swiglu {

constexpr int kTreeTile = 128;   // positions a tile, and rows of a row tile

struct TreeGeom {
    int requests, tokens, kv_heads;
    int group;        // query heads per kv head, 1..128
    int tpt;          // tokens per row tile, 128 / group
    uint32_t recip;   // ceil(2^32 / (2 * tpt)): n / (2 * tpt) for n < 2^24
    int causal;       // 1: no mask, a token sees the new tokens up to itself
    int max_rows;     // positions a block-table row can hold
};
// Limits that keep every unit count in 32 bits (checked on the host):
// tokens below 2^24, and this bound on the units of one call.
SWIGLU_HD uint32_t tree_recip(int tpt) {
    return static_cast<uint32_t>(((1ull << 32) + 2 * tpt - 1) / (2 * tpt));
}
inline bool tree_fits(const TreeGeom &g) {
    const double items = static_cast<double>(g.tokens) / (2 * g.tpt) + g.requests;
    return g.tokens < (1 << 24) &&
           items * g.kv_heads * (g.max_rows / kTreeTile + 1.0) < 2147483648.0;
}

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

// Requests of up to this many rows a kv head are worked on in the kernel's
// narrow form, the others in its wide form, by blocks of their own: each form
// has a line of work with only its requests on it.
// Measured (us, narrow / wide, 2 kv heads of 7 heads of 128): 300 requests of one
// token 17 / 20 at contexts of 100 and 116 / 125 at 2000, of four tokens (28 rows)
// 23 / 20, 48 / 47 at 500 and 125 / 129; 10 requests of four tokens 12.0 / 12.5 and
// 18.4 / 18.6.
constexpr int kTreeNarrow = 32;
SWIGLU_HD bool tree_is_narrow(const TreeGeom &g, const TreeReq &q) {
    return q.n <= kTreeNarrow && q.n * g.group <= kTreeNarrow;
}

SWIGLU_HD int tree_items(const TreeGeom &g, const TreeReq &q) {
    return static_cast<int>(
        (static_cast<uint64_t>(static_cast<uint32_t>(q.n + 2 * g.tpt - 1)) * g.recip) >> 32);
}

// Positions that some token of item `item` may see (>= 1).
SWIGLU_HD int tree_item_len(const TreeGeom &g, const TreeReq &q, int item) {
    return tree_min(q.ctx + (g.causal ? tree_min(q.n, (item + 1) * 2 * g.tpt) : q.n), g.max_rows);
}

SWIGLU_HD int tree_item_tiles(const TreeGeom &g, const TreeReq &q, int item) {
    return (tree_item_len(g, q, item) + kTreeTile - 1) / kTreeTile;
}

// Units of one kv head of a request.
SWIGLU_HD_CALL int tree_head_units(const TreeGeom &g, const TreeReq &q) {
    const int items = tree_items(g, q);
    if (!g.causal) return items * tree_item_tiles(g, q, 0);
    int u = 0;
    for (int i = 0; i < items; ++i) u += tree_item_tiles(g, q, i);
    return u;
}

// What a kv head's `units` cost in the wide form, in quarters of a narrow tile
// (whose time is its bytes'): a tile of an item of one row tile kTreeOneCost,
// of two kTreePairCost, as their products and weights take more than the
// bytes. Measured with half of 64 requests at one token and the others at n, 7
// heads a kv head, contexts of 4000 (us): all at 4 / 5 / 6 / 8, n = 6
// 121 / 118 / 133 / 144, n = 36 (one item of two row tiles) 177 / 163 / 157 / 165.
constexpr int kTreeOneCost = 5, kTreePairCost = 7;
SWIGLU_HD float tree_wide_cost(const TreeGeom &g, const TreeReq &q, int units) {
    const int items = tree_items(g, q);
    float cost = static_cast<float>(units) * kTreePairCost;
    if (q.n - (items - 1) * 2 * g.tpt <= g.tpt)   // the last item has one row tile
        cost -= static_cast<float>(tree_item_tiles(g, q, items - 1)) * (kTreePairCost - kTreeOneCost);
    return cost;
}
// Both lines' units of some requests, and what the wide ones cost.
struct TreeUnits {
    int wide, narrow;
    float cost;
};
SWIGLU_HD void tree_add_units(const TreeGeom &g, const TreeReq &q, TreeUnits *sum) {
    const int per_head = tree_head_units(g, q);
    if (tree_is_narrow(g, q)) {
        sum->narrow += g.kv_heads * per_head;
    } else {
        sum->wide += g.kv_heads * per_head;
        if (per_head) sum->cost += g.kv_heads * tree_wide_cost(g, q, per_head);
    }
}

// How many of `blocks` (>= 2 where both lines have work) blocks take the narrow
// form's line: as its share of the cost.
SWIGLU_HD int tree_narrow_blocks(int narrow, int wide, float wide_cost, int blocks) {
    if (narrow == 0) return 0;
    if (wide == 0) return blocks;
    const float a = 4.f * static_cast<float>(narrow);
    const int n = static_cast<int>(blocks * (a / (a + wide_cost)) + 0.5f);
    return tree_max(1, tree_min(n, blocks - 1));
}

// A line of `total` units cut for `blocks` <= total blocks: the first `more`
// of them take one unit above `each`.
struct TreeCut {
    int each, more;
};
SWIGLU_HD TreeCut tree_cut(int total, int blocks) {
    TreeCut c;
    c.each = static_cast<int>(static_cast<uint32_t>(total) / static_cast<uint32_t>(blocks));
    c.more = total - c.each * blocks;
    return c;
}
SWIGLU_HD int tree_block_begin(const TreeCut &c, int block) {
    return c.each * block + tree_min(block, c.more);
}
// Block that does unit u.
SWIGLU_HD int tree_block_of(const TreeCut &c, int u) {
    const int fat = (c.each + 1) * c.more;
    return u < fat ? u / (c.each + 1) : c.more + (u - fat) / c.each;
}

// Where a block begins: `tile` of item (r, h, item), `units` tiles to do.
struct TreeStart {
    TreeReq q;
    int r, h, item, tile, units;
};

// The place `rem` units into request r.
SWIGLU_HD void tree_locate(const TreeGeom &g, const TreeReq &q, int rem, int per_head, TreeStart *s) {
    s->q = q;
    s->h = static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(per_head));
    rem -= s->h * per_head;
    int item = 0;
    while (true) {
        const int tiles = tree_item_tiles(g, q, item);
        if (rem < tiles) break;
        rem -= tiles;
        ++item;
    }
    s->item = item;
    s->tile = rem;
}

// Unit u0 of one form's line, if it falls to one of the requests r0 .. r1 - 1, whose
// first unit on that line is `at`: sets where it is, and says so.
template <typename Load>   // Load(r) -> TreeReq
SWIGLU_HD bool tree_find(const TreeGeom &g, Load load, bool narrow, int r0, int r1, int at, int u0,
                         TreeStart *s) {
#ifdef __CUDACC__
#pragma unroll 1
#endif
    for (int r = r0; r < r1; ++r) {
        const TreeReq q = load(r);
        if (tree_is_narrow(g, q) != narrow) continue;
        const int per_head = tree_head_units(g, q);
        if (u0 < at + g.kv_heads * per_head) {
            s->r = r;
            tree_locate(g, q, u0 - at, per_head, s);
            return true;
        }
        at += g.kv_heads * per_head;
    }
    return false;
}

// TreePart::flags
enum : int {
    kPartWhole = 1,    // this block does the whole item
    kPartBegins = 2,   // the item begins in this block
    kPartSecond = 4,   // the item's second row tile
};

// One softmax group's part in an entry (below): a row tile and the tiles
// first, first + stride, .. (< end) of its item.
struct TreePart {
    int first, stride, end;
    int edge_from;    // min(ctx, len): tiles that reach past it need a look (new
                      // tokens, or past the end)
    int r, h;         // request, kv head
    int tok;          // first token of the row tile (row of q)
    int place;        // its place among the request's new tokens
    int ntok;         // tokens of the row tile
    int ctx, len;     // of the request; positions of the item
    int flags;

    SWIGLU_HD bool used() const { return first < end; }
    SWIGLU_HD bool active(int step) const { return first + step * stride < end; }
    SWIGLU_HD int tile(int step) const { return first + step * stride; }
    SWIGLU_HD bool edge(int t) const { return (t + 1) * kTreeTile > edge_from; }
};

// What both groups do next. kTreeSplit: an item of one row tile, the groups
// take its even and odd tiles and merge their results. kTreePair: an item of
// two row tiles, one a group, over the same tiles. kTreeDuo: two items of one
// row tile each, one a group; while one group's softmax or result runs, the
// tensor cores work for the other.
enum : int { kTreeSplit = 0, kTreePair = 1, kTreeDuo = 2 };
// Whether two items with this many tiles make a Duo. It saves both results'
// merging and the groups never wait for each other, but the group with fewer
// tiles has nothing to do at the end: so where that is no more than a quarter
// of the longer one, or a few tiles. Measured (us, with / without): 304 requests
// of 9 tokens, 7 heads a kv head, contexts of 100 21 / 29, of 900 69 / 73, of
// 6000 315 / 340; 608 requests of one token, contexts of 100 25 / 33, of 1500
// 158 / 158.
constexpr int kTreeDuoTiles = 4;
SWIGLU_HD bool tree_duo(int a, int b) {
    const int more = tree_max(a, b);
    return more <= kTreeDuoTiles || 4 * (more - tree_min(a, b)) <= more;
}
struct TreeEntry {
    TreePart part[2];
    int kind;
    int steps;        // 0: nothing left
    // for the MMA issuer, each part: its tiles, the first of them that needs a
    // look, and how many 16s of positions the last one has
    int tiles[2], edge[2], tail[2];
    SWIGLU_HD bool two_q() const { return kind != kTreeSplit; }    // a Q tile a group
    // group s has a K and a V tile of its own in a step
    SWIGLU_HD bool own_kv(int step, int s) const {
        return part[s].active(step) && (s == 0 || kind != kTreePair);
    }
};

// The items of one block in order.
struct TreeWalk {
    TreeReq q;
    int r, h, item, items;
    int tokens, len, tiles;   // of the item
    int tb, te;               // this block's tiles of it
    int left;                 // units left, this item's included

    SWIGLU_HD bool pair(const TreeGeom &g) const { return tokens > g.tpt; }

    SWIGLU_HD void set_item(const TreeGeom &g, int from) {
        tokens = tree_min(2 * g.tpt, q.n - item * 2 * g.tpt);
        len = tree_item_len(g, q, item);
        tiles = (len + kTreeTile - 1) / kTreeTile;
        tb = from;
        te = tree_min(tiles, from + left);
    }
    SWIGLU_HD void begin(const TreeGeom &g, const TreeStart &s) {
        q = s.q;
        r = s.r;
        h = s.h;
        item = s.item;
        left = s.units;
        items = tree_items(g, q);
        set_item(g, s.tile);
    }
    // The next item, or left = 0.
    template <typename Load>   // Load(r) -> TreeReq, n = 0: not on this line
    SWIGLU_HD void next(const TreeGeom &g, Load load) {
        left -= te - tb;
        if (left <= 0) return;
        if (++item == items) {
            item = 0;
            if (++h == g.kv_heads) {
                h = 0;
                do {
                    if (++r >= g.requests) {   // (never on a line that was counted right)
                        left = 0;
                        return;
                    }
                    q = load(r);
                } while (q.n == 0);
                items = tree_items(g, q);
            }
        }
        set_item(g, 0);
    }
    SWIGLU_HD TreePart part(const TreeGeom &g) const {
        TreePart p;
        p.r = r;
        p.h = h;
        p.place = item * 2 * g.tpt;
        p.tok = q.t0 + p.place;
        p.ntok = tree_min(g.tpt, tokens);
        p.ctx = q.ctx;
        p.len = len;
        p.edge_from = tree_min(q.ctx, len);
        p.first = tb;
        p.stride = 1;
        p.end = te;
        p.flags = (tb == 0 && te == tiles ? kPartWhole : 0) | (tb == 0 ? kPartBegins : 0);
        return p;
    }
    // The next entry; moves on past its items. steps = 0 at the end.
    template <typename Load>
    SWIGLU_HD void entry(const TreeGeom &g, Load load, TreeEntry *e) {
        e->kind = kTreeSplit;
        e->steps = 0;
        if (left <= 0) return;
        const int mine = te - tb;
        const bool two = pair(g);
        TreePart p = part(g);
        e->part[0] = p;
        if (two) {
            e->kind = kTreePair;
            e->steps = mine;
            p.place += g.tpt;
            p.tok += g.tpt;
            p.ntok = tokens - g.tpt;
            p.flags |= kPartSecond;
        }
        next(g, load);
        if (!two) {
            if (left > 0 && !pair(g) && tree_duo(mine, te - tb)) {
                e->kind = kTreeDuo;
                e->steps = tree_max(mine, te - tb);
                p = part(g);
                next(g, load);
            } else {
                e->steps = (mine + 1) / 2;
                e->part[0].stride = p.stride = 2;
                p.first += 1;
            }
        }
        e->part[1] = p;
        for (int k = 0; k < 2; ++k) {
            const TreePart &x = e->part[k];
            // (strides are 1 or 2)
            const int n = tree_max((x.end - x.first + x.stride - 1) >> (x.stride - 1), 0);
            const int clear = x.edge_from / kTreeTile - x.first;   // tiles before the first edge
            e->tiles[k] = n;
            e->edge[k] = tree_max((clear + x.stride - 1) >> (x.stride - 1), 0);
            e->tail[k] = tree_min(
                (x.len - (x.first + (n - 1) * x.stride) * kTreeTile + 15) >> 4, kTreeTile / 16);
        }
    }
};

}  // namespace swiglu
