// Attention of a step's new tokens over the paged cache.
//
//   o[t, h] = sum_x p_x v_x / sum_x p_x,   p_x = exp(scale * q[t, h] . k_x - max)
//
// over the positions x that token t of request r sees: the request's context
// (x < c) and, of the step's own tokens (x = c + j), those whose bit j is set
// in the token's mask words (without a mask: j <= t's own place). A row that
// sees nothing, or only scores of -inf, is zero. Scores, sums and statistics
// are FP32; the weights p are rounded to BF16 for the second product (the tensor
// cores take both operands in one type, and V is BF16), the result once to BF16: 0.0019 to
// 0.0023 of the values' deviation off 64-bit results, where FP32 weights would
// be 0.0016 to 0.0017 off. The sum below the line is of the rounded weights in the
// narrow form, where it is a product too, and of the unrounded ones in the wide
// form, where it is taken before they are rounded; roundings to nearest average
// out in either.
//
// One persistent block per SM works through its share of the line of tiles
// (tree_schedule.cuh). All query heads of a kv head and many tokens fill the
// 128 rows of a row tile, so each K and V tile is read once for up to two row
// tiles. Roles (20 warps):
//   warps 0-7, 8-15  softmax groups 0 and 1 (below)
//   warp 16          TMA loads: K and V tiles of 128 positions, one box a page,
//                    through one ring of stages in the order of their use
//   warp 17          issues the MMAs
//   warp 18          tiles with new tokens or past a request's end: zeroes V rows
//                    past the end and takes NaN and Inf out of new tokens' V
//                    (0 x NaN would reach rows that do not see them; the rows
//                    that do get them back at the end)
//   warp 19          describes the block's entries (tree_schedule.cuh) ahead of
//                    their use, in a small ring that the other roles read
//
// Two forms, by the rows of a request and kv head (tokens x heads), each with
// blocks of its own (tree_schedule.cuh):
//   wide  S = Q K^T with the rows on the 128-row side (TMEM lanes), two
//       threads a row, 64 positions each. They share the row's maximum; a vote
//       per tile says whether any row of the group has outgrown its own, and
//       only then is it exchanged. The weights go back to TMEM, over the scores,
//       as the A operand of O += P V (V as it lies, MN-major).
//   narrow (up to 32 rows: single tokens, small trees)  S^T = K Q^T with the
//       positions on the 128-row side, one thread a position: a thread has
//       as many exponentials as there are rows, where the wide form would
//       leave 128 to each of a few threads. The weights go to shared memory as
//       the B operand of O^T += V^T P^T, and of a product with ones that sums
//       them; the maximum is common to the group: a vote per tile says whether
//       any score has outgrown it.
// In both the accumulator is only rescaled when the maximum has risen by more
// than 2^8, so most tiles leave it alone and weights stay below 2^8.
// TMEM: scores of the two groups in columns 0-255, the two accumulators in
// 256 + D each (narrow: sums of p v in 32 columns, sums of p in 32). While one
// group's softmax runs, the tensor cores work for the other; how an entry gives
// both groups work is said at TreeEntry.
// Every wait is bounded (sm103_ptx.cuh); a group's barriers are reached by all
// of its warps whatever their waits said.
//
// What bounds it. Narrow, with enough requests: the bytes of K and V (64
// requests of one token, contexts of 4000, 4 kv heads of 128: 5.6 TB/s of
// K and V over the whole call, pages of 64 rows). Wide, two row tiles an item:
// the chain of one tile - scores 512 clocks of the tensor cores, softmax 1900,
// result 512, and some 1000 of waits, barriers and issue between them. While one
// group is in its softmax, the tensor cores have the other group's products to do,
// 1024 clocks, and then wait for it: two tiles of scores would keep them busy if the
// softmax were no longer than that (32 requests of up to 64 tokens, 8 heads a kv
// head, contexts of 2000 to 6000: 271 us, 732 TFLOP/s of products that count).
// No single piece of it is the bound: without the exponentials, or half of either
// product, it takes 4% less. At its 96 registers the kernel spills a little (92 bytes
// of stores and 184 of loads at head size 128, 104 and 196 at 64). Small calls: 6 us are launch, the shares' prologue and the end of the
// kernel, 2 to 3 the join.
//
// Five roles run different code at once, and the SM's instruction cache holds
// some 32 KB: the roles read what they follow from shared memory instead of
// keeping copies, have one call site for each kind of step, and leave loops
// rolled where a step is long anyway (with everything inlined and unrolled,
// 290 KB, a quarter of the fetches missed and warps waited longer for
// instructions than for scores; now 153 KB and a tenth).
#pragma once

#include "epilogue.cuh"
#include "tree_schedule.cuh"

namespace swiglu {

struct TreeAttnArgs {
    TreeGeom geom;
    const int *table;                  // [requests][max_pages]
    const int *ctx_lens;               // [requests]
    const int *query_start;            // [requests + 1]
    const unsigned long long *mask;    // [tokens][mask_words], or null
    const uint16_t *v_cache;           // [pages][kv heads][page rows][D]
    uint16_t *out;                     // [tokens][q heads][D]
    float4 *partial;                   // [2 * grid][D / 4][part_rows], four columns a row
    float2 *stats;                     // [2 * grid][part_rows]: maximum, sum
    int4 *chains;                      // [grid]: an item that goes on in the next block: its blocks
                                       // first | last << 16, first token, kv head, tokens (0: none)
    long long max_pages;
    float scale_log2;                  // scale * log2(e)
    float rise;                        // kTreeRescale / scale_log2: a rise of the maximum, as a score
    int q_heads, num_pages, page_shift, mask_words;
    int part_rows;                     // rows of one partial result: 128 or 256
#ifdef SWIGLU_TEST_FAULT_INJECTION
    int skip_first_fill;               // test build only: never fill the first pipeline stage
#endif
};

constexpr int kTreeEntries = 4;   // entries described ahead of their results
constexpr int kTreeThreads = 640;
constexpr int kTreeGroup = 256;   // threads of a softmax group

// Shared memory of a block, for either form.
template <int D, bool NARROW>
struct TreeCfg {
    static constexpr int HALVES = D / 64;    // 64-column halves of a row
    // A K or V tile: 8-row atoms of 1024 bytes, a row group's halves next to
    // each other, so that a page of both halves is one box and one stretch
    static constexpr int GROUP = HALVES * 1024;
    static constexpr int TILE = kTreeTile / 8 * GROUP;
    // A Q tile: its rows half after half
    static constexpr int Q_HALF = (NARROW ? kTreeNarrow : kTreeTile) * kRowBytes;
    static constexpr int QBUF = HALVES * Q_HALF;
    // Narrow: a group's weights, 128 positions x 32 rows
    static constexpr int W_BYTES = NARROW ? kTreeTile * kTreeNarrow * 2 : 0;
    static constexpr int STAGES = D == 128 ? (NARROW ? 6 : 5) : 11;
    static constexpr int OFF_Q = 0;          // two Q tiles
    static constexpr int OFF_W = 2 * QBUF;   // two groups' weights
    static constexpr int OFF_KV = OFF_W + 2 * W_BYTES;
    static constexpr int END = OFF_KV + STAGES * TILE;
};
// What both forms have in common, behind the larger one.
template <int D>
struct TreeShared {
    static constexpr int BASE =
        TreeCfg<D, true>::END > TreeCfg<D, false>::END ? TreeCfg<D, true>::END : TreeCfg<D, false>::END;
    static constexpr int OFF_STATS = BASE;                  // float2 [2][128]
    static constexpr int OFF_ENTRY = OFF_STATS + 2 * 128 * 8;
    static constexpr int OFF_BAR = OFF_ENTRY + kTreeEntries * static_cast<int>(sizeof(TreeEntry));
    static constexpr int STAGES = D == 128 ? 6 : 11;        // the most a form has
    // ring: full, empty, V fixed; two Q buffers: full, empty; a group: scores,
    // weights, result; entries: full, empty; both groups: statistics, results
    // read; drain
    static constexpr int NUM_BARS = 3 * STAGES + 4 + 6 + 2 * kTreeEntries + 3;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 80;
    static constexpr int TMEM_O = 256;
    static constexpr int TMEM_ONES = 64;    // narrow: 128 x 16 ones
    static_assert(OFF_BAR % 8 == 0 && SMEM_BYTES <= 232448, "shared memory budget");
};

// Addresses of the block's mbarriers.
template <int D>
struct TreeBars {
    using S = TreeShared<D>;
    uint32_t base;
    __device__ uint32_t at(int i) const { return base + S::OFF_BAR + 8u * i; }
    __device__ uint32_t kv_full(int s) const { return at(s); }
    __device__ uint32_t kv_empty(int s) const { return at(S::STAGES + s); }
    __device__ uint32_t v_fixed(int s) const { return at(2 * S::STAGES + s); }
    __device__ uint32_t q_full(int b) const { return at(3 * S::STAGES + b); }
    __device__ uint32_t q_empty(int b) const { return at(3 * S::STAGES + 2 + b); }
    __device__ uint32_t s_full(int s) const { return at(3 * S::STAGES + 4 + s); }
    __device__ uint32_t p_ready(int s) const { return at(3 * S::STAGES + 6 + s); }
    __device__ uint32_t o_full(int s) const { return at(3 * S::STAGES + 8 + s); }
    __device__ uint32_t e_full(int i) const { return at(3 * S::STAGES + 10 + i); }
    __device__ uint32_t e_empty(int i) const { return at(3 * S::STAGES + 10 + kTreeEntries + i); }
    __device__ uint32_t both_ready() const { return at(3 * S::STAGES + 10 + 2 * kTreeEntries); }
    __device__ uint32_t o_done() const { return at(3 * S::STAGES + 11 + 2 * kTreeEntries); }
    __device__ uint32_t drain() const { return at(3 * S::STAGES + 12 + 2 * kTreeEntries); }
};

// The block's share of one form's line, and where things lie.
struct TreeBlock {
    uint8_t *smem;
    uint32_t tmem;
    TreeCut cut;
    int index;       // of the block among its form's
    int base;        // the form's first block
};

// Places in shared memory that several roles use.
template <int D>
__device__ __forceinline__ float *tree_stats(uint8_t *smem) {
    return reinterpret_cast<float *>(smem + TreeShared<D>::OFF_STATS);
}
template <int D>
__device__ __forceinline__ TreeEntry *tree_entries(uint8_t *smem) {
    return reinterpret_cast<TreeEntry *>(smem + TreeShared<D>::OFF_ENTRY);
}
template <int D>
__device__ __forceinline__ volatile int *tree_abort(uint8_t *smem) {
    return reinterpret_cast<volatile int *>(smem + TreeShared<D>::OFF_MISC + 4);
}
// An entry's V had Inf or NaN among its new tokens, [entry][group].
template <int D>
__device__ __forceinline__ volatile int *tree_flags(uint8_t *smem) {
    return reinterpret_cast<volatile int *>(smem + TreeShared<D>::OFF_MISC + 16);
}

constexpr float kTreeRescale = 8.f;   // rise of the maximum (log2) that rescales

// Scores of any finite size. "Has outgrown the maximum" compares scores, score >
// maximum + rise, which holds for every finite score while there is no maximum
// (-inf), and a weight of the maximum itself must not be a rounding error's:
// (score - maximum) * scale is exactly 0 for it. The wide form spends one
// multiply-add a score, score * scale - maximum * scale, whose second product is
// rounded: by up to 64 at 2^31, and past that the rounding alone could take
// weights out of range. There neighbouring scores are 2^7 or more apart, so all
// but the maximum have no weight, which any large factor gives: one that is a power
// of two and takes the maximum to 2^30 rounds nothing.
__device__ __forceinline__ float tree_factor(float max, float scale) {
    constexpr float kLarge = 2147483648.f;
    const uint32_t exponent = (__float_as_uint(max) >> 23) & 255u;
    return max != -INFINITY && fabsf(max * scale) >= kLarge ? __uint_as_float((284u - exponent) << 23)
                                                            : scale;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two products and sums at once.
__device__ __forceinline__ void fma2(float &lo, float &hi, float a_lo, float a_hi, float b, float c) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %4};\n\t"
        "mov.b64 c, {%5, %5};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "f"(a_lo), "f"(a_hi), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float &lo, float &hi, float a_lo, float a_hi) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(lo), "+f"(hi)
        : "f"(a_lo), "f"(a_hi));
}
__device__ __forceinline__ uint32_t mask_of_bits(int n) {   // the n lowest bits, n clamped
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// What decides which positions a token sees.
struct TreeSight {
    const unsigned long long *mask;   // the token's words, or null: causal
    int words;
    int token;                        // its place among the request's new tokens
    int ctx, len;
};

// Which of the 32 positions x0 .. x0 + 31 a token sees (bit b: x0 + b): the
// context, and of the new tokens those in its mask words, or up to itself.
__device__ __forceinline__ uint32_t tree_visible(const TreeSight &t, int x0) {
    uint32_t see = mask_of_bits(t.ctx - x0);
    if (t.mask) {
        // the 32 mask bits from new token j0 on, from one or two words
        const int j0 = x0 - t.ctx;
        uint32_t bits = 0;
        if (j0 > -32) {
            const int from = tree_max(j0, 0), k = from >> 6, sh = from & 63;
            unsigned long long v = k < t.words ? t.mask[k] >> sh : 0ull;
            if (sh > 32 && k + 1 < t.words) v |= t.mask[k + 1] << (64 - sh);
            bits = static_cast<uint32_t>(v);
            if (j0 < 0) bits <<= -j0;
        }
        see |= bits;
    } else {
        see |= mask_of_bits(t.ctx + t.token + 1 - x0);
    }
    return see & mask_of_bits(t.len - x0);
}

// The non-finite V values of the new tokens in positions [x0, x1) that a row
// sees, added to `cols` columns of its result, which this thread has just stored
// (the products took them as zero; nothing finite changes an Inf or a NaN, so
// adding them to the rounded result is the same). V: the column's place in
// the kv head's first page, pages `page_step` elements apart.
template <int D, typename T>
__device__ __noinline__ void tree_add_nonfinite(T *result, int cols, const TreeSight t, int x0, int x1,
                                                const int *table, int page_shift, int num_pages,
                                                long long page_step, const uint16_t *v_col) {
    for (int at = x0 & ~31; at < x1; at += 32) {
        uint32_t see = tree_visible(t, at) & mask_of_bits(x1 - at) & ~mask_of_bits(x0 - at);
        while (see) {
            const int x = at + __ffs(see) - 1;
            see &= see - 1;
            const int page = table[x >> page_shift];
            if (page < 0 || page >= num_pages) continue;
            const uint16_t *v =
                v_col + page * page_step + (x & ((1 << page_shift) - 1)) * static_cast<long long>(D);
            for (int i = 0; i < cols; ++i)
                if ((v[i] & 0x7F80u) == 0x7F80u) {
                    const float add = __uint_as_float(static_cast<uint32_t>(v[i]) << 16);
                    if constexpr (sizeof(T) == 4) {
                        result[i] += add;
                    } else {
                        const __nv_bfloat16 sum = __float2bfloat16_rn(
                            __uint_as_float(static_cast<uint32_t>(result[i]) << 16) + add);
                        result[i] = *reinterpret_cast<const uint16_t *>(&sum);
                    }
                }
        }
    }
}

// mbar_wait with its loop out of line: the first try, which the hardware may
// suspend for a while, mostly succeeds.
__device__ __noinline__ bool tree_wait_on(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
    return mbar_wait(bar, parity, abort_flag);
}
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity,
                                          const volatile int *abort_flag) {
    return mbar_try_wait(bar, parity) || tree_wait_on(bar, parity, abort_flag);
}
// The same by a whole warp: every lane gets the same answer, so that no lane
// is left alone at a later warp-wide instruction.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity,
                                          const volatile int *abort_flag) {
    return __all_sync(~0u, tree_wait(bar, parity, abort_flag));
}
// This thread gave up: says so, and tells the others to leave.
__device__ __noinline__ void tree_give_up(volatile int *abort_flag, unsigned int status) {
    if (!*abort_flag) {
        atomicOr(&g_status_word, status);
        *abort_flag = 1;
    }
}

// Barriers over the eight warps of softmax group s (named barriers 1 and 2).
__device__ __forceinline__ void group_sync(int s) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + s), "n"(kTreeGroup) : "memory");
}
__device__ __forceinline__ bool group_any(int s, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.or.pred q, %1, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(1 + s), "r"(static_cast<uint32_t>(v)), "n"(kTreeGroup)
        : "memory");
    return r != 0;
}

// What the producer, the MMA issuer and the V warp follow: the entries step by
// step, and the ring's stages in the order that all three keep: per step, for
// each group in turn, the V tile of this step and the K tile of the next. The
// step before the first has no V tiles.
template <int D, bool NARROW>
struct TreeCursor {
    using C = TreeCfg<D, NARROW>;
    TreeBars<D> bars;
    const TreeEntry *entries;
    const volatile int *abort_flag;
    const TreeEntry *cur, *nxt;   // entries of this step (null before the first) and the next
    int step, nstep, seq;         // the steps' numbers; entry nxt's
    int stage;
    uint32_t phase;

    __device__ __forceinline__ void advance() {
        if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    }
    // Once entry `seq` is described, the next step is its first.
    __device__ __forceinline__ bool fetch() {
        const int i = seq % kTreeEntries;
        nxt = entries + i;
        nstep = 0;
        return tree_wait(bars.e_full(i), (seq / kTreeEntries) & 1, abort_flag);
    }
    __device__ __forceinline__ bool start() {
        cur = nullptr;
        step = seq = stage = 0;
        phase = 0;
        return fetch();
    }
    // To the next step, giving back the entry that is left.
    __device__ __forceinline__ bool move(bool arrive) {
        if (cur && cur != nxt && arrive) mbar_arrive(bars.e_empty((seq - 1) % kTreeEntries));
        cur = nxt;
        step = nstep;
        nstep = step + 1;
        if (nstep < cur->steps) return true;
        ++seq;
        return fetch();
    }
};

// ---- TMA producer: the whole warp walks, lanes issue pages. Returns which
// stages and Q tiles it filled, and the parity of their last filling, for the
// drain after an abort.
template <int D, bool NARROW>
__device__ __forceinline__ uint2 tree_produce(const CUtensorMap &tmQ, const CUtensorMap &tmK,
                                              const CUtensorMap &tmV, const TreeAttnArgs &a,
                                              const TreeBlock &blk) {
    using C = TreeCfg<D, NARROW>;
    const TreeGeom &g = a.geom;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    const int lane = threadIdx.x & 31;
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    TreeCursor<D, NARROW> k{bars, tree_entries<D>(blk.smem), abort_flag};
    uint32_t issued = 0, parity = 0;   // bits: ring stages, then the two Q tiles
    int qb = 0;
    uint32_t qphase = 0;
    const int pages = kTreeTile >> a.page_shift;   // pages a tile, <= 8
    // this lane's page: of each group's tile in use, and of its next one
    int rows0 = 0, rows1 = 0, ahead0 = 0, ahead1 = 0;
    bool ok = __all_sync(~0u, k.start());
    while (ok && (k.cur || k.nxt->steps)) {
#pragma unroll 1
        for (int op = 0; op < 4; ++op) {   // V of group 0, K of group 0, V and K of group 1
            const bool is_k = op & 1;
            const int s = op >> 1, step = is_k ? k.nstep : k.step;
            const TreeEntry *e = is_k ? k.nxt : k.cur;
            if (!e || step >= e->steps) continue;
            const TreePart &x = e->part[s];
            if (is_k && step == 0 && (s == 0 || e->two_q())) {
                // the row tile's queries (rows past its tokens are not used)
                ok = warp_wait(bars.q_empty(qb), ((qphase >> qb) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                const int toks = (NARROW ? kTreeNarrow : kTreeTile) / g.group;
                if (lane == 0)
                    mbar_arrive_expect_tx(bars.q_full(qb), static_cast<uint32_t>(toks) * g.group *
                                                               kRowBytes * C::HALVES);
                __syncwarp();
                if (lane < C::HALVES)
                    tma_load_3d(bars.base + C::OFF_Q + qb * C::QBUF + lane * C::Q_HALF, &tmQ,
                                bars.q_full(qb), 64 * lane, x.h * g.group, x.tok);
                const int bit = C::STAGES + qb;
                issued |= 1u << bit;
                parity = (parity & ~(1u << bit)) | (((qphase >> qb) & 1u) << bit);
                qphase ^= 1u << qb;
                qb ^= 1;
            }
            if (!e->own_kv(step, s)) continue;
            const int tile = x.tile(step);
            // the tile's pages up to the item's end
            const int count = tree_min(
                pages, (x.len - tile * kTreeTile + (1 << a.page_shift) - 1) >> a.page_shift);
            // a tile's V comes from its K's pages; the next K's are asked for
            // one step ahead (a load of the table takes as long as a tile)
            int row = s ? rows1 : rows0;
            if (is_k) {
                const int *table = a.table + x.r * a.max_pages +
                                   static_cast<long long>(tile) * pages + lane;
                int page = s ? ahead1 : ahead0, next = 0;
                if (step == 0 && lane < count) page = *table;
                const int after = tile + x.stride;
                if (after < x.end &&
                    (after * pages + lane) << a.page_shift < x.len)
                    next = table[static_cast<long long>(x.stride) * pages];
                // outside the cache: a box past its end, filled with zeros
                row = page >= 0 && page < a.num_pages ? page * g.kv_heads + x.h
                                                      : a.num_pages * g.kv_heads;
                if (s) {
                    ahead1 = next;
                    rows1 = row;
                } else {
                    ahead0 = next;
                    rows0 = row;
                }
            }
            ok = warp_wait(bars.kv_empty(k.stage), k.phase ^ 1u, abort_flag);
            if (!ok) break;
#ifdef SWIGLU_TEST_FAULT_INJECTION
            // test build: leave the first stage unfilled, so that the waits for
            // it run out
            if (a.skip_first_fill && k.stage == 0 && k.phase == 0) {
                k.advance();
                continue;
            }
#endif
            if (lane == 0)
                mbar_arrive_expect_tx(bars.kv_full(k.stage), static_cast<uint32_t>(count) *
                                                                 kRowBytes * C::HALVES
                                                                 << a.page_shift);
            __syncwarp();
            if (lane < count)
                tma_load_5d(bars.base + C::OFF_KV + k.stage * C::TILE +
                                (static_cast<uint32_t>(lane) * C::HALVES * kRowBytes << a.page_shift),
                            is_k ? &tmK : &tmV, bars.kv_full(k.stage), 0, 0, 0, 0, row);
            issued |= 1u << k.stage;
            parity = (parity & ~(1u << k.stage)) | (k.phase << k.stage);
            k.advance();
        }
        if (ok && k.nxt->steps == 0) break;
        if (ok) ok = __all_sync(~0u, k.move(lane == 0));
    }
    if (!ok && lane == 0) tree_give_up(abort_flag, kStatusProducerTimeout);
    return make_uint2(issued, parity);
}

// ---- MMA issuer: one thread. It is on every tile's critical path, so unlike
// the other roles it keeps what it follows in registers.
struct TreeIssue {   // of an entry
    int kind, steps, tiles[2], edge[2], tail[2];
    __device__ __forceinline__ void read(const TreeEntry &e) {
        kind = e.kind;
        steps = e.steps;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            tiles[s] = steps ? e.tiles[s] : 0;   // (the last entry has only its steps)
            edge[s] = e.edge[s];
            tail[s] = e.tail[s];
        }
    }
};
template <int D, bool NARROW>
__device__ __forceinline__ void tree_issue(const TreeBlock &blk) {
    using C = TreeCfg<D, NARROW>;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    const TreeEntry *entries = tree_entries<D>(blk.smem);
    // the scores: 128 rows x 128 positions, or 128 positions x 32 rows
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, NARROW ? kTreeNarrow : kTreeTile);
    // the result: 128 rows x D, V as it lies; or D x 32 rows, both as they lie
    constexpr uint32_t idesc_o =
        NARROW ? idesc_bf16_f32(128, kTreeNarrow) | kIdescAMnMajor | kIdescBMnMajor
               : idesc_bf16_f32(128, D) | kIdescBMnMajor;
    // narrow: the weights' sums, as a product with a block of ones, so that they
    // need no registers during the tiles and no exchange between threads
    constexpr uint32_t idesc_l = idesc_bf16_f32(128, kTreeNarrow) | kIdescBMnMajor;
    TreeIssue cur{}, nxt{};   // cur.steps = 0 before the first entry
    int step = 0, nstep = 0, seq = 0;
    // the ring; the stages of the K and V tiles in use; nxt's first Q tile
    int stage = 0, kstage = 0, vstage = 0, qb = 0;
    uint32_t phase = 0, qphase = 0, pphase = 0, fphase = 0;
    auto next_stage = [&](int &at, bool there = false) {   // the ring's next tile, once it is there
        if (!there && !tree_wait(bars.kv_full(stage), phase, abort_flag)) return false;
        at = stage;
        if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
        }
        return true;
    };
    auto fetch = [&] {
        const int i = seq % kTreeEntries;
        nstep = 0;
        if (!tree_wait(bars.e_full(i), (seq / kTreeEntries) & 1, abort_flag)) return false;
        nxt.read(entries[i]);
        return true;
    };
    bool ok = fetch();
    while (ok) {
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
            if (!ok) break;
            bool k_there = false;
            if (step < (s ? cur.tiles[1] : cur.tiles[0])) {   // the result's product
                if (s == 0 || cur.kind != kTreePair) {
                    ok = next_stage(vstage);
                    if (ok && step >= (s ? cur.edge[1] : cur.edge[0])) {
                        ok = tree_wait(bars.v_fixed(vstage), (fphase >> vstage) & 1u, abort_flag);
                        fphase ^= 1u << vstage;
                    }
                }
                // while the weights are due, whether what comes after is there
                k_there = mbar_test_wait(bars.kv_full(stage), phase);
                ok = ok && tree_wait(bars.p_ready(s), (pphase >> s) & 1u, abort_flag);
                if (!ok) break;
                pphase ^= 1u << s;
                tc_fence_after();
                const uint64_t vd = smem_desc(bars.base + C::OFF_KV + vstage * C::TILE,
                                              D == 128 ? 1024 : 0, C::GROUP);
                const uint32_t acc = blk.tmem + TreeShared<D>::TMEM_O + D * s;
                constexpr uint32_t kstep = 2 * C::GROUP >> 4;   // 16 positions of V
                const uint32_t more = step != 0;
                const bool last = step + 1 == (s ? cur.tiles[1] : cur.tiles[0]);
                // positions of the tile, in 16s (the rest has no weight)
                const int count = last ? (s ? cur.tail[1] : cur.tail[0]) : kTreeTile / 16;
#pragma unroll
                for (int i = 0; i < kTreeTile / 16; ++i) {
                    if (i >= count) break;
                    if constexpr (NARROW) {
                        const uint64_t wd =
                            smem_desc(bars.base + C::OFF_W + s * C::W_BYTES, 16, 512, 4);
                        umma_bf16(acc, vd + kstep * i, wd + 64u * i, idesc_o, more || i != 0);
                        umma_bf16_ts(acc + 32, blk.tmem + TreeShared<D>::TMEM_ONES, wd + 64u * i,
                                     idesc_l, more || i != 0);
                    } else {
                        umma_bf16_ts(acc, blk.tmem + 128 * s + 64 * (i >> 2) + 32 + 8 * (i & 3),
                                     vd + kstep * i, idesc_o, more || i != 0);
                    }
                }
                if (s == 1 || cur.kind != kTreePair) umma_commit(bars.kv_empty(vstage));
                if (last) umma_commit(bars.o_full(s));
            }
            if (nstep < (s ? nxt.tiles[1] : nxt.tiles[0])) {   // the next scores
                const bool two_q = nxt.kind != kTreeSplit;
                const int buf = two_q ? qb ^ s : qb;
                if (nstep == 0 && (s == 0 || two_q)) {
                    ok = tree_wait(bars.q_full(buf), (qphase >> buf) & 1u, abort_flag);
                    qphase ^= 1u << buf;
                }
                if (s == 0 || nxt.kind != kTreePair) ok = ok && next_stage(kstage, k_there);
                if (!ok) break;
                tc_fence_after();
                const uint64_t kd =
                    smem_desc(bars.base + C::OFF_KV + kstage * C::TILE, 16, C::GROUP);
                const uint64_t qd = smem_desc(bars.base + C::OFF_Q + buf * C::QBUF, 16, 1024);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t ko = kd + (i >> 2) * (1024 >> 4) + 2u * (i & 3);
                    const uint64_t qo = qd + (i >> 2) * (C::Q_HALF >> 4) + 2u * (i & 3);
                    umma_bf16(blk.tmem + 128 * s, NARROW ? ko : qo, NARROW ? qo : ko, idesc_s,
                              i != 0);
                }
                umma_commit(bars.s_full(s));
                if (s == 1 || nxt.kind != kTreePair) umma_commit(bars.kv_empty(kstage));
                // the last scores that need this Q tile: the part's, in a split
                // those of the entry's last tile
                const bool last = nstep + 1 == (s ? nxt.tiles[1] : nxt.tiles[0]);
                if (two_q ? last : nstep + 1 == nxt.steps && (s == 1 || nstep >= nxt.tiles[1]))
                    umma_commit(bars.q_empty(buf));
            }
        }
        if (!ok || nxt.steps == 0) break;
        if (nstep == 0) {   // into the next entry
            if (seq > 0) mbar_arrive(bars.e_empty((seq - 1) % kTreeEntries));
            cur = nxt;
        }
        step = nstep++;
        if (nstep == cur.steps) {
            if (cur.kind == kTreeSplit) qb ^= 1;
            ++seq;
            ok = fetch();
        }
    }
    if (!ok) tree_give_up(abort_flag, kStatusMmaTimeout);
}

// ---- V rows of edge tiles. Every stage is waited for and given back in ring
// order, K's and those of tiles that need nothing too, so that this warp is
// never a whole pass of the ring away from the others (a wait on a barrier's
// parity cannot tell two passes apart).
template <int D, bool NARROW>
__device__ __forceinline__ void tree_mend_v(const TreeBlock &blk) {
    using C = TreeCfg<D, NARROW>;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    const int lane = threadIdx.x & 31;
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    TreeCursor<D, NARROW> k{bars, tree_entries<D>(blk.smem), abort_flag};
    bool ok = __all_sync(~0u, k.start());
    while (ok && (k.cur || k.nxt->steps)) {
#pragma unroll 1
        for (int op = 0; op < 4; ++op) {
            const bool is_k = op & 1;
            const int s = op >> 1, step = is_k ? k.nstep : k.step;
            const TreeEntry *e = is_k ? k.nxt : k.cur;
            if (!e || step >= e->steps || !e->own_kv(step, s)) continue;
            ok = warp_wait(bars.kv_full(k.stage), k.phase, abort_flag);
            if (!ok) break;
            const TreePart &x = e->part[s];
            const int tile = x.tile(step);
            if (!is_k && x.edge(tile)) {
                // Rows [first, end) hold new tokens, [end, 128) nothing (of
                // which the product reads those up to a multiple of 16). In
                // the order of memory, 256 chunks of 16 bytes at a time, eight
                // loads in flight a lane: with one a tile of new tokens took
                // 6400 clocks, longer than its softmax.
                const int end = tree_min(x.len - tile * kTreeTile, kTreeTile);
                const int first = tree_min(tree_max(x.ctx - tile * kTreeTile, 0), end);
                const int stop = (end + 15) & ~15;
                uint4 *base = reinterpret_cast<uint4 *>(blk.smem + C::OFF_KV + k.stage * C::TILE);
                constexpr int per_group = C::GROUP / 16;   // chunks of eight rows
                auto row_of = [](int m) { return m / per_group * 8 + (m >> 3 & 7); };
                bool bad = false;
#pragma unroll 1
                for (int m0 = ((first >> 3) * per_group & ~255) + lane; row_of(m0) < end; m0 += 256) {
                    uint4 v[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) v[u] = base[m0 + 32 * u];
                    uint32_t any = 0;
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int r = row_of(m0 + 32 * u);
                        // exponent all ones: carry
                        const uint32_t x = ((v[u].x & 0x7F807F80u) + 0x00800080u) |
                                           ((v[u].y & 0x7F807F80u) + 0x00800080u) |
                                           ((v[u].z & 0x7F807F80u) + 0x00800080u) |
                                           ((v[u].w & 0x7F807F80u) + 0x00800080u);
                        any |= r >= first && r < end ? x : 0u;
                    }
                    if (any & 0x80008000u) {
                        bad = true;
#pragma unroll 1
                        for (int u = 0; u < 64; ++u) {   // value u % 8 of chunk u / 8
                            const int m = m0 + 32 * (u >> 3), r = row_of(m);
                            uint16_t *h = reinterpret_cast<uint16_t *>(base + m) + (u & 7);
                            if (r >= first && r < end && (*h & 0x7F80u) == 0x7F80u) *h = 0;
                        }
                    }
                }
#pragma unroll 1
                for (int m = (end >> 3) * per_group + lane; row_of(m) < stop; m += 32)
                    if (row_of(m) >= end) base[m] = make_uint4(0, 0, 0, 0);
                if (bad) {
                    volatile int *flags = tree_flags<D>(blk.smem) + 2 * (e - k.entries);
                    flags[s] = 1;
                    if (e->kind == kTreePair) flags[1] = 1;
                }
                __threadfence_block();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.v_fixed(k.stage));
            }
            if (lane == 0) mbar_arrive(bars.kv_empty(k.stage));
            k.advance();
        }
        if (ok && k.nxt->steps == 0) break;
        if (ok) ok = __all_sync(~0u, k.move(lane == 0));
    }
    if (!ok && lane == 0) tree_give_up(abort_flag, kStatusEpilogueTimeout);
}

// ---- entries, ahead of their use: one thread
template <int D, typename Load>
__device__ __forceinline__ void tree_describe(const TreeAttnArgs &a, const TreeBlock &blk,
                                              const TreeStart &start, Load load) {
    const TreeGeom &g = a.geom;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    volatile int *flags = tree_flags<D>(blk.smem);
    TreeEntry *entries = tree_entries<D>(blk.smem);
    TreeWalk w{};
    if (start.units > 0) w.begin(g, start);
    int4 chain = make_int4(0, 0, 0, 0);
    bool ok = true;
    int seq = 0;
    for (bool more = true; more; ++seq) {
        const int i = seq % kTreeEntries;
        ok = tree_wait(bars.e_empty(i), ((seq / kTreeEntries) & 1) ^ 1, abort_flag);
        if (!ok) break;
        TreeEntry *e = entries + i;
        w.entry(g, load, e);
        flags[2 * i] = flags[2 * i + 1] = 0;
        more = e->steps > 0;
        // an item that goes on in the next block (of a Split or Pair in part 0)
        for (int s = 0; s < (e->kind == kTreeDuo ? 2 : 1) && more; ++s) {
            const TreePart &x = e->part[s];
            const int rest = (x.len + kTreeTile - 1) / kTreeTile - x.end;
            if (rest == 0) continue;
            const int last = tree_block_begin(blk.cut, blk.index + 1) + rest - 1;
            const int first = (x.flags & kPartBegins)
                                  ? blk.index
                                  : tree_block_of(blk.cut, tree_block_begin(blk.cut, blk.index) - x.first);
            chain = make_int4((blk.base + first) | (blk.base + tree_block_of(blk.cut, last)) << 16, x.tok,
                              x.h, x.ntok + (e->kind == kTreePair ? e->part[1].ntok : 0));
        }
        mbar_arrive(bars.e_full(i));
    }
    a.chains[blockIdx.x] = chain;
    if (!ok) tree_give_up(abort_flag, kStatusProducerTimeout);
}

// Where a softmax warp is in the barriers' phases.
struct TreePhase {
    uint32_t scores, own[2], merge, both;   // s_full, o_full of each group, o_done, both_ready
    bool merged;                            // the entry before was shared: o_done is due
};

// The entry before, if the groups shared it: all warps of both have read its
// statistics and accumulators.
template <int D>
__device__ __forceinline__ bool tree_results_read(const TreeBars<D> &bars, TreePhase &ph,
                                                  const volatile int *abort_flag) {
    const bool read = !ph.merged || warp_wait(bars.o_done(), ph.merge ^ 1u, abort_flag);
    ph.merged = false;
    return read;
}

// The largest of a warp's values (NaN left out).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// ---- softmax, narrow form. One entry's part, for the warps of one group: a
// thread is position `row` of each tile, and column d = row of the result.
// False: gave up (the abort flag is set before any group barrier that follows).
// Rows go by eights in loops that are not unrolled: with them unrolled the
// code does not fit the instruction cache beside the other roles' (first
// tiles and results then took 6000 cycles each).
template <int D>
__device__ __forceinline__ bool tree_narrow_part(const TreeAttnArgs &a, const TreeBlock &blk,
                                                 const TreeEntry &entry, int slot, TreePhase &ph) {
    using C = TreeCfg<D, true>;
    const TreeGeom &g = a.geom;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
    const int row = 32 * quad + lane;
    const int c = static_cast<int>(blockIdx.x);
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t ts = blk.tmem + lanes + 128 * s;                            // scores
    const uint32_t to = blk.tmem + lanes + TreeShared<D>::TMEM_O + D * s;      // sums of p v
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    volatile int *flags = tree_flags<D>(blk.smem);
    // a group's statistics: its warps' maxima [4][32], the maximum [32], its
    // last rescale factor [32], what is taken off a score (the maximum, or 0
    // while there is none) [32], and the score above which a row has outgrown
    // its maximum [32]
    constexpr int kMax = 128, kFactor = 160, kBase = 192, kTop = 224;
    float *group_stats = tree_stats<D>(blk.smem) + 256 * s;
    const TreePart &x = entry.part[s];
    const int rows = x.ntok * g.group;
    const bool split = entry.kind == kTreeSplit;
    const bool used1 = entry.part[1].used();
    const float sc = a.scale_log2;
    bool good = true;
    auto give_up = [&] {
        if (lane == 0) tree_give_up(abort_flag, kStatusEpilogueTimeout);
        good = false;
    };
    if (!tree_results_read<D>(bars, ph, abort_flag)) give_up();
    if (warp == 8 * s) {
        group_stats[kMax + lane] = -INFINITY;
        group_stats[kBase + lane] = 0.f;
        group_stats[kTop + lane] = -INFINITY;
    }
    uint8_t *const weights = blk.smem + C::OFF_W + s * C::W_BYTES + row * (2 * kTreeNarrow);
    const int swizzle = 16 * ((row >> 1) & 3);   // 64-byte rows, 64-byte swizzle
    for (int tile = x.first; tile < x.end; tile += x.stride) {
        if (good && !warp_wait(bars.s_full(s), ph.scores, abort_flag)) give_up();
        ph.scores ^= 1u;
        tc_fence_after();
        // bit n: row n sees this position
        uint32_t see = ~0u;
        if (x.edge(tile)) {
            const int pos = tile * kTreeTile + row;
            see = pos < tree_min(x.ctx, x.len) ? ~0u : 0u;
            if (pos >= x.ctx && pos < x.len) {
                const int j = pos - x.ctx;
                const uint32_t heads = mask_of_bits(g.group);
                for (int t = 0; t < x.ntok; ++t) {
                    const bool on =
                        a.mask ? (j >> 6) < a.mask_words &&
                                     ((a.mask[static_cast<long long>(x.tok + t) * a.mask_words +
                                              (j >> 6)] >> (j & 63)) & 1)
                               : j <= x.place + t;
                    if (on) see |= heads << (t * g.group);
                }
            }
        }
        auto scores = [&](int n0, uint32_t (&v)[8]) {
            tmem_ld_32x32b_x8(ts + n0, v);
            tmem_ld_wait();
            reg_fence8(v);
            if (see != ~0u) {
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    if (!((see >> (n0 + n)) & 1u)) v[n] = 0xFF800000u;
            }
        };
        bool first = tile == x.first;
        for (bool again = true;; again = false) {
            // weights by the maximum so far, as if no score had outgrown it
            bool rise = false;
#pragma unroll 1
            for (int n0 = 8 * half; n0 < rows && good; n0 += 16) {
                uint32_t v[8];
                scores(n0, v);
                float base[8], above[8];
#pragma unroll
                for (int n = 0; n < 8; n += 4) {
                    *reinterpret_cast<float4 *>(base + n) =
                        *reinterpret_cast<const float4 *>(group_stats + kBase + n0 + n);
                    *reinterpret_cast<float4 *>(above + n) =
                        *reinterpret_cast<const float4 *>(group_stats + kTop + n0 + n);
                }
                float e[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float score = __uint_as_float(v[n]);
                    e[n] = (score - (first ? 0.f : base[n])) * sc;
                    rise = rise || (n0 + n < rows && score > (first ? -INFINITY : above[n]));
                }
                uint32_t p[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) p[n] = pack_bf16x2(ex2(e[2 * n]), ex2(e[2 * n + 1]));
                *reinterpret_cast<uint4 *>(weights + ((2 * n0) ^ swizzle)) =
                    make_uint4(p[0], p[1], p[2], p[3]);
            }
            // (once a tile: nothing is above the new maximum)
            const bool risen = group_any(s, rise && good && again);
            if (*abort_flag) good = false;
            if (!risen) break;
            // new maxima: each warp's, then the group's
#pragma unroll 1
            for (int n0 = 8 * half; n0 < rows && good; n0 += 16) {
                uint32_t v[8];
                scores(n0, v);
                float top[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) top[n] = warp_max(__uint_as_float(v[n]));
                if (lane == 0) {
                    float4 *at = reinterpret_cast<float4 *>(group_stats + 32 * quad + n0);
                    at[0] = make_float4(top[0], top[1], top[2], top[3]);
                    at[1] = make_float4(top[4], top[5], top[6], top[7]);
                }
            }
            group_sync(s);
            if (warp == 8 * s && lane < rows) {
                const float old = group_stats[kMax + lane];
                const float top = fmaxf(fmaxf(fmaxf(group_stats[lane], group_stats[32 + lane]),
                                              fmaxf(group_stats[64 + lane], group_stats[96 + lane])),
                                        old);
                group_stats[kMax + lane] = top;
                group_stats[kFactor + lane] = top > old ? ex2((old - top) * sc) : 1.f;
                group_stats[kBase + lane] = top == -INFINITY ? 0.f : top;
                group_stats[kTop + lane] = top + a.rise;
            }
            group_sync(s);
            if (!first && tile != x.first) {
                // the sums of p v (columns 0 - 31) and of p (32 - 63)
#pragma unroll 1
                for (int n0 = 8 * half; n0 < rows && good; n0 += 16) {
                    uint32_t o[8], l[8];
                    tmem_ld_32x32b_x8(to + n0, o);
                    tmem_ld_32x32b_x8(to + 32 + n0, l);
                    tmem_ld_wait();
                    reg_fence8(o);
                    reg_fence8(l);
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float f = group_stats[kFactor + n0 + n];
                        o[n] = __float_as_uint(__uint_as_float(o[n]) * f);
                        l[n] = __float_as_uint(__uint_as_float(l[n]) * f);
                    }
                    tmem_st_32x32b_x8(to + n0, o);
                    tmem_st_32x32b_x8(to + 32 + n0, l);
                }
                tmem_st_wait();
            }
            first = false;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (good && lane == 0) mbar_arrive(bars.p_ready(s));
    }

    // ---- this block's result
    if (split) {   // the other group's maxima
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.both_ready());
        if (good && !warp_wait(bars.both_ready(), ph.both, abort_flag)) give_up();
        ph.both ^= 1u;
    }
    if (good && (split || s == 0) && !warp_wait(bars.o_full(0), ph.own[0], abort_flag)) give_up();
    if (good && used1 && (split || s == 1) && !warp_wait(bars.o_full(1), ph.own[1], abort_flag))
        give_up();
    if (!good) return false;
    ph.own[0] ^= 1u;
    if (used1) ph.own[1] ^= 1u;
    tc_fence_after();
    const bool flagged = flags[2 * slot + s] || (split && flags[2 * slot + (s ^ 1)]);
    const bool whole = (x.flags & kPartWhole) != 0;
    const long long part = 2 * c + ((x.flags & kPartBegins) ? 1 : 0);
    const long long prow = part * a.part_rows;
    float4 *const sums = a.partial + part * (D / 4) * a.part_rows;
    const float *m0 = tree_stats<D>(blk.smem) + kMax, *m1 = m0 + 256;
    const uint32_t t0 = blk.tmem + lanes + TreeShared<D>::TMEM_O, t1 = t0 + D;
    // the halves of a group, in a split all four, take the rows in turn
    const int turns = split ? 4 : 2, turn = split ? 2 * s + half : half;
    const long long first_row = static_cast<long long>(x.tok) * a.q_heads + x.h * g.group;
#pragma unroll 1
    for (int r = turn; r < rows; r += turns) {
        uint32_t o, l, y = 0, z = 0;
        tmem_ld_32x32b_x1((split ? t0 : to) + r, o);
        tmem_ld_32x32b_x1((split ? t0 : to) + 32 + r, l);
        if (split && used1) {
            tmem_ld_32x32b_x1(t1 + r, y);
            tmem_ld_32x32b_x1(t1 + 32 + r, z);
        }
        tmem_ld_wait();
        reg_fence4(o, l, y, z);
        float value = __uint_as_float(o), sum = __uint_as_float(l);
        float top = split ? m0[r] : group_stats[kMax + r];
        if (split && used1) {
            const float ma = top, mb = m1[r];
            top = fmaxf(ma, mb);
            const float w0 = ma == -INFINITY ? 0.f : ex2((ma - top) * sc);
            const float w1 = mb == -INFINITY ? 0.f : ex2((mb - top) * sc);
            sum = fmaf(__uint_as_float(z), w1, sum * w0);
            value = fmaf(__uint_as_float(y), w1, value * w0);
        }
        if (row >= D) continue;
        if (whole) {
            const int t = r / g.group;
            const __nv_bfloat16 b = __float2bfloat16_rn(sum == 0.f ? 0.f : __fdividef(value, sum));
            a.out[(first_row + static_cast<long long>(t) * a.q_heads + (r - t * g.group)) * D + row] =
                *reinterpret_cast<const uint16_t *>(&b);
        } else {
            reinterpret_cast<float *>(sums + (row >> 2) * a.part_rows + r)[row & 3] = value;
            if (row == 0) a.stats[prow + r] = make_float2(top, sum);
        }
    }
    if (flagged && row < D) {
        const int x0 = tree_max(x.ctx, (split ? entry.part[0].first : x.first) * kTreeTile);
        const int x1 = tree_min(x.len, x.end * kTreeTile);
        const long long head_step = static_cast<long long>(D) << a.page_shift;
        const uint16_t *vc = a.v_cache + x.h * head_step + row;
        const int *table = a.table + x.r * a.max_pages;
        for (int r = turn; r < rows; r += turns) {
            const int t = r / g.group;
            const TreeSight sight{
                a.mask ? a.mask + static_cast<long long>(x.tok + t) * a.mask_words : nullptr,
                a.mask_words, x.place + t, x.ctx, x.len};
            if (whole)
                tree_add_nonfinite<D>(
                    a.out + (first_row + static_cast<long long>(t) * a.q_heads + r % g.group) * D + row,
                    1, sight, x0, x1, table, a.page_shift, a.num_pages, g.kv_heads * head_step, vc);
            else
                tree_add_nonfinite<D>(
                    reinterpret_cast<float *>(sums + (row >> 2) * a.part_rows + r) + (row & 3), 1,
                    sight, x0, x1, table, a.page_shift, a.num_pages, g.kv_heads * head_step, vc);
        }
    }
    tc_fence_before();
    __syncwarp();
    if (split) {
        if (lane == 0) mbar_arrive(bars.o_done());
        ph.merged = true;
        ph.merge ^= 1u;
    }
    // (no barrier of the group after a way out: tree_softmax has the one that
    // comes before the statistics are used again)
    return true;
}

// ---- softmax, wide form. One entry's part, for the warps of one group: a
// thread is a row and half of each tile's positions. As tree_narrow_part.
template <int D>
__device__ __forceinline__ bool tree_wide_part(const TreeAttnArgs &a, const TreeBlock &blk,
                                               const TreeEntry &entry, int slot, TreePhase &ph) {
    const TreeGeom &g = a.geom;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
    const int row = 32 * quad + lane;
    const int my_tok = row / g.group;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t ts = blk.tmem + lanes + 128 * s;                            // scores, weights
    const uint32_t to = blk.tmem + lanes + TreeShared<D>::TMEM_O + D * s;      // own accumulator
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    volatile int *flags = tree_flags<D>(blk.smem);
    // rows' statistics: the halves' maxima, at the end the maximum and the sum
    float2 *stats = reinterpret_cast<float2 *>(tree_stats<D>(blk.smem)) + 128 * s;
    const TreePart &x = entry.part[s];
    const bool split = entry.kind == kTreeSplit;
    const bool warp_on = 32 * quad < x.ntok * g.group;
    const bool row_on = my_tok < x.ntok;
    const float sc = a.scale_log2;
    bool good = true;
    auto give_up = [&] {
        if (lane == 0) tree_give_up(abort_flag, kStatusEpilogueTimeout);
        good = false;
    };
    auto sight = [&] {
        return TreeSight{
            a.mask ? a.mask + static_cast<long long>(x.tok + my_tok) * a.mask_words : nullptr,
            a.mask_words, x.place + my_tok, x.ctx, x.len};
    };
    if (!tree_results_read<D>(bars, ph, abort_flag)) give_up();
    float m = -INFINITY, l = 0.f;
    for (int tile = x.first; tile < x.end; tile += x.stride) {
        if (good && !warp_wait(bars.s_full(s), ph.scores, abort_flag)) give_up();
        ph.scores ^= 1u;
        tc_fence_after();
        const bool fresh = tile == x.first;
        // The 64 scores, 32 at a time: first their maximum, then the weights, the
        // second 32 from the registers that they are still in, the first 32 read
        // again (all 64 kept would be most of a thread's registers).
        const uint32_t tv = ts + 64 * half;
        unsigned long long see = ~0ull;   // bit j: this half's position j is seen
        if (x.edge(tile)) {
            const TreeSight t = sight();
            see = 0;
#pragma unroll 1
            for (int i = 32; row_on && i >= 0; i -= 32)
                see = see << 32 | tree_visible(t, tile * kTreeTile + 64 * half + i);
        }
        uint32_t v[32];
        auto scores = [&](int i) {
            tmem_ld_32x32b_x32(tv + 32 * i, v);
            tmem_ld_wait();
            reg_fence32(v);
            const uint32_t bits = static_cast<uint32_t>(see >> (32 * i));
            if (bits != ~0u) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (!((bits >> j) & 1u)) v[j] = 0xFF800000u;
            }
        };
        float top = -INFINITY;
        if (warp_on) {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                scores(i);
                float mx[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    mx[(j >> 1) & 3] = fmaxf(mx[(j >> 1) & 3],
                                             fmaxf(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
                top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            }
        }
        const bool rise = fresh || (row_on && top > m + a.rise);
        const bool risen = group_any(s, rise && good);
        if (*abort_flag) good = false;
        if (risen) {
            if (half) stats[row].y = top; else stats[row].x = top;
            group_sync(s);
            const float2 both = stats[row];
            const float now = fmaxf(both.x, both.y);
            float f = 1.f;
            if (now > m && (fresh || now > m + a.rise)) {
                f = ex2((m - now) * sc);
                m = now;
                l *= f;
            }
            if (!fresh && warp_on && __any_sync(~0u, row_on && f != 1.f)) {
#pragma unroll 1
                for (int col = half * (D / 2); col < (half + 1) * (D / 2); col += 8) {
                    uint32_t o[8];
                    tmem_ld_32x32b_x8(to + col, o);
                    tmem_ld_wait();
                    reg_fence8(o);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st_32x32b_x8(to + col, o);
                }
            }
        }
        if (warp_on) {
            // no maximum so far: weights 2^(-inf - 0) = 0
            const float by = tree_factor(m, sc);
            const float base = m == -INFINITY ? 0.f : -m * by;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int i = 1; i >= 0; --i) {
                if (i == 0) scores(0);
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float lo, hi;
                    fma2(lo, hi, __uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), by, base);
                    lo = ex2(lo);
                    hi = ex2(hi);
                    add2(sum[2 * (j & 1)], sum[2 * (j & 1) + 1], lo, hi);
                    p[j] = pack_bf16x2(lo, hi);
                }
                // over this half's own scores, those that are not needed again
                tmem_st_32x32b_x16(tv + 32 + 16 * i, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st_wait();
            tc_fence_before();
        }
        __syncwarp();
        if (good && lane == 0) mbar_arrive(bars.p_ready(s));
    }

    // ---- this block's result: the rows' sums, then (split) the other group's
    group_sync(s);   // (the last maxima have been read)
    if (half) stats[row].y = l;
    group_sync(s);
    if (!half) stats[row] = make_float2(m, l + stats[row].y);
    if (split) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.both_ready());
        if (good && !warp_wait(bars.both_ready(), ph.both, abort_flag)) give_up();
        ph.both ^= 1u;
    } else {
        group_sync(s);
        if (*abort_flag) good = false;
    }
    const bool used1 = entry.part[1].used();
    if (good && (split || s == 0) && !warp_wait(bars.o_full(0), ph.own[0], abort_flag)) give_up();
    if (good && used1 && (split || s == 1) && !warp_wait(bars.o_full(1), ph.own[1], abort_flag))
        give_up();
    if (!good) return false;
    ph.own[0] ^= 1u;
    if (used1) ph.own[1] ^= 1u;
    tc_fence_after();
    if (warp_on) {
        const bool flagged = flags[2 * slot + s] || (split && flags[2 * slot + (s ^ 1)]);
        const bool whole = (x.flags & kPartWhole) != 0;
        // partial results: slot 2c + 1 for an item that begins here, 2c for others
        const long long part =
            2 * static_cast<int>(blockIdx.x) + ((x.flags & kPartBegins) ? 1 : 0);
        const int in_part = ((x.flags & kPartSecond) ? 128 : 0) + row;
        float2 st = stats[row];
        float w0 = 1.f, w1 = 0.f;
        if (split) {
            const float2 *all = reinterpret_cast<const float2 *>(tree_stats<D>(blk.smem));
            const float2 a0 = all[row];
            const float2 a1 = used1 ? all[128 + row] : make_float2(-INFINITY, 0.f);
            const float top = fmaxf(a0.x, a1.x);
            w0 = a0.x == -INFINITY ? 0.f : ex2((a0.x - top) * sc);
            w1 = a1.x == -INFINITY ? 0.f : ex2((a1.x - top) * sc);
            st = make_float2(top, a0.y * w0 + a1.y * w1);
        }
        if (!whole && row_on && half == 0 && (!split || s == 0))
            a.stats[part * a.part_rows + in_part] = st;
        const float inv = whole ? (st.y == 0.f ? 0.f : 1.f / st.y) : 1.f;
        const uint32_t t0 = blk.tmem + lanes + TreeShared<D>::TMEM_O, t1 = t0 + D;
        // this thread's columns: its half of the row, in a split its quarter
        const int width = split ? D / 4 : D / 2;
        const int c0 = (split ? 2 * s + half : half) * width;
        uint16_t *const out = a.out + (static_cast<long long>(x.tok + my_tok) * a.q_heads +
                                       x.h * g.group + (row - my_tok * g.group)) * D;
        // (the lanes' rows next to each other)
        float4 *const sums = a.partial + part * (D / 4) * a.part_rows + in_part;
#pragma unroll 1
        for (int col = c0; col < c0 + width; col += 16) {
            uint32_t o[16];
            if (!split) {
                tmem_ld_32x32b_x16(to + col, o);
                tmem_ld_wait();
                reg_fence16(o);
            } else {
                tmem_ld_32x32b_x16(t0 + col, o);
                uint32_t y[16];
                if (used1) tmem_ld_32x32b_x16(t1 + col, y);
                tmem_ld_wait();
                reg_fence16(o);
                if (used1) {
                    reg_fence16(y);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = __float_as_uint(fmaf(__uint_as_float(y[j]), w1,
                                                    __uint_as_float(o[j]) * w0));
                }
            }
            if (!row_on) continue;
            if (whole) {
                uint4 *dst = reinterpret_cast<uint4 *>(out + col);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        b[i] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * i]) * inv,
                                           __uint_as_float(o[8 * j + 2 * i + 1]) * inv);
                    dst[j] = make_uint4(b[0], b[1], b[2], b[3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sums[(col / 4 + j) * a.part_rows] =
                        make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                    __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
            }
        }
        if (flagged && row_on) {
            const int x0 = tree_max(x.ctx, (split ? entry.part[0].first : x.first) * kTreeTile);
            const int x1 = tree_min(x.len, x.end * kTreeTile);
            const long long head_step = static_cast<long long>(D) << a.page_shift;
            const uint16_t *vc = a.v_cache + x.h * head_step + c0;
            const int *table = a.table + x.r * a.max_pages;
            if (whole)
                tree_add_nonfinite<D>(out + c0, width, sight(), x0, x1, table, a.page_shift,
                                      a.num_pages, g.kv_heads * head_step, vc);
            else
                for (int col = 0; col < width; col += 4)
                    tree_add_nonfinite<D>(
                        reinterpret_cast<float *>(sums + (c0 + col) / 4 * a.part_rows), 4, sight(),
                        x0, x1, table, a.page_shift, a.num_pages, g.kv_heads * head_step, vc + col);
        }
    }
    tc_fence_before();
    __syncwarp();
    if (split) {
        if (lane == 0) mbar_arrive(bars.o_done());
        ph.merged = true;
        ph.merge ^= 1u;
    }
    // (no barrier of the group after a way out: tree_softmax has the one that
    // comes before the statistics are used again)
    return true;
}

// ---- the softmax warps of one group, entry by entry
template <int D, bool NARROW>
__device__ __forceinline__ void tree_softmax(const TreeAttnArgs &a, const TreeBlock &blk) {
    const TreeBars<D> bars{smem_u32(blk.smem)};
    const int s = threadIdx.x / kTreeGroup, lane = threadIdx.x & 31;
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    const TreeEntry *entries = tree_entries<D>(blk.smem);
    TreePhase ph{};
    bool ok = true;
    // rows of no request are zero
    const int used = a.geom.requests > 0
                         ? tree_min(tree_max(a.query_start[a.geom.requests], 0), a.geom.tokens) : 0;
    if (used < a.geom.tokens) {
        const long long per_token = static_cast<long long>(a.q_heads) * D / 8;
        uint4 *o = reinterpret_cast<uint4 *>(a.out);
#pragma unroll 1
        for (long long i = used * per_token + blockIdx.x * (2 * kTreeGroup) + threadIdx.x;
             i < a.geom.tokens * per_token; i += static_cast<long long>(gridDim.x) * (2 * kTreeGroup))
            o[i] = make_uint4(0, 0, 0, 0);
    }
    for (int seq = 0;; ++seq) {
        const int slot = seq % kTreeEntries;
        // The group's warps leave together: one that gave up comes here first,
        // so that none is left alone at a group barrier.
        ok = ok && warp_wait(bars.e_full(slot), (seq / kTreeEntries) & 1, abort_flag);
        if (!ok && lane == 0) tree_give_up(abort_flag, kStatusEpilogueTimeout);
        if (group_any(s, !ok) || entries[slot].steps == 0) break;
        ok = NARROW ? tree_narrow_part<D>(a, blk, entries[slot], slot, ph)
                    : tree_wide_part<D>(a, blk, entries[slot], slot, ph);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bars.e_empty(slot));
    }
}

// ---- one block in one form
template <int D, bool NARROW, typename Load>
__device__ __forceinline__ void tree_block(const CUtensorMap &tmQ, const CUtensorMap &tmK,
                                           const CUtensorMap &tmV, const TreeAttnArgs &a,
                                           const TreeBlock &blk, const TreeStart &start, Load load) {
    using C = TreeCfg<D, NARROW>;
    const TreeBars<D> bars{smem_u32(blk.smem)};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = tree_abort<D>(blk.smem);
    uint2 issued = make_uint2(0, 0);
    if (warp < 16) {
        tree_softmax<D, NARROW>(a, blk);
    } else if (warp == 16) {
        issued = tree_produce<D, NARROW>(tmQ, tmK, tmV, a, blk);
    } else if (warp == 17) {
        if (elect_one()) tree_issue<D, NARROW>(blk);
    } else if (warp == 18) {
        tree_mend_v<D, NARROW>(blk);
    } else if (lane == 0) {
        tree_describe<D>(a, blk, start, load);
    }

    // ---- teardown: every role has left its loop
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 16 && lane == 0) {
            // every TMA load already issued lands before shared memory is reused
            for (int i = 0; i < C::STAGES + 2; ++i)
                if ((issued.x >> i) & 1u)
                    if (!mbar_wait_drain(i < C::STAGES ? bars.kv_full(i) : bars.q_full(i - C::STAGES),
                                         (issued.y >> i) & 1u))
                        atomicOr(&g_status_word, kStatusDrainTimeout);
        }
        if (warp == 17 && elect_one()) {   // (the same lane again)
            umma_commit(bars.drain());
            if (!mbar_wait_drain(bars.drain(), 0)) atomicOr(&g_status_word, kStatusDrainTimeout);
        }
        __syncthreads();
    }
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmQn,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ TreeAttnArgs a) {
    using S = TreeShared<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const TreeBars<D> bars{smem_u32(smem)};
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const TreeGeom &g = a.geom;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + S::OFF_MISC);
    TreeStart *start = reinterpret_cast<TreeStart *>(smem + S::OFF_MISC + 48);
    // the prologue's sums, in the statistics' place
    int2 *warp_sums = reinterpret_cast<int2 *>(tree_stats<D>(smem));
    float *warp_costs = reinterpret_cast<float *>(warp_sums + 32);

    if (warp == 16 && lane == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(bars.kv_full(s), 1);
            mbar_init(bars.kv_empty(s), 2);   // the MMAs' completion and warp 18
            mbar_init(bars.v_fixed(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bars.q_full(s), 1);
            mbar_init(bars.q_empty(s), 1);
            mbar_init(bars.s_full(s), 1);
            mbar_init(bars.p_ready(s), 8);
            mbar_init(bars.o_full(s), 1);
        }
        for (int i = 0; i < kTreeEntries; ++i) {
            mbar_init(bars.e_full(i), 1);
            mbar_init(bars.e_empty(i), 19);   // the softmax warps and warps 16 - 18
        }
        mbar_init(bars.both_ready(), 16);
        mbar_init(bars.o_done(), 16);
        mbar_init(bars.drain(), 1);
        *tree_abort<D>(smem) = 0;
        start->units = 0;
        fence_barrier_init();
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmQn);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (warp == 17) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
        tc_fence_before();
    }
    griddep_launch_dependents();
    griddep_wait();

    // ---- this block's share: both lines' units, summed over the requests, each
    // thread a run of them
    auto load = [&](int r) {
        return tree_request(g, a.query_start[r], a.query_start[r + 1], a.ctx_lens[r]);
    };
    const int per = (g.requests + kTreeThreads - 1) / kTreeThreads;
    const int r0 = tree_min(static_cast<int>(threadIdx.x) * per, g.requests);
    const int r1 = tree_min(r0 + per, g.requests);
    TreeReq q{};
    TreeUnits mine{};
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        q = load(r);
        tree_add_units(g, q, &mine);
    }
    float cost = mine.cost;
    // sums up to this thread, in its warp and then over the warps
    int upto[2] = {mine.wide, mine.narrow};
    auto warp_scan = [&](int (&v)[2]) {
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(~0u, v[0], d), y = __shfl_up_sync(~0u, v[1], d);
            cost += __shfl_xor_sync(~0u, cost, d);
            if (lane >= d) {
                v[0] += x;
                v[1] += y;
            }
        }
    };
    int sums[2] = {0, 0};
    warp_scan(upto);
    if (lane == 31) {
        warp_sums[warp] = make_int2(upto[0], upto[1]);
        warp_costs[warp] = cost;
    }
    __syncthreads();
    cost = 0.f;
    if (lane < kTreeThreads / 32) {
        sums[0] = warp_sums[lane].x;
        sums[1] = warp_sums[lane].y;
        cost = warp_costs[lane];
    }
    warp_scan(sums);
    const int before_w = __shfl_sync(~0u, sums[0], (warp - 1) & 31);
    const int before_n = __shfl_sync(~0u, sums[1], (warp - 1) & 31);
    const int wide = __shfl_sync(~0u, sums[0], 31), narrow = __shfl_sync(~0u, sums[1], 31);

    TreeBlock blk{};
    blk.smem = smem;
    const int c = static_cast<int>(blockIdx.x);
    const int blocks = tree_min(static_cast<int>(gridDim.x), wide + narrow);
    const int nb = tree_min(tree_narrow_blocks(narrow, wide, cost, blocks), narrow);
    const int wb = tree_min(blocks - nb, wide);
    const bool is_narrow = c < nb;
    blk.base = is_narrow ? 0 : nb;
    blk.index = c - blk.base;
    if (blk.index < (is_narrow ? nb : wb)) {
        blk.cut = is_narrow ? tree_cut(narrow, nb) : tree_cut(wide, wb);
        const int u0 = tree_block_begin(blk.cut, blk.index);
        const int own = is_narrow ? mine.narrow : mine.wide;
        const int at =
            (is_narrow ? upto[1] + (warp ? before_n : 0) : upto[0] + (warp ? before_w : 0)) - own;
        // (a thread of one request has it already)
        auto again = [&](int r) { return per > 1 ? load(r) : q; };
        if (u0 >= at && u0 < at + own && tree_find(g, again, is_narrow, r0, r1, at, u0, start))
            start->units = tree_block_begin(blk.cut, blk.index + 1) - u0;
    }
    // (the sums above have passed block barriers: the address is there)
    blk.tmem = *tmem_holder;
    if (is_narrow && warp < 4) {
        uint32_t ones[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) ones[i] = 0x3F803F80u;   // BF16 pairs
        tc_fence_after();
        tmem_st_32x32b_x8(blk.tmem + (static_cast<uint32_t>(32 * warp) << 16) + S::TMEM_ONES, ones);
        tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // a request on one form's line: none of the other form's tokens
    auto on_line = [&](int r) {
        TreeReq x = load(r);
        if (tree_is_narrow(g, x) != is_narrow) x.n = 0;
        return x;
    };
    if (is_narrow)
        tree_block<D, true>(tmQn, tmK, tmV, a, blk, *start, on_line);
    else
        tree_block<D, false>(tmQ, tmK, tmV, a, blk, *start, on_line);
    if (warp == 17) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(blk.tmem, 512);
    }
}

// ---------------------------------------------------------------- partial results
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kJoinBlocks = 8;   // for each block whose item goes on in the next

// Items that several blocks worked on: out = sum_b w_b o_b / sum_b w_b l_b,
// w_b = exp(scale * (m_b - max m)), in an order that depends on the item alone,
// not on which block finished first. A task is 32 rows (a lane each: partial
// results lie with the rows next to each other) and eight columns. An item of p
// blocks has kJoinBlocks * (p - 1) blocks here, and as these grow more than its
// tasks, up to eight warps share a task's partial results, and with few rows the
// lanes that these leave over. Measured, one request of 2 kv heads with 7 heads
// each, context 16000 (76 blocks an item), the call: one token 46 us with
// kJoinBlocks blocks an item and one warp a task, 20 with the warps, 17 with the
// lanes too; 18 tokens 77 and 23.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeAttnArgs a) {
    __shared__ float shares[kJoinWarps][10][32];   // maximum, sum, eight columns
    griddep_launch_dependents();
    griddep_wait();
    const int4 chain = a.chains[blockIdx.x];
    if (chain.w == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = chain.x & 0xFFFF, parts = (chain.x >> 16) - c + 1;
    const int tpt = a.geom.tpt, group = a.geom.group;
    const int rows = chain.w * group;
    const int groups = (rows + 31) / 32, tasks = groups * (D / 8);
    const int helpers = kJoinBlocks * (parts - 1);
    const int helper = kJoinBlocks * (static_cast<int>(blockIdx.x) - c) + static_cast<int>(blockIdx.y);
    // warps a task: as there is room, each with two partial results at least
    int sharers = 1;
    while (2 * sharers <= kJoinWarps && 4 * sharers <= parts && 2 * sharers * tasks <= kJoinWarps * helpers)
        sharers *= 2;
    const int at_once = kJoinWarps / sharers, part = warp % sharers;
    // and the lanes that the rows leave over, as long as two are left for each:
    // adding up a share costs about as much as reading a partial result
    int slots = 32;
    if (sharers > 1)
        while (slots >= 2 * rows && sharers * (32 / slots) * 4 <= parts) slots >>= 1;
    const int lane_row = lane & (slots - 1), stride = sharers * (32 / slots);
    const int first = part * (32 / slots) + lane / slots;
    for (int base = helper * at_once; base < tasks; base += helpers * at_once) {
        const int task = base + warp / sharers;
        const int col = task / groups * 8, i = (task % groups) * 32 + lane_row;
        const int tok = i / group, head = i - tok * group;
        const int second = tok >= tpt;
        const int row = 128 * second + (tok - second * tpt) * group + head;
        const bool on = task < tasks && i < rows;
        // part 0 is the slot of an item that begins in c, the others' of one that goes on
        float top = -INFINITY;
        for (int b = first; on && b < parts; b += stride) {
            const long long slot = b == 0 ? 2 * c + 1 : 2 * (c + b);
            top = fmaxf(top, a.stats[slot * a.part_rows + row].x);
        }
        float acc[8] = {}, l = 0.f;
#pragma unroll 1
        for (int b = first; on && b < parts; b += stride) {
            const long long slot = b == 0 ? 2 * c + 1 : 2 * (c + b);
            const float2 st = a.stats[slot * a.part_rows + row];
            const float4 *o = a.partial + (slot * (D / 4) + col / 4) * a.part_rows + row;
            const float4 x = o[0], y = o[a.part_rows];
            const float f = st.x == -INFINITY ? 0.f : ex2((st.x - top) * a.scale_log2);
            l = fmaf(st.y, f, l);
            acc[0] = fmaf(x.x, f, acc[0]);
            acc[1] = fmaf(x.y, f, acc[1]);
            acc[2] = fmaf(x.z, f, acc[2]);
            acc[3] = fmaf(x.w, f, acc[3]);
            acc[4] = fmaf(y.x, f, acc[4]);
            acc[5] = fmaf(y.y, f, acc[5]);
            acc[6] = fmaf(y.z, f, acc[6]);
            acc[7] = fmaf(y.w, f, acc[7]);
        }
        if (sharers > 1) {   // the first of them adds the others' shares
            float(*mine)[32] = shares[warp];
            mine[0][lane] = top;
            mine[1][lane] = l;
#pragma unroll
            for (int e = 0; e < 8; ++e) mine[2 + e][lane] = acc[e];
            __syncthreads();
            if (part == 0 && lane < slots) {
                float now = top;
                for (int w = 0; w < stride; ++w)
                    now = fmaxf(now, mine[10 * (w & (sharers - 1))][lane + w / sharers * slots]);
                l = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 1
                for (int w = 0; w < stride; ++w) {
                    const int other = 10 * (w & (sharers - 1)), at = lane + w / sharers * slots;
                    const float m = mine[other][at];
                    const float fw = m == -INFINITY ? 0.f : ex2((m - now) * a.scale_log2);
                    l = fmaf(mine[other + 1][at], fw, l);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(mine[other + 2 + e][at], fw, acc[e]);
                }
            }
            __syncthreads();
        }
        if (!on || part || lane >= slots) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        *reinterpret_cast<uint4 *>(
            a.out + (static_cast<long long>(chain.y + tok) * a.q_heads + chain.z * group + head) * D +
            col) = make_uint4(p[0], p[1], p[2], p[3]);
    }
}

}  // namespace swiglu
