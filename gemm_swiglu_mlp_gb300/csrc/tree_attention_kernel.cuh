// Attention of a step's new tokens over the paged cache.
//
//   o[t, h] = sum_x p_x v_x / sum_x p_x,   p_x = exp(scale * q[t, h] . k_x - max)
//
// over the positions x that token t of request r sees: the request's context
// (x < c) and, of the step's own tokens (x = c + j), those whose bit j is set
// in the token's mask words (without a mask: j <= t's own place). A row that
// sees nothing, or only scores of -inf, is zero. Scores, sums and statistics
// are FP32; the weights p are rounded to BF16 for the second product (the
// tensor cores take BF16 pairs), the result once to BF16.
//
// One persistent block per SM works through its share of the line of tiles
// (tree_schedule.cuh). All query heads of a kv head and many tokens fill the
// 128 rows of a row tile, so each K and V tile is read once for up to two row
// tiles. Roles (12 warps):
//   warps 0-3, 4-7  softmax groups 0 and 1, one thread per row: scores from
//                   TMEM, mask, running maximum and sum, weights back to TMEM
//                   as the A operand of the second product; at an item's end
//                   the result to memory. The accumulator is only rescaled when
//                   the maximum has risen by more than 2^8, so most tiles leave
//                   it alone and weights stay below 2^8.
//   warp 8          TMA loads: K and V tiles of 128 positions, page by page,
//                   through one ring of stages in the order of their use
//   warp 9          issues the MMAs: S = Q K^T (both K-major), O += P V with P
//                   from TMEM and V as it lies (MN-major)
//   warp 10         tiles with new tokens or past a request's end: zeroes V rows
//                   past the end and takes NaN and Inf out of new tokens' V
//                   (0 x NaN would reach rows that do not see them; the rows
//                   that do get them back at the end)
//   warp 11         describes the block's entries (tree_schedule.cuh) ahead of
//                   their use, in a small ring that the other roles read
// TMEM: scores of the two groups in columns 0-255 (weights alias them), the
// two accumulators in 256 + D each.
//
// While one group's softmax runs, the tensor cores work for the other; how an
// entry gives both groups work is said at TreeEntry.
// Every wait is bounded (sm103_ptx.cuh).
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
    float *partial;                    // [2 * grid][part_rows][D]
    float2 *stats;                     // [2 * grid][part_rows]: maximum, sum
    int4 *chains;                      // [grid]: items that begin in a block and go on
    long long max_pages;
    float scale_log2;                  // scale * log2(e)
    int q_heads, num_pages, page_shift, mask_words;
    int part_rows;                     // rows of one partial result: 128 or 256
    int min_units;                     // tiles a block, at least
    int q_one;                         // up to this many tokens: Q token by token
};

constexpr int kTreeEntries = 4;   // entries described ahead of their results

template <int D>
struct TreeCfg {
    static constexpr int HALVES = D / 64;                  // 64-column halves of a row
    static constexpr int BLOCK = kTreeTile * kRowBytes;    // one half of a tile: 16 KB
    static constexpr int TILE = HALVES * BLOCK;            // a Q, K or V tile
    static constexpr int STAGES = D == 128 ? 5 : 11;
    static constexpr int OFF_Q = 0;                        // two row tiles
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_STATS = OFF_KV + STAGES * TILE;   // float2 [2][128]
    static constexpr int OFF_ENTRY = OFF_STATS + 2 * 128 * 8;
    static constexpr int OFF_BAR = OFF_ENTRY + kTreeEntries * static_cast<int>(sizeof(TreeEntry));
    // ring: full, empty, V fixed; two Q tiles: full, empty; a group: scores,
    // weights, result; a warp pair: statistics, results read; entries: full,
    // empty; drain
    static constexpr int NUM_BARS = 3 * STAGES + 4 + 6 + 8 + 2 * kTreeEntries + 1;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 80;
    static constexpr int TMEM_O = 256;
    static_assert(OFF_BAR % 8 == 0 && SMEM_BYTES <= 232448, "shared memory budget");
};

constexpr int kTreeThreads = 384;
// Registers a thread after the split: the softmax groups hold a row of 128
// scores; 2 * 128 threads of 216 and 128 of 72 are the 384 * 168 of the launch.
constexpr int kTreeSoftmaxRegs = 216, kTreeOtherRegs = 72;
constexpr float kTreeRescale = 8.f;   // rise of the maximum (log2) that rescales

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

// What a token's row of the mask is judged by.
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
// sees, added to 32 columns of its result, which this thread has just stored
// (the products took them as zero; nothing finite changes an Inf or a NaN, so
// adding them to the rounded result is the same). V: the column's place in
// the kv head's first page, pages `page_step` elements apart.
template <int D, typename T>
__device__ __noinline__ void tree_add_nonfinite(T *result, const TreeSight t, int x0, int x1,
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
            for (int i = 0; i < 32; ++i)
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

// A bounded wait by a whole warp: every lane gets the same answer, so that no
// lane is left alone at a later warp-wide instruction.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity,
                                          const volatile int *abort_flag) {
    return __all_sync(~0u, mbar_wait(bar, parity, abort_flag));
}

// Sum over the block of one number a thread: before this thread, and in all.
struct TreeScan {
    long long before, total;
};
__device__ __forceinline__ TreeScan tree_block_scan(long long mine, long long *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long in = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(~0u, in, d);
        if (lane >= d) in += x;
    }
    if (lane == 31) warp_sums[warp] = in;
    __syncthreads();
    TreeScan s{in - mine, 0};
    for (int w = 0; w < kTreeThreads / 32; ++w) {
        if (w < warp) s.before += warp_sums[w];
        s.total += warp_sums[w];
    }
    return s;
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmQ1,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ TreeAttnArgs a) {
    using C = TreeCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const TreeGeom &g = a.geom;

    auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * i; };
    auto kv_full = [&](int s) { return bar(s); };
    auto kv_empty = [&](int s) { return bar(C::STAGES + s); };
    auto v_fixed = [&](int s) { return bar(2 * C::STAGES + s); };
    auto q_full = [&](int b) { return bar(3 * C::STAGES + b); };
    auto q_empty = [&](int b) { return bar(3 * C::STAGES + 2 + b); };
    auto s_full = [&](int s) { return bar(3 * C::STAGES + 4 + s); };
    auto p_ready = [&](int s) { return bar(3 * C::STAGES + 6 + s); };
    auto o_full = [&](int s) { return bar(3 * C::STAGES + 8 + s); };
    auto st_ready = [&](int w) { return bar(3 * C::STAGES + 10 + w); };
    auto o_done = [&](int w) { return bar(3 * C::STAGES + 14 + w); };
    auto e_full = [&](int i) { return bar(3 * C::STAGES + 18 + i); };
    auto e_empty = [&](int i) { return bar(3 * C::STAGES + 18 + kTreeEntries + i); };
    const uint32_t drain_bar = bar(3 * C::STAGES + 18 + 2 * kTreeEntries);
    float2 *row_stats = reinterpret_cast<float2 *>(smem + C::OFF_STATS);
    TreeEntry *entries = reinterpret_cast<TreeEntry *>(smem + C::OFF_ENTRY);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    // an entry's V had Inf or NaN among its new tokens, for each group
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 16);
    TreeStart *start = reinterpret_cast<TreeStart *>(smem + C::OFF_MISC + 48);
    // the prologue's sums, in the statistics' place
    long long *warp_sums = reinterpret_cast<long long *>(smem + C::OFF_STATS);

    if (warp == 8 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
            mbar_init(v_fixed(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
            mbar_init(s_full(s), 1);
            mbar_init(p_ready(s), 4);
            mbar_init(o_full(s), 1);
        }
        for (int w = 0; w < 4; ++w) {
            mbar_init(st_ready(w), 2);
            mbar_init(o_done(w), 2);
        }
        for (int i = 0; i < kTreeEntries; ++i) {
            mbar_init(e_full(i), 1);
            mbar_init(e_empty(i), 8);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        start->units = 0;
        fence_barrier_init();
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmQ1);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    griddep_launch_dependents();
    griddep_wait();

    // ---- this block's share: sums over the requests, each thread a run of them
    auto load = [&](int r) {
        return tree_request(g, a.query_start[r], a.query_start[r + 1], a.ctx_lens[r]);
    };
    const int c = static_cast<int>(blockIdx.x);
    TreeCut cut{};
    {
        const int per = (g.requests + kTreeThreads - 1) / kTreeThreads;
        const int r0 = tree_min(static_cast<int>(threadIdx.x) * per, g.requests);
        const int r1 = tree_min(r0 + per, g.requests);
        long long mine = 0;
        for (int r = r0; r < r1; ++r) mine += g.kv_heads * tree_head_units(g, load(r));
        const TreeScan scan = tree_block_scan(mine, warp_sums);
        const int blocks = static_cast<int>(
            max(1ll, min(static_cast<long long>(gridDim.x), tree_div(scan.total, a.min_units))));
        cut = tree_cut(scan.total, blocks);
        const long long u0 = tree_block_begin(cut, c);
        if (c < blocks && u0 >= scan.before && u0 < scan.before + mine) {
            long long at = scan.before;
            for (int r = r0; r < r1; ++r) {
                const TreeReq q = load(r);
                const long long u = g.kv_heads * tree_head_units(g, q);
                if (u0 < at + u) {
                    start->r = r;
                    start->units = tree_block_begin(cut, c + 1) - u0;
                    tree_locate(g, q, u0 - at, start);
                    break;
                }
                at += u;
            }
        }
    }
    // rows of no request are zero
    {
        const int used = g.requests > 0
                             ? tree_min(tree_max(a.query_start[g.requests], 0), g.tokens) : 0;
        const long long per_token = static_cast<long long>(a.q_heads) * D / 8;
        uint4 *o = reinterpret_cast<uint4 *>(a.out);
        for (long long i = used * per_token + c * kTreeThreads + threadIdx.x;
             i < g.tokens * per_token; i += static_cast<long long>(gridDim.x) * kTreeThreads)
            o[i] = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // entry `seq`, once it is described (false: gave up)
    auto fetch = [&](int seq, TreeEntry &e) {
        const int i = seq % kTreeEntries;
        const bool got = mbar_wait(e_full(i), (seq / kTreeEntries) & 1, abort_flag);
        e = entries[i];
        return got;
    };
    // producer bookkeeping for the drain after an abort
    uint32_t issued = 0, parity = 0;   // bits: ring stages, then the two Q tiles

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTreeOtherRegs));
        // The ring's order, the same for warps 8, 9 and 10: per step, for each
        // group in turn, the V tile of this step and the K tile of the next.
        TreeEntry cur{}, nxt{};
        int step = 0, seq = 0, nstep = 0;
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        auto advance = [&] {
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        };
        auto follow = [&] {   // nxt, nstep: the step after (cur, step)
            nxt = cur;
            nstep = step + 1;
            if (nstep < cur.steps) return true;
            nstep = 0;
            return fetch(++seq, nxt);
        };
        auto own_kv = [](const TreeEntry &e, int st, int s) {   // group s has tiles of its own
            return e.part[s].active(st) && (s == 0 || e.two_kv());
        };

        if (warp == 8) {
            // ---- TMA producer: the whole warp walks, lanes issue pages
            int qb = 0;
            uint32_t qphase = 0;
            const int pages = kTreeTile >> a.page_shift;   // pages a tile, <= 8
            auto load_tile = [&](const CUtensorMap &tm, const TreePart &x, int tile) {
                const int left = x.len - tile * kTreeTile;   // positions of the tile, > 0
                const int count = tree_min(pages, (left + (1 << a.page_shift) - 1) >> a.page_shift);
                int row = 0;
                if (lane < count) {
                    const int page = a.table[x.r * a.max_pages +
                                             static_cast<long long>(tile) * pages + lane];
                    // outside the cache: a box past its end, filled with zeros
                    row = page >= 0 && page < a.num_pages ? page * g.kv_heads + x.h
                                                          : a.num_pages * g.kv_heads;
                }
                if (!warp_wait(kv_empty(stage), phase ^ 1u, abort_flag)) return false;
                const uint32_t bytes = static_cast<uint32_t>(count) * kRowBytes * C::HALVES
                                       << a.page_shift;
                if (lane == 0) mbar_arrive_expect_tx(kv_full(stage), bytes);
                __syncwarp();
                const uint32_t dst = sbase + C::OFF_KV + stage * C::TILE +
                                     (static_cast<uint32_t>(lane) * kRowBytes << a.page_shift);
                if (lane < count) {
#pragma unroll
                    for (int b = 0; b < C::HALVES; ++b)
                        tma_load_3d(dst + b * C::BLOCK, &tm, kv_full(stage), 64 * b, 0, row);
                }
                issued |= 1u << stage;
                parity = (parity & ~(1u << stage)) | (phase << stage);
                advance();
                return true;
            };
            auto load_q = [&](const TreePart &x) {
                if (!warp_wait(q_empty(qb), ((qphase >> qb) & 1u) ^ 1u, abort_flag)) return false;
                const bool one = x.ntok <= a.q_one;
                if (lane == 0)
                    mbar_arrive_expect_tx(q_full(qb), static_cast<uint32_t>(one ? x.ntok : g.tpt) *
                                                          g.group * kRowBytes * C::HALVES);
                __syncwarp();
                const uint32_t dst = sbase + C::OFF_Q + qb * C::TILE;
                if (one) {
                    if (lane < x.ntok)
#pragma unroll
                        for (int b = 0; b < C::HALVES; ++b)
                            tma_load_3d(dst + b * C::BLOCK + lane * g.group * kRowBytes, &tmQ1,
                                        q_full(qb), 64 * b, x.h * g.group, x.tok + lane);
                } else if (lane < C::HALVES) {
                    tma_load_3d(dst + lane * C::BLOCK, &tmQ, q_full(qb), 64 * lane, x.h * g.group,
                                x.tok);
                }
                const int bit = C::STAGES + qb;
                issued |= 1u << bit;
                parity = (parity & ~(1u << bit)) | (((qphase >> qb) & 1u) << bit);
                qphase ^= 1u << qb;
                qb ^= 1;
                return true;
            };
            // group s's K tile of a step (Q too at an entry's first)
            auto load_k = [&](const TreeEntry &e, int st, int s) {
                if (st == 0 && e.steps > 0 && (s == 0 || e.two_q()) && !load_q(e.part[s]))
                    return false;
                return !own_kv(e, st, s) || load_tile(tmK, e.part[s], e.part[s].tile(st));
            };
            ok = __all_sync(~0u, fetch(0, cur));
            if (ok && cur.steps) ok = load_k(cur, 0, 0) && load_k(cur, 0, 1);
            while (ok && cur.steps) {
                ok = __all_sync(~0u, follow());
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!ok) break;
                    if (own_kv(cur, step, s)) ok = load_tile(tmV, cur.part[s], cur.part[s].tile(step));
                    if (nxt.steps) ok = ok && load_k(nxt, nstep, s);
                }
                cur = nxt;
                step = nstep;
            }
            if (!ok && lane == 0 && !*abort_flag) {
                atomicOr(&g_status_word, kStatusProducerTimeout);
                *abort_flag = 1;
            }
        } else if (warp == 9) {
            // ---- MMA issuer
            if (lane == 0) {
                constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kTreeTile);
                constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D) | kIdescBMnMajor;
                int qb = 0, kstage = 0, vstage = 0;
                uint32_t qphase = 0, pphase = 0, fphase = 0;
                // scores of group s for a step
                auto scores = [&](const TreeEntry &e, int st, int s) {
                    const TreePart &x = e.part[s];
                    if (!x.active(st)) return true;
                    const int buf = qb ^ (e.two_q() ? s : 0);
                    if (st == 0 && (s == 0 || e.two_q())) {
                        if (!mbar_wait(q_full(buf), (qphase >> buf) & 1u, abort_flag)) return false;
                        qphase ^= 1u << buf;
                    }
                    if (s == 0 || e.two_kv()) {
                        if (!mbar_wait(kv_full(stage), phase, abort_flag)) return false;
                        kstage = stage;
                        advance();
                    }
                    tc_fence_after();
                    const uint64_t qd = smem_desc_k128(sbase + C::OFF_Q + buf * C::TILE);
                    const uint64_t kd = smem_desc_k128(sbase + C::OFF_KV + kstage * C::TILE);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * (C::BLOCK >> 4) + 2u * (k & 3);
                        umma_bf16(tmem + 128 * s, qd + off, kd + off, idesc_qk, k != 0);
                    }
                    umma_commit(s_full(s));
                    if (s == 1 || e.two_kv()) umma_commit(kv_empty(kstage));
                    // the last scores that need this Q tile
                    if (x.tile(st) + 1 == x.end) {
                        umma_commit(q_empty(buf));
                        if (!e.two_q()) qb ^= 1;
                    }
                    return true;
                };
                ok = fetch(0, cur);
                if (ok && cur.steps) ok = scores(cur, 0, 0) && scores(cur, 0, 1);
                while (ok && cur.steps) {
                    ok = follow();
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!ok) break;
                        const TreePart &x = cur.part[s];
                        if (x.active(step)) {
                            if (s == 0 || cur.two_kv()) {
                                ok = mbar_wait(kv_full(stage), phase, abort_flag);
                                vstage = stage;
                                advance();
                                if (ok && x.edge(x.tile(step))) {
                                    ok = mbar_wait(v_fixed(vstage), (fphase >> vstage) & 1u,
                                                   abort_flag);
                                    fphase ^= 1u << vstage;
                                }
                            }
                            ok = ok && mbar_wait(p_ready(s), (pphase >> s) & 1u, abort_flag);
                            if (!ok) break;
                            pphase ^= 1u << s;
                            tc_fence_after();
                            const uint64_t vd =
                                smem_desc_mn128(sbase + C::OFF_KV + vstage * C::TILE, C::BLOCK);
#pragma unroll
                            for (int k = 0; k < kTreeTile / 16; ++k)
                                umma_bf16_ts(tmem + C::TMEM_O + D * s, tmem + 128 * s + 8 * k,
                                             vd + 128u * k, idesc_pv, step != 0 || k != 0);
                            if (s == 1 || cur.two_kv()) umma_commit(kv_empty(vstage));
                            if (x.last(step)) umma_commit(o_full(s));
                        }
                        if (nxt.steps) ok = scores(nxt, nstep, s);
                    }
                    cur = nxt;
                    step = nstep;
                }
                if (!ok && !*abort_flag) {
                    atomicOr(&g_status_word, kStatusMmaTimeout);
                    *abort_flag = 1;
                }
            }
        } else if (warp == 10) {
            // ---- V rows of edge tiles. Every stage is waited for in ring
            // order, K's and those of tiles that need nothing too: a wait on a
            // stage a whole pass ahead would take the pass before for it.
            auto pass = [&] {
                const bool full = warp_wait(kv_full(stage), phase, abort_flag);
                advance();
                return full;
            };
            ok = __all_sync(~0u, fetch(0, cur));
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (ok && cur.steps && own_kv(cur, 0, s)) ok = pass();
            while (ok && cur.steps) {
                const int slot = seq % kTreeEntries;
                ok = __all_sync(~0u, follow());
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!ok) break;
                    if (own_kv(cur, step, s)) {
                        const int at = stage;
                        ok = pass();
                        if (!ok) break;
                        const TreePart &x = cur.part[s];
                        if (x.edge(x.tile(step))) {
                            const int x0 = x.tile(step) * kTreeTile;
                            // rows [first, end) hold new tokens, [end, 128) nothing;
                            // a row's 16-byte chunks are permuted within its 128 bytes
                            const int end = tree_min(x.len - x0, kTreeTile);
                            const int first = tree_min(tree_max(x.ctx - x0, 0), end);
                            bool bad = false;
                            for (int b = 0; b < C::HALVES; ++b) {
                                uint4 *base = reinterpret_cast<uint4 *>(
                                    smem + C::OFF_KV + at * C::TILE + b * C::BLOCK);
                                for (int i = end * 8 + lane; i < kTreeTile * 8; i += 32)
                                    base[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 4
                                for (int i = first * 8 + lane; i < end * 8; i += 32) {
                                    uint4 v = base[i];
                                    uint32_t any = 0;   // exponent all ones: carry
                                    any |= (v.x & 0x7F807F80u) + 0x00800080u;
                                    any |= (v.y & 0x7F807F80u) + 0x00800080u;
                                    any |= (v.z & 0x7F807F80u) + 0x00800080u;
                                    any |= (v.w & 0x7F807F80u) + 0x00800080u;
                                    if (any & 0x80008000u) {
                                        uint32_t *e = reinterpret_cast<uint32_t *>(base + i);
                                        for (int k = 0; k < 4; ++k) {
                                            uint32_t z = e[k];
                                            if ((z & 0x7F80u) == 0x7F80u) z &= 0xFFFF0000u;
                                            if ((z & 0x7F800000u) == 0x7F800000u) z &= 0xFFFFu;
                                            e[k] = z;
                                        }
                                        bad = true;
                                    }
                                }
                            }
                            if (bad) {
                                flags[2 * slot + s] = 1;
                                if (!cur.two_kv()) flags[2 * slot + 1] = 1;
                            }
                            __threadfence_block();
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(v_fixed(at));
                        }
                    }
                    if (nxt.steps && own_kv(nxt, nstep, s)) ok = ok && pass();
                }
                cur = nxt;
                step = nstep;
            }
            if (!ok && lane == 0 && !*abort_flag) {
                atomicOr(&g_status_word, kStatusEpilogueTimeout);
                *abort_flag = 1;
            }
        } else if (lane == 0) {
            // ---- entries, ahead of their use
            TreeWalk w{};
            w.begin(g, *start, load);
            int4 chain = make_int4(0, 0, 0, 0);
            for (bool more = true; more && ok; ++seq) {
                const int i = seq % kTreeEntries;
                const TreeEntry e = w.entry(g, load);
                more = e.steps > 0;
                ok = mbar_wait(e_empty(i), ((seq / kTreeEntries) & 1) ^ 1, abort_flag);
                if (!ok) break;
                entries[i] = e;
                flags[2 * i] = flags[2 * i + 1] = 0;
                mbar_arrive(e_full(i));
                // an item that begins here and goes on in the next blocks
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!more) break;
                    const TreePart &x = e.part[s];
                    if ((x.flags & (kPartWhole | kPartBegins | kPartSecond)) != kPartBegins) continue;
                    const int rest = (x.len + kTreeTile - 1) / kTreeTile - x.end;
                    chain = make_int4(tree_block_of(cut, tree_block_begin(cut, c + 1) + rest - 1),
                                      x.tok, x.h,
                                      x.ntok + (e.kind == kTreePair ? e.part[1].ntok : 0));
                }
            }
            a.chains[c] = chain;
            if (!ok && !*abort_flag) {
                atomicOr(&g_status_word, kStatusProducerTimeout);
                *abort_flag = 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTreeSoftmaxRegs));
        // ---- softmax group s, one thread a row
        const int s = warp >> 2, quad = warp & 3;
        const int row = 32 * quad + lane;
        const int my_tok = row / g.group, my_head = row - my_tok * g.group;
        const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
        const uint32_t ts = tmem + lanes + 128 * s;                  // scores, weights
        const uint32_t to = tmem + lanes + C::TMEM_O + D * s;        // own accumulator
        uint32_t sphase = 0, ophase0 = 0, ophase1 = 0, xphase = 0;
        bool ok = true, merged = false;   // merged: results were shared, o_done is due
        for (int seq = 0;; ++seq) {
            const int slot = seq % kTreeEntries;
            ok = warp_wait(e_full(slot), (seq / kTreeEntries) & 1, abort_flag);
            if (!ok) break;
            const TreeEntry &entry = entries[slot];
            if (entry.steps == 0) break;
            // most of it stays in shared memory: the scores need the registers
            const TreePart &x = entry.part[s];
            const bool warp_on = 32 * quad < x.ntok * g.group;
            const bool row_on = my_tok < x.ntok;
            auto sight = [&] {
                return TreeSight{a.mask ? a.mask + static_cast<long long>(x.tok + my_tok) *
                                                       a.mask_words
                                        : nullptr,
                                 a.mask_words, x.place + my_tok, x.ctx, x.len};
            };
            float m = -INFINITY, l = 0.f;
            bool fresh = true;
            for (int tile = x.first; tile < x.end; tile += x.stride) {
                ok = warp_wait(s_full(s), sphase, abort_flag);
                if (!ok) break;
                sphase ^= 1u;
                if (warp_on) {
                    tc_fence_after();
                    uint32_t v[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, v[i]);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 4; ++i) reg_fence32(v[i]);
                    if (x.edge(tile)) {
                        const TreeSight t = sight();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t see =
                                row_on ? tree_visible(t, tile * kTreeTile + 32 * i) : 0u;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((see >> j) & 1u)) v[i][j] = 0xFF800000u;
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            mx[(j >> 1) & 3] = fmaxf(mx[(j >> 1) & 3],
                                                     fmaxf(__uint_as_float(v[i][j]),
                                                           __uint_as_float(v[i][j + 1])));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (fresh) {
                        m = top;
                        fresh = false;
                    } else {
                        const bool rise = top * a.scale_log2 > m * a.scale_log2 + kTreeRescale;
                        if (__any_sync(~0u, rise && row_on)) {
                            const float f = rise ? ex2((m - top) * a.scale_log2) : 1.f;
                            m = rise ? top : m;
                            l *= f;
#pragma unroll 1
                            for (int i = 0; i < D / 32; ++i) {
                                uint32_t o[32];
                                tmem_ld_32x32b_x32(to + 32 * i, o);
                                tmem_ld_wait();
                                reg_fence32(o);
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st_32x32b_x32(to + 32 * i, o);
                            }
                        }
                    }
                    // an all-masked row so far: weights 2^(-inf - 0) = 0
                    const float base = m == -INFINITY ? 0.f : -m * a.scale_log2;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float lo, hi;
                            fma2(lo, hi, __uint_as_float(v[i][2 * j]),
                                 __uint_as_float(v[i][2 * j + 1]), a.scale_log2, base);
                            lo = ex2(lo);
                            hi = ex2(hi);
                            add2(sum[2 * (j & 1)], sum[2 * (j & 1) + 1], lo, hi);
                            p[j] = pack_bf16x2(lo, hi);
                        }
                        tmem_st_32x32b_x16(ts + 16 * i, p);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                // the accumulator of the entry before has been read by both groups
                if (merged) {
                    ok = warp_wait(o_done(quad), xphase ^ 1u, abort_flag);
                    if (!ok) break;
                    merged = false;
                }
                if (warp_on) {
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready(s));
            }
            if (!ok) break;

            // ---- the entry's end: this block's result
            const bool whole = (x.flags & kPartWhole) != 0;
            // partial results: slot 2c + 1 for an item that begins here, 2c for others
            const long long prow =
                static_cast<long long>(2 * c + ((x.flags & kPartBegins) ? 1 : 0)) * a.part_rows +
                ((x.flags & kPartSecond) ? 128 : 0) + row;
            const bool split = entry.kind == kTreeSplit;
            const bool used1 = entry.part[1].used();
            int first = x.first;              // this block's tiles of the item
            float w0 = 1.f, w1 = 0.f;
            int c0 = 0, c1 = D;               // columns that this thread writes
            if (split) {
                // merge the groups' statistics; each writes half of the columns
                first = entry.part[0].first;
                if (x.used()) row_stats[128 * s + row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(st_ready(quad));
                ok = warp_wait(st_ready(quad), xphase, abort_flag);
                if (!ok) break;
                const float2 a0 = row_stats[row];
                const float2 a1 = used1 ? row_stats[128 + row] : make_float2(-INFINITY, 0.f);
                m = fmaxf(a0.x, a1.x);
                w0 = a0.x == -INFINITY ? 0.f : ex2((a0.x - m) * a.scale_log2);
                w1 = a1.x == -INFINITY ? 0.f : ex2((a1.x - m) * a.scale_log2);
                l = a0.y * w0 + a1.y * w1;
                c0 = s * (D / 2);
                c1 = c0 + D / 2;
            }
            if (split || s == 0) ok = warp_wait(o_full(0), ophase0, abort_flag);
            if (ok && used1 && (split || s == 1)) ok = warp_wait(o_full(1), ophase1, abort_flag);
            if (!ok) break;
            ophase0 ^= 1u;
            if (used1) ophase1 ^= 1u;
            tc_fence_after();
            const bool flagged = flags[2 * slot + s] || (split && flags[2 * slot + (s ^ 1)]);
            if (warp_on) {
                if (!whole && row_on && (!split || s == 0)) a.stats[prow] = make_float2(m, l);
                const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                const uint32_t t0 = tmem + lanes + C::TMEM_O, t1 = t0 + D;
#pragma unroll 1
                for (int col = c0; col < c1; col += 32) {
                    uint32_t o[32];
                    if (!split) {
                        tmem_ld_32x32b_x32(to + col, o);
                        tmem_ld_wait();
                        reg_fence32(o);
                    } else {
                        tmem_ld_32x32b_x32(t0 + col, o);
                        uint32_t y[32];
                        if (used1) tmem_ld_32x32b_x32(t1 + col, y);
                        tmem_ld_wait();
                        reg_fence32(o);
                        if (used1) {
                            reg_fence32(y);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                o[j] = __float_as_uint(fmaf(__uint_as_float(y[j]), w1,
                                                            __uint_as_float(o[j]) * w0));
                        }
                    }
                    if (!row_on) continue;
                    uint16_t *const out = a.out + (static_cast<long long>(x.tok + my_tok) * a.q_heads +
                                                   x.h * g.group + my_head) * D + col;
                    float *const sums = a.partial + prow * D + col;
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(out);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t b[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                b[k] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * k]) * inv,
                                                   __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
                            dst[j] = make_uint4(b[0], b[1], b[2], b[3]);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(sums);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                    if (flagged) {
                        const int x0 = tree_max(x.ctx, first * kTreeTile);
                        const int x1 = tree_min(x.len, x.end * kTreeTile);
                        const long long head_step = static_cast<long long>(D) << a.page_shift;
                        const uint16_t *vc = a.v_cache + x.h * head_step + col;
                        const int *table = a.table + x.r * a.max_pages;
                        if (whole)
                            tree_add_nonfinite<D>(out, sight(), x0, x1, table, a.page_shift,
                                                  a.num_pages, g.kv_heads * head_step, vc);
                        else
                            tree_add_nonfinite<D>(sums, sight(), x0, x1, table, a.page_shift,
                                                  a.num_pages, g.kv_heads * head_step, vc);
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (split) {
                if (lane == 0) mbar_arrive(o_done(quad));
                merged = true;
                xphase ^= 1u;
            }
            if (lane == 0) mbar_arrive(e_empty(slot));
        }
        if (!ok && lane == 0 && !*abort_flag) {
            atomicOr(&g_status_word, kStatusEpilogueTimeout);
            *abort_flag = 1;
        }
    }

    // ---- teardown: every role has left its loop
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 8 && lane == 0) {
            // every TMA load already issued lands before shared memory is reused
            for (int i = 0; i < C::STAGES + 2; ++i)
                if ((issued >> i) & 1u)
                    if (!mbar_wait_drain(i < C::STAGES ? kv_full(i) : q_full(i - C::STAGES),
                                         (parity >> i) & 1u))
                        atomicOr(&g_status_word, kStatusDrainTimeout);
        }
        if (warp == 9 && lane == 0) {
            umma_commit(drain_bar);
            if (!mbar_wait_drain(drain_bar, 0)) atomicOr(&g_status_word, kStatusDrainTimeout);
        }
        __syncthreads();
    }
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- partial results
constexpr int kJoinThreads = 256;

// Items that several blocks worked on: out = sum_b w_b o_b / sum_b w_b l_b,
// w_b = exp(scale * (m_b - max m)), in block order, so that the result does
// not depend on which block finished first. One warp a row; the rows of all
// such items are dealt evenly over the grid's warps, each of which adds up
// the items' row counts for itself.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeAttnArgs a, int blocks) {
    constexpr int V = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int warps = static_cast<int>(gridDim.x) * (kJoinThreads / 32);
    const int tpt = a.geom.tpt, group = a.geom.group;
    // consecutive rows on different SMs
    int task = (threadIdx.x >> 5) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    for (int chunk = 0; chunk < blocks; chunk += 32) {
        // items that begin in blocks chunk .. chunk + 31: last block, first
        // token, head, tokens (0: none)
        const int4 mine = chunk + lane < blocks ? a.chains[chunk + lane] : make_int4(0, 0, 0, 0);
        int upto = mine.w * group;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += x;
        }
        const int rows = __shfl_sync(~0u, upto, 31);
        for (; task < rows; task += warps) {
            const int from = __popc(__ballot_sync(~0u, upto <= task));
            const int c = chunk + from;
            const int last = __shfl_sync(~0u, mine.x, from), tok0 = __shfl_sync(~0u, mine.y, from);
            const int h = __shfl_sync(~0u, mine.z, from), tokens = __shfl_sync(~0u, mine.w, from);
            const int i = task - (__shfl_sync(~0u, upto, from) - tokens * group);
            const int tok = i / group, head = i - tok * group;
            const int rt = tok >= tpt;
            const long long row = 128 * rt + (tok - rt * tpt) * group + head;
            const int parts = last - c + 1;
            // part 0 is the slot of an item that begins in c, the others' of one that goes on
            auto slot = [&](int b) {
                return static_cast<long long>(b == 0 ? 2 * c + 1 : 2 * (c + b)) * a.part_rows + row;
            };
            float top = -INFINITY;
            for (int b = lane; b < parts; b += 32) top = fmaxf(top, a.stats[slot(b)].x);
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            float acc[V] = {}, l = 0.f;
#pragma unroll 4
            for (int b = 0; b < parts; ++b) {
                const float2 st = a.stats[slot(b)];
                const float f = st.x == -INFINITY ? 0.f : ex2((st.x - top) * a.scale_log2);
                const float *o = a.partial + slot(b) * D + V * lane;
                float v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = o[e];
                l = fmaf(st.y, f, l);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(v[e], f, acc[e]);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint32_t *dst = reinterpret_cast<uint32_t *>(
                a.out +
                (static_cast<long long>(tok0 + tok) * a.q_heads + h * group + head) * D + V * lane);
#pragma unroll
            for (int e = 0; e < V / 2; ++e)
                dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        }
        task -= rows;
    }
}

}  // namespace swiglu
