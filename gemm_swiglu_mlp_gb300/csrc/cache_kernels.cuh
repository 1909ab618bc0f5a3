// The paged key/value cache of a serving step: block tables, slot map,
// positions and tree masks from the requests' lengths (cache_plan_kernel),
// the step's new rows into the cache (cache_write_kernel), and the accepted
// path's rows moved behind the context (cache_accept_kernel).
//
// Cache: K and V each [pages][kv heads][page rows][head size] BF16, so one
// page of one head is a contiguous block (4 KB at 16 rows of 128) that the
// attention kernel fetches as one 5-D tensor-map box. Position
// x of request r is row x % P of page table[r][x / P]; its slot is
// page * P + x % P.
#pragma once

#include <climits>

#include "sm103_ptx.cuh"

namespace swiglu {

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 512;
// Requests of one plan: two 4-byte prefix sums a request in shared memory.
constexpr int kPlanMaxRequests = 16384;

struct CachePlanArgs {
    const int *ctx_lens, *new_lens, *pages_held;   // [requests]
    int *table;                                    // [requests][max_pages]
    const int *free_pages;                         // [num_free]
    const int *free_head;                          // first unused entry; null: 0
    const int *parents;                            // [requests][tree_width]; null: chains
    int *query_start;                              // [requests + 1]
    int *slots, *positions;                        // [max_tokens]
    int *held_out;                                 // [requests]
    int *counts;                                   // [3]
    unsigned long long *mask;                      // [max_tokens][mask_words]
    long long max_pages, num_free;
    int requests, page_shift, tree_width, mask_words, max_tokens;
};

__device__ __forceinline__ int saturate_int(long long v) {
    return v > INT_MAX ? INT_MAX : static_cast<int>(v);
}

// New tokens of request r: none for a negative count, no more than the tree
// has columns.
__device__ __forceinline__ int plan_new_tokens(const CachePlanArgs &a, int r) {
    int n = max(a.new_lens[r], 0);
    return a.parents ? min(n, a.tree_width) : n;
}

// Pages a request holds, and the pages it wants after this step.
__device__ __forceinline__ int plan_held(const CachePlanArgs &a, int r) {
    return static_cast<int>(min(static_cast<long long>(max(a.pages_held[r], 0)), a.max_pages));
}
__device__ __forceinline__ int plan_wanted(const CachePlanArgs &a, int r, int n, int held) {
    const long long rows = static_cast<long long>(max(a.ctx_lens[r], 0)) + n;
    const long long pages = (rows + (1ll << a.page_shift) - 1) >> a.page_shift;
    return max(held, static_cast<int>(min(pages, a.max_pages)));
}

// Every block computes both prefix sums over the requests (tokens, new
// pages) for itself in shared memory: a few loads a thread, against a second
// launch or a wait between blocks. Then tokens are spread over all threads of
// the grid and requests' new pages over its warps. A chain of dependent loads
// bounds it (lengths, the request's table, the parents up a tree), not the bytes:
// 64 requests of one token 3.5 us, 192 trees of up to 60 tokens 5.3, of which an
// empty launch is 2.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const CachePlanArgs a) {
    extern __shared__ int plan_smem[];
    int *start = plan_smem;                    // [requests + 1]
    int *first = plan_smem + a.requests + 1;   // [requests]: new pages of earlier requests
    __shared__ long long warp_tok[kPlanThreads / 32], warp_pag[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    griddep_wait();
    const long long head = a.free_head ? max(*a.free_head, 0) : 0;

    // this thread's requests [r0, r1), their sums, and the sums before them
    const int per = (a.requests + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
    long long tok = 0, pag = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = plan_new_tokens(a, r), held = plan_held(a, r);
        tok += n;
        pag += plan_wanted(a, r, n, held) - held;
    }
    long long tok_in = tok, pag_in = pag;   // inclusive over the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(~0u, tok_in, d), y = __shfl_up_sync(~0u, pag_in, d);
        if (lane >= d) {
            tok_in += x;
            pag_in += y;
        }
    }
    if (lane == 31) {
        warp_tok[warp] = tok_in;
        warp_pag[warp] = pag_in;
    }
    __syncthreads();
    long long tok_at = tok_in - tok, pag_at = pag_in - pag, tok_all = 0, pag_all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            tok_at += warp_tok[w];
            pag_at += warp_pag[w];
        }
        tok_all += warp_tok[w];
        pag_all += warp_pag[w];
    }
    for (int r = r0; r < r1; ++r) {
        const int n = plan_new_tokens(a, r), held = plan_held(a, r);
        start[r] = saturate_int(tok_at);
        first[r] = saturate_int(pag_at);
        tok_at += n;
        pag_at += plan_wanted(a, r, n, held) - held;
    }
    if (tid == 0) start[a.requests] = saturate_int(tok_all);
    __syncthreads();

    const long long avail = max(a.num_free - head, 0ll);
    if (blockIdx.x == 0) {
        for (int r = tid; r <= a.requests; r += kPlanThreads) a.query_start[r] = start[r];
        if (tid == 0) {
            a.counts[0] = saturate_int(tok_all);
            a.counts[1] = saturate_int(pag_all);
            a.counts[2] = saturate_int(head + min(pag_all, avail));
        }
    }

    // new pages, one warp a request
    const int warps = static_cast<int>(gridDim.x) * (kPlanThreads / 32);
    for (int r = static_cast<int>(blockIdx.x) * (kPlanThreads / 32) + warp; r < a.requests;
         r += warps) {
        const int held = plan_held(a, r);
        const int want = plan_wanted(a, r, plan_new_tokens(a, r), held) - held;
        int *row = a.table + static_cast<long long>(r) * a.max_pages + held;
        const long long from = first[r];
        for (int i = lane; i < want; i += 32)
            row[i] = from + i < avail ? a.free_pages[head + from + i] : -1;
        if (lane == 0)
            a.held_out[r] =
                held + static_cast<int>(min(static_cast<long long>(want), max(avail - from, 0ll)));
    }

    // tokens, one thread each
    const int total = start[a.requests];
    const long long page_rows = 1ll << a.page_shift;
    for (long long t64 = static_cast<long long>(blockIdx.x) * kPlanThreads + tid;
         t64 < a.max_tokens; t64 += static_cast<long long>(gridDim.x) * kPlanThreads) {
        const int t = static_cast<int>(t64);
        unsigned long long *words = a.mask + t64 * a.mask_words;
        if (t >= total) {   // past the last request: no slot, sees nothing
            a.slots[t] = -1;
            a.positions[t] = 0;
            for (int w = 0; w < a.mask_words; ++w) words[w] = 0;
            continue;
        }
        int lo = 0, hi = a.requests;   // the last request with start <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= t) lo = mid; else hi = mid;
        }
        const int r = lo, i = t - start[r];
        const int ctx = max(a.ctx_lens[r], 0), held = plan_held(a, r);
        const long long x = static_cast<long long>(ctx) + i, p = x >> a.page_shift;
        long long page = -1;
        if (p < held)
            page = a.table[static_cast<long long>(r) * a.max_pages + p];
        else if (p < a.max_pages && first[r] + (p - held) < avail)
            page = a.free_pages[head + first[r] + (p - held)];
        const long long slot = page * page_rows + (x & (page_rows - 1));
        a.slots[t] = page >= 0 && slot <= INT_MAX ? static_cast<int>(slot) : -1;
        int depth = i;
        if (a.parents) {
            const int *par = a.parents + static_cast<long long>(r) * a.tree_width;
            // up the tree: an index only ever falls, so the walk ends
            for (int w = 0; w < a.mask_words; ++w) {
                unsigned long long bits = 0;
                int steps = 0;
                for (int j = i;; ++steps) {
                    if ((j >> 6) == w) bits |= 1ull << (j & 63);
                    const int up = par[j];
                    if (up < 0 || up >= j) break;
                    j = up;
                }
                words[w] = bits;
                depth = steps;
            }
        }
        a.positions[t] = saturate_int(static_cast<long long>(ctx) + depth);
    }
}

// ---------------------------------------------------------------- write
constexpr int kWriteThreads = 256;

struct CacheWriteArgs {
    const uint4 *k, *v;                // rows of head_size values, strides below
    uint4 *k_cache, *v_cache;
    const int *slots;                  // [tokens]; out of range: the row is dropped
    long long k_tok, k_head, v_tok, v_head;   // strides in 16-byte chunks
    long long num_slots;
    int tokens, kv_heads, row_shift, page_shift;   // 2^row_shift chunks a row
    int tokens_per_block;
};

// One 16-byte chunk of K and the same one of V a thread: both loads are in
// flight before either store; consecutive threads take consecutive chunks of
// a row on both sides (128 or 256 contiguous bytes). Its bytes bound it: 10
// prompts of up to 2000 tokens, 8 kv heads of 128, 22.6 us, 6.2 TB/s read and
// written; small calls are an empty launch's 2 us.
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const CacheWriteArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int row = 1 << a.row_shift;
    const int per_token = a.kv_heads << a.row_shift;
    const int t0 = static_cast<int>(blockIdx.x) * a.tokens_per_block;
    const int count = min(a.tokens_per_block, a.tokens - t0) * per_token;
    for (int i = threadIdx.x; i < count; i += kWriteThreads) {
        const int tl = i / per_token, rest = i - tl * per_token;
        const int h = rest >> a.row_shift, c = rest & (row - 1);
        const long long t = t0 + tl;
        const int slot = a.slots[t];
        const uint4 kx = a.k[t * a.k_tok + h * a.k_head + c];
        const uint4 vx = a.v[t * a.v_tok + h * a.v_head + c];
        if (slot < 0 || slot >= a.num_slots) continue;
        const long long page = slot >> a.page_shift;
        const int off = slot & ((1 << a.page_shift) - 1);
        const long long at =
            ((((page * a.kv_heads + h) << a.page_shift) + off) << a.row_shift) + c;
        a.k_cache[at] = kx;
        a.v_cache[at] = vx;
    }
}

// ---------------------------------------------------------------- accept
constexpr int kAcceptThreads = 128;
constexpr int kAcceptBatch = 8;    // rows loaded before any of them is stored

struct CacheAcceptArgs {
    uint4 *k_cache, *v_cache;          // [layers][pages][kv heads][page rows][head size]
    const int *table, *ctx_lens, *paths, *path_lens;
    int *ctx_out;
    long long max_pages, num_pages;
    long long layer_chunks;            // 16-byte chunks of one layer's cache
    long long columns;                 // layers * 2 * kv heads * chunks a row
    int path_width, kv_heads, row_shift, page_shift;
};

// Row c + i of a request takes the old value of row c + path[i], in every
// layer and head of K and V. A thread owns whole columns (one 16-byte chunk
// of one head of one cache) and walks the path in order. Paths increase, so
// path[j] >= j > i for j > i: no row is written before it has been read,
// neither within a batch (all of its loads come first) nor by an earlier one.
// The addresses (path, then table, then rows) are its time, not the bytes: one
// layer of 8 requests 2.3 us, 28 layers of 48 requests 3.5.
__global__ void __launch_bounds__(kAcceptThreads) cache_accept_kernel(const CacheAcceptArgs a) {
    __shared__ long long src[32], dst[32];   // chunk offsets at head 0 of a layer
    __shared__ int moves;
    griddep_launch_dependents();
    griddep_wait();
    const int r = blockIdx.x, tid = threadIdx.x;
    const long long ctx = max(a.ctx_lens[r], 0);
    const int len = min(max(a.path_lens[r], 0), a.path_width);
    if (blockIdx.y == 0 && tid == 0) a.ctx_out[r] = saturate_int(ctx + len);
    const int *table = a.table + static_cast<long long>(r) * a.max_pages;
    const int *path = a.paths + static_cast<long long>(r) * a.path_width;
    const int row = 1 << a.row_shift;
    const long long head_chunks = 1ll << (a.page_shift + a.row_shift);

    // chunk offset of a position's row at head 0, or -1
    auto place = [&](long long x) -> long long {
        const long long p = x >> a.page_shift;
        if (p >= a.max_pages) return -1;
        const long long page = table[p];
        if (page < 0 || page >= a.num_pages) return -1;
        return page * a.kv_heads * head_chunks +
               ((x & ((1ll << a.page_shift) - 1)) << a.row_shift);
    };
    for (int base = 0; base < len; base += 32) {
        __syncthreads();
        if (tid < 32) {
            const int i = base + tid;
            const int from = i < len ? path[i] : -1;
            long long s = -1, d = -1;
            if (from > i) {
                s = place(ctx + from);
                d = place(ctx + i);
            }
            const bool move = s >= 0 && d >= 0;
            const unsigned who = __ballot_sync(~0u, move);
            if (move) {
                const int at = __popc(who & ((1u << tid) - 1));
                src[at] = s;
                dst[at] = d;
            }
            if (tid == 0) moves = __popc(who);
        }
        __syncthreads();
        const int m = moves;
        if (m == 0) continue;
        for (long long col = static_cast<long long>(blockIdx.y) * kAcceptThreads + tid;
             col < a.columns; col += static_cast<long long>(gridDim.y) * kAcceptThreads) {
            const int c = static_cast<int>(col & (row - 1));
            const long long lh = col >> a.row_shift;         // (layer, cache, head)
            const long long lc = lh / a.kv_heads;
            const int h = static_cast<int>(lh - lc * a.kv_heads);
            uint4 *cache = ((lc & 1) ? a.v_cache : a.k_cache) + (lc >> 1) * a.layer_chunks +
                           h * head_chunks + c;
            for (int b = 0; b < m; b += kAcceptBatch) {
                uint4 x[kAcceptBatch];
#pragma unroll
                for (int u = 0; u < kAcceptBatch; ++u)
                    if (b + u < m) x[u] = cache[src[b + u]];
#pragma unroll
                for (int u = 0; u < kAcceptBatch; ++u)
                    if (b + u < m) cache[dst[b + u]] = x[u];
            }
        }
    }
}

}  // namespace swiglu
