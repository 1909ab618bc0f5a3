// Attention of a step's new tokens over the paged cache.
//
//   o[t, h] = sum_x p_x v_x / sum_x p_x,   p_x = exp(scale * q[t, h] . k_x - max)
//
// over the positions x that token t of request r sees: the request's context
// (x < c) and, of the step's own tokens (x = c + j), those whose bit j is set
// in the token's mask words (without a mask: j <= t's own place). A row that
// sees nothing, or only scores of -inf, is zero. Sums and statistics are
// FP32; the result is rounded once to BF16.
#pragma once

#include <cuda_bf16.h>

#include "sm103_ptx.cuh"

namespace swiglu {

struct TreeAttnArgs {
    const uint16_t *q;                 // [tokens][q heads][D], strides in elements
    const uint16_t *k_cache, *v_cache; // [pages][kv heads][page rows][D]
    const int *table;                  // [requests][max_pages]
    const int *ctx_lens;               // [requests]
    const int *query_start;            // [requests + 1]
    const unsigned long long *mask;    // [tokens][mask_words], or null
    uint16_t *out;                     // [tokens][q heads][D]
    long long q_tok, q_head;
    long long max_pages, num_pages;
    float scale;
    int tokens, requests, q_heads, kv_heads, page_shift, mask_words;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

constexpr int kRowAttnThreads = 128;

// One warp a (token, q head): lane i holds D / 32 values of q and of the sum.
template <int D>
__global__ void __launch_bounds__(kRowAttnThreads) tree_attention_rows_kernel(const TreeAttnArgs a) {
    constexpr int V = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    const long long row = static_cast<long long>(blockIdx.x) * (kRowAttnThreads / 32) +
                          (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= static_cast<long long>(a.tokens) * a.q_heads) return;
    const int t = static_cast<int>(row / a.q_heads), h = static_cast<int>(row % a.q_heads);
    float acc[V] = {}, q[V], m = -INFINITY, l = 0.f;
    int r = -1, ctx = 0, n = 0, i = 0;
    if (a.requests > 0 && t < a.query_start[a.requests]) {
        int lo = 0, hi = a.requests;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.query_start[mid] <= t) lo = mid; else hi = mid;
        }
        r = lo;
        ctx = max(a.ctx_lens[r], 0);
        i = t - a.query_start[r];
        n = a.query_start[r + 1] - a.query_start[r];
    }
    const int kh = h / (a.q_heads / a.kv_heads);
#pragma unroll
    for (int e = 0; e < V; ++e)
        q[e] = bf16_lo(a.q[t * a.q_tok + h * a.q_head + V * lane + e]) * a.scale;
    const long long L = r < 0 ? 0 : min(static_cast<long long>(ctx) + n,
                                        a.max_pages << a.page_shift);
    for (long long x = 0; x < L; ++x) {
        if (x >= ctx) {
            const int j = static_cast<int>(x - ctx);
            const bool see = a.mask ? (j >> 6) < a.mask_words &&
                                          (a.mask[static_cast<long long>(t) * a.mask_words +
                                                  (j >> 6)] >> (j & 63) & 1)
                                    : j <= i;
            if (!see) continue;
        }
        const long long page = a.table[r * a.max_pages + (x >> a.page_shift)];
        if (page < 0 || page >= a.num_pages) continue;
        const long long at =
            ((((page * a.kv_heads + kh) << a.page_shift) + (x & ((1 << a.page_shift) - 1))) * D) +
            V * lane;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) s += q[e] * bf16_lo(a.k_cache[at + e]);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        const float m_new = fmaxf(m, s);
        if (m_new == -INFINITY && s == s) continue;
        const float keep = __expf(m - m_new), p = __expf(s - m_new);
        m = m_new;
        l = l * keep + p;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = acc[e] * keep + p * bf16_lo(a.v_cache[at + e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const __nv_bfloat16 o = __float2bfloat16_rn(acc[e] * inv);
        a.out[row * D + V * lane + e] = *reinterpret_cast<const uint16_t *>(&o);
    }
}

}  // namespace swiglu
