// Verification of drafted tokens against the target's probabilities, from
// given random numbers. Request r brings a tree of tokens (token 0 is known to
// hold); from the last token that holds, node a, its children are tried in
// the order of their indices:
//
//   w = p_a, Z = 1            what is left of the target's distribution, and its sum
//   child c, token x: holds if u_c * q_a(x) * Z < w(x)
//   else                      w = max(w - Z q_a, 0), Z = sum of w
//
// (q_a: what the children were drawn from; without it, 1 at x and 0 elsewhere. A w
// that would sum to 0 stays as it was.) When no child holds, the token that
// follows is drawn from w: the least i whose w_0 + .. + w_i exceeds u_0 * sum of w.
// The tokens that come out are distributed as the target's own.
//
// As max(max(p - b, 0) - c, 0) = max(p - b - c, 0) for c >= 0, the w after
// several refusals is max(p - S q, 0) with S the sum of the Zs so far: one row of p
// and one of q are all there is to read, whatever the number of children.
//
// Sums are whole units of 2^-50 between lanes: with 32-bit sums (2^-24) one draw in
// some hundreds would give a neighbour of the token. A lane adds its values up as pairs of
// FP32 numbers, each addition's error kept: conversions of every value to a 64-bit integer,
// which go at a rate of two a clock and SM, were most of the time of a batch (64 rows of 128000
// 52 us), and digits taken off by additions of constants half as many instructions again as
// the pairs. The pairs' second numbers are rounded: by at most 2^-43 of the lane's sum for the
// 16 values between two settlings, 2^-36 for the 2048 values that a lane has of 2^20 over one
// CTA; the lanes' own units come to 2^-37 and the draw's to 2^-38 more. So a row's borders are
// held to 2^-35, and those of a softmax's rows, whose roundings go both ways, to about
// 2^-44 (without settling a row of .55 and 2^20 equal values was off by 2^-31).
//
// Measured (device time): 64 chains of 6 over 128000 values with a draft 17.5 us, of which the rows
// that are read (45 MB) need 6.7 at the copy rate; 32 trees of 60 over 152000 without one 18.1
// (several rows one after the other); one chain of 5 over 32000 6.8; greedy 2.6. About 8 us are
// the launch, three dependent loads before the walk (starts, tokens, their probabilities), the
// exchange of the sums and the draw, each waiting for the one before.
#pragma once

#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "verify_split.cuh"

namespace swiglu {

constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxWidth = 4096;    // tokens a request: the tree lies in shared memory
constexpr int kVerifyMaxVocab = 1 << 20;
constexpr int kVerifyUnroll = 4;         // loads of p (and q) a lane has in flight, 4 values each

struct VerifyArgs {
    const int *tokens;                   // [rows]
    const int *query_start;              // [requests + 1]
    const int *parents;                  // [requests][width]; null: chains
    const void *target, *draft;          // [rows][vocab] FP32 or BF16; draft may be null
    const int *following;                // [rows]: the target's greedy tokens (greedy kernel)
    const float *uniform;                // [rows]
    int *paths, *path_lens, *next;       // [requests][width], [requests], [requests]
    long long target_stride, draft_stride;
    int rows, width, vocab;
#ifdef SWIGLU_TEST_FAULT_INJECTION
    int skip_first_fill;                 // test build only: a cluster's last CTA sends nothing
#endif
};

// Request r's rows: [first, first + n), inside the arrays whatever query_start says.
__device__ __forceinline__ int verify_tokens(const VerifyArgs &a, int r, int *first) {
    const int t0 = a.query_start[r], t1 = a.query_start[r + 1];
    *first = t0;
    if (t0 < 0 || t0 >= a.rows || t1 <= t0) return 0;
    return min(min(t1, a.rows) - t0, a.width);
}

// Parent of token i (an earlier one of the request), or -1.
__device__ __forceinline__ int verify_parent(const VerifyArgs &a, int r, int i) {
    const int p = a.parents ? a.parents[static_cast<long long>(r) * a.width + i] : i - 1;
    return p >= 0 && p < i ? p : -1;
}

// The next token after `from` whose parent is `cur`, or n. All 32 lanes.
__device__ __forceinline__ int verify_child(const int *parent, int from, int n, int cur, int lane) {
    for (int j = from + 1; j < n; j += 32) {
        const unsigned hit = __ballot_sync(~0u, j + lane < n && parent[j + lane] == cur);
        if (hit) return j + __ffs(hit) - 1;
    }
    return n;
}

__device__ __forceinline__ float verify_load(const float *p) { return __ldg(p); }
__device__ __forceinline__ float verify_load(const __nv_bfloat16 *p) {
    return __bfloat162float(__ldg(p));
}

// f in units of 2^-50, |f| < 2^9, by 32-bit conversions.
__device__ __forceinline__ long long verify_fixed(float f) {
    const float x = f * 0x1p22f;
    const int high = __float2int_rn(x);
    const int low = __float2int_rn((x - static_cast<float>(high)) * 0x1p28f);
    return (static_cast<long long>(high) << 28) + low;
}
// s + c in units of 2^-50, s >= 0 and |c| small beside it (or both nearly 0); at most 2^8.
__device__ __forceinline__ unsigned long long verify_units(float s, float c) {
    const long long u = verify_fixed(fminf(s, 0x1p8f)) + verify_fixed(c);
    return u > 0 ? static_cast<unsigned long long>(u) : 0;
}
// Sums over a warp, by 32-bit sums of 22 bits at a time. (At most 2^9 = 2^59 units: only rows that
// are no probabilities come to more, and no sum of up to 32 such sums passes 64 bits.)
__device__ __forceinline__ unsigned long long verify_warp_sum(unsigned long long x) {
    const unsigned a = __reduce_add_sync(~0u, static_cast<unsigned>(x) & 0x3FFFFFu);
    const unsigned b = __reduce_add_sync(~0u, static_cast<unsigned>(x >> 22) & 0x3FFFFFu);
    const unsigned c = __reduce_add_sync(~0u, static_cast<unsigned>(x >> 44));
    const unsigned long long sum = a + (static_cast<unsigned long long>(b) << 22) +
                                   (static_cast<unsigned long long>(c) << 44);
    return min(sum, 1ull << 59);
}
// The first lane whose values up to it and its own come to more than `want`, and `want` less those
// before it. Where rounding leaves no such lane (or none at all: -1), the last that has any.
__device__ __forceinline__ int verify_pick(unsigned long long x, unsigned long long *want, int lane) {
    unsigned long long in = x;           // inclusive over the lanes
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(~0u, in, d);
        if (lane >= d) in += y;
    }
    const unsigned over = __ballot_sync(~0u, in > *want), some = __ballot_sync(~0u, x > 0);
    const int at = over ? __ffs(over) - 1 : 31 - __clz(some);
    const unsigned long long before = __shfl_sync(~0u, in - x, at & 31);
    const unsigned long long own = __shfl_sync(~0u, x, at & 31);
    *want = over ? *want - before : own - 1;
    return some ? at : -1;
}

// Stores v to a CTA of the cluster and counts its 8 bytes on that CTA's barrier.
__device__ __forceinline__ void st_async_u64(uint32_t addr, unsigned long long v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(
                     addr),
                 "l"(v), "r"(bar)
                 : "memory");
}

// A sum of values as a pair of FP32 numbers.
struct VerifySum {
    float s, c;
    // Adds w + e, |e| at most half of w's last place: w exactly, by the error of its addition.
    __device__ __forceinline__ void add(float w, float e) {
        const float t = __fadd_rn(s, w), v = __fsub_rn(t, s);
        const float err = __fadd_rn(__fsub_rn(s, __fsub_rn(t, v)), __fsub_rn(w, v));
        s = t;
        c = __fadd_rn(c, __fadd_rn(err, e));
    }
    // The pair with s as near to the sum as it gets, so that c is small and its own additions lose
    // less: over n values without it c grows by n half steps of s and loses n^2 2^-50.
    __device__ __forceinline__ void settle() {
        const float t = __fadd_rn(s, c);
        c = __fsub_rn(c, __fsub_rn(t, s));
        s = t;
    }
    __device__ __forceinline__ unsigned long long units() const { return verify_units(s, c); }
};

// What is left of the target's row at one value: max(p - S q, 0), probabilities clamped to
// [0, 1], NaN as 0.
template <typename T>
struct VerifyLeft {
    const T *p, *q;                      // rows of the node; q null: no draft, or nothing refused
    float S, S_low;                      // sum of the Zs, as a pair; 1 after the first refusal
    // DRAFT: 0 without q, 1 with S = 1, 2 with any S
    template <int DRAFT>
    __device__ __forceinline__ void pair(float pv, float qv, float &w, float &e) const {
        w = __saturatef(pv);
        e = 0.f;
        if (DRAFT == 0) return;
        const float p1 = w, q1 = __saturatef(qv);
        const float y = DRAFT == 1 ? q1 : __fmul_rn(S, q1);
        const float d = __fsub_rn(p1, y);
        e = __fsub_rn(__fsub_rn(p1, d), y);       // exact where d >= 0
        if (DRAFT == 2) e = __fsub_rn(e, __fmaf_rn(S_low, q1, __fmaf_rn(S, q1, -y)));
        const bool some = d > 0.f && (DRAFT == 1 || __fadd_rn(d, e) > 0.f);
        w = some ? d : 0.f;
        e = some ? e : 0.f;
    }
    __device__ __forceinline__ int draft() const { return !q ? 0 : S == 1.f && S_low == 0.f ? 1 : 2; }
    // (with q or without)
    __device__ __forceinline__ float2 both(float pv, float qv) const {
        float w, e;
        if (q)
            pair<2>(pv, qv, w, e);
        else
            pair<0>(pv, qv, w, e);
        return make_float2(w, e);
    }
    __device__ __forceinline__ unsigned long long at(float pv, float qv) const {
        const float2 w = both(pv, qv);
        return verify_units(w.x, w.y);
    }
};

// Four values in a row from [lo, hi), 0 past its end; VEC: the row is aligned to them.
template <bool VEC>
__device__ __forceinline__ float4 verify_load4(const float *row, int i, int hi) {
    if (VEC && i + 4 <= hi) return __ldg(reinterpret_cast<const float4 *>(row + i));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < hi) v.x = __ldg(row + i);
    if (i + 1 < hi) v.y = __ldg(row + i + 1);
    if (i + 2 < hi) v.z = __ldg(row + i + 2);
    if (i + 3 < hi) v.w = __ldg(row + i + 3);
    return v;
}
template <bool VEC>
__device__ __forceinline__ float4 verify_load4(const __nv_bfloat16 *row, int i, int hi) {
    if (VEC && i + 4 <= hi) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(row + i));
        return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                           __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < hi) v.x = verify_load(row + i);
    if (i + 1 < hi) v.y = verify_load(row + i + 1);
    if (i + 2 < hi) v.z = verify_load(row + i + 2);
    if (i + 3 < hi) v.w = verify_load(row + i + 3);
    return v;
}

// This lane's sum over [lo, hi), a warp's range; lanes in a row have four values each in a row.
template <bool VEC, int DRAFT, typename T>
__device__ __forceinline__ unsigned long long verify_range(const VerifyLeft<T> &left, int lo, int hi,
                                                           int lane) {
    VerifySum sum{0.f, 0.f};
    for (int base = lo + 4 * lane; base < hi; base += 128 * kVerifyUnroll) {
        float4 p[kVerifyUnroll], q[kVerifyUnroll];
#pragma unroll
        for (int u = 0; u < kVerifyUnroll; ++u) {
            p[u] = verify_load4<VEC>(left.p, base + 128 * u, hi);
            if (DRAFT) q[u] = verify_load4<VEC>(left.q, base + 128 * u, hi);
        }
#pragma unroll
        for (int u = 0; u < kVerifyUnroll; ++u) {
            float w[4], e[4];
            left.template pair<DRAFT>(p[u].x, q[u].x, w[0], e[0]);
            left.template pair<DRAFT>(p[u].y, q[u].y, w[1], e[1]);
            left.template pair<DRAFT>(p[u].z, q[u].z, w[2], e[2]);
            left.template pair<DRAFT>(p[u].w, q[u].w, w[3], e[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum.add(w[i], e[i]);
        }
        sum.settle();
    }
    return sum.units();
}

// What is left at value i < hi (0 past it, and at the `skips` values of skip), as a pair.
template <typename T>
__device__ __forceinline__ float2 verify_pair(const VerifyLeft<T> &left, int i, int hi, const int *skip,
                                              int skips) {
    if (i >= hi) return make_float2(0.f, 0.f);
    for (int j = 0; j < skips; ++j)
        if (skip[j] == i) return make_float2(0.f, 0.f);
    return left.both(verify_load(left.p + i), left.q ? verify_load(left.q + i) : 0.f);
}
template <typename T>
__device__ __forceinline__ unsigned long long verify_value(const VerifyLeft<T> &left, int i, int hi,
                                                           const int *skip, int skips) {
    const float2 w = verify_pair(left, i, hi, skip, skips);
    return verify_units(w.x, w.y);
}

// The first value of [lo, hi) of which anything is left, or -1. All 32 lanes.
template <typename T>
__device__ __noinline__ int verify_first(const VerifyLeft<T> &left, int lo, int hi, const int *skip,
                                         int skips, int lane) {
    for (int base = lo; base < hi; base += 32) {
        const float w = verify_pair(left, base + lane, hi, skip, skips).x;
        const unsigned some = __ballot_sync(~0u, w > 0.f);
        if (some) return base + __ffs(some) - 1;
    }
    return -1;
}

// What warp 0 wants of its CTA's warps.
template <typename T>
struct VerifyOrder {
    VerifyLeft<T> left;
    int piece;      // -1: sums of every warp's piece of the row; else: of parts of that piece; -2: end
    int skips;
};

// One cluster a request; each CTA's warps have a piece of the row each, in the order of the
// vocabulary. Warp 0 of every CTA walks the tree, from shared memory, and comes to the same
// results; when it needs the sum of a row, all warps sum their pieces, and the CTAs send
// each other their sums (each knows then where its own begins: a draw falls into one of them).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyArgs a) {
    extern __shared__ int verify_smem[];
    __shared__ unsigned long long warp_sum[kVerifyWarps], part_sum[kVerifyWarps];
    __shared__ unsigned long long cta_sum[2][kVerifyMaxCluster];
    __shared__ unsigned long long arrived[2];   // barriers: the cluster's sums of one pass
    __shared__ VerifyOrder<T> order;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    int ctas;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int r = static_cast<int>(blockIdx.x) / ctas;
    int *parent = verify_smem, *token = parent + a.width, *skip = token + a.width;
    float *up = reinterpret_cast<float *>(skip + a.width), *uq = up + a.width, *uu = uq + a.width;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&arrived[0]), 1);
        mbar_init(smem_u32(&arrived[1]), 1);
        fence_barrier_init();
    }
    cluster_arrive();
    griddep_launch_dependents();
    griddep_wait();

    const T *target = static_cast<const T *>(a.target);
    const T *draft = static_cast<const T *>(a.draft);
    int first;
    const int n = verify_tokens(a, r, &first);
    for (int i = threadIdx.x; i < n; i += kVerifyThreads) {
        const int x = a.tokens[first + i], p = verify_parent(a, r, i);
        const bool known = x >= 0 && x < a.vocab;
        parent[i] = p;
        token[i] = known ? x : -1;
        uu[i] = fminf(__saturatef(a.uniform[first + i]), 1.f - 0x1p-24f);
        float pv = 0.f, qv = 1.f;
        if (p >= 0 && known) {
            pv = verify_load(target + (first + p) * a.target_stride + x);
            if (draft) qv = verify_load(draft + (first + p) * a.draft_stride + x);
        }
        up[i] = __saturatef(pv);
        uq[i] = __saturatef(qv);
    }
    const int pieces = ctas * kVerifyWarps;
    const int piece = ((a.vocab + pieces - 1) / pieces + 3) & ~3;   // (whole vectors)
    const int part = (piece + kVerifyWarps - 1) / kVerifyWarps;     // of a piece, a warp's
    __syncwarp();
    cluster_wait();                          // the cluster's CTAs run, their barriers are there
    __syncthreads();                         // (and this one's tree)

    // this warp's share of an order, its sum to warp_sum or part_sum
    auto obey = [&] {
        const VerifyLeft<T> left = order.left;
        const int of = order.piece;
        if (of < 0) {
            const int lo = min((rank * kVerifyWarps + warp) * piece, a.vocab);
            const int hi = min(lo + piece, a.vocab), form = left.draft();
            const unsigned long long s = form == 0   ? verify_range<VEC, 0>(left, lo, hi, lane)
                                         : form == 1 ? verify_range<VEC, 1>(left, lo, hi, lane)
                                                     : verify_range<VEC, 2>(left, lo, hi, lane);
            const unsigned long long all = verify_warp_sum(s);
            if (lane == 0) warp_sum[warp] = all;
        } else {
            const int b0 = of * piece + warp * part;
            const int b1 = min(min(b0 + part, (of + 1) * piece), a.vocab);
            unsigned long long s = 0;
            for (int i = b0 + lane; i < b1; i += 32)
                s += verify_value(left, i, b1, skip, order.skips);
            s = verify_warp_sum(s);
            if (lane == 0) part_sum[warp] = s;
        }
    };
    if (warp != 0) {
        while (true) {
            __syncthreads();                 // an order
            if (order.piece == -2) return;
            obey();
            __syncthreads();                 // obeyed
        }
    }

    // ---- warp 0
    auto command = [&](const VerifyLeft<T> &left, int of, int skips) {
        if (lane == 0) {
            order.left = left;
            order.piece = of;
            order.skips = skips;
        }
        __syncthreads();
        if (of == -2) return;
        obey();
        __syncthreads();
    };
    int *path = a.paths + static_cast<long long>(r) * a.width;
    const bool writes = rank == 0 && lane == 0;
    int cur = 0, len = n > 0 ? 1 : 0, at = 0;   // node, tokens that hold, last child tried
    if (writes && n > 0) path[0] = 0;
    int skips = 0, pass = 0;
    bool summed = false;                     // the sums are those of the present w
    bool counts = false;                     // Z is the sum of w (else it counts as one)
    unsigned long long Z = 0, S = 0;         // in units; S: sum of the Zs of the refusals
    VerifyLeft<T> left{nullptr, nullptr, 0.f, 0.f};
    const int never = 0;
    bool gave_up = false;                    // a wait ran out (reported as such)

    // sum of w over the row, every CTA's in cta_sum[(pass - 1) & 1]
    auto sum_row = [&]() -> unsigned long long {
        command(left, -1, 0);
        const unsigned long long all = verify_warp_sum(lane < kVerifyWarps ? warp_sum[lane] : 0);
        unsigned long long *sums = cta_sum[pass & 1];
        if (ctas == 1) {
            if (lane == 0) sums[0] = all;
            __syncwarp();
        } else {
            const uint32_t bar = smem_u32(&arrived[pass & 1]);
            if (lane == 0) mbar_arrive_expect_tx(bar, 8u * static_cast<uint32_t>(ctas));
            __syncwarp();
            bool sends = lane < ctas;
#ifdef SWIGLU_TEST_FAULT_INJECTION
            sends = sends && !(a.skip_first_fill && rank == ctas - 1);
#endif
            if (sends)
                st_async_u64(mapa_shared(smem_u32(sums + rank), static_cast<uint32_t>(lane)), all,
                             mapa_shared(bar, static_cast<uint32_t>(lane)));
            if (!__all_sync(~0u, mbar_wait_cluster(bar, (pass >> 1) & 1, &never))) {
                if (lane == 0) atomicOr(&g_status_word, kStatusEpilogueTimeout);
                gave_up = true;
            }
        }
        ++pass;
        return verify_warp_sum(lane < ctas ? sums[lane] : 0);
    };

    while (n > 0 && !gave_up) {
        const T *row_p = target + (first + cur) * a.target_stride;
        const int c = verify_child(parent, at, n, cur, lane);
        if (c >= n) {
            if (!summed) {
                left = {row_p, nullptr, 0.f, 0.f};
                Z = sum_row();
            }
            break;
        }
        at = c;
        const int x = token[c];
        // w at x, in units, and whether u * q * Z < w
        bool holds = false, gone = x < 0;
        unsigned long long w = 0;
        if (x >= 0) {
            if (!draft)
                for (int j = 0; j < skips; ++j) gone |= skip[j] == x;
            w = gone ? 0 : left.at(up[c], uq[c]);
            const double bar = static_cast<double>(uu[c]) * static_cast<double>(uq[c]);
            holds = counts ? bar * static_cast<double>(Z) < static_cast<double>(w)
                           : bar < static_cast<double>(up[c]);
        }
        if (holds) {
            if (writes) path[len] = c;
            ++len;
            cur = c;
            S = Z = 0;
            summed = counts = false;
            skips = 0;
            left = {nullptr, nullptr, 0.f, 0.f};
            continue;
        }
        if (draft) {
            const VerifyLeft<T> before = left;
            const unsigned long long with = S + (counts ? Z : 1ull << 50);
            const double of_q = static_cast<double>(with) * 0x1p-50;
            const float of_q_high = static_cast<float>(of_q);
            left = {row_p, draft + (first + cur) * a.draft_stride, of_q_high,
                    static_cast<float>(of_q - static_cast<double>(of_q_high))};
            const unsigned long long sum = sum_row();
            if (sum > 0) {
                S = with;
                Z = sum;
                summed = counts = true;
            } else {
                // nothing would be left: w stays, but the pieces' sums are gone
                left = before;
                if (counts && !gave_up) Z = sum_row();
            }
            continue;
        }
        if (!summed) {
            left = {row_p, nullptr, 0.f, 0.f};
            Z = sum_row();
            summed = true;
        }
        if (Z > w) {
            if (!gone) {
                // out of the piece and of the CTA that hold it
                const int owner = x / piece;
                if (lane == 0) {
                    skip[skips] = x;
                    unsigned long long &cs = cta_sum[(pass - 1) & 1][owner / kVerifyWarps];
                    cs -= min(cs, w);
                    if (owner / kVerifyWarps == rank) {
                        unsigned long long &ws = warp_sum[owner % kVerifyWarps];
                        ws -= min(ws, w);
                    }
                }
                __syncwarp();
                ++skips;
                Z -= w;
            }
            counts = true;
        }
    }

    // the draw: the CTA, then the warp's piece, its part, then the value
    int found = -1;
    bool mine = rank == 0;                   // without a draw CTA 0 writes
    if (n > 0 && Z > 0 && !gave_up) {
        unsigned long long want = static_cast<unsigned long long>(
            static_cast<double>(Z) * static_cast<double>(uu[0]));
        want = min(want, Z - 1);
        const int owner = verify_pick(lane < ctas ? cta_sum[(pass - 1) & 1][lane] : 0, &want, lane);
        mine = owner < 0 ? rank == 0 : owner == rank;
        const int of = mine ? verify_pick(lane < kVerifyWarps ? warp_sum[lane] : 0, &want, lane) : -1;
        if (of >= 0) {
            command(left, rank * kVerifyWarps + of, skips);
            const int sub = verify_pick(lane < kVerifyWarps ? part_sum[lane] : 0, &want, lane);
            const int b0 = (rank * kVerifyWarps + of) * piece + max(sub, 0) * part;
            const int b1 = min(min(b0 + part, (rank * kVerifyWarps + of + 1) * piece), a.vocab);
            for (int base = b0; base < b1 && found < 0; base += 32) {
                const unsigned long long w = verify_value(left, base + lane, b1, skip, skips);
                const unsigned long long all = verify_warp_sum(w);
                if (want < all) found = base + verify_pick(w, &want, lane);
                else want -= all;
            }
            // None of the piece's values counts by itself (all of them are below 2^-51), though the
            // lanes' sums of them do: the first that is not 0.
            if (sub < 0) found = verify_first(left, b0, min(b0 + piece, a.vocab), skip, skips, lane);
        }
    }
    command(left, -2, 0);
    if (mine && lane == 0) a.next[r] = found;
    if (rank == 0) {
        for (int i = len + lane; i < a.width; i += 32) path[i] = -1;
        if (lane == 0) a.path_lens[r] = len;
    }
    // All that others send to this CTA it has waited for, so it may leave. Where a wait ran out, they
    // may still be about to, for one pass: its shared memory stays while they wait in turn.
    if (gave_up && ctas > 1) {
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitLimitCycles) {
        }
    }
}

// Greedy: a child holds if it is the token that the target puts after its parent; one
// warp a request.
__global__ void __launch_bounds__(32) verify_greedy_kernel(const VerifyArgs a) {
    extern __shared__ int verify_smem[];
    const int lane = threadIdx.x, r = blockIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    int first;
    const int n = verify_tokens(a, r, &first);
    for (int i = lane; i < n; i += 32) {
        const int p = verify_parent(a, r, i);
        verify_smem[i] = p >= 0 && a.following[first + p] == a.tokens[first + i] ? p : -1;
    }
    __syncwarp();
    int *path = a.paths + static_cast<long long>(r) * a.width;
    int len = 0, cur = 0;
    for (int c = 0; c < n; c = verify_child(verify_smem, c, n, c, lane)) {
        if (lane == 0) path[len] = c;
        ++len;
        cur = c;
    }
    for (int i = len + lane; i < a.width; i += 32) path[i] = -1;
    if (lane == 0) {
        a.path_lens[r] = len;
        a.next[r] = n > 0 ? a.following[first + cur] : -1;
    }
}

}  // namespace swiglu
