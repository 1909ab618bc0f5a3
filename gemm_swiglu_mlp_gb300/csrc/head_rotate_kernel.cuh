// Norms of each query and key head with the position rotation, in one pass
// over them; with a paged cache (cache_kernels.cuh) the rotated keys and the
// values go straight to their slots.
//
//   y = x * w / sqrt(mean(x^2) + eps)          (w null: y = x)
//   a_i = position * inv_freq[i], i < n        (pairs (i, i + n) or (2i, 2i + 1))
//   (y1, y2) -> (y1 cos a - y2 sin a, y1 sin a + y2 cos a), the rest of y as it is
//
// FP32 throughout, one rounding to BF16 at the end. The angle is reduced to a
// part of a turn in 64-bit fixed point, where whole turns fall off the top of a
// wrapping product: position * (inv_freq / 2 pi * 2^64). In FP32 the product
// alone would be off by 2^-24 of itself, 0.06 radians at position 1000000. The part of a turn
// that is left, in units of 2^-32, is rounded to FP32 (2^-26 turns) for its sine and cosine.
#pragma once

#include <cuda_bf16.h>

#include "epilogue.cuh"

namespace swiglu {

constexpr int kRotateThreads = 256;
constexpr int kRotateWarps = kRotateThreads / 32;
constexpr int kRotateBlocks = 2;       // of one SM at once
constexpr int kRotateAhead = 4;        // steps of a warp on their way

struct HeadRotateArgs {
    const uint4 *q, *k, *v;            // v: only with a cache
    uint4 *q_out, *k_out;              // k_out: only without a cache
    uint4 *k_cache, *v_cache;          // null without a cache
    const int *positions, *slots;      // [tokens]
    const float *inv_freq;             // [freqs]
    const uint4 *q_weight, *k_weight;  // [head size] BF16; null: no norm
    long long q_tok, q_head, k_tok, k_head, v_tok, v_head;   // strides in 16-byte chunks
    long long qo_tok, qo_head, ko_tok, ko_head;
    long long num_slots;
    float eps;
    int tokens, q_heads, kv_heads, page_shift;
    int freqs;                         // a multiple of 8, at most half a head
    int parts;                         // warps a token: 1, 2, 4 or 8
};

// inv_freq / 2 pi in units of 2^-64 turns, modulo whole turns: the FP32 value's
// 24 significant bits times 2^64 / 2 pi (62 bits). Not finite: 0.
__device__ __forceinline__ unsigned long long rotate_turns(float f) {
    constexpr unsigned long long kTurn = 2935890503282001226ull;   // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(f);
    const int e = static_cast<int>((bits >> 23) & 255u);
    const unsigned long long m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    if (e == 255) return 0;
    const int down = 150 - (e ? e : 1);   // f = m * 2^-down
    const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);
    unsigned long long t;
    if (down <= 0)
        t = down > -64 ? lo << -down : 0;
    else if (down < 64)
        t = (lo >> down) | (hi << (64 - down));
    else
        t = down < 128 ? hi >> (down - 64) : 0;
    return bits >> 31 ? 0ull - t : t;
}

// Two FP32 numbers worked on by one instruction.
struct F32x2 {
    float x, y;
};
__device__ __forceinline__ F32x2 mul2(F32x2 a, F32x2 b) {
    F32x2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ F32x2 fma2(F32x2 a, F32x2 b, F32x2 c) {
    F32x2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// Two 16-byte chunks of BF16 as pairs.
__device__ __forceinline__ void unpack_chunks(const uint4 &lo, const uint4 &hi, F32x2 (&f)[8]) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)};
}

// 16 bytes from global memory to this thread's own place in shared memory, in the background.
__device__ __forceinline__ void copy_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a lane does with its two chunks of a head: norm and rotation.
template <int D, bool NEIGHBOURS>
struct HeadRotator {
    static constexpr int LANES = D / 16, ROWS = 32 / LANES;
    F32x2 w[8];            // the norm's weights
    float cs[8], sn[8];
    bool norm, rotates;
    float eps;

    __device__ __forceinline__ void set_weight(const uint4 *weight, int c0, int c1) {
        norm = weight != nullptr;
        if (norm) unpack_chunks(weight[c0], weight[c1], w);
    }
    // All lanes of the warp.
    __device__ __forceinline__ void turn(uint4 &lo, uint4 &hi) const {
        F32x2 f[8];
        unpack_chunks(lo, hi, f);
        if (norm) {
            F32x2 sum = mul2(f[0], f[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) sum = fma2(f[i], f[i], sum);
            float all = sum.x + sum.y;
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) all += __shfl_xor_sync(~0u, all, d);
            const float r = rsqrtf(fmaf(all, 1.f / D, eps));
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = mul2(mul2(f[i], {r, r}), w[i]);
        } else if (!rotates) {
            return;                       // as it is, bit for bit
        }
        if (rotates) {                    // (a product with a sine of 0 would spread Inf)
            if (NEIGHBOURS) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = fma2({f[i].x, f[i].x}, {cs[i], sn[i]},
                                mul2({f[i].y, f[i].y}, {-sn[i], cs[i]}));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F32x2 c = {cs[2 * i], cs[2 * i + 1]}, n = {sn[2 * i], sn[2 * i + 1]};
                    const F32x2 x = f[i], y = f[i + 4];
                    f[i] = fma2(x, c, mul2(y, {-n.x, -n.y}));
                    f[i + 4] = fma2(x, n, mul2(y, c));
                }
            }
        }
        lo = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                        pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
        hi = make_uint4(pack_bf16x2(f[4].x, f[4].y), pack_bf16x2(f[5].x, f[5].y),
                        pack_bf16x2(f[6].x, f[6].y), pack_bf16x2(f[7].x, f[7].y));
    }
};

// A lane's way through heads of one kind: its first chunk's address at the present step, and
// how much further on the next step's is.
struct HeadWalk {
    uint4 *at;
    long long on;
    int h, heads;
    template <int ROWS>
    __device__ __forceinline__ void seek(const uint4 *base, long long head, int heads_of, int step,
                                         int own, int c0) {
        h = step * ROWS + own;
        heads = heads_of;
        at = const_cast<uint4 *>(base) + h * head + c0;
        on = ROWS * head;
    }
    template <int ROWS>
    __device__ __forceinline__ void next() {
        h += ROWS;
        at += on;
    }
};

// A block takes kRotateWarps / parts tokens at a time: its threads make their cosines and
// sines, one each, in shared memory, and each warp takes one token's heads (or one of `parts`
// shares of them): LANES = D / 16 lanes a head, ROWS = 32 / LANES heads a step. A lane holds two
// 16-byte chunks of a head whose values rotate with one another: chunks s and s + n/8 (halves),
// or 2s and 2s + 1 (neighbours); either way its angles are those of frequencies 8s .. 8s + 7, the
// same for every head of the token. The steps ahead, of the next token too, are on their way to
// the lane's own places in shared memory, kRotateAhead of them: registers for as many would
// leave too few warps.
//
// Bytes bound it: 16384 tokens of 64 + 8 heads of 128 with norms 98 us, 6.2 TB/s read and
// written, 91% of the copy rate (two steps in registers instead: 117; a third block an SM, whose
// registers spill: 125). 832 tokens of 28 + 4 + 4 heads into the cache 5.9 us, one token 1.9,
// as much as an empty launch.
template <int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRotateThreads, kRotateBlocks)
    head_rotate_kernel(const HeadRotateArgs a) {
    using R = HeadRotator<D, NEIGHBOURS>;
    // [tile's parity][token][cosines, sines][freqs / 4]
    __shared__ float4 tables[2][kRotateWarps][2][D / 8];
    __shared__ uint4 ahead[kRotateAhead][2][kRotateThreads];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = lane & (R::LANES - 1), own = lane / R::LANES;
    griddep_launch_dependents();
    griddep_wait();

    R rot;
    rot.eps = a.eps;
    const int turned = a.freqs >> 3;          // slots of a head that rotate
    rot.rotates = s < turned;
    const bool apart = !NEIGHBOURS && rot.rotates;
    const int c0 = apart ? s : 2 * s, c1 = apart ? s + turned : 2 * s + 1;   // this lane's chunks
    // a token's steps: queries, then keys, then (with a cache) values, each in whole steps
    auto steps = [](int heads) { return (heads + R::ROWS - 1) / R::ROWS; };
    const int k_at = steps(a.q_heads), v_at = k_at + steps(a.kv_heads);
    const int all = v_at + (a.k_cache ? steps(a.kv_heads) : 0);
    const int tokens = kRotateWarps / a.parts;               // of the block at a time
    const int local = warp / a.parts, part = warp - local * a.parts;
    const int i0 = all * part / a.parts, i1 = all * (part + 1) / a.parts;
    const int stride = static_cast<int>(gridDim.x) * tokens;
    const int t_first = static_cast<int>(blockIdx.x) * tokens + local;

    // the next step to ask for
    const int apart_by = c1 - c0;
    int ask_t = t_first, ask_i = i0;
    uint32_t ask_to = smem_u32(&ahead[0][0][threadIdx.x]);
    const uint32_t place = sizeof(ahead[0]), first_place = ask_to;
    const uint32_t end_place = first_place + kRotateAhead * place;
    HeadWalk from{};
    bool seek_from = true;
    auto ask = [&] {
        if (ask_t < a.tokens) {
            if (seek_from || ask_i == k_at || ask_i == v_at) {
                if (ask_i < k_at)
                    from.template seek<R::ROWS>(a.q + ask_t * a.q_tok, a.q_head, a.q_heads, ask_i, own,
                                                c0);
                else if (ask_i < v_at)
                    from.template seek<R::ROWS>(a.k + ask_t * a.k_tok, a.k_head, a.kv_heads,
                                                ask_i - k_at, own, c0);
                else
                    from.template seek<R::ROWS>(a.v + ask_t * a.v_tok, a.v_head, a.kv_heads,
                                                ask_i - v_at, own, c0);
            }
            if (from.h < from.heads) {
                copy_async_16(ask_to, from.at);
                copy_async_16(ask_to + sizeof(ahead[0][0]), from.at + apart_by);
            }
            from.template next<R::ROWS>();
            seek_from = ++ask_i == i1;
            if (seek_from) {
                ask_i = i0;
                ask_t += stride;
            }
        }
        copy_async_commit();
        ask_to = ask_to + place == end_place ? first_place : ask_to + place;
    };
#pragma unroll
    for (int i = 0; i < kRotateAhead - 1; ++i) ask();
    uint32_t take = first_place;              // place of the step that comes
    int weight_of = -1;                       // whose weight is there: 0 q's, 1 k's

    for (int t0 = static_cast<int>(blockIdx.x) * tokens, tile = 0; t0 < a.tokens; t0 += stride, ++tile) {
        // (a warp still at the tile before reads the other table)
        auto table = tables[tile & 1];
        // cosines and sines of the block's tokens
        for (int i = threadIdx.x; i < tokens * a.freqs; i += kRotateThreads) {
            const int of = i / a.freqs, f = i - of * a.freqs;
            if (t0 + of < a.tokens) {
                const long long pos = a.positions[t0 + of];
                const int ph = static_cast<int>(
                    (static_cast<unsigned long long>(pos) * rotate_turns(a.inv_freq[f])) >> 32);
                float sn, cs;
                sincospif(static_cast<float>(ph) * 0x1p-31f, &sn, &cs);   // half turns in [-1, 1)
                reinterpret_cast<float *>(&table[of][0][0])[f] = cs;
                reinterpret_cast<float *>(&table[of][1][0])[f] = sn;
            }
        }
        const int t = t0 + local;
        const bool there = local < tokens && t < a.tokens;
        // keys and values of a token without a slot are dropped
        const int slot = there && a.k_cache && i1 > k_at ? a.slots[t] : 0;
        __syncthreads();
        if (there) {
            if (rot.rotates) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 c = table[local][0][2 * s + i], n = table[local][1][2 * s + i];
                    rot.cs[4 * i] = c.x, rot.cs[4 * i + 1] = c.y;
                    rot.cs[4 * i + 2] = c.z, rot.cs[4 * i + 3] = c.w;
                    rot.sn[4 * i] = n.x, rot.sn[4 * i + 1] = n.y;
                    rot.sn[4 * i + 2] = n.z, rot.sn[4 * i + 3] = n.w;
                }
            }
            const bool kept = slot >= 0 && slot < a.num_slots;
            const long long page = slot >> a.page_shift;
            const long long at = (((page * a.kv_heads) << a.page_shift) +
                                  (slot & ((1 << a.page_shift) - 1))) * (D / 8);
            const long long cache_head = static_cast<long long>(D / 8) << a.page_shift;
            HeadWalk to{};
#pragma unroll 1
            for (int i = i0; i < i1; ++i) {
                ask();
                copy_async_wait<kRotateAhead - 1>();
                uint4 lo = ld_shared_v4(take), hi = ld_shared_v4(take + sizeof(ahead[0][0]));
                take = take + place == end_place ? first_place : take + place;
                if (i == i0 || i == k_at || i == v_at) {
                    // another kind of heads
                    if (i < k_at) {
                        to.template seek<R::ROWS>(a.q_out + t * a.qo_tok, a.qo_head, a.q_heads, i, own,
                                                  c0);
                    } else {
                        const int step = i - (i < v_at ? k_at : v_at);
                        if (a.k_cache)
                            to.template seek<R::ROWS>((i < v_at ? a.k_cache : a.v_cache) + at,
                                                      cache_head, kept ? a.kv_heads : 0, step, own, c0);
                        else
                            to.template seek<R::ROWS>(a.k_out + t * a.ko_tok, a.ko_head, a.kv_heads,
                                                      step, own, c0);
                    }
                    if (i < v_at && weight_of != (i < k_at ? 0 : 1)) {
                        weight_of = i < k_at ? 0 : 1;
                        rot.set_weight(weight_of ? a.k_weight : a.q_weight, c0, c1);
                    }
                }
                if (i < v_at) rot.turn(lo, hi);
                if (to.h < to.heads) {
                    to.at[0] = lo;
                    to.at[apart_by] = hi;
                }
                to.template next<R::ROWS>();
            }
        }
    }
}

}  // namespace swiglu
