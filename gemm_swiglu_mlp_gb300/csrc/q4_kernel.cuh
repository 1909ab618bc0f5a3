// Products of few token rows with 4-bit weights and group scales:
//
//   W[n, k] = (code[n, k] - 8) * scale[k / G, n]
//   out = A W^T, or the gated up-projection out = SiLU(A W1^T) (.) (A W2^T)
//
// ("Tile-Level Activation Overlap for Efficient LLM Inference", Section 1
// Introduction, has the gated MLP; at the few rows of a decode step its BF16
// kernels read the weights at the memory's rate, so only fewer bytes make it faster.)
//
// The operands' roles are swapped as in the decode down-projection: 16 output
// columns are the matrix instruction's 16-row side, 8 tokens its 8-column side
// (mma.sync m16n8k16, BF16 in, FP32 sums). Codes become BF16 in registers, where
// code - 8 is exact; a group's products are summed as they are and the sum is
// multiplied by the scale in FP32, so no weight is rounded. tcgen05 would take
// the weights from shared or tensor memory, a write and a wait more for each of
// them: up to 8 tokens its rate is not what is missing. From 9 on instructions bound
// this kernel, and weights unpacked into tensor memory would take about half of them;
// that form is not built.
//
// A CTA computes 128 columns of weights (the gated form: 64 output columns of both) for
// up to 8 NT tokens over a share of K, in steps of 256 values of k. One warp loads a
// step's codes (128-byte rows as they lie in memory, [N, K/2]), scales and tokens by bulk
// copies through a ring of shared memory. Eight warps multiply: four take the even steps
// and four the odd ones, each 64 columns of weights by 128 values of k, so that what a warp
// does once a step (waits, addresses, the tokens' values) is shared by 32 products
// of 16 x 8 x 16. What the CTAs share out, by the host's rule:
//   tiles that run at once: each by a cluster, whose CTAs have a share of K each and add
//   their sums in shared memory, in the order of k;
//   more of them: the steps of all tiles lie in one line that is cut evenly over the CTAs
//   (462 tiles on 152 SMs are 3.04 each, but 4 for the slowest); a tile that is cut leaves FP32
//   sums in the workspace, which q4_join_kernel adds in the order of k.
#pragma once

#include "epilogue.cuh"

namespace swiglu {

constexpr int kQ4Cols = 128;              // columns of weights a CTA
constexpr int kQ4Step = 256;              // values of k a ring stage
constexpr int kQ4Warps = 8;               // that multiply
// The line has a warp of its own for the loads. A tile's share of K is short, and there the first
// warps of the even and of the odd steps fill their stages themselves: fewer threads to start,
// and more registers for each (one token of 512 x 16384 4.8 -> 4.0 us; 462 tiles of 16 tokens
// in a line 69 us, but 75 that way).
constexpr int kQ4Threads = 32 * kQ4Warps, kQ4LineThreads = kQ4Threads + 32;
constexpr int kQ4MaxSplits = 16;          // shares of K: CTAs of a cluster

// GROUPS: a warp's groups in its 128 values of k of a step, which it sums apart: 4 for groups of 32,
// 2 for 64, 1 for 128 (one token of 8192 -> 2 x 29568 49.4 -> 47.0 us, with its halves apart before);
// for more than 8 tokens, whose sums take the registers, still 2, a group's halves.
template <int NT, bool GATED, int GROUPS>
struct Q4Cfg {
    static constexpr int MATS = GATED ? 2 : 1;
    static constexpr int COLS = kQ4Cols / MATS;                   // output columns
    static constexpr int TOKENS = 8 * NT;
    // two CTAs an SM; 32 tokens' sums need more registers than that leaves, and 16 tokens with
    // short groups more shared memory
    static constexpr int CTAS = NT == 4 || (NT == 2 && GROUPS == 4) ? 1 : 2;
    static constexpr int CODE_BYTES = kQ4Cols * kQ4Step / 2;      // a weight's 128-byte rows
    static constexpr int TOKEN_BYTES = TOKENS * kQ4Step * 2;      // four boxes of 64 values
    static constexpr int SCALE_BYTES = kQ4Cols * 2 * (GROUPS == 4 ? 8 : 4);   // groups a step, at most
    static constexpr int STAGE_BYTES = CODE_BYTES + SCALE_BYTES + TOKEN_BYTES;
    // FP32 sums: rows of a token's 128 columns, over the ring when it is idle ...
    static constexpr int PART_ROW = kQ4Cols + 8;                  // (no bank conflicts)
    static constexpr int PART_VALUES = TOKENS * PART_ROW;
    // ... and those that the cluster's CTAs send to the one that adds them
    // (up to as many places too many as there are CTAs, for shares are rounded up; or, of the
    // line, one tile's sums while the ring goes on)
    static constexpr int SENT_BYTES = (TOKENS * COLS / 4 + kQ4MaxSplits) * MATS * 16;
    static constexpr int RECEIVE_BYTES = SENT_BYTES > PART_VALUES * 4 ? SENT_BYTES : PART_VALUES * 4;
    // an even number, so that a stage is always the same warps': warps that had not waited for
    // its last filling could take the barrier's phase before it for the one after
    static constexpr int STAGES =
        ((CTAS == 2 ? 111 : 200) * 1024 - RECEIVE_BYTES) / STAGE_BYTES / 2 * 2;
    static constexpr int OFF_CODES = 0;
    static constexpr int OFF_TOKENS = OFF_CODES + STAGES * CODE_BYTES;
    static constexpr int OFF_SCALES = OFF_TOKENS + STAGES * TOKEN_BYTES;
    static constexpr int OFF_RECEIVE = OFF_SCALES + STAGES * SCALE_BYTES;
    static constexpr int OFF_BAR = OFF_RECEIVE + RECEIVE_BYTES;
    static constexpr int OFF_ABORT = OFF_BAR + 16 * STAGES;
    static constexpr int SMEM_BYTES = OFF_ABORT + 16 + 1024;      // + alignment slack
    static_assert(4 * 4 * PART_VALUES <= OFF_RECEIVE, "the sums fit in the ring");
    static_assert(STAGES >= 4 && STAGES % 2 == 0, "two groups of warps take turns");
    static_assert(CTAS * (SMEM_BYTES + 1024) <= 228 * 1024, "CTAs an SM");
};

struct Q4Args {
    uint16_t *out;               // [M][N] BF16
    int M, N;
    int steps;                   // of kQ4Step values of k
    int splits;                  // shares of K: the cluster's CTAs
    int tiles;                   // of the columns (the line: the first block of tokens', then on)
    int units;                   // the line: the steps of all tiles
    float *partial;              // the line's cut tiles: [CTA][its first, its last][token][128]
    int group_shift;             // log2 of the group: 5, 6 or 7
#ifdef SWIGLU_TEST_FAULT_INJECTION
    int skip_first_fill;         // test build only: never fill the first ring stage
#endif
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, const float4 &v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x),
                 "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
// d = a b + c, 16 x 8 x 16.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Eight codes (a nibble each, the first lowest) as BF16 numbers, pairs (0, 4), (1, 5), (2, 6),
// (3, 7). The bits 0 .. 7 of a BF16 number with nothing above them count units of 2^-133
// (subnormals, then the first binade: the same step), so a nibble masked out at bits 0 .. 3 is
// that many units, and one at bits 4 .. 7 that many sixteens of units: five integer
// instructions a word, where a shift for every nibble takes seven, and the integer pipe was what
// the kernel ran into. From there two ways, by what bounds the kernel then:
//   more than 8 tokens (matrix instructions): one exact multiply-add makes them (code - 8) / 64;
//   up to 8 (instructions issued): they are used as they are. The tokens are multiplied by 2^60,
//   or 2^56 where they meet sixteens, which takes the products into FP32's range, and a
//   group's sums start from -8 times the tokens' sum: a multiply-add less for every code
//   pair, 4 matrix instructions more for 16 (one token, 2 weights of 3584 x 18944: 15.0 -> 14.3 us,
//   of 8192 x 29568 52.3 -> 47.1; 16 tokens, 2 of 8192 x 29568: 69 us, but 73 this way).
//   All sums are 2^-73 of what they stand for then, so FP32's smallest step is 2^-76 of it, and
//   values from 2^68 on pass FP32's range: the contract says so. (Scales times 2^57 would leave
//   that step to a group's sums only; it is an instruction for every two scales, 14.25 -> 14.40 us,
//   5 tokens of 4864 x 896 with groups of 32 4.23 -> 4.46.)
template <int NT>
struct Q4Form {
    static constexpr bool DIRECT = NT == 1;
    static constexpr float UNIT = DIRECT ? 0x1p73f : 64.f;        // of the sums
};
template <bool DIRECT>
__device__ __forceinline__ void q4_unpack(uint32_t x, uint32_t (&w)[4]) {
    const uint32_t y = x >> 8;
    w[0] = x & 0x000F000Fu;
    w[1] = x & 0x00F000F0u;
    w[2] = y & 0x000F000Fu;
    w[3] = y & 0x00F000F0u;
    if constexpr (!DIRECT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float by = i & 1 ? 0x1p123f : 0x1p127f;
            const __nv_bfloat162 d =
                __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]),
                        __floats2bfloat162_rn(by, by), __floats2bfloat162_rn(-0.125f, -0.125f));
            w[i] = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}
constexpr uint32_t kQ4Less8 = 0x80088008u;     // -8 units, twice
constexpr uint32_t kQ4Less128 = 0x80808080u;   // -8 sixteens
// Eight of a token's values of k in the same pairs.
template <bool DIRECT>
__device__ __forceinline__ void q4_pairs(const uint4 &v, uint32_t (&b)[4]) {
    b[0] = __byte_perm(v.x, v.z, 0x5410);
    b[1] = __byte_perm(v.x, v.z, 0x7632);
    b[2] = __byte_perm(v.y, v.w, 0x5410);
    b[3] = __byte_perm(v.y, v.w, 0x7632);
    if constexpr (DIRECT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float by = i & 1 ? 0x1p56f : 0x1p60f;
            const __nv_bfloat162 d = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&b[i]),
                                             __floats2bfloat162_rn(by, by));
            b[i] = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

// Where CTA `cta` of `ctas` begins in the line of all tiles' steps.
__device__ __forceinline__ int q4_line_at(int units, int cta, int ctas) {
    return static_cast<int>(static_cast<long long>(units) * cta / ctas);
}

// One output chunk: four columns from `at` on of one token.
template <bool GATED>
__device__ __forceinline__ void q4_store(const Q4Args &args, int token, int at, float4 v, float4 up) {
    if constexpr (GATED) {
        v.x = silu_mul(v.x, up.x);
        v.y = silu_mul(v.y, up.y);
        v.z = silu_mul(v.z, up.z);
        v.w = silu_mul(v.w, up.w);
    }
    *reinterpret_cast<uint2 *>(args.out + static_cast<size_t>(token) * args.N + at) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void add4(float4 &x, const float4 &y) {
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
}

// A warp's sums to their places: the CTA's columns of the first weight, then the second's.
// ADD: on top of those that are there, if `more`.
template <int NT, bool GATED, bool ADD>
__device__ __forceinline__ void q4_shares(const float (&acc)[4][NT][4], float *sums, int tile, int g,
                                          int t, bool more) {
    constexpr int ROW = kQ4Cols + 8, COLS = kQ4Cols / 2;
    const int c0 = 2 * g + (g >> 2), c1 = c0 ^ 1;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int col = GATED ? (r >> 1) * COLS + 32 * tile + 16 * (r & 1) : 64 * tile + 16 * r;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // fragment columns 2t and 2t + 1 are tokens t and t + 4
            float *p = sums + (8 * nt + t) * ROW + col;
            const float (&x)[4] = acc[r][nt];
            const bool add = ADD && more;
            p[c0] = x[0] + (add ? p[c0] : 0.f);
            p[4 * ROW + c0] = x[1] + (add ? p[4 * ROW + c0] : 0.f);
            p[c1] = x[2] + (add ? p[c1] : 0.f);
            p[4 * ROW + c1] = x[3] + (add ? p[4 * ROW + c1] : 0.f);
        }
    }
}

// LINE: this CTA's share of the line of all tiles' steps; else of one tile's (splits of them).
template <int NT, bool GATED, int GROUPS, bool LINE>
__global__ void __launch_bounds__(LINE ? kQ4LineThreads : kQ4Threads,
                                 Q4Cfg<NT, GATED, GROUPS>::CTAS)
    q4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmQ1,
              const __grid_constant__ CUtensorMap tmQ2, const __grid_constant__ CUtensorMap tmS1,
              const __grid_constant__ CUtensorMap tmS2, const Q4Args args) {
    using C = Q4Cfg<NT, GATED, GROUPS>;
    constexpr bool DIRECT = Q4Form<NT>::DIRECT;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x);
    const int splits = LINE ? 1 : args.splits;
    const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    // first column and token of a tile; the line counts them from 0, else there is one
    int own_n0 = 0, own_m0 = 0, u0, u1;
    if (LINE) {
        u0 = q4_line_at(args.units, cta, static_cast<int>(gridDim.x));
        u1 = q4_line_at(args.units, cta + 1, static_cast<int>(gridDim.x));
    } else {
        const int tile = splits > 1 ? cta / splits : cta, block = tile / args.tiles;
        own_n0 = (tile - block * args.tiles) * C::COLS;
        own_m0 = block * C::TOKENS;
        u0 = static_cast<int>(static_cast<long long>(args.steps) * rank / splits);
        u1 = static_cast<int>(static_cast<long long>(args.steps) * (rank + 1) / splits);
    }
    auto columns = [&](int tile) { return LINE ? tile % args.tiles * C::COLS : own_n0; };
    auto token_rows = [&](int tile) { return LINE ? tile / args.tiles * C::TOKENS : own_m0; };
    auto full = [&](int s) { return base + C::OFF_BAR + 8u * s; };
    auto empty = [&](int s) { return base + C::OFF_BAR + 8u * (C::STAGES + s); };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_ABORT);
    const int per_step = kQ4Step >> args.group_shift;   // groups a step

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kQ4Warps / 2);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (splits > 1) cluster_arrive();         // (waited for before anything is sent)
    __syncthreads();
    griddep_launch_dependents();

    const int tile = warp & 1, half = (warp >> 1) & 1, odd = LINE ? (warp >> 2) & 1 : warp >> 2;
    // Loads: by lane 0 of the line's ninth warp, or of the first warp of the even and of the odd steps.
    constexpr int EVERY = LINE ? 1 : 2;                 // steps from one load to a loader's next
    const bool loads = lane == 0 && (LINE ? warp == kQ4Warps : (warp & 3) == 0);
    int load_u = u0 + (LINE ? 0 : odd);                 // the next one's step, as its tile's
    int load_of = LINE ? load_u / args.steps : 0, load_s = load_u - load_of * args.steps;
    uint32_t issued = 0, parity = 0;                    // for the drain after an abort
    auto forward = [&] {
        load_u += EVERY;
        load_s += EVERY;
        if (LINE && load_s == args.steps) {
            load_s = 0;
            ++load_of;
        }
    };
    auto load = [&](int stage, uint32_t phase) {
#ifdef SWIGLU_TEST_FAULT_INJECTION
        if (args.skip_first_fill && load_u == u0) {
            forward();
            return;
        }
#endif
        const uint32_t bar = full(stage);
        const int n0 = columns(load_of), m0 = token_rows(load_of);
        mbar_arrive_expect_tx(bar, C::CODE_BYTES + per_step * kQ4Cols * 2 + C::TOKEN_BYTES);
#pragma unroll
        for (int m = 0; m < C::MATS; ++m) {
            tma_load_2d(base + C::OFF_CODES + stage * C::CODE_BYTES + m * (C::CODE_BYTES / C::MATS),
                        m ? &tmQ2 : &tmQ1, bar, load_s * (kQ4Step / 2), n0);
            tma_load_2d(base + C::OFF_SCALES + stage * C::SCALE_BYTES + m * (C::SCALE_BYTES / C::MATS),
                        m ? &tmS2 : &tmS1, bar, n0, load_s * per_step);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
            tma_load_2d(base + C::OFF_TOKENS + stage * C::TOKEN_BYTES + b * C::TOKENS * 128, &tmA, bar,
                        load_s * kQ4Step + 64 * b, m0);
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        forward();
    };
    if (loads) {
        // the ring's first codes, while the launch before this one ends
        const int u_first = load_u, s_first = load_s, of_first = load_of;
        for (int i = 0; i < C::STAGES / EVERY && load_u < u1; ++i, forward()) {
            tma_prefetch_2d(&tmQ1, load_s * (kQ4Step / 2), columns(load_of));
            if constexpr (GATED) tma_prefetch_2d(&tmQ2, load_s * (kQ4Step / 2), columns(load_of));
        }
        load_u = u_first;
        load_s = s_first;
        load_of = of_first;
    }
    griddep_wait();
    if (loads)
        for (int i = 0; i < C::STAGES / EVERY && load_u < u1; ++i) load(LINE ? i : odd + 2 * i, 0);

    float acc[4][NT][4];                                // [16-column tile][8 tokens][fragment]
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][t][i] = 0.f;
    const int g = lane >> 2, t = lane & 3;
    if (LINE && warp == kQ4Warps) {
        if (loads) {
            int st = 0;
            for (uint32_t ph = 0; load_u < u1;) {
                if (!mbar_wait(empty(st), ph, abort_flag)) {
                    if (!*abort_flag) {
                        atomicOr(&g_status_word, kStatusProducerTimeout);
                        *abort_flag = 1;
                    }
                    break;
                }
                load(st, ph ^ 1u);
                if (++st == C::STAGES) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
    } else {
        // A warp has the even or the odd steps (warp / 4), 128 values of k of them (bit 1), and 64
        // columns of weights (bit 0): for the gated form columns 32 * bit 0 .. of both.
        // token of fragment column g: its low bit taken for the highest, so that the two rows of
        // a quarter-warp's loads lie in different halves of the swizzled 128 bytes
        const uint32_t tok = ((g & 1) << 2) | (g >> 1);
        // row of fragment row i of a 16-column tile (the other eight rows are those + 1 or - 1):
        // 0, 2, 4, 6, 9, 11, 13, 15, so that eight rows still differ in their last three bits (by
        // which 16-byte chunks are swizzled) and a lane's two columns have their scales in one word
        auto row_of = [](int i) { return i < 8 ? 2 * i + (i >> 2) : 2 * (i - 8) + 1 - ((i - 8) >> 2); };
        const int first = 64 / C::MATS * tile;         // of the first weight's rows
        const uint32_t row = first + row_of(lane & 15);
        const uint32_t code_at = base + C::OFF_CODES + row * 128u;
        const uint32_t chunk = (4u * half + (lane >> 4)) ^ (row & 7u);
        const uint32_t scale_at = base + C::OFF_SCALES + 2u * (first + 2 * g) +
                                  ((128u * half) >> args.group_shift) * (C::COLS * 2);
        const uint32_t low = g < 4 ? 0x1044u : 0x3244u, high = g < 4 ? 0x3244u : 0x1044u;
        const uint32_t tok_at = base + C::OFF_TOKENS + (2 * half * C::TOKENS + tok) * 128u;
        const uint32_t chunk0 = (t ^ tok) << 4, chunk1 = ((4u + t) ^ tok) << 4;
        // from the scales of one of its groups to the next's (halves of a group have the same)
        const uint32_t next_group = args.group_shift == 7 ? 0u : C::COLS * 2u;
        int st = odd, before = -1;             // this step's stage, and the last one's, to load again
        uint32_t ph = 0, before_ph = 0;
        bool ok = true;
        auto give_up = [&](unsigned status) {
            ok = false;
            if (lane == 0 && !*abort_flag) {
                atomicOr(&g_status_word, status);
                *abort_flag = 1;
            }
        };
        int u = u0 + odd;
        // one tile's steps after the other (without the line there is one)
        int of = LINE ? u0 / args.steps : 0;
        for (int from = u0; from < u1; ++of) {
            const int to = LINE ? min(u1, (of + 1) * args.steps) : u1;
            for (; u < to; u += 2) {
                if (!LINE && (warp & 3) == 0 && before >= 0 && ok) {
                    bool freed = true;
                    if (loads && load_u < u1) {
                        freed = mbar_wait(empty(before), before_ph, abort_flag);
                        if (freed) load(before, before_ph ^ 1u);
                    }
                    if (!__all_sync(~0u, freed)) give_up(kStatusProducerTimeout);
                }
                if (ok && !__all_sync(~0u, mbar_wait(full(st), ph, abort_flag)))
                    give_up(kStatusMmaTimeout);
                if (!ok) continue;   // (the line's other warps still meet this one below)
                constexpr int SPAN = 4 / GROUPS;              // blocks of 32 values a group
                constexpr int AHEAD = SPAN == 4 ? 2 : 1;      // 64s of values that a group takes
                uint32_t b[2 * AHEAD][NT][4];                 // tokens' values
                float start[AHEAD == 2 || SPAN == 2 ? 1 : 2][NT][4];
                float part[SPAN == 4 ? 4 : 1][NT][4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {                 // 64 values of k each
                    if (q % AHEAD == 0) {
#pragma unroll
                        for (int h = 0; h < AHEAD; ++h)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t toks = tok_at + st * C::TOKEN_BYTES +
                                                      (q + h) * C::TOKENS * 128 + nt * 1024;
                                q4_pairs<DIRECT>(ld_shared_v4(toks + chunk0), b[2 * h][nt]);
                                q4_pairs<DIRECT>(ld_shared_v4(toks + chunk1), b[2 * h + 1][nt]);
                            }
                        // what each group's sums start from: -8 times the tokens' sum, or 0
#pragma unroll
                        for (int blk = 0; blk < 2 * AHEAD; ++blk)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float(&p)[4] = start[blk / SPAN][nt];
                                if (blk % SPAN == 0) p[0] = p[1] = p[2] = p[3] = 0.f;
                                if constexpr (DIRECT) {
                                    const uint32_t(&k)[4] = b[blk][nt];
                                    mma_bf16(p, kQ4Less8, kQ4Less8, kQ4Less128, kQ4Less128, k[0], k[1],
                                             p[0], p[1], p[2], p[3]);
                                    mma_bf16(p, kQ4Less8, kQ4Less8, kQ4Less128, kQ4Less128, k[2], k[3],
                                             p[0], p[1], p[2], p[3]);
                                }
                            }
                    }
                    const uint32_t codes = code_at + st * C::CODE_BYTES + ((chunk ^ (2u * q)) << 4);
                    const uint32_t scales = scale_at + st * C::SCALE_BYTES +
                                            (SPAN == 4 ? 0 : q * (2 / SPAN)) * next_group;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // the gated form's third and fourth tiles are the second weight's
                        const uint32_t m = GATED && r >= 2, rr = GATED ? r & 1 : r;
                        uint32_t x[4];
                        ldmatrix_x4(x, codes + m * (C::CODE_BYTES / 2) + rr * 16 * 128);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int blk = 2 * (q % AHEAD) + i;      // of b
                            const bool begins = blk % SPAN == 0, ends = (blk + 1) % SPAN == 0;
                            uint32_t lo[4], hi[4];
                            q4_unpack<DIRECT>(x[2 * i], lo);
                            q4_unpack<DIRECT>(x[2 * i + 1], hi);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float(&p)[4] = part[SPAN == 4 ? r : 0][nt];
                                const uint32_t(&k)[4] = b[blk][nt];
                                const float(&c)[4] = begins ? start[blk / SPAN][nt] : p;
                                mma_bf16(p, lo[0], hi[0], lo[1], hi[1], k[0], k[1], c[0], c[1], c[2], c[3]);
                                mma_bf16(p, lo[2], hi[2], lo[3], hi[3], k[2], k[3], p[0], p[1], p[2], p[3]);
                            }
                            if (!ends) continue;
                            const uint32_t two = ld_shared_u32(scales + m * (C::SCALE_BYTES / 2) + rr * 32 +
                                                               (SPAN == 1 ? i * C::COLS * 2 : 0));
                            const float sl = __uint_as_float(__byte_perm(two, 0, low));
                            const float sh = __uint_as_float(__byte_perm(two, 0, high));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const float(&p)[4] = part[SPAN == 4 ? r : 0][nt];
                                acc[r][nt][0] = fmaf(sl, p[0], acc[r][nt][0]);
                                acc[r][nt][1] = fmaf(sl, p[1], acc[r][nt][1]);
                                acc[r][nt][2] = fmaf(sh, p[2], acc[r][nt][2]);
                                acc[r][nt][3] = fmaf(sh, p[3], acc[r][nt][3]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(st));
                before = st;
                before_ph = ph;
                st += 2;
                if (st >= C::STAGES) {
                    st -= C::STAGES;
                    ph ^= 1u;
                }
            }
            if constexpr (LINE) {
                // the tile's four shares one after the other, beside the ring, then its result; or its
                // sums to the workspace, where other CTAs have the rest of it
                float *sums = reinterpret_cast<float *>(smem + C::OFF_RECEIVE);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    if ((warp >> 1) == q) q4_shares<NT, GATED, true>(acc, sums, tile, g, t, q > 0);
                    named_barrier(1, kQ4Threads);
                }
                constexpr float unit = Q4Form<NT>::UNIT;
                const bool whole = from == of * args.steps && to == (of + 1) * args.steps;
                const int n0 = columns(of), m0 = token_rows(of), tokens = min(C::TOKENS, args.M - m0);
                constexpr int PER = C::COLS / 4;
                float *partial = args.partial + (2 * static_cast<size_t>(cta) + (from != u0)) *
                                                    C::TOKENS * kQ4Cols;
                for (int c = threadIdx.x; c < tokens * PER && ok; c += kQ4Threads) {
                    const int token = c / PER, at = 4 * (c % PER);
                    float4 v[2];
#pragma unroll
                    for (int m = 0; m < C::MATS; ++m) {
                        v[m] = *reinterpret_cast<const float4 *>(sums + token * C::PART_ROW +
                                                                 m * C::COLS + at);
                        v[m] = {unit * v[m].x, unit * v[m].y, unit * v[m].z, unit * v[m].w};
                        if (!whole)
                            *reinterpret_cast<float4 *>(partial + token * kQ4Cols + m * C::COLS + at) = v[m];
                    }
                    if (whole && n0 + at < args.N)
                        q4_store<GATED>(args, m0 + token, n0 + at, v[0], v[C::MATS - 1]);
                }
                named_barrier(1, kQ4Threads);      // (the sums have been read)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[r][nt][0] = acc[r][nt][1] = acc[r][nt][2] = acc[r][nt][3] = 0.f;
            }
            from = to;
        }
    }

    __syncthreads();
    if (*abort_flag) {
        // every copy already issued lands before the ring is reused
        if (loads)
            for (int s = 0; s < C::STAGES; ++s)
                if ((issued >> s) & 1u)
                    if (!mbar_wait_drain(full(s), (parity >> s) & 1u))
                        atomicOr(&g_status_word, kStatusDrainTimeout);
        __syncthreads();
    }
    if constexpr (LINE) return;
    float *sums = reinterpret_cast<float *>(smem);
    q4_shares<NT, GATED, false>(acc, sums + (warp >> 1) * C::PART_VALUES, tile, g, t, false);
    __syncthreads();
    if (splits > 1) cluster_wait();           // every CTA of the cluster has started
    // Chunks of 4 columns of the tokens that there are. Each is summed over this CTA's four shares
    // and sent to the CTA of the cluster that adds it up: CTA r has `most` of them from most * r on
    // (the gated form's: of both weights), and a place for those of every CTA.
    constexpr int PER = C::COLS / 4;          // chunks a token (and weight)
    const int n0 = own_n0, m0 = own_m0;
    const int chunks = min(C::TOKENS, args.M - m0) * PER;
    const int most = (chunks + splits - 1) / splits;
    float4 *received = reinterpret_cast<float4 *>(smem + C::OFF_RECEIVE);   // [chunk][CTA][weight]
    for (int i = threadIdx.x; i < C::MATS * chunks; i += kQ4Threads) {
        const int c = i / C::MATS, m = i % C::MATS;
        const float *p = sums + (c / PER) * C::PART_ROW + m * C::COLS + 4 * (c % PER);
        float4 x = *reinterpret_cast<const float4 *>(p);
#pragma unroll
        for (int q = 1; q < 4; ++q)
            add4(x, *reinterpret_cast<const float4 *>(p + q * C::PART_VALUES));
        constexpr float unit = Q4Form<NT>::UNIT;
        x = make_float4(unit * x.x, unit * x.y, unit * x.z, unit * x.w);
        const int to = c / most;              // (every CTA but the last has `most` of them)
        float4 *place = received + ((c - to * most) * splits + rank) * C::MATS + m;
        if (splits > 1)
            st_cluster_f32x4(mapa_shared(smem_u32(place), static_cast<uint32_t>(to)), x);
        else
            *place = x;
    }
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    if (*abort_flag) return;
    const int c0 = min(chunks, most * rank), c1 = min(chunks, c0 + most);
    for (int c = c0 + static_cast<int>(threadIdx.x); c < c1; c += kQ4Threads) {
        const int token = c / PER, col = n0 + 4 * (c % PER);
        if (col >= args.N) continue;          // (N % 8 == 0: all four or none)
        const float4 *p = received + (c - c0) * splits * C::MATS;
        float4 v[C::MATS];
#pragma unroll
        for (int m = 0; m < C::MATS; ++m) v[m] = p[m];
        for (int q = 1; q < splits; ++q)
#pragma unroll
            for (int m = 0; m < C::MATS; ++m) add4(v[m], p[q * C::MATS + m]);
        q4_store<GATED>(args, m0 + token, col, v[0], v[C::MATS - 1]);
    }
}

// The line's cut tiles: block b is the cut between CTAs b and b + 1; the first cut inside a
// tile adds up the sums of all CTAs that have steps of it.
constexpr int kQ4JoinThreads = 128;
template <bool GATED>
__global__ void __launch_bounds__(kQ4JoinThreads) q4_join_kernel(const Q4Args args, int ctas,
                                                                 int tile_tokens) {
    constexpr int MATS = GATED ? 2 : 1, COLS = kQ4Cols / MATS, PER = COLS / 4;
    griddep_launch_dependents();
    griddep_wait();
    const int first = static_cast<int>(blockIdx.x);
    const int cut = q4_line_at(args.units, first + 1, ctas), tile = cut / args.steps;
    const int begins = tile * args.steps, ends = begins + args.steps;
    const int from = q4_line_at(args.units, first, ctas);
    if (cut == begins || from > begins) return;
    int last = first + 1;
    while (q4_line_at(args.units, last + 1, ctas) < ends) ++last;
    const int n0 = tile % args.tiles * COLS, m0 = tile / args.tiles * tile_tokens;
    const int tokens = min(tile_tokens, args.M - m0);
    const size_t size = static_cast<size_t>(tile_tokens) * kQ4Cols;
    // (CTA `first` began with this tile or came to it after another; the others began with it)
    const float *mine = args.partial + (2 * static_cast<size_t>(first) + (from < begins)) * size;
    for (int c = threadIdx.x; c < tokens * PER; c += kQ4JoinThreads) {
        const int token = c / PER, at = 4 * (c % PER);
        if (n0 + at >= args.N) continue;
        float4 v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            const size_t place = static_cast<size_t>(token) * kQ4Cols + m * COLS + at;
            v[m] = *reinterpret_cast<const float4 *>(mine + place);
            for (int q = first + 1; q <= last; ++q)
                add4(v[m], *reinterpret_cast<const float4 *>(args.partial + 2 * size * q + place));
        }
        q4_store<GATED>(args, m0 + token, n0 + at, v[0], v[MATS - 1]);
    }
}

}  // namespace swiglu
