// Host side of the decode step's other entry points declared in
// include/swiglu.h (head norm and rotation, draft verification, 4-bit
// products): argument validation, tensor maps and launches. Included by
// swiglu_api.cu after cache_api.cuh, whose helpers it shares.
#pragma once

#include "head_rotate_kernel.cuh"
#include "q4_kernel.cuh"
#include "verify_kernel.cuh"

namespace swiglu {
namespace {

struct Range {
    const void *p;
    size_t n;
};
bool overlaps_any(const Range &x, const Range *others, size_t count) {
    for (size_t i = 0; i < count; ++i)
        if (x.p && others[i].p && x.n && others[i].n && overlaps(x.p, x.n, others[i].p, others[i].n))
            return true;
    return false;
}

// [tokens, heads, head_dim] BF16 rows of one argument, strides in elements.
struct Heads {
    const void *p;
    int64_t tok, head;
};
bool heads_ok(const Heads &x, int64_t tokens) {
    return (tokens == 0 || x.p) && aligned16(x.p) && strides_ok(x.tok, x.head);
}
Range heads_range(const Heads &x, int64_t tokens, int64_t heads, int64_t dim) {
    return {x.p, tokens > 0 ? rows_extent(tokens, heads, dim, x.tok, x.head) : 0};
}
// No two rows share an element: heads lie within a token's stride, or tokens within a head's.
bool rows_apart(const Heads &x, int64_t tokens, int64_t heads, int64_t dim) {
    const bool by_token = (heads == 1 || x.head >= dim) &&
                          (tokens == 1 || x.tok >= (heads - 1) * x.head + dim);
    const bool by_head = (tokens == 1 || x.tok >= dim) &&
                         (heads == 1 || x.head >= (tokens - 1) * x.tok + dim);
    return by_token || by_head;
}

// The cache that a rotation writes into.
struct RotateCache {
    Heads v;
    const int32_t *slots;
    void *k_cache, *v_cache;
    int64_t num_pages, page_size;
};

int head_rotate(const Heads &q, const Heads &k, const int32_t *positions, int64_t tokens,
                int64_t q_heads, int64_t kv_heads, int64_t head_dim, const float *inv_freq,
                int64_t freqs, int interleaved, const void *q_weight, const void *k_weight,
                float eps, const Heads &q_out, const Heads &k_out, const RotateCache *cache,
                void *stream) {
    if (tokens < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || !(eps >= 0.f) ||
        !(eps - eps == 0.f))
        return SWIGLU_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || q_heads >= (1 << 20) || kv_heads >= (1 << 20) ||
        tokens >= kMaxI32 || tokens * (q_heads + 2 * kv_heads) >= (kMaxI32 >> 2))
        return SWIGLU_ERR_UNSUPPORTED;
    if (freqs < 0 || (freqs > 0) != (inv_freq != nullptr) || freqs % 8 != 0 || 2 * freqs > head_dim)
        return SWIGLU_ERR_INVALID_ARG;
    if (!heads_ok(q, tokens) || !heads_ok(k, tokens) || !heads_ok(q_out, tokens) ||
        !rows_apart(q_out, tokens, q_heads, head_dim) || (tokens > 0 && !positions) ||
        !aligned4(positions) || !aligned4(inv_freq) || !aligned16(q_weight) || !aligned16(k_weight))
        return SWIGLU_ERR_INVALID_ARG;
    const size_t T = static_cast<size_t>(tokens), D = static_cast<size_t>(head_dim);
    CacheShape shape{};
    Range in[8] = {heads_range(q, tokens, q_heads, head_dim),
                   heads_range(k, tokens, kv_heads, head_dim),
                   {positions, 4 * T},
                   {inv_freq, 4 * static_cast<size_t>(freqs)},
                   {q_weight, 2 * D},
                   {k_weight, 2 * D},
                   {nullptr, 0},
                   {nullptr, 0}};
    Range out[3] = {heads_range(q_out, tokens, q_heads, head_dim), {nullptr, 0}, {nullptr, 0}};
    if (cache) {
        const int c = cache_shape(cache->num_pages, kv_heads, cache->page_size, head_dim, &shape);
        if (c != SWIGLU_OK) return c;
        if (!heads_ok(cache->v, tokens) || !cache->k_cache || !cache->v_cache ||
            !aligned16(cache->k_cache) || !aligned16(cache->v_cache) ||
            (tokens > 0 && !cache->slots) || !aligned4(cache->slots))
            return SWIGLU_ERR_INVALID_ARG;
        in[6] = heads_range(cache->v, tokens, kv_heads, head_dim);
        in[7] = {cache->slots, 4 * T};
        out[1] = {cache->k_cache, shape.layer_bytes};
        out[2] = {cache->v_cache, shape.layer_bytes};
    } else {
        if (!heads_ok(k_out, tokens) || !rows_apart(k_out, tokens, kv_heads, head_dim))
            return SWIGLU_ERR_INVALID_ARG;
        out[1] = heads_range(k_out, tokens, kv_heads, head_dim);
    }
    // in place: the same rows, each read and written by the same lanes. The views of one fused
    // tensor interleave, so their extents say nothing about each other then.
    auto same = [](const Heads &a, const Heads &b) {
        return a.p == b.p && a.tok == b.tok && a.head == b.head;
    };
    const bool q_in_place = same(q, q_out), k_in_place = !cache && same(k, k_out);
    if (q_in_place ? overlaps_any(out[0], in + 2, 4) || overlaps_any(out[0], in + 7, 1)
                   : overlaps_any(out[0], in, 8))
        return SWIGLU_ERR_INVALID_ARG;
    if (k_in_place ? overlaps_any(out[1], in + 2, 4) : overlaps_any(out[1], in, 8))
        return SWIGLU_ERR_INVALID_ARG;
    if (cache && (overlaps_any(out[2], in, 8) || overlaps_any(out[2], out, 2)))
        return SWIGLU_ERR_INVALID_ARG;
    if (!(q_in_place && k_in_place) && overlaps_any(out[1], out, 1)) return SWIGLU_ERR_INVALID_ARG;
    int dev;
    DeviceState *st;
    const int s = device_setup(&dev, &st);
    if (s != SWIGLU_OK) return s;
    if (tokens == 0) return SWIGLU_OK;
    HeadRotateArgs a{};
    a.q = static_cast<const uint4 *>(q.p);
    a.k = static_cast<const uint4 *>(k.p);
    a.q_out = static_cast<uint4 *>(const_cast<void *>(q_out.p));
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_weight = static_cast<const uint4 *>(q_weight);
    a.k_weight = static_cast<const uint4 *>(k_weight);
    a.q_tok = q.tok / 8;
    a.q_head = q.head / 8;
    a.k_tok = k.tok / 8;
    a.k_head = k.head / 8;
    a.qo_tok = q_out.tok / 8;
    a.qo_head = q_out.head / 8;
    if (cache) {
        a.v = static_cast<const uint4 *>(cache->v.p);
        a.v_tok = cache->v.tok / 8;
        a.v_head = cache->v.head / 8;
        a.slots = cache->slots;
        a.k_cache = static_cast<uint4 *>(cache->k_cache);
        a.v_cache = static_cast<uint4 *>(cache->v_cache);
        a.page_shift = shape.page_shift;
        a.num_slots = cache->num_pages << shape.page_shift;
    } else {
        a.k_out = static_cast<uint4 *>(const_cast<void *>(k_out.p));
        a.ko_tok = k_out.tok / 8;
        a.ko_head = k_out.head / 8;
    }
    a.eps = eps;
    a.tokens = static_cast<int>(tokens);
    a.q_heads = static_cast<int>(q_heads);
    a.kv_heads = static_cast<int>(kv_heads);
    a.freqs = static_cast<int>(freqs);
    // two warps a token (more blocks' worth of work to share out evenly: 16384 tokens 98 us), and
    // more for few tokens, as long as the blocks run at once
    const int64_t at_once = 512 / head_dim, room = int64_t(kRotateBlocks) * st->sm_count;
    auto steps = [at_once](int64_t heads) { return (heads + at_once - 1) / at_once; };
    const int64_t all = steps(q_heads) + steps(kv_heads) * (cache ? 2 : 1);
    a.parts = all >= 2 ? 2 : 1;
    while (a.parts < kRotateWarps && 2 * a.parts <= all && tokens * 2 * a.parts <= room * kRotateWarps)
        a.parts *= 2;
    const int64_t blocks =
        std::min<int64_t>((tokens * a.parts + kRotateWarps - 1) / kRotateWarps, room);
    void (*const kernel)(HeadRotateArgs) =
        head_dim == 64 ? (interleaved ? head_rotate_kernel<64, true> : head_rotate_kernel<64, false>)
                       : (interleaved ? head_rotate_kernel<128, true> : head_rotate_kernel<128, false>);
    return launch_overlapped(kernel, dim3(static_cast<unsigned>(blocks)), kRotateThreads, 0, stream, a);
}

// Once a device: the widest tree's shared memory, clusters of more than the portable 8, and the
// largest cluster (a power of two) of which one can run with that much of it: *fits at most.
template <typename T, bool VEC>
bool verify_setup_one(int *fits) {
    auto kernel = verify_kernel<T, VEC>;
    constexpr int bytes = 6 * 4 * kVerifyMaxWidth;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    for (; *fits > 1; *fits /= 2) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(*fits);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(*fits));
        cfg.blockDim = dim3(kVerifyThreads);
        cfg.dynamicSmemBytes = bytes;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0)
            break;
        cudaGetLastError();
    }
    return true;
}
bool verify_setup(DeviceState &st) {
    st.verify_cluster = kVerifyMaxCluster;
    int *fits = &st.verify_cluster;
    return verify_setup_one<float, true>(fits) && verify_setup_one<float, false>(fits) &&
           verify_setup_one<__nv_bfloat16, true>(fits) && verify_setup_one<__nv_bfloat16, false>(fits);
}
// device_setup and, with that device's first verification of probabilities, its own.
int verify_device(DeviceState **st) {
    int dev;
    const int s = device_setup(&dev, st);
    if (s != SWIGLU_OK) return s;
    DeviceState &d = **st;
    std::call_once(d.verify_once, [&d] {
        if (verify_setup(d)) return;
        cudaGetLastError();
        d.verify_status = SWIGLU_ERR_CUDA;
    });
    return d.verify_status;
}

// One 4-bit product: out [M, N] from A [M, K], or the gated form with Q2 and S2.
struct Q4Problem {
    const void *A, *Q1, *S1, *Q2, *S2;
    void *out;
    int64_t M, N, K, group;
    void *workspace;             // optional: without it whole tiles
    size_t workspace_bytes;
    size_t code_bytes() const { return static_cast<size_t>(N) * static_cast<size_t>(K / 2); }
    size_t scale_bytes() const {
        return static_cast<size_t>((K + group - 1) / group) * static_cast<size_t>(N) * 2;
    }
};

int q4_check(const Q4Problem &p, bool gated) {
    if (!p.A || !p.Q1 || !p.S1 || !p.out || (gated && (!p.Q2 || !p.S2)) || p.M < 1 || p.N < 8 ||
        p.K < 32 || p.N % 8 != 0 || p.K % 32 != 0)
        return SWIGLU_ERR_INVALID_ARG;
    for (const void *x : {p.A, p.Q1, p.S1, p.Q2, p.S2, static_cast<const void *>(p.out)})
        if (!aligned16(x)) return SWIGLU_ERR_INVALID_ARG;
    if (p.group != 32 && p.group != 64 && p.group != 128) return SWIGLU_ERR_UNSUPPORTED;
    if (p.N >= kMaxI32 || p.K >= kMaxI32 || p.M > (1 << 20)) return SWIGLU_ERR_UNSUPPORTED;
    const Range in[] = {{p.A, static_cast<size_t>(p.M) * static_cast<size_t>(p.K) * 2},
                        {p.Q1, p.code_bytes()}, {p.S1, p.scale_bytes()},
                        {p.Q2, p.code_bytes()}, {p.S2, p.scale_bytes()}};
    const Range out{p.out, static_cast<size_t>(p.M) * static_cast<size_t>(p.N) * 2};
    const Range ws{p.workspace, p.workspace ? p.workspace_bytes : 0};
    if ((reinterpret_cast<uintptr_t>(p.workspace) & 255u) != 0 || overlaps_any(out, in, 5) ||
        overlaps_any(ws, in, 5) || overlaps_any(ws, &out, 1))
        return SWIGLU_ERR_INVALID_ARG;
    return SWIGLU_OK;
}

// Tensor map over scales [groups][columns] BF16; a box has one step's groups.
bool encode_scales(CUtensorMap *m, const void *base, uint64_t columns, uint64_t groups,
                   uint32_t box_columns, uint32_t box_groups) {
    EncodeTiledFn enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[2] = {columns, groups};
    const cuuint64_t strides[1] = {2 * columns};
    const cuuint32_t box[2] = {box_columns, box_groups};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shares of K of each of `tiles` tiles: the most that let all CTAs run at once, of two steps at
// least (one token of 18944 x 3584: 1 share 39.1 us, 4 17.2, 8 10.9, 10 10.0; 76 tiles of 4
// steps: 1 share 3.7 us, 2 3.4, 4, whose clusters no longer run at once, 6.5).
int q4_splits(int64_t tiles, int steps, const int *clusters) {
    for (int j = std::min(kQ4MaxSplits, steps / 2); j > 1; --j)
        if (tiles <= clusters[j]) return j;
    return 1;
}

// How one product is shared out.
struct Q4Plan {
    int tiles, blocks, splits;   // tiles of columns, blocks of tokens, shares of K of each
    int line_ctas;               // more than 0: one line of steps, over so many CTAs ...
    size_t workspace;            // ... with this much workspace
};
template <int NT, bool GATED, int GROUPS>
Q4Plan q4_plan(const Q4Problem &p, const DeviceState &st) {
    using C = Q4Cfg<NT, GATED, GROUPS>;
    const int *clusters = C::CTAS == 1 ? st.q4_clusters_1 : st.q4_clusters_2;
    const int steps = static_cast<int>((p.K + kQ4Step - 1) / kQ4Step);
    Q4Plan x{};
    x.tiles = static_cast<int>((p.N + C::COLS - 1) / C::COLS);
    x.blocks = static_cast<int>((p.M + C::TOKENS - 1) / C::TOKENS);
    const int64_t all = int64_t(x.tiles) * x.blocks, sms = st.sm_count;
    x.splits = q4_splits(all, steps, clusters);
    // Whole tiles: the SMs with one more than the average decide. Where that is worth more than
    // cutting the line costs (a launch, cut tiles' sums: 3 us, an SM's time for 8 steps), the line
    // (462 tiles of 32 steps, 16 tokens: 77 -> 69 us; of one, with halves of groups of 128 summed
    // apart, 55 -> 49, and 188 of 16 steps 15.7 -> 15.2; both 47 and 14.5 now).
    if (x.splits == 1 && all * steps < (int64_t(1) << 30) && clusters[1] > 1 &&
        ((all + sms - 1) / sms * sms - all) * steps > 8 * sms) {
        x.line_ctas = clusters[1];
        x.workspace = static_cast<size_t>(x.line_ctas) * 2 * C::TOKENS * kQ4Cols * sizeof(float);
    }
    return x;
}

template <int NT, bool GATED, int GROUPS>
int q4_launch(const Q4Problem &p, const DeviceState &st, void *stream) {
    using C = Q4Cfg<NT, GATED, GROUPS>;
    CUtensorMap tmA, tmQ1, tmQ2, tmS1, tmS2;
    const uint64_t N = static_cast<uint64_t>(p.N), K = static_cast<uint64_t>(p.K);
    const uint64_t groups = (K + p.group - 1) / p.group;
    const uint32_t per_step = static_cast<uint32_t>(kQ4Step / p.group);
    if (!encode_2d(&tmA, p.A, K, static_cast<uint64_t>(p.M), 64, C::TOKENS) ||
        !encode_2d(&tmQ1, p.Q1, K / 2, N, kQ4Step / 2, C::COLS, true) ||
        !encode_scales(&tmS1, p.S1, N, groups, C::COLS, per_step))
        return SWIGLU_ERR_CUDA;
    tmQ2 = tmQ1;                 // (used by the gated form only)
    tmS2 = tmS1;
    if (GATED && (!encode_2d(&tmQ2, p.Q2, K / 2, N, kQ4Step / 2, C::COLS, true) ||
                  !encode_scales(&tmS2, p.S2, N, groups, C::COLS, per_step)))
        return SWIGLU_ERR_CUDA;
    Q4Args a{};
    a.out = static_cast<uint16_t *>(p.out);
    a.M = static_cast<int>(p.M);
    a.N = static_cast<int>(p.N);
    a.steps = static_cast<int>((p.K + kQ4Step - 1) / kQ4Step);
    a.group_shift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
#ifdef SWIGLU_TEST_FAULT_INJECTION
    a.skip_first_fill = g_test_skip_first_fill;
#endif
    const Q4Plan plan = q4_plan<NT, GATED, GROUPS>(p, st);
    a.tiles = plan.tiles;
    a.splits = plan.splits;
    const int64_t all = int64_t(plan.tiles) * plan.blocks;
    if (all * a.splits >= kMaxI32) return SWIGLU_ERR_UNSUPPORTED;
    const bool line = plan.line_ctas > 0 && p.workspace && p.workspace_bytes >= plan.workspace;
    a.units = line ? static_cast<int>(all * a.steps) : 0;
    a.partial = static_cast<float *>(p.workspace);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    cfg.gridDim = dim3(static_cast<unsigned>(line ? plan.line_ctas : all * a.splits));
    cfg.blockDim = dim3(line ? kQ4LineThreads : kQ4Threads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaError_t err =
        cudaLaunchKernelEx(&cfg, line ? q4_kernel<NT, GATED, GROUPS, true>
                                      : q4_kernel<NT, GATED, GROUPS, false>,
                           tmA, tmQ1, tmQ2, tmS1, tmS2, a);
    if (err == cudaSuccess && line) {
        cfg.gridDim = dim3(static_cast<unsigned>(plan.line_ctas - 1));
        cfg.blockDim = dim3(kQ4JoinThreads);
        cfg.dynamicSmemBytes = 0;
        cfg.numAttrs = 1;
        err = cudaLaunchKernelEx(&cfg, q4_join_kernel<GATED>, a, plan.line_ctas,
                                 static_cast<int>(C::TOKENS));
    }
    if (err != cudaSuccess) {
        cudaGetLastError();
        return SWIGLU_ERR_CUDA;
    }
    return SWIGLU_OK;
}

// By the token rows of a CTA (8, 16 or 32) and the group: f(the kernel's template arguments).
template <int NT, int GROUPS>
struct Q4Choice {
    static constexpr int nt = NT, groups = GROUPS;
};
template <typename F>
auto q4_choose(int64_t M, int64_t group, F f) {
    if (group == 32)
        return M <= 8 ? f(Q4Choice<1, 4>{}) : M <= 16 ? f(Q4Choice<2, 4>{}) : f(Q4Choice<4, 4>{});
    if (M <= 8) return group == 64 ? f(Q4Choice<1, 2>{}) : f(Q4Choice<1, 1>{});
    return M <= 16 ? f(Q4Choice<2, 2>{}) : f(Q4Choice<4, 2>{});
}
template <bool GATED>
int q4_forward(const Q4Problem &p, const DeviceState &st, void *stream) {
    return q4_choose(p.M, p.group, [&](auto c) {
        return q4_launch<decltype(c)::nt, GATED, decltype(c)::groups>(p, st, stream);
    });
}

// Once a device: the kernels' shared memory and cluster sizes, and how many clusters of j CTAs
// run at once, two CTAs an SM (16 tokens' kernel) or one (32 tokens').
template <int NT, bool GATED, int GROUPS>
bool q4_setup_one() {
    auto kernel = q4_kernel<NT, GATED, GROUPS, false>;
    constexpr int bytes = Q4Cfg<NT, GATED, GROUPS>::SMEM_BYTES;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
               cudaSuccess &&
           cudaFuncSetAttribute(q4_kernel<NT, GATED, GROUPS, true>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
               cudaSuccess;
}
template <int NT>
bool q4_setup_rows(int sms, int *clusters) {
    using C = Q4Cfg<NT, true, 2>;
    if (!q4_setup_one<NT, true, 2>() || !q4_setup_one<NT, true, 4>() ||
        !q4_setup_one<NT, false, 2>() || !q4_setup_one<NT, false, 4>())
        return false;
    if (!clusters) return true;
    for (int j = 1; j <= kQ4MaxSplits; ++j) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(j);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(j * std::max(1, C::CTAS * sms / j)));
        cfg.blockDim = dim3(kQ4Threads);
        cfg.dynamicSmemBytes = C::SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&clusters[j], q4_kernel<NT, true, 2, false>,
                                           &cfg) != cudaSuccess) {
            cudaGetLastError();
            clusters[j] = 0;
        }
    }
    return true;
}
bool q4_setup(DeviceState &st) {
    return q4_setup_one<1, true, 1>() && q4_setup_one<1, false, 1>() &&
           q4_setup_rows<1>(st.sm_count, nullptr) && q4_setup_rows<2>(st.sm_count, st.q4_clusters_2) &&
           q4_setup_rows<4>(st.sm_count, st.q4_clusters_1);
}
// device_setup and, with that device's first 4-bit product (or its workspace's size), its own.
int q4_device(DeviceState **st) {
    int dev;
    const int s = device_setup(&dev, st);
    if (s != SWIGLU_OK) return s;
    DeviceState &d = **st;
    std::call_once(d.q4_once, [&d] {
        if (q4_setup(d)) return;
        cudaGetLastError();
        d.q4_status = SWIGLU_ERR_CUDA;
    });
    return d.q4_status;
}

// Workspace of one product on the current device.
template <bool GATED>
size_t q4_workspace(int64_t M, int64_t N, int64_t K, int64_t group) {
    if (M < 1 || M > (1 << 20) || N < 8 || K < 32 || N >= kMaxI32 || K >= kMaxI32 ||
        (group != 32 && group != 64 && group != 128))
        return 0;
    DeviceState *st;
    if (q4_device(&st) != SWIGLU_OK) return 0;
    Q4Problem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.group = group;
    return q4_choose(M, group, [&](auto c) {
        return q4_plan<decltype(c)::nt, GATED, decltype(c)::groups>(p, *st).workspace;
    });
}

}  // namespace
}  // namespace swiglu

extern "C" {

int swiglu_head_rotate(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                       const void *k, int64_t k_token_stride, int64_t k_head_stride,
                       const int32_t *positions, int64_t tokens, int64_t q_heads,
                       int64_t kv_heads, int64_t head_dim, const float *inv_freq, int64_t freqs,
                       int interleaved, const void *q_weight, const void *k_weight, float eps,
                       void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                       void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                       void *stream) {
    return head_rotate({q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                       positions, tokens, q_heads, kv_heads, head_dim, inv_freq, freqs, interleaved,
                       q_weight, k_weight, eps, {q_out, q_out_token_stride, q_out_head_stride},
                       {k_out, k_out_token_stride, k_out_head_stride}, nullptr, stream);
}

int swiglu_head_rotate_write(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                             const void *k, int64_t k_token_stride, int64_t k_head_stride,
                             const void *v, int64_t v_token_stride, int64_t v_head_stride,
                             const int32_t *positions, const int32_t *slots, int64_t tokens,
                             int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                             const float *inv_freq, int64_t freqs, int interleaved,
                             const void *q_weight, const void *k_weight, float eps, void *q_out,
                             int64_t q_out_token_stride, int64_t q_out_head_stride,
                             void *k_cache, void *v_cache, int64_t num_pages, int64_t page_size,
                             void *stream) {
    const RotateCache cache{{v, v_token_stride, v_head_stride}, slots, k_cache, v_cache, num_pages,
                            page_size};
    return head_rotate({q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                       positions, tokens, q_heads, kv_heads, head_dim, inv_freq, freqs, interleaved,
                       q_weight, k_weight, eps, {q_out, q_out_token_stride, q_out_head_stride},
                       {nullptr, 0, 0}, &cache, stream);
}

int swiglu_verify_drafts(const int32_t *tokens, int64_t rows, const int32_t *query_start,
                         int64_t requests, const int32_t *parents, int64_t tree_width,
                         const void *target, int64_t target_stride, int value_type,
                         const void *draft, int64_t draft_stride, int64_t vocab,
                         const float *uniform, int32_t *paths, int32_t *path_lens,
                         int32_t *next_tokens, void *stream) {
    if (rows < 0 || requests < 0 || tree_width < 1 || value_type < SWIGLU_TARGET_FP32 ||
        value_type > SWIGLU_TARGET_TOKENS || !query_start)
        return SWIGLU_ERR_INVALID_ARG;
    const bool greedy = value_type == SWIGLU_TARGET_TOKENS;
    if (greedy ? draft || uniform || vocab || target_stride || draft_stride
               : vocab < 1 || target_stride < vocab || (draft ? draft_stride < vocab : draft_stride != 0))
        return SWIGLU_ERR_INVALID_ARG;
    if ((rows > 0 && (!tokens || !target || (!greedy && !uniform))) ||
        (requests > 0 && (!paths || !path_lens || !next_tokens)))
        return SWIGLU_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(tokens), static_cast<const void *>(query_start),
                          static_cast<const void *>(parents), static_cast<const void *>(uniform),
                          static_cast<const void *>(paths), static_cast<const void *>(path_lens),
                          static_cast<const void *>(next_tokens)})
        if (!aligned4(p)) return SWIGLU_ERR_INVALID_ARG;
    const uintptr_t odd = value_type == SWIGLU_TARGET_BF16 ? 1 : 3;
    if ((reinterpret_cast<uintptr_t>(target) & odd) || (reinterpret_cast<uintptr_t>(draft) & odd))
        return SWIGLU_ERR_INVALID_ARG;
    if (rows >= kMaxI32 || requests >= (1 << 27) || tree_width > kVerifyMaxWidth ||
        vocab > kVerifyMaxVocab || target_stride >= kMaxI32 || draft_stride >= kMaxI32)
        return SWIGLU_ERR_UNSUPPORTED;
    const size_t T = static_cast<size_t>(rows), R = static_cast<size_t>(requests),
                 W = static_cast<size_t>(tree_width), size = value_type == SWIGLU_TARGET_BF16 ? 2 : 4;
    auto table = [&](const void *p, int64_t stride) -> Range {
        return {p, T ? size * ((T - 1) * static_cast<size_t>(stride) + static_cast<size_t>(vocab)) : 0};
    };
    const Range in[] = {{tokens, 4 * T}, {query_start, 4 * (R + 1)}, {parents, 4 * R * W},
                        greedy ? Range{target, 4 * T} : table(target, target_stride),
                        table(draft, draft_stride), {uniform, 4 * T}};
    const Range out[] = {{paths, 4 * R * W}, {path_lens, 4 * R}, {next_tokens, 4 * R}};
    for (int i = 0; i < 3; ++i)
        if (overlaps_any(out[i], in, 6) || overlaps_any(out[i], out, i)) return SWIGLU_ERR_INVALID_ARG;
    int dev;
    DeviceState *st;
    const int s = greedy ? device_setup(&dev, &st) : verify_device(&st);
    if (s != SWIGLU_OK) return s;
    if (requests == 0) return SWIGLU_OK;
    VerifyArgs a{};
    a.tokens = tokens;
    a.query_start = query_start;
    a.parents = parents;
    a.target = greedy ? nullptr : target;
    a.draft = draft;
    a.following = greedy ? static_cast<const int *>(target) : nullptr;
    a.uniform = uniform;
    a.paths = paths;
    a.path_lens = path_lens;
    a.next = next_tokens;
    a.target_stride = target_stride;
    a.draft_stride = draft_stride;
    a.rows = static_cast<int>(rows);
    a.width = static_cast<int>(tree_width);
    a.vocab = static_cast<int>(vocab);
#ifdef SWIGLU_TEST_FAULT_INJECTION
    a.skip_first_fill = g_test_skip_first_fill;
#endif
    if (greedy)
        return launch_overlapped(verify_greedy_kernel, dim3(static_cast<unsigned>(requests)), 32,
                                 sizeof(int) * W, stream, a);
    // rows that lie on whole vectors of four values: read by them
    const uintptr_t vec = 4 * size - 1;
    const bool by_four = ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) &
                          vec) == 0 && target_stride % 4 == 0 && draft_stride % 4 == 0;
    const int ctas = verify_ctas(requests, vocab, st->sm_count, st->verify_cluster);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(static_cast<unsigned>(requests * ctas));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = 6 * sizeof(int) * W;
    const bool bf16 = value_type == SWIGLU_TARGET_BF16;
    void (*const kernel)(VerifyArgs) =
        by_four ? (bf16 ? verify_kernel<__nv_bfloat16, true> : verify_kernel<float, true>)
                : (bf16 ? verify_kernel<__nv_bfloat16, false> : verify_kernel<float, false>);
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return SWIGLU_ERR_CUDA;
    }
    return SWIGLU_OK;
}

size_t swiglu_up_q4_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t group) {
    return q4_workspace<true>(M, N, K, group);
}

size_t swiglu_down_q4_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t group) {
    return q4_workspace<false>(M, K, N, group);
}

size_t swiglu_mlp_q4_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t group) {
    return std::max(q4_workspace<true>(M, N, K, group), q4_workspace<false>(M, K, N, group));
}

int swiglu_up_forward_q4(const void *A, const void *Q1, const void *S1, const void *Q2,
                         const void *S2, void *Y, int64_t M, int64_t N, int64_t K, int64_t group,
                         void *workspace, size_t workspace_bytes, void *stream) {
    const Q4Problem up{A, Q1, S1, Q2, S2, Y, M, N, K, group, workspace, workspace_bytes};
    DeviceState *st;
    int s = q4_check(up, true);
    if (s == SWIGLU_OK) s = q4_device(&st);
    return s == SWIGLU_OK ? q4_forward<true>(up, *st, stream) : s;
}

int swiglu_down_forward_q4(const void *Y, const void *Q3, const void *S3, void *out, int64_t M,
                           int64_t N, int64_t K, int64_t group, void *workspace,
                           size_t workspace_bytes, void *stream) {
    const Q4Problem down{Y, Q3, S3, nullptr, nullptr, out, M, K, N, group, workspace,
                         workspace_bytes};
    DeviceState *st;
    int s = q4_check(down, false);
    if (s == SWIGLU_OK) s = q4_device(&st);
    return s == SWIGLU_OK ? q4_forward<false>(down, *st, stream) : s;
}

int swiglu_mlp_forward_q4(const void *A, const void *Q1, const void *S1, const void *Q2,
                          const void *S2, const void *Q3, const void *S3, void *Y, void *out,
                          int64_t M, int64_t N, int64_t K, int64_t group, void *workspace,
                          size_t workspace_bytes, void *stream) {
    const Q4Problem up{A, Q1, S1, Q2, S2, Y, M, N, K, group, workspace, workspace_bytes};
    const Q4Problem down{Y, Q3, S3, nullptr, nullptr, out, M, K, N, group, workspace,
                         workspace_bytes};
    int s = q4_check(up, true);
    if (s == SWIGLU_OK) s = q4_check(down, false);
    if (s != SWIGLU_OK) return s;
    // neither output on what the other product reads
    const Range of_up[] = {{A, static_cast<size_t>(M) * static_cast<size_t>(K) * 2},
                           {Q1, up.code_bytes()}, {S1, up.scale_bytes()},
                           {Q2, up.code_bytes()}, {S2, up.scale_bytes()}};
    const Range of_down[] = {{Q3, down.code_bytes()}, {S3, down.scale_bytes()}};
    if (overlaps_any({out, static_cast<size_t>(M) * static_cast<size_t>(K) * 2}, of_up, 5) ||
        overlaps_any({Y, static_cast<size_t>(M) * static_cast<size_t>(N) * 2}, of_down, 2))
        return SWIGLU_ERR_INVALID_ARG;
    DeviceState *st;
    s = q4_device(&st);
    if (s == SWIGLU_OK) s = q4_forward<true>(up, *st, stream);
    return s == SWIGLU_OK ? q4_forward<false>(down, *st, stream) : s;
}

}  // extern "C"
