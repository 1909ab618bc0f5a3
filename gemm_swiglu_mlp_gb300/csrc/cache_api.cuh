// Host side of the paged-cache entry points declared in include/swiglu.h:
// argument validation, tensor maps and launches. Included by swiglu_api.cu
// (the library is one translation unit) after its shared helpers.
#pragma once

#include "cache_kernels.cuh"
#include "tree_attention_kernel.cuh"

namespace swiglu {
namespace {

constexpr int64_t kMaxI32 = int64_t(1) << 31;

// log2 of a supported page size (16, 32, 64 or 128 rows), or -1.
int page_shift_of(int64_t page_size) {
    for (int s = 4; s <= 7; ++s)
        if (page_size == (int64_t(1) << s)) return s;
    return -1;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The cache's shape: checked sizes, log2s, and one layer's bytes.
struct CacheShape {
    int page_shift, row_shift;   // log2 of the rows a page and the 16-byte chunks a row
    size_t layer_bytes;
};
int cache_shape(int64_t num_pages, int64_t kv_heads, int64_t page_size, int64_t head_dim,
                CacheShape *out) {
    if (num_pages < 1 || kv_heads < 1 || head_dim < 1 || page_size < 1)
        return SWIGLU_ERR_INVALID_ARG;
    out->page_shift = page_shift_of(page_size);
    if (out->page_shift < 0 || (head_dim != 64 && head_dim != 128) || kv_heads > 65535 ||
        num_pages >= (kMaxI32 >> out->page_shift) || num_pages * kv_heads >= kMaxI32)
        return SWIGLU_ERR_UNSUPPORTED;
    out->row_shift = head_dim == 64 ? 3 : 4;
    out->layer_bytes = static_cast<size_t>(num_pages) * static_cast<size_t>(kv_heads) *
                       static_cast<size_t>(page_size) * static_cast<size_t>(head_dim) * 2;
    return SWIGLU_OK;
}

// Launches `kernel` on `stream` so that its blocks may start while the
// previous launch finishes (every kernel here waits before it touches memory).
template <typename Args>
int launch_overlapped(void (*kernel)(Args), dim3 grid, unsigned threads, size_t smem, void *stream,
                      const Args &args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return SWIGLU_ERR_CUDA;
    }
    return SWIGLU_OK;
}

// Workspace of one attention call: which items go on in another block, and
// two partial results a block (of the item it takes over and of the one it
// leaves).
struct TreeWorkspace {
    int rows;   // of one partial result
    size_t stats, partial, bytes;
};
TreeWorkspace tree_workspace(int64_t tokens, int group, int head_dim, int sms) {
    TreeWorkspace w;
    w.rows = tokens <= kTreeTile / group ? 128 : 256;
    const size_t parts = static_cast<size_t>(2) * sms * w.rows;
    w.stats = static_cast<size_t>(round_up(16 * int64_t(sms), 256));
    w.partial = w.stats + parts * sizeof(float2);
    w.bytes = w.partial + parts * head_dim * sizeof(float);
    return w;
}

// 3-D tensor map over BF16 [d2][d1][d0] with strides s1 and s2 (elements) and
// a 128-byte-swizzled box of 64 x b1 x b2.
bool encode_3d(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
               uint64_t s1, uint64_t s2, uint32_t b1, uint32_t b2) {
    EncodeTiledFn enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {2 * s1, 2 * s2};
    const cuuint32_t box[3] = {64, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over one cache, [pages * heads][page rows][head size] as 5-D
// [pages * heads][groups of 8 rows][64-column halves][8 rows][64]: a box is
// one page of one head and lands as TreeCfg's K and V tiles lie.
bool encode_pages(CUtensorMap *m, const void *base, int64_t head_dim, int64_t page_size,
                  uint64_t pages_heads) {
    EncodeTiledFn enc = get_encode();
    if (!enc) return false;
    const cuuint64_t halves = static_cast<cuuint64_t>(head_dim / 64);
    const cuuint64_t groups = static_cast<cuuint64_t>(page_size / 8);
    const cuuint64_t row = static_cast<cuuint64_t>(head_dim) * 2;
    const cuuint64_t dims[5] = {64, 8, halves, groups, pages_heads};
    const cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(page_size) * row};
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(halves),
                               static_cast<cuuint32_t>(groups), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The attention kernel, one block per SM, and the sums of shared items.
template <int D>
int tree_launch(const CUtensorMap &tmQ, const CUtensorMap &tmQn, const CUtensorMap &tmK,
                const CUtensorMap &tmV, const TreeAttnArgs &a, int sms, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(sms));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = TreeShared<D>::SMEM_BYTES;
    cudaError_t err = cudaLaunchKernelEx(&cfg, tree_attention_kernel<D>, tmQ, tmQn, tmK, tmV, a);
    if (err == cudaSuccess) {
        cfg.gridDim = dim3(static_cast<unsigned>(sms), kJoinBlocks);
        cfg.blockDim = dim3(kJoinThreads);
        cfg.dynamicSmemBytes = 0;
        err = cudaLaunchKernelEx(&cfg, tree_join_kernel<D>, a);
    }
    if (err != cudaSuccess) {
        cudaGetLastError();
        return SWIGLU_ERR_CUDA;
    }
    return SWIGLU_OK;
}

// Bytes from the first to the last element of a [tokens, heads, head_dim]
// BF16 view with the given strides (in elements, not negative).
size_t rows_extent(int64_t tokens, int64_t heads, int64_t head_dim, int64_t tok, int64_t head) {
    return 2 * (static_cast<size_t>(tokens - 1) * tok + static_cast<size_t>(heads - 1) * head +
                head_dim);
}
bool strides_ok(int64_t tok, int64_t head) {
    return tok >= 0 && head >= 0 && (tok % 8) == 0 && (head % 8) == 0 && tok < kMaxI32 &&
           head < kMaxI32;
}

}  // namespace
}  // namespace swiglu

extern "C" {

int swiglu_cache_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *pages_held,
                      int32_t *block_table, int64_t requests, int64_t max_pages,
                      const int32_t *free_pages, int64_t num_free, const int32_t *free_head,
                      int64_t page_size, const int32_t *parents, int64_t tree_width,
                      int64_t max_tokens, int32_t *query_start, int32_t *slots,
                      int32_t *positions, int32_t *pages_held_out, int32_t *counts,
                      int64_t *mask, void *stream) {
    if (requests < 0 || max_tokens < 0 || max_pages < 1 || num_free < 0 || page_size < 1)
        return SWIGLU_ERR_INVALID_ARG;
    if (!query_start || !counts || (max_tokens > 0 && (!slots || !positions)) ||
        (requests > 0 &&
         (!ctx_lens || !new_lens || !pages_held || !block_table || !pages_held_out)) ||
        (num_free > 0 && !free_pages))
        return SWIGLU_ERR_INVALID_ARG;
    if ((parents != nullptr) != (tree_width > 0) || tree_width < 0 ||
        (parents && max_tokens > 0 && !mask))
        return SWIGLU_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(ctx_lens), static_cast<const void *>(new_lens),
                          static_cast<const void *>(pages_held),
                          static_cast<const void *>(block_table),
                          static_cast<const void *>(free_pages),
                          static_cast<const void *>(free_head),
                          static_cast<const void *>(parents),
                          static_cast<const void *>(query_start),
                          static_cast<const void *>(slots), static_cast<const void *>(positions),
                          static_cast<const void *>(pages_held_out),
                          static_cast<const void *>(counts)})
        if (!aligned4(p)) return SWIGLU_ERR_INVALID_ARG;
    if (!aligned8(mask)) return SWIGLU_ERR_INVALID_ARG;
    const int shift = page_shift_of(page_size);
    if (shift < 0 || requests > kPlanMaxRequests || max_tokens >= kMaxI32 ||
        max_pages >= (kMaxI32 >> shift) || num_free >= kMaxI32 || tree_width > (1 << 20))
        return SWIGLU_ERR_UNSUPPORTED;
    // blocks read the inputs while others write outputs
    struct Range { const void *p; size_t n; };
    const size_t R = static_cast<size_t>(requests), T = static_cast<size_t>(max_tokens);
    const int64_t words = parents ? (tree_width + 63) / 64 : 0;
    const Range in[] = {{ctx_lens, 4 * R}, {new_lens, 4 * R}, {pages_held, 4 * R},
                        {free_pages, 4 * static_cast<size_t>(num_free)}, {free_head, 4},
                        {parents, 4 * R * static_cast<size_t>(tree_width)}};
    const Range out[] = {{block_table, 4 * R * static_cast<size_t>(max_pages)},
                         {query_start, 4 * (R + 1)}, {slots, 4 * T}, {positions, 4 * T},
                         {pages_held_out, 4 * R}, {counts, 12},
                         {parents ? mask : nullptr, 8 * T * static_cast<size_t>(words)}};
    const int nout = static_cast<int>(sizeof out / sizeof out[0]);
    for (int i = 0; i < nout; ++i) {
        if (!out[i].p) continue;
        for (const Range &x : in)
            if (x.p && overlaps(out[i].p, out[i].n, x.p, x.n)) return SWIGLU_ERR_INVALID_ARG;
        for (int j = i + 1; j < nout; ++j)
            if (out[j].p && overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
                return SWIGLU_ERR_INVALID_ARG;
    }
    int dev;
    DeviceState *st;
    const int s = device_setup(&dev, &st);
    if (s != SWIGLU_OK) return s;
    CachePlanArgs a{};
    a.ctx_lens = ctx_lens;
    a.new_lens = new_lens;
    a.pages_held = pages_held;
    a.table = block_table;
    a.free_pages = free_pages;
    a.free_head = free_head;
    a.parents = parents;
    a.query_start = query_start;
    a.slots = slots;
    a.positions = positions;
    a.held_out = pages_held_out;
    a.counts = counts;
    a.mask = reinterpret_cast<unsigned long long *>(mask);
    a.max_pages = max_pages;
    a.num_free = num_free;
    a.requests = static_cast<int>(requests);
    a.page_shift = shift;
    a.tree_width = static_cast<int>(tree_width);
    a.mask_words = static_cast<int>(words);
    a.max_tokens = static_cast<int>(max_tokens);
    const int64_t token_blocks = (max_tokens + kPlanThreads - 1) / kPlanThreads;
    const int64_t request_blocks = (requests + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    const int64_t blocks = std::min<int64_t>(
        std::max<int64_t>({token_blocks, request_blocks, 1}), 2 * st->sm_count);
    return launch_overlapped(cache_plan_kernel, dim3(static_cast<unsigned>(blocks)), kPlanThreads,
                             (2 * R + 1) * sizeof(int), stream, a);
}

int swiglu_cache_write(const void *k, const void *v, int64_t tokens, int64_t kv_heads,
                       int64_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                       int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots,
                       void *k_cache, void *v_cache, int64_t num_pages, int64_t page_size,
                       void *stream) {
    if (tokens < 0) return SWIGLU_ERR_INVALID_ARG;
    CacheShape shape;
    const int c = cache_shape(num_pages, kv_heads, page_size, head_dim, &shape);
    if (c != SWIGLU_OK) return c;
    if (!k_cache || !v_cache || (tokens > 0 && (!k || !v || !slots)))
        return SWIGLU_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned4(slots) || !strides_ok(k_token_stride, k_head_stride) ||
        !strides_ok(v_token_stride, v_head_stride))
        return SWIGLU_ERR_INVALID_ARG;
    if (tokens >= kMaxI32) return SWIGLU_ERR_UNSUPPORTED;
    if (overlaps(k_cache, shape.layer_bytes, v_cache, shape.layer_bytes))
        return SWIGLU_ERR_INVALID_ARG;
    if (tokens > 0) {
        const size_t kb = rows_extent(tokens, kv_heads, head_dim, k_token_stride, k_head_stride);
        const size_t vb = rows_extent(tokens, kv_heads, head_dim, v_token_stride, v_head_stride);
        for (const void *cache : {k_cache, v_cache})
            if (overlaps(cache, shape.layer_bytes, k, kb) ||
                overlaps(cache, shape.layer_bytes, v, vb) ||
                overlaps(cache, shape.layer_bytes, slots, 4 * static_cast<size_t>(tokens)))
                return SWIGLU_ERR_INVALID_ARG;
    }
    int dev;
    DeviceState *st;
    const int s = device_setup(&dev, &st);
    if (s != SWIGLU_OK) return s;
    if (tokens == 0) return SWIGLU_OK;
    CacheWriteArgs a{};
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.k_cache = static_cast<uint4 *>(k_cache);
    a.v_cache = static_cast<uint4 *>(v_cache);
    a.slots = slots;
    a.k_tok = k_token_stride / 8;
    a.k_head = k_head_stride / 8;
    a.v_tok = v_token_stride / 8;
    a.v_head = v_head_stride / 8;
    a.num_slots = num_pages << shape.page_shift;
    a.tokens = static_cast<int>(tokens);
    a.kv_heads = static_cast<int>(kv_heads);
    a.row_shift = shape.row_shift;
    a.page_shift = shape.page_shift;
    const int64_t per_token = kv_heads << shape.row_shift;
    a.tokens_per_block = static_cast<int>(std::max<int64_t>(1, kWriteThreads / per_token));
    const int64_t blocks = (tokens + a.tokens_per_block - 1) / a.tokens_per_block;
    return launch_overlapped(cache_write_kernel, dim3(static_cast<unsigned>(blocks)),
                             kWriteThreads, 0, stream, a);
}

int swiglu_cache_accept(void *k_cache, void *v_cache, int64_t layers, int64_t num_pages,
                        int64_t kv_heads, int64_t page_size, int64_t head_dim,
                        const int32_t *block_table, int64_t requests, int64_t max_pages,
                        const int32_t *ctx_lens, const int32_t *paths, int64_t path_width,
                        const int32_t *path_lens, int32_t *ctx_out, void *stream) {
    if (layers < 1 || requests < 0 || max_pages < 1 || path_width < 0)
        return SWIGLU_ERR_INVALID_ARG;
    CacheShape shape;
    const int c = cache_shape(num_pages, kv_heads, page_size, head_dim, &shape);
    if (c != SWIGLU_OK) return c;
    if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache) ||
        (requests > 0 && (!block_table || !ctx_lens || !path_lens || !ctx_out ||
                          (path_width > 0 && !paths))))
        return SWIGLU_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(block_table),
                          static_cast<const void *>(ctx_lens), static_cast<const void *>(paths),
                          static_cast<const void *>(path_lens), static_cast<const void *>(ctx_out)})
        if (!aligned4(p)) return SWIGLU_ERR_INVALID_ARG;
    if (requests >= kMaxI32 || max_pages >= (kMaxI32 >> shape.page_shift) ||
        path_width >= kMaxI32 || layers > 65535)
        return SWIGLU_ERR_UNSUPPORTED;
    const size_t bytes = shape.layer_bytes * static_cast<size_t>(layers);
    const size_t R = static_cast<size_t>(requests);
    if (overlaps(k_cache, bytes, v_cache, bytes)) return SWIGLU_ERR_INVALID_ARG;
    if (requests > 0) {
        struct Range { const void *p; size_t n; };
        const Range in[] = {{block_table, 4 * R * static_cast<size_t>(max_pages)},
                            {ctx_lens, 4 * R}, {path_lens, 4 * R},
                            {paths, 4 * R * static_cast<size_t>(path_width)}};
        for (const Range &x : in)
            if (overlaps(ctx_out, 4 * R, x.p, x.n) || overlaps(k_cache, bytes, x.p, x.n) ||
                overlaps(v_cache, bytes, x.p, x.n))
                return SWIGLU_ERR_INVALID_ARG;
        if (overlaps(ctx_out, 4 * R, k_cache, bytes) || overlaps(ctx_out, 4 * R, v_cache, bytes))
            return SWIGLU_ERR_INVALID_ARG;
    }
    int dev;
    DeviceState *st;
    const int s = device_setup(&dev, &st);
    if (s != SWIGLU_OK) return s;
    if (requests == 0) return SWIGLU_OK;
    CacheAcceptArgs a{};
    a.k_cache = static_cast<uint4 *>(k_cache);
    a.v_cache = static_cast<uint4 *>(v_cache);
    a.table = block_table;
    a.ctx_lens = ctx_lens;
    a.paths = paths;
    a.path_lens = path_lens;
    a.ctx_out = ctx_out;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.layer_chunks = static_cast<long long>(shape.layer_bytes / 16);
    a.columns = (layers * 2 * kv_heads) << shape.row_shift;
    a.path_width = static_cast<int>(path_width);
    a.kv_heads = static_cast<int>(kv_heads);
    a.row_shift = shape.row_shift;
    a.page_shift = shape.page_shift;
    // about eight blocks a SM over all requests, never more than the columns fill
    const int64_t fill = (a.columns + kAcceptThreads - 1) / kAcceptThreads;
    const int64_t want = (8 * int64_t(st->sm_count) + requests - 1) / requests;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({fill, want, 65535}));
    return launch_overlapped(cache_accept_kernel,
                             dim3(static_cast<unsigned>(requests), static_cast<unsigned>(parts)),
                             kAcceptThreads, 0, stream, a);
}

size_t swiglu_tree_attention_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t kv_heads,
                                             int64_t head_dim) {
    if (tokens < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 ||
        q_heads / kv_heads > kTreeTile || (head_dim != 64 && head_dim != 128))
        return 0;
    return tree_workspace(tokens, static_cast<int>(q_heads / kv_heads),
                          static_cast<int>(head_dim), current_sm_count()).bytes;
}

int swiglu_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                          const void *k_cache, const void *v_cache, int64_t num_pages,
                          int64_t page_size, const int32_t *block_table, int64_t requests,
                          int64_t max_pages, const int32_t *ctx_lens, const int32_t *query_start,
                          const int64_t *mask, int64_t mask_words, float scale, void *out,
                          int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (tokens < 0 || requests < 0 || q_heads < 1 || max_pages < 1 || mask_words < 0 ||
        (mask != nullptr) != (mask_words > 0))
        return SWIGLU_ERR_INVALID_ARG;
    CacheShape shape;
    const int c = cache_shape(num_pages, kv_heads, page_size, head_dim, &shape);
    if (c != SWIGLU_OK) return c;
    if (q_heads % kv_heads != 0 || !(scale > 0.f) || !(scale - scale == 0.f)) return SWIGLU_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !query_start || (tokens > 0 && (!q || !out)) ||
        (requests > 0 && (!block_table || !ctx_lens)))
        return SWIGLU_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned4(block_table) || !aligned4(ctx_lens) || !aligned4(query_start) ||
        !aligned8(mask) || !strides_ok(q_token_stride, q_head_stride))
        return SWIGLU_ERR_INVALID_ARG;
    const int64_t group = q_heads / kv_heads;
    if (tokens >= kMaxI32 / 2 || q_heads > 65535 || tokens * q_heads >= kMaxI32 ||
        requests >= kMaxI32 || max_pages >= (kMaxI32 / 2 >> shape.page_shift) ||
        mask_words > (1 << 20) || group > kTreeTile)
        return SWIGLU_ERR_UNSUPPORTED;
    // a tensor map's strides step over whole rows
    if ((tokens > 1 && q_token_stride < head_dim) || (q_heads > 1 && q_head_stride < head_dim))
        return SWIGLU_ERR_INVALID_ARG;
    // what the kernels read while others of their blocks write
    struct Range { const void *p; size_t n; };
    const size_t R = static_cast<size_t>(requests), T = static_cast<size_t>(tokens);
    const size_t obytes = T * static_cast<size_t>(q_heads) * static_cast<size_t>(head_dim) * 2;
    const Range in[] = {
        {q, tokens > 0 ? rows_extent(tokens, q_heads, head_dim, q_token_stride, q_head_stride) : 0},
        {k_cache, shape.layer_bytes},
        {v_cache, shape.layer_bytes},
        {block_table, 4 * R * static_cast<size_t>(max_pages)},
        {ctx_lens, 4 * R},
        {query_start, 4 * (R + 1)},
        {mask, 8 * T * static_cast<size_t>(mask_words)}};
    auto on_input = [&](const void *p, size_t n) {
        for (const Range &x : in)
            if (x.p && overlaps(p, n, x.p, x.n)) return true;
        return false;
    };
    if (tokens > 0 && on_input(out, obytes)) return SWIGLU_ERR_INVALID_ARG;
    int dev;
    DeviceState *st;
    const int s = device_setup(&dev, &st);
    if (s != SWIGLU_OK) return s;
    if (tokens == 0) return SWIGLU_OK;
    const TreeWorkspace ws = tree_workspace(tokens, static_cast<int>(group),
                                            static_cast<int>(head_dim), st->sm_count);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < ws.bytes)
        return SWIGLU_ERR_INVALID_ARG;
    if (overlaps(workspace, ws.bytes, out, obytes) || on_input(workspace, ws.bytes))
        return SWIGLU_ERR_INVALID_ARG;
    TreeAttnArgs a{};
    a.geom.requests = static_cast<int>(requests);
    a.geom.tokens = static_cast<int>(tokens);
    a.geom.kv_heads = static_cast<int>(kv_heads);
    a.geom.group = static_cast<int>(group);
    a.geom.tpt = kTreeTile / static_cast<int>(group);
    a.geom.recip = tree_recip(a.geom.tpt);
    a.geom.causal = mask == nullptr;
    a.geom.max_rows = static_cast<int>(max_pages << shape.page_shift);
    if (!tree_fits(a.geom)) return SWIGLU_ERR_UNSUPPORTED;
    a.table = block_table;
    a.ctx_lens = ctx_lens;
    a.query_start = query_start;
    a.mask = reinterpret_cast<const unsigned long long *>(mask);
    a.v_cache = static_cast<const uint16_t *>(v_cache);
    a.out = static_cast<uint16_t *>(out);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.chains = reinterpret_cast<int4 *>(base);
    a.stats = reinterpret_cast<float2 *>(base + ws.stats);
    a.partial = reinterpret_cast<float4 *>(base + ws.partial);
    a.max_pages = max_pages;
    // (finite, also from the largest and the smallest scales)
    a.scale_log2 = std::min(scale * 1.4426950408889634f, FLT_MAX);   // log2(e)
    a.rise = std::min(kTreeRescale / a.scale_log2, FLT_MAX);
    a.q_heads = static_cast<int>(q_heads);
    a.num_pages = static_cast<int>(num_pages);
    a.page_shift = shape.page_shift;
    a.mask_words = static_cast<int>(mask_words);
    a.part_rows = ws.rows;
#ifdef SWIGLU_TEST_FAULT_INJECTION
    a.skip_first_fill = g_test_skip_first_fill;
#endif
    const uint64_t pages_heads = static_cast<uint64_t>(num_pages) * static_cast<uint64_t>(kv_heads);
    CUtensorMap tmQ, tmQn, tmK, tmV;
    const uint64_t D = static_cast<uint64_t>(head_dim);
    const uint64_t qh = q_heads > 1 ? q_head_stride : D, qt = tokens > 1 ? q_token_stride : D;
    if (!encode_3d(&tmQ, q, D, q_heads, tokens, qh, qt, static_cast<uint32_t>(group),
                   static_cast<uint32_t>(a.geom.tpt)) ||
        !encode_3d(&tmQn, q, D, q_heads, tokens, qh, qt, static_cast<uint32_t>(group),
                   static_cast<uint32_t>(std::max<int64_t>(1, kTreeNarrow / group))) ||
        !encode_pages(&tmK, k_cache, head_dim, page_size, pages_heads) ||
        !encode_pages(&tmV, v_cache, head_dim, page_size, pages_heads))
        return SWIGLU_ERR_CUDA;
    return head_dim == 64 ? tree_launch<64>(tmQ, tmQn, tmK, tmV, a, st->sm_count, stream)
                          : tree_launch<128>(tmQ, tmQn, tmK, tmV, a, st->sm_count, stream);
}

}  // extern "C"
