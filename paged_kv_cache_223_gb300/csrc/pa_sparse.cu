// pa_sparse.cu -- the sparse decode step's part of the C ABI declared in include/pagedattn.h: argument validation and
// kernel launches. The kernels are those of tables.cu, select_blocks.cu and selected.cu.
#include <algorithm>
#include <cmath>

#include "pa_pool.h"
#include "pa_sparse.h"

using namespace pa;

pa_status pa::group_map(pa_pool *pool, const void *cache, CUtensorMap *out) {
    std::lock_guard<std::mutex> lk(pool->mu);
    const auto it = pool->group_maps.find(cache);
    if (it != pool->group_maps.end()) {
        *out = it->second;
        return PA_OK;
    }
    const auto fn = encode_fn();
    if (!fn) return PA_ERR_CUDA;
    const pa_pool_config &c = pool->cfg;
    const cuuint64_t row = (cuuint64_t)c.head_dim * 2, halves = (cuuint64_t)c.head_dim / 64;
    const cuuint64_t dims[4] = {64, 8, halves, (cuuint64_t)c.num_blocks * c.num_kv_heads * c.block_size / 8};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)halves, TILE_TOKENS / 8}, estr[4] = {1, 1, 1, 1};
    CUtensorMap m;
    if (fn(&m, c.dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
           const_cast<void *>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return PA_ERR_CUDA;
    keep_map(pool->group_maps, cache, m);
    *out = m;
    return PA_OK;
}

namespace {

constexpr int64_t MAX_CONTEXT = (int64_t)1 << 29;

struct Span {
    const void *at;
    uint64_t bytes;
};

bool meet(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.bytes && b.bytes && (x <= y ? y - x < a.bytes : x - y < b.bytes);
}

bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

int max_len_of(const pa_pool_config &c, int32_t stride) {
    return (int)std::min((int64_t)stride * c.block_size, MAX_CONTEXT);
}

pa_status launched(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    cudaGetLastError();                                // not left behind for the next caller that asks for the last error
    return PA_ERR_CUDA;
}

uint64_t bounds_codes(const pa_pool_config &c) { return (uint64_t)c.num_blocks * c.num_kv_heads * 2 * c.head_dim; }
uint64_t bounds_bytes(const pa_pool_config &c) { return bounds_codes(c) + (uint64_t)c.num_blocks * c.num_kv_heads * 4; }

// The sizes that selection and attention share.
pa_status row_sizes(const pa_pool_config &c, int32_t stride, int32_t num_seqs, int32_t num_q_heads, int32_t q_len,
                    int32_t budget) {
    if (stride < 1 || num_seqs < 0 || num_q_heads < 1 || num_q_heads % c.num_kv_heads != 0 || q_len < 1 || budget < 1)
        return PA_ERR_INVALID_ARG;
    if ((int64_t)(num_q_heads / c.num_kv_heads) * q_len > MAX_ROWS || budget > PA_SELECT_MAX_BUDGET ||
        (int64_t)num_seqs * c.num_kv_heads >= (int64_t)1 << 27)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_step_tables(pa_pool *pool, const pa_tables_args *a, void *stream) {
    if (!pool || !a || a->num_seqs < 0 || a->num_tokens < 0 || a->block_table_stride < 1) return PA_ERR_INVALID_ARG;
    if (a->num_seqs > PA_TABLES_MAX_SEQS || a->num_tokens > PA_TABLES_MAX_TOKENS) return PA_ERR_UNSUPPORTED;
    const pa_pool_config &c = pool->cfg;
    const uint64_t n = a->num_seqs, t = a->num_tokens;
    if (!a->cu_q || !a->num_free || !a->free_blocks || (n && (!a->new_lens || !a->context_lens || !a->block_tables)) ||
        (t && (!a->positions || !a->slot_mapping)))
        return PA_ERR_INVALID_ARG;
    const Span in[] = {{a->new_lens, 4 * n}, {a->keep_lens, a->keep_lens ? 4 * n : 0}};
    const Span out[] = {{a->context_lens, 4 * n}, {a->block_tables, 4 * n * a->block_table_stride},
                        {a->free_blocks, 4 * (uint64_t)c.num_blocks}, {a->num_free, 4}, {a->cu_q, 4 * (n + 1)},
                        {a->positions, 4 * t}, {a->slot_mapping, 8 * t}};
    for (const Span &s : in) {
        if (!aligned(s.at, 4)) return PA_ERR_INVALID_ARG;
        for (const Span &o : out)
            if (meet(s, o) && !(o.at == a->context_lens && s.at == o.at)) return PA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 7; ++i) {
        if (!aligned(out[i].at, i == 6 ? 8 : 4)) return PA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return PA_ERR_INVALID_ARG;
    }
    TablesParams p;
    p.num_seqs = a->num_seqs;
    p.num_tokens = a->num_tokens;
    p.block_tables = a->block_tables;
    p.stride = a->block_table_stride;
    p.context_lens = a->context_lens;
    p.keep_lens = a->keep_lens;
    p.new_lens = a->new_lens;
    p.free_blocks = a->free_blocks;
    p.num_free = a->num_free;
    p.cu_q = a->cu_q;
    p.positions = a->positions;
    p.slots = a->slot_mapping;
    p.bs_shift = c.block_size == 16 ? 4 : 5;
    p.num_blocks = c.num_blocks;
    p.max_len = max_len_of(c, a->block_table_stride);
    p.status = pool->status;
    DeviceGuard g(c.device);
    if (!g.ok) return PA_ERR_CUDA;
    return launched(launch_tables(p, pool->sm_count, static_cast<cudaStream_t>(stream)));
}

pa_status pa_key_bounds_size(const pa_pool *pool, uint64_t *bytes) {
    if (!pool || !bytes) return PA_ERR_INVALID_ARG;
    *bytes = bounds_bytes(pool->cfg);
    return PA_OK;
}

pa_status pa_key_bounds(pa_pool *pool, const void *k_cache, const int32_t *cu_q, const int32_t *block_tables,
                        int32_t block_table_stride, const int32_t *context_lens, int32_t num_tokens, int32_t num_seqs,
                        void *bounds, void *stream) {
    if (!pool || num_tokens < 0 || num_seqs < 0 || block_table_stride < 1) return PA_ERR_INVALID_ARG;
    if (num_seqs > PA_TABLES_MAX_SEQS) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    const pa_pool_config &c = pool->cfg;
    if (!k_cache) k_cache = pool->k_cache;
    if (!cu_q || !block_tables || !context_lens || !bounds || !aligned16(k_cache) || !aligned(bounds, 32) ||
        !aligned(cu_q, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    const Span out = {bounds, bounds_bytes(c)};
    const uint64_t n = num_seqs;
    if (meet(out, {k_cache, pool->cache_bytes}) || meet(out, {cu_q, 4 * (n + 1)}) || meet(out, {context_lens, 4 * n}) ||
        meet(out, {block_tables, 4 * n * block_table_stride}))
        return PA_ERR_INVALID_ARG;
    BoundsParams p;
    p.k_cache = k_cache;
    p.k_scales = c.kv_format == PA_KV_FP8_E4M3
                     ? reinterpret_cast<const float *>(static_cast<const uint8_t *>(k_cache) + bounds_codes(c) / 2 * c.block_size)
                     : nullptr;
    p.cu_q = cu_q;
    p.block_tables = block_tables;
    p.stride = block_table_stride;
    p.context_lens = context_lens;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.Hkv = c.num_kv_heads;
    p.bs = c.block_size;
    p.num_blocks = c.num_blocks;
    p.max_len = max_len_of(c, block_table_stride);
    p.codes = static_cast<int8_t *>(bounds);
    p.steps = reinterpret_cast<float *>(static_cast<uint8_t *>(bounds) + bounds_codes(c));
    p.status = pool->status;
    DeviceGuard g(c.device);
    if (!g.ok) return PA_ERR_CUDA;
    return launched(launch_key_bounds(p, c.dtype, c.head_dim, pool->sm_count, static_cast<cudaStream_t>(stream)));
}

pa_status pa_select_blocks(pa_pool *pool, const void *q, const void *bounds, const int32_t *block_tables,
                           int32_t block_table_stride, const int32_t *context_lens, int32_t num_seqs,
                           int32_t num_q_heads, int32_t q_len, int32_t budget, int32_t num_first, int32_t num_last,
                           int32_t *selected, void *stream) {
    if (!pool || num_first < 0 || num_last < 0) return PA_ERR_INVALID_ARG;
    const pa_pool_config &c = pool->cfg;
    const pa_status st = row_sizes(c, block_table_stride, num_seqs, num_q_heads, q_len, budget);
    if (st != PA_OK) return st;
    if (block_table_stride > PA_SELECT_MAX_BLOCKS) return PA_ERR_UNSUPPORTED;
    if (num_last < (q_len - 2 + c.block_size) / c.block_size + 1 || (int64_t)num_first + num_last > budget)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!q || !bounds || !block_tables || !context_lens || !selected || !aligned16(q) || !aligned(bounds, 32) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(selected, 4))
        return PA_ERR_INVALID_ARG;
    const uint64_t n = num_seqs;
    const Span out = {selected, 4 * n * c.num_kv_heads * budget};
    if (meet(out, {q, 2 * n * q_len * num_q_heads * c.head_dim}) || meet(out, {bounds, bounds_bytes(c)}) ||
        meet(out, {context_lens, 4 * n}) || meet(out, {block_tables, 4 * n * block_table_stride}))
        return PA_ERR_INVALID_ARG;
    SelectParams p;
    p.q = q;
    p.codes = static_cast<const int8_t *>(bounds);
    p.steps = reinterpret_cast<const float *>(static_cast<const uint8_t *>(bounds) + bounds_codes(c));
    p.block_tables = block_tables;
    p.stride = block_table_stride;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.Hq = num_q_heads;
    p.Hkv = c.num_kv_heads;
    p.G = num_q_heads / c.num_kv_heads;
    p.q_len = q_len;
    p.rows = p.G * q_len;
    p.bs = c.block_size;
    p.num_blocks = c.num_blocks;
    p.max_len = max_len_of(c, block_table_stride);
    p.budget = budget;
    p.num_first = num_first;
    p.num_last = num_last;
    p.selected = selected;
    p.status = pool->status;
    DeviceGuard g(c.device);
    if (!g.ok) return PA_ERR_CUDA;
    return launched(launch_select(p, c.dtype, c.head_dim, pool->sm_count, static_cast<cudaStream_t>(stream)));
}

pa_status pa_decode_selected(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *selected, int32_t budget, const int32_t *block_tables,
                             int32_t block_table_stride, const int32_t *context_lens, int32_t num_seqs,
                             int32_t num_q_heads, int32_t q_len, float scale, void *out, void *stream) {
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!pool || !std::isfinite(scale_log2) || (k_cache == nullptr) != (v_cache == nullptr)) return PA_ERR_INVALID_ARG;
    const pa_pool_config &c = pool->cfg;
    pa_status st = row_sizes(c, block_table_stride, num_seqs, num_q_heads, q_len, budget);
    if (st != PA_OK) return st;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache) {
        k_cache = pool->k_cache;
        v_cache = pool->v_cache;
    }
    if (!q || !out || !selected || !block_tables || !context_lens || !aligned16(q) || !aligned16(out) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !aligned(selected, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    const uint64_t n = num_seqs, q_bytes = 2 * n * q_len * num_q_heads * c.head_dim;
    const Span o = {out, q_bytes};
    if (meet(o, {q, q_bytes}) || meet(o, {k_cache, pool->cache_bytes}) || meet(o, {v_cache, pool->cache_bytes}) ||
        meet(o, {selected, 4 * n * c.num_kv_heads * budget}) || meet(o, {context_lens, 4 * n}) ||
        meet(o, {block_tables, 4 * n * block_table_stride}))
        return PA_ERR_INVALID_ARG;
    SelectedParams p;
    p.q = q;
    p.out = out;
    p.k_scales = p.v_scales = nullptr;
    if (c.kv_format == PA_KV_FP8_E4M3) {
        const uint64_t codes = (uint64_t)c.num_blocks * c.num_kv_heads * c.block_size * c.head_dim;
        p.k_scales = reinterpret_cast<const float *>(static_cast<const uint8_t *>(k_cache) + codes);
        p.v_scales = reinterpret_cast<const float *>(static_cast<const uint8_t *>(v_cache) + codes);
    }
    p.selected = selected;
    p.budget = budget;
    p.block_tables = block_tables;
    p.stride = block_table_stride;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.Hq = num_q_heads;
    p.Hkv = c.num_kv_heads;
    p.G = num_q_heads / c.num_kv_heads;
    p.q_len = q_len;
    p.rows = p.G * q_len;
    p.bs = c.block_size;
    p.num_blocks = c.num_blocks;
    p.max_len = max_len_of(c, block_table_stride);
    p.scale_log2 = scale_log2;
    p.wait_ns = pool->wait_ns;
    p.status = pool->status;
    DeviceGuard g(c.device);
    if (!g.ok) return PA_ERR_CUDA;
    CUtensorMap tmk, tmv;
    const auto map = p.k_scales ? tensor_map : group_map;
    if ((st = map(pool, k_cache, &tmk)) != PA_OK || (st = map(pool, v_cache, &tmv)) != PA_OK) return st;
    return launched(launch_selected(p, c.dtype, c.head_dim, tmk, tmv, pool->sm_count, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
