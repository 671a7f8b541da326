// pa_serving.cu -- the serving operators' part of the C ABI declared in include/pagedattn.h: rotary
// frequencies, argument validation, TMA descriptor encoding and kernel launches. The kernels are those of
// rope_append.cu, prompt.cu and logits.cu.
#include <algorithm>
#include <cmath>
#include <new>

#include "pa_pool.h"
#include "pa_serving.h"

using namespace pa;

struct pa_rope {
    uint64_t *freq = nullptr;    // device [rot_dim / 2], 2^-64 turns per position
    int rot = 0, interleaved = 0, device = 0;
    float scale = 1.f;
};

extern "C" {

// A launch's result as a status; an error is not left behind for the next caller that asks CUDA for the last one.
static pa_status launched(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    cudaGetLastError();
    return PA_ERR_CUDA;
}

using wide = __int128;                                // strides are the caller's: no product of them overflows

// Do n rows of a_row bytes at a, a_stride bytes apart, share a byte with such rows at b? Rows of different strides
// count as sharing where their spans meet.
static bool rows_meet(const void *a, wide a_row, wide a_stride, const void *b, wide b_row, wide b_stride, wide n) {
    const wide x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (x + (n - 1) * a_stride + a_row <= y || y + (n - 1) * b_stride + b_row <= x) return false;
    if (n == 1 || a_stride != b_stride) return true;
    const wide d = ((y - x) % a_stride + a_stride) % a_stride;     // b's column, with a's at 0
    return d < a_row || d + b_row > a_stride;
}

pa_status pa_rope_create(const double *inv_freq, int32_t rot_dim, int32_t interleaved, float scale, int32_t device,
                         pa_rope **out) {
    if (!out) return PA_ERR_INVALID_ARG;
    *out = nullptr;
    if (!inv_freq || rot_dim < 16 || rot_dim > 128 || rot_dim % 16 != 0 || (interleaved != 0 && interleaved != 1) ||
        !std::isfinite(scale) || device < 0)
        return PA_ERR_INVALID_ARG;
    uint64_t f[64];
    // 1 / 2 pi as the sum of two doubles: the nearest double and what is left of it
    const double inv_2pi = 0.15915494309189535, inv_2pi_lo = -9.839338337591243e-18;
    for (int i = 0; i < rot_dim / 2; ++i) {
        if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > PA_ROPE_MAX_FREQ) return PA_ERR_INVALID_ARG;
        // of the magnitude: hi - floor(hi) is exact from 0 on, but rounds for a small negative hi
        const double w = std::fabs(inv_freq[i]), hi = w * inv_2pi;
        const double lo = std::fma(w, inv_2pi, -hi) + w * inv_2pi_lo;
        const double units = std::ldexp(hi - std::floor(hi), 64), whole = std::floor(units);   // below 2^64
        f[i] = (uint64_t)whole + (uint64_t)(int64_t)std::llrint((units - whole) + std::ldexp(lo, 64));
        if (inv_freq[i] < 0) f[i] = 0 - f[i];
    }
    DeviceGuard g(device);
    if (!g.ok) return PA_ERR_CUDA;
    pa_rope *r = new (std::nothrow) pa_rope();
    if (!r) return PA_ERR_OOM;
    r->rot = rot_dim;
    r->interleaved = interleaved;
    r->scale = scale;
    r->device = device;
    if (cudaMalloc(&r->freq, sizeof(f)) != cudaSuccess) {
        cudaGetLastError();
        delete r;
        return PA_ERR_OOM;
    }
    // a copy from pageable memory may return before it has landed: streams that do not wait for the default one read it
    if (cudaMemcpy(r->freq, f, sizeof(uint64_t) * (rot_dim / 2), cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(r->freq);
        delete r;
        return PA_ERR_CUDA;
    }
    *out = r;
    return PA_OK;
}

void pa_rope_destroy(pa_rope *rope) {
    if (!rope) return;
    DeviceGuard g(rope->device);
    cudaFree(rope->freq);
    delete rope;
}

pa_status pa_rope_append(pa_pool *pool, const pa_rope *rope, const void *q, int64_t q_stride, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                         const int64_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads, void *q_out,
                         int64_t q_out_stride, void *k_cache, void *v_cache, void *stream) {
    if (!pool || !rope || num_tokens < 0 || num_q_heads < 0 || num_q_heads > 65536) return PA_ERR_INVALID_ARG;
    const pa_pool_config &c = pool->cfg;
    if (rope->rot > c.head_dim || rope->device != c.device) return PA_ERR_INVALID_ARG;
    if (num_q_heads + 2LL * c.num_kv_heads > 262144) return PA_ERR_UNSUPPORTED;
    if ((k_cache == nullptr) != (v_cache == nullptr)) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !positions || !slot_mapping || (num_q_heads > 0 && (!q || !q_out))) return PA_ERR_INVALID_ARG;
    if (!k_cache) {
        k_cache = pool->k_cache;
        v_cache = pool->v_cache;
    }
    const int64_t kv_row = (int64_t)c.num_kv_heads * c.head_dim, q_row = (int64_t)num_q_heads * c.head_dim;
    if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 != 0 || v_stride % 8 != 0) return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (q_stride < q_row || q_out_stride < q_row || q_stride % 8 != 0 || q_out_stride % 8 != 0 ||
                            (q == q_out && q_stride != q_out_stride) || !aligned16(q) || !aligned16(q_out)))
        return PA_ERR_INVALID_ARG;
    const auto meets_out = [&](const void *x, int64_t row, int64_t stride) {
        return rows_meet(q_out, 2 * q_row, (wide)2 * q_out_stride, x, 2 * row, (wide)2 * stride, num_tokens);
    };
    if (num_q_heads > 0 &&
        ((q != q_out && meets_out(q, q_row, q_stride)) || meets_out(k, kv_row, k_stride) || meets_out(v, kv_row, v_stride)))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PA_ERR_INVALID_ARG;
    RopeParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.positions = positions;
    p.slots = slot_mapping;
    p.freq = rope->freq;
    p.mscale = rope->scale;
    p.rot = rope->rot;
    p.interleaved = rope->interleaved;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.status = pool->status;
    p.num_tokens = num_tokens;
    p.num_blocks = c.num_blocks;
    p.Hq = num_q_heads;
    p.Hkv = c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.bs = c.block_size;
    p.fp8 = c.kv_format == PA_KV_FP8_E4M3;
    DeviceGuard g(c.device);
    if (!g.ok) return PA_ERR_CUDA;
    return launched(launch_rope_append(p, c.dtype, pool->sm_count, static_cast<cudaStream_t>(stream)));
}

// The checks of pa_prefill_packed's sizes, shared with the workspace query.
static pa_status packed_params(const pa_pool *pool, int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                               int32_t stride, PromptParams &p) {
    const pa_pool_config &c = pool->cfg;
    if (num_tokens < 0 || num_seqs < 0 || num_q_heads < 1 || num_q_heads % c.num_kv_heads != 0 || stride < 1)
        return PA_ERR_INVALID_ARG;
    if (c.kv_format != PA_KV_16BIT) return PA_ERR_UNSUPPORTED;
    const int G = num_q_heads / c.num_kv_heads;
    if (G > 128 || num_seqs > PA_PACKED_MAX_SEQS || (int64_t)num_tokens * num_q_heads >= (int64_t)1 << 31)
        return PA_ERR_UNSUPPORTED;
    int64_t max_ctx = (int64_t)stride * c.block_size;
    if (max_ctx > PA_PACKED_MAX_CONTEXT) max_ctx = PA_PACKED_MAX_CONTEXT;
    p.stride = stride;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.Hq = num_q_heads;
    p.Hkv = c.num_kv_heads;
    p.G = G;
    p.bs = c.block_size;
    p.num_blocks = c.num_blocks;
    p.max_ctx = (int)max_ctx;
    p.P = 128 / G;
    // Items behind long contexts are cut along the keys only where num_tokens rows, if all of them belong to
    // sequences, make too few items for two rounds of blocks (the lengths are on the device, which decides again), and
    // not into key ranges of a few tiles. So one long context beside enough other rows, or in a call padded to as
    // many, is one block's work per KV head: 4096 fresh tokens with one behind 65536, 32 / 8 heads, take 843 us, and
    // apart 106 and 58.
    const int64_t least_items = ((int64_t)num_tokens + 2 * p.P - 1) / (2 * p.P) * c.num_kv_heads;
    p.max_units = least_items < 2 * pool->sm_count && max_ctx > 4 * 128 ? 2 * pool->sm_count : 0;
    p.status = pool->status;
    // The kernel's longest waits last as long as a unit's work (the next unit's Q takes the place of its Q): 1.5 to 2 us
    // per key tile of what may be a whole context. Four times that, where it is above the pool's limit.
    p.wait_ns = std::max(pool->wait_ns, (uint64_t)(max_ctx / 128) * 8000);
    return PA_OK;
}

// The pool as a 4-D tensor for copies of whole blocks: [8 tokens x 64 dimensions], the dimension halves, groups of
// eight tokens. One box is a block's rows of one KV head, 128-byte swizzled.
static pa_status block_map(const pa_pool_config &c, const void *cache, CUtensorMap *out) {
    auto fn = encode_fn();
    if (!fn) return PA_ERR_CUDA;
    const cuuint64_t row = (cuuint64_t)c.head_dim * 2, groups = (cuuint64_t)c.num_blocks * c.num_kv_heads * c.block_size / 8;
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)c.head_dim / 64, groups};
    cuuint64_t strides[3] = {row, 128, 8 * row};
    cuuint32_t box[4] = {64, 8, (cuuint32_t)c.head_dim / 64, (cuuint32_t)c.block_size / 8};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(out, c.dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
              const_cast<void *>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PA_OK
               : PA_ERR_CUDA;
}

// q [num_tokens, Hq, head_dim] for boxes of P positions x G heads x 64 dimensions.
static pa_status q_map(const PromptParams &p, int dtype, int head_dim, CUtensorMap *out) {
    auto fn = encode_fn();
    if (!fn) return PA_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)p.Hq, (cuuint64_t)p.num_tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)p.Hq * head_dim * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.P};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(out, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(p.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status pa_prefill_packed_workspace(const pa_pool *pool, int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                      int32_t block_table_stride, uint64_t *bytes) {
    if (!pool || !bytes) return PA_ERR_INVALID_ARG;
    PromptParams p;
    const pa_status st = packed_params(pool, num_tokens, num_seqs, num_q_heads, block_table_stride, p);
    if (st != PA_OK) return st;
    // a state for each unit of a call that may be cut, for each block of one that is not but whose sums may be long
    const uint64_t slots = p.max_units > 0 ? p.max_units : p.max_ctx > 128 * PROMPT_FOLD_TILES ? pool->sm_count : 0;
    *bytes = slots == 0 ? 0 : 256 + (uint64_t)p.max_units * PROMPT_ITEM_BYTES + slots * prompt_slot_bytes(pool->cfg.head_dim);
    return PA_OK;
}

pa_status pa_prefill_packed(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *cu_q, const int32_t *block_tables, int32_t block_table_stride,
                            const int32_t *context_lens, int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                            float scale, void *workspace, uint64_t workspace_bytes, void *out, void *stream) {
    if (!pool || !std::isfinite(scale) || !(scale > 0.f)) return PA_ERR_INVALID_ARG;
    if ((k_cache == nullptr) != (v_cache == nullptr)) return PA_ERR_INVALID_ARG;
    PromptParams p;
    const pa_status st = packed_params(pool, num_tokens, num_seqs, num_q_heads, block_table_stride, p);
    if (st != PA_OK) return st;
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    uint64_t need = 0;
    pa_prefill_packed_workspace(pool, num_tokens, num_seqs, num_q_heads, block_table_stride, &need);
    if (!q || !out || !cu_q || !block_tables || !context_lens || (need > 0 && !workspace) || workspace_bytes < need)
        return PA_ERR_INVALID_ARG;
    const pa_pool_config &c = pool->cfg;
    if (!k_cache) {
        k_cache = pool->k_cache;
        v_cache = pool->v_cache;
    }
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_q) & 3u))
        return PA_ERR_INVALID_ARG;
    const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
    if ((qa < oa ? oa - qa : qa - oa) < (uintptr_t)num_tokens * num_q_heads * c.head_dim * 2)
        return PA_ERR_INVALID_ARG;                    // a unit's rows would be written while another still reads them
    p.q = q;
    p.out = out;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.cu_q = cu_q;
    p.context_lens = context_lens;
    p.scale_log2 = scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_total = reinterpret_cast<int *>(ws);
    p.ws_items = reinterpret_cast<PromptItem *>(ws + 256);
    p.ws_slots = ws + 256 + (size_t)p.max_units * PROMPT_ITEM_BYTES;
    DeviceGuard g(c.device);
    if (!g.ok) return PA_ERR_CUDA;
    CUtensorMap tmq, tmk, tmv;
    pa_status ms;
    if ((ms = q_map(p, c.dtype, c.head_dim, &tmq)) != PA_OK || (ms = block_map(c, k_cache, &tmk)) != PA_OK ||
        (ms = block_map(c, v_cache, &tmv)) != PA_OK)
        return ms;
    return launched(
        launch_prompt(p, c.dtype, c.head_dim, tmq, tmk, tmv, pool->sm_count, static_cast<cudaStream_t>(stream)));
}

static pa_status logits_call(const pa_logits_args *a, bool probs, void *stream) {
    if (!a || a->num_seqs < 0 || a->rows_per_seq < 1 || a->num_bias < 0 || a->vocab < 1 || a->seq_stride < 0 ||
        a->row_stride < 0 || a->history_stride < 0)
        return PA_ERR_INVALID_ARG;
    if (a->dtype != PA_LOGITS_FP16 && a->dtype != PA_LOGITS_BF16 && a->dtype != PA_LOGITS_FP32)
        return PA_ERR_INVALID_ARG;
    if (a->vocab > PA_LOGITS_MAX_VOCAB || a->history_stride > PA_LOGITS_MAX_HISTORY ||
        a->num_bias > PA_LOGITS_MAX_BIAS || a->rows_per_seq > PA_LOGITS_MAX_ROWS ||
        (int64_t)a->num_seqs * a->rows_per_seq >= (int64_t)1 << 24)
        return PA_ERR_UNSUPPORTED;
    if (a->num_seqs == 0) return PA_OK;
    const bool has_history = a->history && a->history_stride > 0;
    if (!a->logits || !a->out || (probs && !a->temperature) || (has_history && !a->history_lens) ||
        (a->num_bias > 0 && (!a->bias_tokens || !a->bias_values)))
        return PA_ERR_INVALID_ARG;
    const uintptr_t esize = a->dtype == PA_LOGITS_FP32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(a->logits) % esize != 0) return PA_ERR_INVALID_ARG;
    const void *words[] = {a->history,     a->history_lens, a->prompt_lens, a->draft, a->repetition, a->presence, a->frequency,
                           a->bias_tokens, a->bias_values,  a->mask,        a->temperature, a->out};
    for (const void *x : words)
        if (reinterpret_cast<uintptr_t>(x) & 3u) return PA_ERR_INVALID_ARG;
    const int64_t V = a->vocab, R = a->rows_per_seq;
    const bool in_place = a->logits == static_cast<const void *>(a->out);
    if (in_place && (a->dtype != PA_LOGITS_FP32 || (R > 1 && a->row_stride != V) ||
                     (a->num_seqs > 1 && a->seq_stride != R * V)))
        return PA_ERR_INVALID_ARG;
    const wide span = (wide)(a->num_seqs - 1) * a->seq_stride + (wide)(R - 1) * a->row_stride + V;
    if (!in_place && rows_meet(a->logits, span * (int)esize, 0, a->out, 4 * a->num_seqs * R * V, 0, 1))
        return PA_ERR_INVALID_ARG;
    LogitsParams p;
    p.logits = a->logits;
    p.dtype = a->dtype;
    p.B = a->num_seqs;
    p.R = a->rows_per_seq;
    p.V = (int)V;
    p.seq_stride = a->seq_stride;
    p.row_stride = a->row_stride;
    p.history = has_history ? a->history : nullptr;
    p.history_stride = a->history_stride;
    p.history_cap = (int)a->history_stride;
    p.history_lens = a->history_lens;
    p.prompt_lens = a->prompt_lens;
    p.draft = R > 1 ? a->draft : nullptr;
    p.repetition = a->repetition;
    p.presence = a->presence;
    p.frequency = a->frequency;
    p.bias_tokens = a->bias_tokens;
    p.bias_values = a->bias_values;
    p.num_bias = a->num_bias;
    p.mask = a->mask;
    p.temperature = a->temperature;
    p.out = a->out;
    return launched(launch_logits(p, probs, static_cast<cudaStream_t>(stream)));
}

pa_status pa_adjust_logits(const pa_logits_args *args, void *stream) { return logits_call(args, false, stream); }

pa_status pa_token_probs(const pa_logits_args *args, void *stream) { return logits_call(args, true, stream); }

}  // extern "C"
