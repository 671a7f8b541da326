// pa_serving.h -- types and launchers of the serving operators: rotation and append, packed prompts, logits.
#pragma once

#include "pa_internal.h"

namespace pa {

struct RopeParams {
    const void *q, *k, *v;      // token rows of [heads, head_dim], strides in elements
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const int32_t *positions;
    const int64_t *slots;
    const uint64_t *freq;       // [rot / 2], 2^-64 turns per position
    float mscale;               // factor on every cosine and sine
    int rot;                    // rotated dimensions of a head (a multiple of 16)
    int interleaved;            // pairs are neighbours, not halves
    void *q_out;
    void *k_cache, *v_cache;
    int *status;
    int64_t num_tokens;
    int64_t num_blocks;
    int Hq, Hkv, head_dim, bs;
    int fp8;                    // the pool holds E4M3 codes and scales
};

struct PromptParams {
    const void *q;              // [num_tokens, Hq, D]
    void *out;
    const void *v_cache;        // for the values that are no numbers; K and V come through the tensor maps
    const int32_t *block_tables;
    const int32_t *cu_q;        // [num_seqs + 1]
    const int32_t *context_lens;
    int *status;
    int64_t stride;             // block-table row stride (entries)
    int num_tokens, num_seqs;
    int Hq, Hkv, G;
    int bs, num_blocks;
    int max_ctx;                // longest context the tables hold
    int P;                      // positions of a row tile: 128 / G
    int max_units;              // units that a call may be cut into; 0: nothing is cut
    int *ws_total;              // workspace: number of items to join, the items, the states of units or blocks
    struct PromptItem *ws_items;
    uint8_t *ws_slots;
    float scale_log2;
    uint64_t wait_ns;
};

struct LogitsParams {
    const void *logits;
    int dtype;
    int B, R;
    int V;
    int64_t seq_stride, row_stride;
    const int32_t *history;
    int64_t history_stride;
    int history_cap;            // entries of a history row
    const int32_t *history_lens, *prompt_lens;
    const int32_t *draft;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_tokens;
    const float *bias_values;
    int num_bias;
    const int32_t *mask;
    const float *temperature;
    float *out;
};

cudaError_t launch_rope_append(const RopeParams &p, int dtype, int sm_count, cudaStream_t stream);
cudaError_t launch_prompt(const PromptParams &p, int dtype, int head_dim, const CUtensorMap &tmq,
                          const CUtensorMap &tmk, const CUtensorMap &tmv, int sm_count, cudaStream_t stream);
cudaError_t setup_prompt(int dtype, int head_dim);
size_t prompt_slot_bytes(int head_dim);
constexpr int PROMPT_ITEM_BYTES = 32;   // of the workspace per unit, beside its state
constexpr int PROMPT_FOLD_TILES = 128;  // key tiles (of 128 keys) that a unit sums up without a state in the workspace
cudaError_t launch_logits(const LogitsParams &p, bool probs, cudaStream_t stream);

}  // namespace pa
