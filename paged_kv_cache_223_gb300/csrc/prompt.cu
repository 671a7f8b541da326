// prompt.cu -- causal attention of packed prompts of different lengths through the block tables.
//
// Sequence b's new tokens are rows cu_q[b] .. cu_q[b+1] of q; row i of them sits at position
// p = context_lens[b] - n_b + i and attends to tokens 0..p:
//   out = sum_t softmax_t(scale q . K_t) V_t.
//
// Simple form: one warp per (token, query head), one pass over its keys with the running maximum and
// sum of the softmax.
#include "pa_device.cuh"

namespace pa {

template <typename T, int D>
__global__ void __launch_bounds__(128) prompt_simple_kernel(const PromptParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
    if (w >= (int64_t)p.num_tokens * p.Hq) return;
    const int tok = (int)(w / p.Hq), h = (int)(w % p.Hq), g = h / p.G;
    int b = 0;
    while (b < p.num_seqs && __ldg(p.cu_q + b + 1) <= tok) ++b;
    if (b == p.num_seqs || __ldg(p.cu_q + b) > tok) return;          // behind the last sequence
    const int n = __ldg(p.cu_q + b + 1) - __ldg(p.cu_q + b);
    int L = __ldg(p.context_lens + b);
    if (L < n || L > p.max_ctx) {
        if (lane == 0) set_status(p.status, STATUS_BOUNDS);
        L = L > p.max_ctx ? p.max_ctx : L;
    }
    const int last = L - n + (tok - __ldg(p.cu_q + b));
    const T *q = static_cast<const T *>(p.q) + w * D + lane * E;
    float qv[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) qv[e] = (float)q[e], o[e] = 0.f;
    for (int t = 0; t <= last; ++t) {
        int id = __ldg(p.block_tables + (int64_t)b * p.stride + t / p.bs);
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) set_status(p.status, STATUS_BOUNDS);
            id = 0;
        }
        const int64_t row = (((int64_t)id * p.Hkv + g) * p.bs + t % p.bs) * D + lane * E;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += qv[e] * (float)static_cast<const T *>(p.k_cache)[row + e];
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), a = exp2f(m - mn), x = exp2f(s - mn);
        l = l * a + x;
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + x * (float)static_cast<const T *>(p.v_cache)[row + e];
        m = mn;
    }
    T *out = static_cast<T *>(p.out) + w * D + lane * E;
    for (int e = 0; e < E; ++e) out[e] = (T)(l > 0.f ? o[e] / l : o[e]);
}

cudaError_t launch_prompt(const PromptParams &p, int dtype, int head_dim, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)p.num_tokens * p.Hq + 3) / 4);
    if (dtype == PA_FP16) {
        if (head_dim == 64) prompt_simple_kernel<__half, 64><<<grid, 128, 0, stream>>>(p);
        else prompt_simple_kernel<__half, 128><<<grid, 128, 0, stream>>>(p);
    } else {
        if (head_dim == 64) prompt_simple_kernel<__nv_bfloat16, 64><<<grid, 128, 0, stream>>>(p);
        else prompt_simple_kernel<__nv_bfloat16, 128><<<grid, 128, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace pa
