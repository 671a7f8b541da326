// logits.cu -- penalties for repeated tokens, biases and grammar masks on logits, and the softmax with
// temperature that makes a token distribution of them (the p of pa_spec_verify).
//
// Row j of sequence b (j < rows_per_seq; row j of a verify follows drafts 0..j-1), token t:
//   count = occurrences of t among the outputs history[b][prompt_lens[b]..history_lens[b]) and
//           draft[b][0..j);  seen = count > 0 or t occurs in history[b][0..prompt_lens[b])
//   x = logit;  seen: x = x > 0 ? x / repetition : x * repetition
//   x = x - frequency * count;  count > 0: x = x - presence;  x = x + bias
//   mask bit 0: x = -inf
//   probability = exp((x - max x) / temperature) / sum (temperature 0: 1 at the largest x, lowest index)
// The steps on x are single fp32 operations in this order, none contracted.
//
// Simple form: one block per row; the token counts are found by walking the lists for every token.
#include "pa_device.cuh"

namespace pa {

__device__ __forceinline__ float load_logit(const LogitsParams &p, int64_t i) {
    if (p.dtype == PA_LOGITS_FP32) return static_cast<const float *>(p.logits)[i];
    if (p.dtype == PA_LOGITS_FP16) return __half2float(static_cast<const __half *>(p.logits)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[i]);
}

__device__ float adjusted(const LogitsParams &p, int b, int j, int t, int hist, int prompt) {
    float x = load_logit(p, b * p.seq_stride + j * p.row_stride + t);
    int count = 0;
    bool seen = false;
    for (int i = 0; i < hist; ++i)
        if (__ldg(p.history + b * p.history_stride + i) == t) {
            seen = true;
            count += i >= prompt;
        }
    if (p.draft)
        for (int i = 0; i < j; ++i) count += __ldg(p.draft + (int64_t)b * (p.R - 1) + i) == t;
    if (p.repetition && (seen || count > 0)) {
        const float r = __ldg(p.repetition + b);
        x = x > 0.f ? __fdiv_rn(x, r) : __fmul_rn(x, r);
    }
    if (count > 0) {
        if (p.frequency) x = __fsub_rn(x, __fmul_rn(__ldg(p.frequency + b), (float)count));
        if (p.presence) x = __fsub_rn(x, __ldg(p.presence + b));
    }
    for (int i = p.num_bias - 1; i >= 0; --i)
        if (__ldg(p.bias_tokens + (int64_t)b * p.num_bias + i) == t) {
            x = __fadd_rn(x, __ldg(p.bias_values + (int64_t)b * p.num_bias + i));
            break;
        }
    if (p.mask && !((__ldg(p.mask + ((int64_t)b * p.R + j) * ((p.V + 31) / 32) + t / 32) >> (t & 31)) & 1))
        x = -INFINITY;
    return x;
}

template <bool PROBS>
__global__ void __launch_bounds__(1024) logits_simple_kernel(const LogitsParams p) {
    __shared__ float red[32];
    __shared__ int ired[32];
    const int b = blockIdx.x / p.R, j = blockIdx.x % p.R, tid = threadIdx.x;
    int hist = p.history ? __ldg(p.history_lens + b) : 0;
    hist = hist < 0 ? 0 : (hist > p.history_cap ? p.history_cap : hist);
    const int prompt = p.prompt_lens ? __ldg(p.prompt_lens + b) : 0;
    float *out = p.out + (int64_t)blockIdx.x * p.V;
    float m = -INFINITY;
    for (int t = tid; t < p.V; t += 1024) {
        const float x = adjusted(p, b, j, t, hist, prompt);
        out[t] = x;
        m = fmaxf(m, x);
    }
    if constexpr (PROBS) {
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = red[tid & 31];
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        __syncthreads();
        const float T = __ldg(p.temperature + b);
        const bool greedy = T == 0.f;
        const float inv = T > 0.f ? fminf(__fdiv_rn(1.f, T), 3.402823466e38f) : __int_as_float(0x7fc00000);
        float sum = 0.f;
        int best = 0x7fffffff;
        for (int t = tid; t < p.V; t += 1024) {
            const float x = out[t];
            float e;
            if (greedy) {
                if (x == m && x > -INFINITY) best = min(best, t);
                e = x != x ? x : 0.f;
            } else {
                e = x == -INFINITY ? 0.f : expf((x - m) * inv);
            }
            out[t] = e;
            sum += e;
        }
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        }
        if ((tid & 31) == 0) red[tid >> 5] = sum, ired[tid >> 5] = best;
        __syncthreads();
        sum = red[tid & 31];
        best = ired[tid & 31];
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        }
        const float r = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
        for (int t = tid; t < p.V; t += 1024)
            out[t] = greedy ? (sum != sum ? sum : (t == best ? 1.f : 0.f)) : out[t] * r;
    }
}

cudaError_t launch_logits(const LogitsParams &p, bool probs, cudaStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)p.B * p.R);
    if (probs) logits_simple_kernel<true><<<grid, 1024, 0, stream>>>(p);
    else logits_simple_kernel<false><<<grid, 1024, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
