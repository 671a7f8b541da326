// rope_append.cu -- rotate the new tokens' q and k rows by their positions and append k, v to the
// paged cache, in one pass over the rows.
//
// Rotary position embedding: dimension pair i of a row at position p turns by the angle p f_i,
//   (a, b) -> (a cos - b sin, b cos + a sin),
// with (a, b) = dimensions (i, i + rot/2) ("halves") or (2i, 2i + 1) (neighbours), i < rot/2;
// dimensions from rot on pass through. v is copied. The cache row is 16-bit words, or E4M3 codes
// with one scale per (slot, head), as pa_cache_write lays them out.
//
// Angles: pa_rope_create turns f_i into turns per token as a 64-bit fixed-point fraction,
// F_i = f_i / 2 pi mod 1 in units of 2^-64. The phase p F_i mod 2^64 is then exact integer
// arithmetic at any 32-bit position (its error is p 2^-64 turns plus that of f_i / 2 pi), and only the
// reduced angle, in [-1/2, 1/2) turns, is rounded to fp32 for sincospif. A position table of cosines
// and sines would cost 4 rot bytes of reads per token instead.
//
// Rotation is fp32; q' and k' are rounded once, to the model type (FP8 pools: k' is quantised from
// the fp32 values, without a 16-bit rounding in between).
//
// Simple form: one thread per pair or element position of a (token, head) row.
#include <cmath>
#include <new>

#include "pa_device.cuh"

namespace pa {

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// cos and sin of pos * freq, freq in 2^-64 turns per position.
__device__ __forceinline__ void phase_sincos(int32_t pos, uint64_t freq, float &s, float &c) {
    const int64_t ph = (int64_t)((uint64_t)(int64_t)pos * freq);       // turns mod 1, signed, 2^-64 units
    sincospif(__ll2float_rn(ph) * 1.08420217248550443e-19f, &s, &c);   // 2^-63: half turns
}

// One block per token, one thread per dimension of a head, heads in turn.
template <typename T>
__global__ void rope_append_kernel(const RopeParams p) {
    __shared__ float red[4];
    const int64_t tok = blockIdx.x;
    const int d = threadIdx.x, D = p.head_dim;
    const int64_t s = __ldg(p.slots + tok);
    const bool bad = s >= p.num_blocks * p.bs, keep = s >= 0 && !bad;
    if (bad && d == 0) set_status(p.status, STATUS_BOUNDS);
    float cs = 1.f, sn = 0.f;
    int partner = d;
    if (d < p.rot) {
        const int half = p.rot / 2;
        const int i = p.interleaved ? d / 2 : d % half;
        phase_sincos(__ldg(p.positions + tok), p.freq[i], sn, cs);
        cs *= p.mscale;
        sn *= p.mscale;
        const bool first = p.interleaved ? (d & 1) == 0 : d < half;
        partner = p.interleaved ? d ^ 1 : (first ? d + half : d - half);
        if (first) sn = -sn;
    }
    const int64_t codes = p.num_blocks * p.Hkv * p.bs * D;
    for (int h = 0; h < p.Hq + 2 * p.Hkv; ++h) {
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        const int hk = is_q ? 0 : (is_v ? h - p.Hq - p.Hkv : h - p.Hq);
        const T *src = static_cast<const T *>(is_q ? p.q : (is_v ? p.v : p.k)) +
                       tok * (is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride)) + (is_q ? h : hk) * D;
        const float x = (float)src[d];
        float y = x;
        if (!is_v && d < p.rot) y = x * cs + (float)src[partner] * sn;
        if (is_q) {
            __syncthreads();                                          // q_out may be q
            static_cast<T *>(p.q_out)[tok * p.q_out_stride + h * D + d] = from_float<T>(y);
        } else if (keep) {
            const int64_t srow = ((s / p.bs) * p.Hkv + hk) * p.bs + s % p.bs;
            if (!p.fp8) {
                static_cast<T *>(is_v ? p.v_cache : p.k_cache)[srow * D + d] = from_float<T>(y);
            } else {
                uint8_t *cache = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache);
                float a = fabsf(y);
                for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                __syncthreads();
                if ((d & 31) == 0) red[d >> 5] = a;
                __syncthreads();
                a = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
                const float scale = a > 0.f ? __fdiv_rn(a, 448.f) : 1.f;
                cache[srow * D + d] = __nv_cvt_float_to_fp8(__fdiv_rn(y, scale), __NV_SATFINITE, __NV_E4M3);
                if (d == 0) reinterpret_cast<float *>(cache + codes)[srow] = scale;
            }
        }
    }
}

cudaError_t launch_rope_append(const RopeParams &p, int dtype, cudaStream_t stream) {
    if (dtype == PA_FP16)
        rope_append_kernel<__half><<<(unsigned)p.num_tokens, p.head_dim, 0, stream>>>(p);
    else
        rope_append_kernel<__nv_bfloat16><<<(unsigned)p.num_tokens, p.head_dim, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pa
