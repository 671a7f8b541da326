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
// Bound: memory, 2 d (2 Hq + 4 Hkv) bytes a token. A thread owns two 16-byte vectors of one head's row
// that hold eight whole pairs (halves: vectors j and j + rot/16; neighbours: 2j and 2j + 1), so every
// load and store is a full vector and the pass-through dimensions take the same path; d / 16 threads
// cover a head. The tile's sines and cosines are computed once per token into shared memory, in 16-byte
// columns that the threads of a head read without bank conflicts. The first row of each thread is in
// flight while they are computed, the next one while a row is rotated. Measured: 8192 tokens of 64 / 8 heads
// of 128, slices of one projection's output, 56 us, 6.0 TB/s (0.89 of the copy rate; one element per thread,
// heads in turn: 207 us); one token 2 us in a captured graph.
#include <type_traits>

#include "pa_device.cuh"
#include "pa_serving.h"

namespace pa {

constexpr int RA_THREADS = 256;

// cos and sin of pos * freq, freq in 2^-64 turns per position.
__device__ __forceinline__ void phase_sincos(int32_t pos, uint64_t freq, float &s, float &c) {
    const int64_t ph = (int64_t)((uint64_t)(int64_t)pos * freq);       // turns mod 1, signed, 2^-64 units
    sincospif(__ll2float_rn(ph) * 1.08420217248550443e-19f, &s, &c);   // 2^-63: half turns
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {                                                       // a bf16 is the top half of an fp32
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float scale) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Block (x, y): tokens [x TOK, (x + 1) TOK), every gridDim.y-th group of RA_THREADS / TPH rows of them.
template <typename T, int D, int TOK, bool FP8>
__global__ void __launch_bounds__(RA_THREADS) rope_append_kernel(const RopeParams p) {
    constexpr int TPH = D / 16, RPP = RA_THREADS / TPH;                // threads per head row, rows per pass
    __shared__ float4 trig[TOK][4][TPH];                               // [token][cos lo, cos hi, sin lo, sin hi][j]
    const int tid = threadIdx.x, j = tid % TPH, rsub = tid / TPH;
    const int H = p.Hq + 2 * p.Hkv, rj = p.rot / 16;
    const int64_t tok0 = (int64_t)blockIdx.x * TOK;
    const int ntok = (int)(p.num_tokens - tok0 < TOK ? p.num_tokens - tok0 : TOK);
    const int rows = ntok * H, step = RPP * (int)gridDim.y;
    // vectors of this thread in a q or k row: a pair of vectors with eight whole pairs, or two that pass through
    const bool turned = j < rj;
    const int v0 = turned && !p.interleaved ? j : 2 * j, v1 = turned && !p.interleaved ? j + rj : 2 * j + 1;
    pdl_wait();
    auto source = [&](int r, int &t, int &h) -> const uint4 * {
        t = r / H;
        h = r - t * H;
        const int64_t tok = tok0 + t;
        if (h < p.Hq) return reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + tok * p.q_stride + h * D);
        if (h < p.Hq + p.Hkv)
            return reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k) + tok * p.k_stride + (h - p.Hq) * D);
        return reinterpret_cast<const uint4 *>(static_cast<const T *>(p.v) + tok * p.v_stride + (h - p.Hq - p.Hkv) * D);
    };
    int r = (int)blockIdx.y * RPP + rsub, t = 0, h = 0;
    uint4 a = {}, b = {};
    if (r < rows) {
        const uint4 *src = source(r, t, h);
        a = src[v0];
        b = src[v1];
    }
    for (int i = tid; i < ntok * (p.rot / 2); i += RA_THREADS) {
        const int tt = i / (p.rot / 2), f = i - tt * (p.rot / 2);
        float s, c;
        phase_sincos(__ldg(p.positions + tok0 + tt), __ldg(p.freq + f), s, c);
        float *col = reinterpret_cast<float *>(&trig[tt][(f & 4) ? 1 : 0][f >> 3]) + (f & 3);
        col[0] = c * p.mscale;
        col[2 * TPH * 4] = s * p.mscale;
    }
    __syncthreads();
    const int64_t codes = p.num_blocks * p.Hkv * p.bs * D;
    // (all lanes of a head's group agree on the row, so the shuffles of an FP8 row's maximum are whole groups)
    for (; r < rows; r += step) {
        const uint4 a0 = a, b0 = b;
        const int t0 = t, h0 = h;
        if (r + step < rows) {
            const uint4 *src = source(r + step, t, h);
            a = src[v0];
            b = src[v1];
        }
        const bool is_q = h0 < p.Hq, is_v = h0 >= p.Hq + p.Hkv;
        uint4 ya = a0, yb = b0;
        float x[8], y[8];
        if ((turned && !is_v) || (FP8 && !is_q)) {
            unpack8<T>(a0, x);
            unpack8<T>(b0, y);
        }
        if (turned && !is_v) {
            const float4 c0 = trig[t0][0][j], c1 = trig[t0][1][j], s0 = trig[t0][2][j], s1 = trig[t0][3][j];
            const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float xa = x[2 * i], xb = x[2 * i + 1], za = y[2 * i], zb = y[2 * i + 1];
                    x[2 * i] = xa * c[i] - xb * s[i];
                    x[2 * i + 1] = xb * c[i] + xa * s[i];
                    y[2 * i] = za * c[4 + i] - zb * s[4 + i];
                    y[2 * i + 1] = zb * c[4 + i] + za * s[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xa = x[i], xb = y[i];
                    x[i] = xa * c[i] - xb * s[i];
                    y[i] = xb * c[i] + xa * s[i];
                }
            }
            if (!FP8 || is_q) {
                ya = pack8<T>(x);
                yb = pack8<T>(y);
            }
        }
        if (is_q) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.q_out) + (tok0 + t0) * p.q_out_stride + h0 * D);
            dst[v0] = ya;
            dst[v1] = yb;
            continue;
        }
        const int64_t slot = __ldg(p.slots + tok0 + t0);
        if (slot < 0) continue;                                        // padding token
        if (slot >= p.num_blocks * p.bs) {                             // outside the pool: skip, flag
            if (j == 0) set_status(p.status, STATUS_BOUNDS);
            continue;
        }
        const int hk = is_v ? h0 - p.Hq - p.Hkv : h0 - p.Hq;
        const int64_t blk = slot / p.bs, srow = (blk * p.Hkv + hk) * p.bs + (slot - blk * p.bs);
        void *cache = is_v ? p.v_cache : p.k_cache;
        if constexpr (FP8) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(y[i])));
            const unsigned group = ((1u << TPH) - 1u) << ((tid & 31) / TPH * TPH);
#pragma unroll
            for (int o = TPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, o));
            const float unit = __fdiv_rn(m, 448.f);                    // 0 for rows below 448 of the smallest number, too
            const float scale = unit > 0.f ? unit : 1.f;
            uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + srow * D);
            dst[v0] = e4m3x8(x, scale);
            dst[v1] = e4m3x8(y, scale);
            if (j == 0) reinterpret_cast<float *>(static_cast<uint8_t *>(cache) + codes)[srow] = scale;
        } else {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(cache) + srow * D);
            dst[v0] = ya;
            dst[v1] = yb;
        }
    }
}

template <typename T, int D, bool FP8>
static cudaError_t launch_t(const RopeParams &p, int sm_count, cudaStream_t stream) {
    constexpr int RPP = RA_THREADS / (D / 16);
    const int H = p.Hq + 2 * p.Hkv;
    // Few tokens: one per block, and its rows over several blocks, so that a row waits for no other (the sines
    // are computed once per block). From two blocks of four tokens per SM on, four tokens share a block: a
    // quarter of the blocks' start-up and waits for one round of sines.
    if (p.num_tokens >= 8LL * sm_count) {
        return launch_pdl(rope_append_kernel<T, D, 4, FP8>, dim3((unsigned)((p.num_tokens + 3) / 4)), dim3(RA_THREADS),
                          0, stream, p);
    }
    const int groups = (H + RPP - 1) / RPP;
    return launch_pdl(rope_append_kernel<T, D, 1, FP8>, dim3((unsigned)p.num_tokens, (unsigned)groups),
                      dim3(RA_THREADS), 0, stream, p);
}

cudaError_t launch_rope_append(const RopeParams &p, int dtype, int sm_count, cudaStream_t stream) {
    if (p.fp8)
        return dtype == PA_FP16 ? launch_t<__half, 128, true>(p, sm_count, stream)
                                : launch_t<__nv_bfloat16, 128, true>(p, sm_count, stream);
    if (p.head_dim == 64)
        return dtype == PA_FP16 ? launch_t<__half, 64, false>(p, sm_count, stream)
                                : launch_t<__nv_bfloat16, 64, false>(p, sm_count, stream);
    return dtype == PA_FP16 ? launch_t<__half, 128, false>(p, sm_count, stream)
                            : launch_t<__nv_bfloat16, 128, false>(p, sm_count, stream);
}

}  // namespace pa
