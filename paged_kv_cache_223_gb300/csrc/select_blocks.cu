// select_blocks.cu -- the bounds of each block's keys, and the blocks that a cheap score selects for each query.
//
// Bounds. Per block and KV head, over the tokens that a block holds: hi_d = max K_d, lo_d = min K_d, step = the smallest
// power of two with max |hi|, |lo| <= 127 step, codes = hi / step and lo / step, rounded to the nearest whole number (even
// ones of two). Dividing by a power of two is exact, so the codes have one rounding and no choice in them.
//
// Score. A query row is taken to whole numbers c_d the same way, with a step of its own. The largest product that a key
// within the bounds can have with it is estimated by sum_d max(c_d hi_d, c_d lo_d): hi_d where c_d is positive, lo_d where
// it is negative, so one product of [hi, lo] with [c+, c-]. These are sums of at most 256 whole numbers below 2^14, exact
// in fp32 in any order; times the two steps, exact again. The score of a block is the largest over the query rows that
// read the KV head (the group's heads, the rows of a verify). No rounding can turn two blocks around, so the selection is
// the definition's, ties going to the lowest index.
#include <algorithm>
#include <cfloat>

#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_sparse.h"

namespace pa {

namespace {

constexpr uint32_t INF_BITS = 0x7F800000u;

// The smallest power of two s (at least the smallest number of fp32) with |x| <= 127 s, from the bits of |x|, which is
// finite; 0 for 0.
__device__ __forceinline__ float step_of(uint32_t bits) {
    if (bits == 0) return 0.f;
    int e = (int)(bits >> 23);
    uint32_t m = bits & 0x7FFFFFu;
    if (e == 0) {                                      // subnormal: leading one to bit 23
        const int up = __clz(m) - 8;
        m = (m << up) & 0x7FFFFFu;
        e = 1 - up;
    }
    const int s = e - 6 + (m > 0x7E0000u);             // biased exponent: |x| / 2^(e - 133) is 64 (1 + m / 2^23)
    return s >= 1 ? __uint_as_float((uint32_t)s << 23) : __uint_as_float(s > -22 ? 1u << (22 + s) : 1u);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// x / step, rounded to the nearest whole number; exact but for that rounding.
__device__ __forceinline__ int code_of(float x, float step, float inv) {
    return step == 0.f ? 0 : __float2int_rn(inv != 0.f ? x * inv : x / step);
}

// 1 / step where it is a number, else 0 (subnormal steps).
__device__ __forceinline__ float inverse_of(float step) { return step >= FLT_MIN ? 1.f / step : 0.f; }

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __half) {
    const __half2 r = __hmin2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float2 unpack2(uint32_t x, __half) { return __half22float2(*reinterpret_cast<__half2 *>(&x)); }
__device__ __forceinline__ float2 unpack2(uint32_t x, __nv_bfloat16) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&x));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 0xFF) | (uint32_t)(b & 0xFF) << 8 | (uint32_t)(c & 0xFF) << 16 | (uint32_t)d << 24;
}

// max with NaN kept
__device__ __forceinline__ float max_nan(float a, float b) { return a != a ? a : (a > b || b != b ? (b != b ? b : a) : b); }
__device__ __forceinline__ float min_nan(float a, float b) { return a != a ? a : (a < b || b != b ? (b != b ? b : a) : b); }

}  // namespace

// ------------------------------------------------------------------ bounds

constexpr int BND_WARPS = 4;

// One warp per (touched block, KV head): 16 bytes of a key row per lane, several rows a step, the lanes that hold the
// same dimensions joined at the end. Every CTA makes the list of touched blocks for itself: their sums over the sequences.
template <typename T, int D, bool KV8>
__global__ void __launch_bounds__(BND_WARPS * 32) bounds_kernel(const BoundsParams p) {
    extern __shared__ int bsm[];
    const int B = p.num_seqs;
    int *start = bsm, *first = start + B + 1;          // sums of B + 1; first touched block
    __shared__ int wsum[BND_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    int carry = 0;
    for (int b0 = 0; b0 < B; b0 += BND_WARPS * 32) {
        const int b = b0 + tid;
        int n = 0;
        if (b < B) {
            const int lo = __ldg(p.cu_q + b), hi = __ldg(p.cu_q + b + 1), len = __ldg(p.context_lens + b);
            if (lo < 0 || hi < lo || hi > p.num_tokens || len < hi - lo || len > p.max_len) {
                if (blockIdx.x == 0) set_status(p.status, STATUS_BOUNDS);
            } else if (hi > lo) {
                first[b] = (len - (hi - lo)) / p.bs;
                n = (len - 1) / p.bs - first[b] + 1;
            }
        }
        int s = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < BND_WARPS; ++w) {
            if (w < warp) before += wsum[w];
            carry += wsum[w];
        }
        if (b < B) start[b] = before + s - n;
        __syncthreads();
    }
    if (tid == 0) start[B] = carry;
    __syncthreads();

    constexpr int LPR = KV8 ? D / 16 : D / 8;          // lanes per row
    constexpr int RPS = 32 / LPR;                      // rows a step
    constexpr int EL = KV8 ? 16 : 8;                   // dimensions per lane
    const int sub = lane % LPR, grp = lane / LPR;
    const int64_t items = (int64_t)carry * p.Hkv;
    for (int64_t item = (int64_t)blockIdx.x * BND_WARPS + warp; item < items; item += (int64_t)gridDim.x * BND_WARPS) {
        const int i = (int)(item / p.Hkv), h = (int)(item - (int64_t)i * p.Hkv);
        int lo = 0, hi = B;                            // the last sequence that starts at or before i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int j = first[lo] + i - start[lo];
        const int rows = min(p.bs, __ldg(p.context_lens + lo) - j * p.bs);
        const int id = __ldg(p.block_tables + lo * p.stride + j);
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) set_status(p.status, STATUS_BOUNDS);
            continue;
        }
        const int64_t unit = (int64_t)id * p.Hkv + h;
        float vmax[EL], vmin[EL];
        if constexpr (KV8) {
            const uint8_t *k = static_cast<const uint8_t *>(p.k_cache) + unit * p.bs * D + sub * 16;
            const float *sc = p.k_scales + unit * p.bs;
#pragma unroll
            for (int e = 0; e < EL; ++e) vmax[e] = -INFINITY, vmin[e] = INFINITY;
            for (int r = grp; r < rows; r += RPS) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(k + (int64_t)r * D));
                const float f = __ldg(sc + r);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(ww[c >> 1] >> ((c & 1) * 16)));
                    const float2 x = unpack2(h2, __half());
                    const float a = x.x * f, b = x.y * f;
                    vmax[2 * c] = max_nan(vmax[2 * c], a), vmin[2 * c] = min_nan(vmin[2 * c], a);
                    vmax[2 * c + 1] = max_nan(vmax[2 * c + 1], b), vmin[2 * c + 1] = min_nan(vmin[2 * c + 1], b);
                }
            }
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < EL; ++e) {
                    vmax[e] = max_nan(vmax[e], __shfl_xor_sync(0xffffffffu, vmax[e], o));
                    vmin[e] = min_nan(vmin[e], __shfl_xor_sync(0xffffffffu, vmin[e], o));
                }
        } else {
            const uint16_t *k = static_cast<const uint16_t *>(p.k_cache) + unit * p.bs * D + sub * 8;
            // rows behind the last repeat row 0, which every group may count
            uint4 w = __ldg(reinterpret_cast<const uint4 *>(k + (int64_t)(grp < rows ? grp : 0) * D));
            uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll 4
            for (int r = grp + RPS; r < rows; r += RPS) {
                w = __ldg(reinterpret_cast<const uint4 *>(k + (int64_t)r * D));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) a[c] = max2(a[c], ww[c], T()), b[c] = min2(b[c], ww[c], T());
            }
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    a[c] = max2(a[c], __shfl_xor_sync(0xffffffffu, a[c], o), T());
                    b[c] = min2(b[c], __shfl_xor_sync(0xffffffffu, b[c], o), T());
                }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 x = unpack2(a[c], T()), y = unpack2(b[c], T());
                vmax[2 * c] = x.x, vmax[2 * c + 1] = x.y;
                vmin[2 * c] = y.x, vmin[2 * c + 1] = y.y;
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < EL; ++e) top = max(top, max(abs_bits(vmax[e]), abs_bits(vmin[e])));
        top = __reduce_max_sync(0xffffffffu, top);
        const bool number = top < INF_BITS;            // else: codes 0 and an infinite step, a block that is always wanted
        const float step = number ? step_of(top) : INFINITY, inv = number ? inverse_of(step) : 0.f;
        if (grp < 2) {
            uint32_t out[EL / 4];
#pragma unroll
            for (int c = 0; c < EL / 4; ++c) {
                int q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[e] = number ? code_of(grp == 0 ? vmax[4 * c + e] : vmin[4 * c + e], step, inv) : 0;
                out[c] = pack4(q[0], q[1], q[2], q[3]);
            }
            int8_t *dst = p.codes + (unit * 2 + grp) * D + sub * EL;
            if constexpr (KV8) *reinterpret_cast<uint4 *>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
            else *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
        }
        if (lane == 0) p.steps[unit] = step;
    }
}

cudaError_t launch_key_bounds(const BoundsParams &p, int dtype, int head_dim, int sm_count, cudaStream_t stream) {
    // touched blocks: at most one for each new token, and the full ones plus two ends of each sequence
    const int64_t blocks = std::min<int64_t>(p.num_tokens, p.num_tokens / p.bs + 2LL * p.num_seqs);
    const int64_t ctas = (blocks * p.Hkv + BND_WARPS - 1) / BND_WARPS, most = 8LL * sm_count;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min(ctas, most));
    const size_t smem = (size_t)(2 * p.num_seqs + 1) * sizeof(int);
    const auto launch = [&](auto kernel) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(BND_WARPS * 32), smem, stream, p);
    };
    if (p.k_scales) return launch(bounds_kernel<__half, 128, true>);
    if (dtype == PA_FP16) return head_dim == 128 ? launch(bounds_kernel<__half, 128, false>) : launch(bounds_kernel<__half, 64, false>);
    return head_dim == 128 ? launch(bounds_kernel<__nv_bfloat16, 128, false>) : launch(bounds_kernel<__nv_bfloat16, 64, false>);
}

// ------------------------------------------------------------------ selection

constexpr int SEL_WARPS = 8;
constexpr int SEL_THREADS = SEL_WARPS * 32;

__host__ __device__ constexpr int sel_q_stride(int D) { return 4 * D + 8; }   // bytes of a row [c+, c-] in fp16, and a pad
__host__ __device__ constexpr size_t sel_smem(int D, int NT, int chunk) {
    return (size_t)NT * 8 * (sel_q_stride(D) + 8) + (4 * 256 + 2 + SEL_WARPS * 2) * 4 + (size_t)chunk * 4;
}

// Whole numbers of four bytes as two pairs of fp16: the byte plus 128, under the exponent of 1024, less 1152.
__device__ __forceinline__ void bytes_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = x ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));        // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x0 = __hsub2(*reinterpret_cast<__half2 *>(&a), off), x1 = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x0);
    hi = *reinterpret_cast<const uint32_t *>(&x1);
}

// fp32 in an order of unsigned integers
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One cluster per (sequence, KV head); its CTAs hold the keys (ordered scores) of `chunk` blocks each in shared memory.
// Scores: 16 blocks per warp and step, the rows of an m16n8k16 product whose columns are 8 query rows; the codes go from
// global memory to the fragments without shared memory, 16 bytes per lane: a lane's 4 bytes are its four values of one
// 16-deep step, so the contraction's order is the bytes' own, and the query rows are laid out to match.
// Then the budget-th largest key, by its four bytes from the top (histograms in shared memory, summed over the cluster),
// and the indices of the keys above it and of the first ones equal to it, in order.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const SelectParams p) {
    constexpr int RP = NT * 8, LOADS = D / 32;         // 64-byte pieces of [hi, lo]
    constexpr int QS = sel_q_stride(D);
    extern __shared__ __align__(16) uint8_t ssm[];
    uint8_t *qsm = ssm;                                // [RP][QS]
    float *qmul = reinterpret_cast<float *>(qsm + RP * QS), *qadd = qmul + RP;   // a row's step; 0, or -inf: does not count
    int *hist = reinterpret_cast<int *>(qadd + RP);    // [4][256]
    int *counts = hist + 4 * 256;                      // keys above and equal to the threshold
    int *wcount = counts + 2;                          // [warps][2]
    uint32_t *keys = reinterpret_cast<uint32_t *>(wcount + SEL_WARPS * 2);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int unit = (int)(blockIdx.x / ranks), g = unit % p.Hkv, b = unit / p.Hkv;
    pdl_trigger();
    pdl_wait();

    int len = __ldg(p.context_lens + b);
    if (len < 0 || len > p.max_len || (len > 0 && len < p.q_len)) {
        if (tid == 0 && rank == 0) set_status(p.status, STATUS_BOUNDS);
        len = len < 0 ? 0 : min(len, p.max_len);
    }
    const int n = (len + p.bs - 1) / p.bs;
    int32_t *out = p.selected + (int64_t)unit * p.budget;
    if (n <= p.budget) {                               // all of them (the same in every CTA of the cluster)
        for (int i = rank * SEL_THREADS + tid; i < p.budget; i += ranks * SEL_THREADS) out[i] = i < n ? i : -1;
        return;
    }

    // ---- query rows
    for (int r = warp; r < RP; r += SEL_WARPS) {
        constexpr int PL = D / 32;
        float x[PL];
        uint32_t top = 0;
        if (r < p.rows) {
            const int qi = r / p.G, hh = r - qi * p.G;
            const T *q = static_cast<const T *>(p.q) + (((int64_t)b * p.q_len + qi) * p.Hq + g * p.G + hh) * D;
#pragma unroll
            for (int e = 0; e < PL; e += 2) {
                const float2 v = unpack2(__ldg(reinterpret_cast<const uint32_t *>(q + lane * PL + e)), T());
                x[e] = v.x, x[e + 1] = v.y;
                top = max(top, max(abs_bits(v.x), abs_bits(v.y)));
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const bool counts_row = r < p.rows && top < INF_BITS;
        const float step = counts_row ? step_of(top) : 0.f, inv = inverse_of(step);
        __half *row = reinterpret_cast<__half *>(qsm + r * QS);
#pragma unroll
        for (int e = 0; e < PL; ++e) {
            const int c = counts_row ? code_of(x[e], step, inv) : 0;
            row[lane * PL + e] = __int2half_rn(max(c, 0));
            row[D + lane * PL + e] = __int2half_rn(min(c, 0));
        }
        if (lane == 0) qmul[r] = step, qadd[r] = counts_row ? 0.f : -INFINITY;
    }
    for (int i = tid; i < 4 * 256; i += SEL_THREADS) hist[i] = 0;
    __syncthreads();

    // ---- scores
    const int i0 = rank * p.chunk, mine = max(0, min(p.chunk, n - i0));
    const int gq = lane >> 2, tq = lane & 3;
    const int32_t *trow = p.block_tables + b * p.stride;
    float mul[NT][2], add[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mul[nt][e] = qmul[nt * 8 + 2 * tq + e], add[nt][e] = qadd[nt * 8 + 2 * tq + e];
    for (int t = warp * 16; t < mine; t += SEL_WARPS * 16) {
        int id[2];
        bool ok[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = t + gq + 8 * e;
            id[e] = i < mine ? __ldg(trow + i0 + i) : 0;
            ok[e] = id[e] >= 0 && id[e] < p.num_blocks;
            if (!ok[e]) {
                set_status(p.status, STATUS_BOUNDS);
                id[e] = 0;
            }
        }
        uint4 w[2][LOADS];
        float step[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t u = (int64_t)id[e] * p.Hkv + g;
            const uint4 *src = reinterpret_cast<const uint4 *>(p.codes + u * 2 * D) + tq;
#pragma unroll
            for (int l = 0; l < LOADS; ++l) w[e][l] = __ldg(src + 4 * l);
            step[e] = __ldg(p.steps + u);
        }
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const uint32_t x[4] = {w[0][l].x, w[0][l].y, w[0][l].z, w[0][l].w};
            const uint32_t y[4] = {w[1][l].x, w[1][l].y, w[1][l].z, w[1][l].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t a0, a1, a2, a3;
                bytes_to_f16(x[c], a0, a2);
                bytes_to_f16(y[c], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(qsm + (nt * 8 + gq) * QS + (64 * l + 16 * tq + 4 * c) * 2);
                    mma_16816<__half>(acc[nt], a0, a1, a2, a3, q.x, q.y);
                }
            }
        }
        float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                best[0] = fmaxf(best[0], acc[nt][e] * mul[nt][e] + add[nt][e]);
                best[1] = fmaxf(best[1], acc[nt][2 + e] * mul[nt][e] + add[nt][e]);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], 1));
            best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], 2));
            const int i = t + gq + 8 * e, at = i0 + i;
            // a zero's sign must not order blocks; a step that is no number wants its block
            const float score = step[e] == INFINITY ? INFINITY : step[e] == 0.f ? 0.f : __fadd_rn(__fmul_rn(best[e], step[e]), 0.f);
            if (tq == e && i < mine)
                keys[i] = at < p.num_first || at >= n - p.num_last ? 0xFFFFFFFFu : ok[e] ? ordered(score) : 0u;
        }
    }
    __syncthreads();

    // ---- the budget-th largest key
    uint32_t prefix = 0, mask = 0;
    int need = p.budget;
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        int *h = hist + pass * 256;
        for (int i = tid; i < mine; i += SEL_THREADS)
            if ((keys[i] & mask) == prefix) atomicAdd(h + ((keys[i] >> shift) & 255), 1);
        cluster_sync();
        // warp 0: lane l sums bins 8 (31 - l) .. + 7, from the top
        if (warp == 0) {
            int bin[8], sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) bin[k] = 0;
            for (int r = 0; r < ranks; ++r) {
                const uint32_t src = map_rank(smem_u32(h + 8 * (31 - lane)), r);
#pragma unroll
                for (int k = 0; k < 8; ++k) bin[k] += ld_cluster_int(src + 4 * k);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += bin[k];
            int above = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, above, d);
                if (lane >= d) above += u;
            }
            above -= sum;
            if (above < need && above + sum >= need) {
                int k = 7;
                while (above + bin[k] < need) above += bin[k--];
                wcount[0] = 8 * (31 - lane) + k;
                wcount[1] = need - above;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)wcount[0] << shift;
        mask |= 0xFFu << shift;
        need = wcount[1];
        __syncthreads();
    }

    // ---- the keys above the threshold, and the first `need` equal to it
    if (tid == 0) counts[0] = counts[1] = 0;
    __syncthreads();
    int gt = 0, eq = 0;
    for (int i = tid; i < mine; i += SEL_THREADS) gt += keys[i] > prefix, eq += keys[i] == prefix;
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        if (gt) atomicAdd(counts, gt);
        if (eq) atomicAdd(counts + 1, eq);
    }
    cluster_sync();
    int gts = 0, eqs = 0;                              // before this CTA's blocks, then before this round's
    for (int r = 0; r < rank; ++r) {
        const uint32_t src = map_rank(smem_u32(counts), r);
        gts += ld_cluster_int(src);
        eqs += ld_cluster_int(src + 4);
    }
    cluster_arrive();                                  // this CTA reads no other one's memory any more
    for (int base = 0; base < mine; base += SEL_THREADS) {
        const int i = base + tid;
        const uint32_t key = i < mine ? keys[i] : 0u;
        const bool is_gt = i < mine && key > prefix, is_eq = i < mine && key == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
        if (lane == 0) wcount[2 * warp] = __popc(mg), wcount[2 * warp + 1] = __popc(me);
        __syncthreads();
        int g0 = gts, e0 = eqs;
        for (int w = 0; w < SEL_WARPS; ++w) {
            if (w < warp) g0 += wcount[2 * w], e0 += wcount[2 * w + 1];
            gts += wcount[2 * w], eqs += wcount[2 * w + 1];
        }
        const uint32_t below = (1u << lane) - 1u;
        g0 += __popc(mg & below);
        e0 += __popc(me & below);
        if (is_gt || (is_eq && e0 < need)) out[g0 + min(e0, need)] = i0 + i;
        __syncthreads();
    }
    cluster_wait();
}

template <typename T, int D>
static cudaError_t launch_select_t(SelectParams p, int sm_count, cudaStream_t stream) {
    const int blocks = (p.max_len + p.bs - 1) / p.bs, tiles = (blocks + 15) / 16;
    const int64_t units = (int64_t)p.num_seqs * p.Hkv;
    // CTAs of a cluster: enough for two on each SM, each with a tile for every warp
    int ranks = 1;
    while (ranks < 8 && ((units * ranks < 2LL * sm_count && tiles > ranks * SEL_WARPS) || tiles > ranks * 2048)) ranks *= 2;
    p.chunk = (tiles + ranks - 1) / ranks * 16;
    const auto launch = [&](auto kernel, int nt) {
        const size_t smem = sel_smem(D, nt, p.chunk);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return e != cudaSuccess ? e : launch_clusters(kernel, (unsigned)(units * ranks), SEL_THREADS, smem, ranks, stream, p);
    };
    switch ((p.rows + 7) / 8) {
        case 1: return launch(select_kernel<T, D, 1>, 1);
        case 2: return launch(select_kernel<T, D, 2>, 2);
        case 3: return launch(select_kernel<T, D, 3>, 3);
        default: return launch(select_kernel<T, D, 4>, 4);
    }
}

cudaError_t launch_select(SelectParams p, int dtype, int head_dim, int sm_count, cudaStream_t stream) {
    if (dtype == PA_FP16)
        return head_dim == 128 ? launch_select_t<__half, 128>(p, sm_count, stream) : launch_select_t<__half, 64>(p, sm_count, stream);
    return head_dim == 128 ? launch_select_t<__nv_bfloat16, 128>(p, sm_count, stream)
                           : launch_select_t<__nv_bfloat16, 64>(p, sm_count, stream);
}

}  // namespace pa
