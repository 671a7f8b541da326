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

}  // namespace

// ------------------------------------------------------------------ bounds

constexpr int BND_WARPS = 4;
// A lane's rows on their way at once: four. Eight take registers from other warps (14600 tokens of prompts 7.4 -> 8.9 us,
// 33 sequences of an FP8 pool 6.8 -> 7.6).
constexpr int BND_STEPS = 4;

// One warp per (touched block, KV head): 16 bytes of a key row per lane, several rows a step, the lanes that hold the
// same dimensions joined at the end. Every CTA makes the list of touched blocks for itself: their sums over the sequences.
// Bound by the chain before the first key (lengths, sums, search, table: 3.5 us) and then by memory: a decode step of 64
// sequences, 8 heads of 128 bf16, 3.5 us; 14600 tokens of prompts (33 MB) 7.4 us, 4.5 TB/s; 33 sequences of an FP8 pool 6.8.
template <typename T, int D, bool KV8>
__global__ void __launch_bounds__(BND_WARPS * 32) bounds_kernel(const BoundsParams p) {
    extern __shared__ int bsm[];
    const int B = p.num_seqs;
    int *start = bsm, *first = start + B + 1;          // sums of B + 1; first touched block
    __shared__ long long wsum[BND_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    long long carry = 0;
    for (int b0 = 0; b0 < B; b0 += BND_WARPS * 32) {
        const int b = b0 + tid;
        int n = 0;
        if (b < B) {
            const int lo = p.cu_q[b], hi = p.cu_q[b + 1], len = p.context_lens[b];
            if (lo < 0 || hi < lo || hi > p.num_tokens || len < hi - lo || len > p.max_len) {
                if (blockIdx.x == 0) set_status(p.status, STATUS_BOUNDS);
            } else if (hi > lo) {
                first[b] = (len - (hi - lo)) / p.bs;
                n = (len - 1) / p.bs - first[b] + 1;
            }
        }
        long long s = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        long long before = carry;
        for (int w = 0; w < BND_WARPS; ++w) {
            if (w < warp) before += wsum[w];
            carry += wsum[w];
        }
        if (b < B) start[b] = (int)(before + s - n);
        __syncthreads();
    }
    // more than num_tokens tokens can touch: sequences share rows of cu_q (one decreases, which is flagged); the sums of 32
    // bits and the work would have no bound
    if (carry > p.num_tokens / p.bs + 2LL * B) return;
    if (tid == 0) start[B] = (int)carry;
    __syncthreads();

    constexpr int LPR = KV8 ? D / 16 : D / 8;          // lanes per row
    constexpr int RPS = 32 / LPR;                      // rows a step
    constexpr int EL = KV8 ? 16 : 8;                   // dimensions per lane
    const int sub = lane % LPR, grp = lane / LPR;
    const int64_t items = carry * p.Hkv;
    for (int64_t item = (int64_t)blockIdx.x * BND_WARPS + warp; item < items; item += (int64_t)gridDim.x * BND_WARPS) {
        const int i = (int)(item / p.Hkv), h = (int)(item - (int64_t)i * p.Hkv);
        int lo = 0, hi = B;                            // the last sequence that starts at or before i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int j = first[lo] + i - start[lo];
        const int rows = min(p.bs, p.context_lens[lo] - j * p.bs);
        const int id = p.block_tables[lo * p.stride + j];
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) set_status(p.status, STATUS_BOUNDS);
            continue;
        }
        const int64_t unit = (int64_t)id * p.Hkv + h;
        float vmax[EL], vmin[EL];
        bool odd = false;                              // FP8: a NaN code, or a scale that is no number
        if constexpr (KV8) {
            const uint8_t *k = static_cast<const uint8_t *>(p.k_cache) + unit * p.bs * D + sub * 16;
            const float *sc = p.k_scales + unit * p.bs;
#pragma unroll
            for (int e = 0; e < EL; ++e) vmax[e] = -INFINITY, vmin[e] = INFINITY;
            for (int r0 = grp; r0 < rows; r0 += BND_STEPS * RPS) {
                uint4 w[BND_STEPS];
                float f[BND_STEPS];
#pragma unroll
                for (int s = 0; s < BND_STEPS; ++s) {
                    const int r = r0 + s * RPS;
                    if (r >= rows) break;
                    w[s] = *reinterpret_cast<const uint4 *>(k + (int64_t)r * D);
                    f[s] = sc[r];
                }
#pragma unroll
                for (int s = 0; s < BND_STEPS; ++s) {
                    if (r0 + s * RPS >= rows) break;
                    odd |= !(fabsf(f[s]) < INFINITY);
                    const uint32_t ww[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        odd |= __vcmpeq4(ww[c] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 x = unpack2(e4m3x2_to_f16x2((uint16_t)(ww[c] >> (16 * e))), __half());
                            const int i = 4 * c + 2 * e;
                            vmax[i] = fmaxf(vmax[i], x.x * f[s]), vmin[i] = fminf(vmin[i], x.x * f[s]);
                            vmax[i + 1] = fmaxf(vmax[i + 1], x.y * f[s]), vmin[i + 1] = fminf(vmin[i + 1], x.y * f[s]);
                        }
                    }
                }
            }
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < EL; ++e) {
                    vmax[e] = fmaxf(vmax[e], __shfl_xor_sync(0xffffffffu, vmax[e], o));
                    vmin[e] = fminf(vmin[e], __shfl_xor_sync(0xffffffffu, vmin[e], o));
                }
        } else {
            const uint16_t *k = static_cast<const uint16_t *>(p.k_cache) + unit * p.bs * D + sub * 8;
            uint32_t a[4], b[4];
            for (int r0 = grp; r0 < rows || r0 == grp; r0 += BND_STEPS * RPS) {
                uint4 w[BND_STEPS];                    // rows behind the last repeat row 0, which every group may count
#pragma unroll
                for (int s = 0; s < BND_STEPS; ++s) {
                    const int r = r0 + s * RPS;
                    if (s == 0 || r < rows) w[s] = *reinterpret_cast<const uint4 *>(k + (int64_t)(r < rows ? r : 0) * D);
                }
#pragma unroll
                for (int s = 0; s < BND_STEPS; ++s) {
                    if (s > 0 && r0 + s * RPS >= rows) break;
                    const uint32_t ww[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const bool begin = s == 0 && r0 == grp;
                        a[c] = begin ? ww[c] : max2(a[c], ww[c], T());
                        b[c] = begin ? ww[c] : min2(b[c], ww[c], T());
                    }
                }
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
        // else: codes 0 and an infinite step, a block that is always wanted
        const bool number = top < INF_BITS && !(KV8 && __any_sync(0xffffffffu, odd));
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
    const int64_t ctas = (blocks * p.Hkv + BND_WARPS - 1) / BND_WARPS, most = 16LL * sm_count;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min(ctas, most));
    const size_t smem = (size_t)(2 * p.num_seqs + 1) * sizeof(int);
    const auto launch = [&](auto kernel) {
        // the most that any call takes: the attribute is the kernel's, and other threads' calls set it too
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (2 * PA_TABLES_MAX_SEQS + 1) * (int)sizeof(int));
        return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(BND_WARPS * 32), smem, stream, p);
    };
    if (p.k_scales) return launch(bounds_kernel<__half, 128, true>);
    if (dtype == PA_FP16) return head_dim == 128 ? launch(bounds_kernel<__half, 128, false>) : launch(bounds_kernel<__half, 64, false>);
    return head_dim == 128 ? launch(bounds_kernel<__nv_bfloat16, 128, false>) : launch(bounds_kernel<__nv_bfloat16, 64, false>);
}

// ------------------------------------------------------------------ selection

constexpr int SEL_WARPS = 8;
constexpr int SEL_THREADS = SEL_WARPS * 32;
// Per SM: 64 registers a thread, of which heads of 128 spill 4 bytes with up to 8 query rows, 16 with 17 to 24 and 72 with more,
// heads of 64 12 bytes with 17 to 24. Three CTAs, which spill nothing: 64 sequences of 1024 blocks 27.0 -> 36.5 us.
constexpr int SEL_CTAS = 4;
constexpr int SEL_BINS = 256;
static_assert(SEL_BINS == SEL_THREADS, "one bin per thread");
constexpr int SEL_MAX_RANKS = 16;
constexpr int SEL_MAX_TILES = PA_SELECT_MAX_BLOCKS / 16 / SEL_MAX_RANKS;   // of 16 blocks, per CTA: 64 KB of keys
// Words of shared memory in front of the keys: histograms, ends (4), the digit (4), sums and counts of the warps.
constexpr int SEL_WORDS = 4 * SEL_BINS + 4 + 4 + SEL_WARPS * 3;

__host__ __device__ constexpr int sel_q_stride(int D) { return 4 * D + 32; }   // bytes of a row [c+, c-] in fp16, and a pad
// Where value i of a row lies: the four values of each of a quad's lanes in one step side by side.
__device__ __forceinline__ int sel_q_at(int i) { return (((i >> 7) * 8 + ((i & 31) >> 2)) * 4 + ((i >> 5) & 3)) * 4 + (i & 3); }
__host__ __device__ constexpr size_t sel_smem(int D, int NT, int chunk) {
    return (size_t)NT * 8 * (sel_q_stride(D) + 8) + SEL_WORDS * 4 + (size_t)chunk * 4;
}

// 32 bytes that no other CTA of this call reads (the bounds of a step are larger than what L2 could keep for the next).
__device__ __forceinline__ void ldg256(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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
// global memory to the fragments without shared memory, 32 bytes per lane: a lane's 4 bytes are its four values of one
// 16-deep step, so the contraction's order is the bytes' own, and the query rows are laid out to match.
//
// Then the threshold, the least key that is taken beside the blocks that always are: digits of 8 bits, from the highest
// bit in which the keys differ, by histograms that every CTA sums over the cluster for itself; it ends where a bin is
// taken whole, after two digits as a rule, after all of them only among equal scores. What the CTAs before this one hold
// above and at the threshold comes out of the same histograms, so the indices are written in order without another round.
//
// Bound by memory while it scores (64 sequences of 1024 blocks, 64 / 8 heads of 128: 132 MB in 18 us), with 2 us before it
// and 4 us behind it in which all CTAs, resident at once, are at the same point: 25.7 us, 5.1 TB/s. One sequence of 8192 blocks:
// 14.8 us, of which the barriers and histograms of 16 CTAs take 7. L2 is told to let the codes go first: 31.4 -> 29.9 us.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(SEL_THREADS, SEL_CTAS) select_kernel(const SelectParams p) {
    constexpr int W = SEL_WARPS, THREADS = SEL_THREADS;
    constexpr int RP = NT * 8, LOADS = D / 64;         // 128-byte pieces of [hi, lo]
    constexpr int QS = sel_q_stride(D);
    extern __shared__ __align__(16) uint8_t ssm[];
    uint8_t *qsm = ssm;                                // [RP][QS]
    float *qmul = reinterpret_cast<float *>(qsm + RP * QS), *qadd = qmul + RP;   // a row's step; 0, or -inf: does not count
    int *hist = reinterpret_cast<int *>(qadd + RP);    // [4][256]
    uint32_t *ends = reinterpret_cast<uint32_t *>(hist + 4 * SEL_BINS);   // least and largest key, of the CTA and of the cluster
    int *digit = reinterpret_cast<int *>(ends + 4);    // the digit, what is needed of its bin, the bin's size
    int *wtot = digit + 4;                             // [warps] sums; [warps][2] counts
    uint32_t *keys = reinterpret_cast<uint32_t *>(hist + SEL_WORDS);   // the block ids, then the keys in their place
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int unit = (int)(blockIdx.x / ranks), g = unit % p.Hkv, b = unit / p.Hkv;
    pdl_trigger();
    pdl_wait();

    int len = p.context_lens[b];
    // ---- query rows, on their way together
    constexpr int PL = D / 32, QR = (RP + W - 1) / W;  // values per lane; rows per warp
    uint32_t x[QR][PL / 2];
#pragma unroll
    for (int i = 0; i < QR; ++i) {
        const int r = warp + i * W;
#pragma unroll
        for (int e = 0; e < PL / 2; ++e) x[i][e] = 0u;
        if (r < p.rows) {
            const int qi = r / p.G, hh = r - qi * p.G;
            const T *q = static_cast<const T *>(p.q) + (((int64_t)b * p.q_len + qi) * p.Hq + g * p.G + hh) * D;
#pragma unroll
            for (int e = 0; e < PL / 2; ++e) x[i][e] = *reinterpret_cast<const uint32_t *>(q + lane * PL + 2 * e);
        }
    }
    // One CTA to a unit holds its blocks whatever the length is: their ids, and the codes of a warp's first tile as far as L2, a
    // line of 128 bytes a lane, are on their way before the query rows are taken to whole numbers (64 sequences 26.4 -> 25.7
    // us, in a graph 28.6 -> 26.6; two tiles 26.5; in clusters, where the memory is not what bounds it, 11.15 -> 11.3).
    const int32_t *trow = p.block_tables + b * p.stride;
    if (ranks == 1) {
        const int count = min(p.chunk, (int)p.stride);
        for (int i = tid; i < count; i += THREADS) keys[i] = (uint32_t)trow[i];
        const int i = warp * 16 + lane / 2;
        const int id = i < count ? trow[i] : -1;
        if (id >= 0 && id < p.num_blocks && (lane & 1) * 128 < 2 * D)
            prefetch_l2(p.codes + ((int64_t)id * p.Hkv + g) * 2 * D + (lane & 1) * 128);
    }
    if (len < 0 || len > p.max_len || (len > 0 && len < p.q_len)) {
        if (tid == 0 && rank == 0) set_status(p.status, STATUS_BOUNDS);
        len = len < 0 ? 0 : min(len, p.max_len);
    }
    const int n = (len + p.bs - 1) / p.bs;
    int32_t *out = p.selected + (int64_t)unit * p.budget;
    if (n <= p.budget) {                               // all of them (the same in every CTA of the cluster)
        for (int i = rank * THREADS + tid; i < p.budget; i += ranks * THREADS) {
            out[i] = i < n ? i : -1;
            const int id = i >= n ? 0 : ranks == 1 ? (int)keys[i] : trow[i];   // keys[i]: this thread's own
            if (id < 0 || id >= p.num_blocks) set_status(p.status, STATUS_BOUNDS);
        }
        return;
    }
    // blocks of this CTA, shared out evenly in tiles of 16; those of [lo, hi) are chosen by score, the others always
    const int per = ((n + 15) / 16 + ranks - 1) / ranks * 16;
    const int i0 = rank * per, mine = max(0, min(per, n - i0));
    const int lo = min(max(0, p.num_first - i0), mine), hi = max(lo, min(mine, n - p.num_last - i0));
    if (ranks > 1)
        for (int i = tid; i < mine; i += THREADS) keys[i] = (uint32_t)trow[i0 + i];
#pragma unroll
    for (int i = 0; i < QR; ++i) {
        const int r = warp + i * W;
        if (r >= RP) break;
        float v[PL];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < PL / 2; ++e) {
            const float2 f = unpack2(x[i][e], T());
            v[2 * e] = f.x, v[2 * e + 1] = f.y;
            top = max(top, max(abs_bits(f.x), abs_bits(f.y)));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const bool counts_row = r < p.rows && top < INF_BITS;
        const float step = counts_row ? step_of(top) : 0.f, inv = inverse_of(step);
        __half *row = reinterpret_cast<__half *>(qsm + r * QS);
#pragma unroll
        for (int e = 0; e < PL; ++e) {
            const int c = counts_row ? code_of(v[e], step, inv) : 0;
            row[sel_q_at(lane * PL + e)] = __int2half_rn(max(c, 0));
            row[sel_q_at(D + lane * PL + e)] = __int2half_rn(min(c, 0));
        }
        if (lane == 0) qmul[r] = step, qadd[r] = counts_row ? 0.f : -INFINITY;
    }
    for (int i = tid; i < 4 * SEL_BINS; i += THREADS) hist[i] = 0;
    if (tid < 2) ends[2 * tid] = 0xFFFFFFFFu, ends[2 * tid + 1] = 0u;
    __syncthreads();
    if (ranks > 1) cluster_arrive();

    // ---- scores
    const int gq = lane >> 2, tq = lane & 3;
    uint32_t least = 0xFFFFFFFFu, most = 0u;
    float mul[NT][2], add[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mul[nt][e] = qmul[nt * 8 + 2 * tq + e], add[nt][e] = qadd[nt * 8 + 2 * tq + e];
    for (int t = warp * 16; t < mine; t += W * 16) {
        int id[2];
        bool ok[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = t + gq + 8 * e;
            id[e] = i < mine ? (int)keys[i] : 0;
            ok[e] = id[e] >= 0 && id[e] < p.num_blocks;
            if (!ok[e]) {
                set_status(p.status, STATUS_BOUNDS);
                id[e] = 0;
            }
        }
        uint32_t w[2][LOADS][8];
        float step[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t u = (int64_t)id[e] * p.Hkv + g;
            const int8_t *src = p.codes + u * 2 * D + 32 * tq;
#pragma unroll
            for (int l = 0; l < LOADS; ++l) ldg256(src + 128 * l, w[e][l]);
            step[e] = p.steps[u];
        }
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t a0, a1, a2, a3;
                bytes_to_f16(w[0][l][c], a0, a2);
                bytes_to_f16(w[1][l][c], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 q = *reinterpret_cast<const uint2 *>(qsm + (nt * 8 + gq) * QS + (8 * l + c) * 32 + tq * 8);
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
            const int i = t + gq + 8 * e;
            // a zero's sign must not order blocks; a step that is no number wants its block
            const float score = step[e] == INFINITY ? INFINITY : step[e] == 0.f ? 0.f : __fadd_rn(__fmul_rn(best[e], step[e]), 0.f);
            if (tq == e && i >= lo && i < hi) {
                const uint32_t key = ok[e] ? ordered(score) : 0u;
                keys[i] = key;
                least = min(least, key), most = max(most, key);
            }
        }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMin(ends, least), atomicMax(ends + 1, most);
    __syncthreads();
    least = ends[0], most = ends[1];
    if (ranks > 1) {                                   // this CTA's to every CTA: no load waits for another one's memory
        cluster_wait();                                // their words are set
        if (tid < ranks) {
            const uint32_t to = map_rank(smem_u32(ends + 2), tid);
            red_cluster_min(to, least);
            red_cluster_max(to + 4, most);
        }
        cluster_sync();
        least = ends[2], most = ends[3];
    }

    // ---- the threshold: a key is taken if its digits so far are above `prefix`, or equal and among the first `need` of those
    int need = p.budget - (p.num_first + p.num_last);
    // what the CTAs before this one hold: above the threshold (the first blocks and, as the last CTA may, the last ones),
    // and at it
    int gt_before = min(i0, p.num_first) + max(0, min(i0, n) - (n - p.num_last)), eq_before = 0;
    int bits = 32 - __clz(least ^ most);               // bits in which the keys differ
    uint32_t mask = bits == 32 ? 0u : 0xFFFFFFFFu << bits, prefix = most & mask;
    if (need == 0) mask = prefix = 0xFFFFFFFFu, bits = 0;   // above every key
    else if (bits == 0) eq_before = max(0, min(i0, n - p.num_last) - p.num_first);   // equal keys
    for (int pass = 0; bits > 0; ++pass) {
        const int shift = max(0, bits - 8);
        const uint32_t digits = (1u << (bits - shift)) - 1u;
        int *h = hist + pass * SEL_BINS;
        for (int i = lo + tid; i < hi; i += THREADS) {
            const uint32_t key = keys[i];
            if ((key & mask) == prefix) atomicAdd(h + ((key >> shift) & digits), 1);
        }
        const int bin = SEL_BINS - 1 - tid;            // this thread's, from the top
        int sum = 0, before = 0;
        if (ranks > 1) {
            cluster_sync();
            const uint32_t src = smem_u32(h + bin);
            int v[SEL_MAX_RANKS];                      // all on their way before the first is added
#pragma unroll
            for (int r = 0; r < SEL_MAX_RANKS; ++r) v[r] = r < ranks ? ld_cluster_int(map_rank(src, r)) : 0;
#pragma unroll
            for (int r = 0; r < SEL_MAX_RANKS; ++r) sum += v[r], before += r < rank ? v[r] : 0;
        } else {
            __syncthreads();
            sum = h[bin];
        }
        int above = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, above, d);
            if (lane >= d) above += u;
        }
        if (lane == 31) wtot[warp] = above;
        above -= sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) above += wtot[w];
        if (above < need && above + sum >= need) digit[0] = bin, digit[1] = need - above, digit[2] = sum;
        __syncthreads();
        const int d = digit[0], size = digit[2];
        need = digit[1];
        if (ranks > 1) {                               // what lies before this CTA in the bins above and in this one
            int *cnt = wtot + SEL_WARPS;               // [warps][2]
            const int up = __reduce_add_sync(0xffffffffu, bin > d ? before : 0);
            const int at = __reduce_add_sync(0xffffffffu, bin == d ? before : 0);
            if (lane == 0) cnt[2 * warp] = up, cnt[2 * warp + 1] = at;
            __syncthreads();
            eq_before = 0;
#pragma unroll
            for (int w = 0; w < SEL_WARPS; ++w) gt_before += cnt[2 * w], eq_before += cnt[2 * w + 1];
        }
        prefix |= (uint32_t)d << shift;
        mask = shift == 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << shift;
        bits = size == need ? 0 : shift;               // a bin that is taken whole ends it
    }
    if (ranks > 1) cluster_arrive();                   // this CTA reads no other one's memory any more

    // ---- the indices, in order: a stretch of blocks per warp, counted and then written
    const int stretch = (mine + THREADS - 1) / THREADS * 32, s0 = min(mine, warp * stretch), s1 = min(mine, s0 + stretch);
    const auto taken = [&](int i, bool &is_gt, bool &is_eq) {
        const uint32_t key = i < s1 ? keys[i] & mask : 0u;
        const bool scored = i >= lo && i < hi;
        is_gt = i < s1 && (!scored || key > prefix);
        is_eq = i < s1 && scored && key == prefix;
    };
    __syncthreads();                                   // the sums' words are free
    int gt = 0, eq = 0;
    for (int i = s0 + lane; i < s0 + stretch; i += 32) {
        bool a, e;
        taken(i, a, e);
        gt += __popc(__ballot_sync(0xffffffffu, a)), eq += __popc(__ballot_sync(0xffffffffu, e));
    }
    if (lane == 0) wtot[2 * warp] = gt, wtot[2 * warp + 1] = eq;
    __syncthreads();
    for (int w = 0; w < warp; ++w) gt_before += wtot[2 * w], eq_before += wtot[2 * w + 1];
    for (int i = s0 + lane; i < s0 + stretch; i += 32) {
        bool a, e;
        taken(i, a, e);
        const uint32_t ma = __ballot_sync(0xffffffffu, a), me = __ballot_sync(0xffffffffu, e), below = (1u << lane) - 1u;
        const int ga = gt_before + __popc(ma & below), ee = eq_before + __popc(me & below);
        if (a || (e && ee < need)) out[ga + min(ee, need)] = i0 + i;
        gt_before += __popc(ma);
        eq_before += __popc(me);
    }
    if (ranks > 1) cluster_wait();
}

template <typename T, int D>
static cudaError_t launch_select_t(SelectParams p, int sm_count, cudaStream_t stream) {
    const int blocks = (p.max_len + p.bs - 1) / p.bs, tiles = (blocks + 15) / 16;
    const int64_t units = (int64_t)p.num_seqs * p.Hkv;
    // CTAs of a cluster, by what one takes, in units of 5 ns: a warp's tiles of 16 blocks, 1 us each, for every round of resident
    // CTAs; 2 us for the barriers and histograms of a cluster; and what the CTAs that start and meet cost, of all units and of one.
    // Over 290 shapes (8 to 512 units, 130 to 8192 blocks, 4 to 32 rows, heads of 64 and 128) this picks the best of 1, 2, 4, 8, 16
    // but for 1.2% on average, 22% at most. "Two CTAs on each SM, each with a tile for every warp" lost 15% and up to 72%: 128
    // units of 160 blocks take 7.2 us as single CTAs, 10.7 as clusters of two; 64 of 4096 48 and, of eight, 23.6; 8 of 8192 71
    // and, of sixteen, 14.8.
    int ranks = SEL_MAX_RANKS;
    int64_t best = -1;
    for (int r = 1; r <= SEL_MAX_RANKS; r *= 2) {
        if (tiles > r * SEL_MAX_TILES) continue;       // no room for the keys
        const int64_t rounds = (units * r + SEL_CTAS * sm_count - 1) / (SEL_CTAS * sm_count);
        const int64_t cost = 200 * rounds * ((tiles + r * SEL_WARPS - 1) / (r * SEL_WARPS)) + (r > 1 ? 400 : 0) + (units + 24) * r;
        if (best < 0 || cost < best) best = cost, ranks = r;
    }
    p.chunk = (tiles + ranks - 1) / ranks * 16;
    const auto launch = [&](auto kernel, int nt) {
        static_assert(sel_smem(D, 4, SEL_MAX_TILES * 16) <= MAX_SMEM_PER_CTA, "the keys of the longest row");
        const size_t smem = sel_smem(D, nt, p.chunk);
        // the most that any call takes: the attribute is the kernel's, and other threads' calls set it too
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sel_smem(D, nt, SEL_MAX_TILES * 16));
        if (e == cudaSuccess && ranks > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
