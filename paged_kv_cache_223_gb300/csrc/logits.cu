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
// Bound: memory, one read of the logits and one fp32 write. So a row is read once and stays in registers:
// it is cut into slices, one block each; for probabilities the row's (up to 8) blocks are a cluster that
// exchanges each warp's (max, sum, first index of the max) through distributed shared memory, in one
// barrier. A thread
// holds 4 NG values; its loads are all in flight before the block turns to the lists.
// The lists (history, drafts, biases) are sparse, so they are worked on entry by entry: each block counts
// the entries of its slice in a table in shared memory, one word per token (bits 0..19 count the outputs,
// bit 20 marks a prompt token, bits 21..31 hold 1 + the index of the last bias entry naming the token;
// integer atomics, so the order of arrival changes nothing), and the first entry to claim a token's bit
// replaces the token's word by the adjusted logit. The pass over the values only looks at the bits.
//
// Measured, 64 x 6 rows of 128256 fp32 logits: adjusting without lists 59 us (0.99 of the copy rate), with a history
// of up to 4096 tokens, biases, drafts and masks 87 us; probabilities without lists 91 us, with them 141 us (0.42), of
// which counting takes about 22 and the adjusted logits 16 (entries kept in one list of the block, with the positions
// from shared atomics, and eight entries held per thread, which spilled: 151 us).
// What is left is a block's chain of barriers (three for the lists, one of the cluster) with two blocks per SM to
// overlap it: registers bound those (64 a thread with 8 groups, 8 to 16 bytes spilled). Rows above 131072 tokens
// take the kernel of 24 groups, one block per SM and up to 284 bytes spilled: 64 x 6 rows with lists of 151936 fp32
// logits 329 us (0.21), of 262144 409 us (0.30). Not kept: penalties computed in the pass over the values (200 us),
// slices dealt out in pieces of 128 or 2048 tokens so that the lists even out (lists 5 to 10 us less, the rest 13
// to 20 us more), the logits prefetched into L2 one round of blocks ahead and loaded behind the lists (150 us), the
// lists read once for six rows that a cluster takes in turn (161 us), asynchronous copies of the listed logits and
// of the biases into shared memory (160 us).
#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_serving.h"

namespace pa {

constexpr int LG_THREADS = 512;
constexpr int LG_GROUP = 4 * LG_THREADS;              // values of a block per group of four per thread
constexpr uint32_t LG_PROMPT = 1u << 20, LG_COUNT = LG_PROMPT - 1u;
constexpr int LG_BIAS_SHIFT = 21;
static_assert(PA_LOGITS_MAX_HISTORY + PA_LOGITS_MAX_ROWS <= (int)LG_COUNT, "an output count fits its field");
static_assert(PA_LOGITS_MAX_BIAS + 1 < (1 << (32 - LG_BIAS_SHIFT)), "a bias index fits its field");
constexpr int LG_MAX_SLICES = 8;                      // blocks of a row: a portable cluster
constexpr int LG_KEPT = 384;                          // entries of a slice that a warp keeps in shared memory
constexpr int LG_KEPT_BYTES = LG_THREADS / 32 * LG_KEPT * 2;
static_assert(PA_LOGITS_MAX_VOCAB <= 8 * 65536, "a token within a slice fits 16 bits of an entry");
static_assert(PA_LOGITS_MAX_VOCAB <= 8 * 24 * LG_GROUP, "a cluster holds the largest row");

struct RowPart {
    float m, s;
    int best;
};

// The lists of a row, and this thread's first entries of them, loaded before the logits are (behind those, a
// list's latency would be theirs too).
constexpr int LG_HELD = 6;
struct RowLists {
    int len, prompt, bias0, draft0, hist0[LG_HELD];
};

__device__ __forceinline__ void load_lists(const LogitsParams &p, int b, int j, int tid, RowLists &l) {
    const int cap = p.history ? p.history_cap : 0;
    l.len = cap > 0 ? __ldg(p.history_lens + b) : 0;
    l.prompt = cap > 0 && p.prompt_lens ? __ldg(p.prompt_lens + b) : 0;
    l.bias0 = tid < p.num_bias ? __ldg(p.bias_tokens + (int64_t)b * p.num_bias + tid) : -1;
    l.draft0 = p.draft && tid < j ? __ldg(p.draft + b * (p.R - 1) + tid) : -1;
    const int32_t *hist = p.history + b * p.history_stride;
#pragma unroll
    for (int k = 0; k < LG_HELD; ++k)
        l.hist0[k] = tid + k * LG_THREADS < cap ? __ldg(hist + tid + k * LG_THREADS) : -1;
}

__device__ __forceinline__ float load_logit(const LogitsParams &p, int64_t i) {
    if (p.dtype == PA_LOGITS_FP32) return static_cast<const float *>(p.logits)[i];
    if (p.dtype == PA_LOGITS_FP16) return __half2float(static_cast<const __half *>(p.logits)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[i]);
}

// Adjusted logits of the listed tokens of the slice [base, base + n) (entries that name another slice's token,
// or none, are left to others): bit t of `bits` set, the fp32 word in table[t]. `off`: the slice's first logit.
// Each warp keeps the tokens that its entries named for the last step; one with more than LG_KEPT of them (a long
// history of few different tokens) reads its entries again for it. table and bits come zeroed.
__device__ __forceinline__ void adjust_listed(const LogitsParams &p, RowLists &l, int b, int j, int base, int n, int64_t off,
                                              uint32_t *table, uint32_t *bits, uint16_t *kept, int tid) {
    const float rep = p.repetition ? __ldg(p.repetition + b) : 1.f;
    const float freq = p.frequency ? __ldg(p.frequency + b) : 0.f, pres = p.presence ? __ldg(p.presence + b) : 0.f;
    const int lane = tid & 31, first = tid - lane;
    const int cap = p.history ? p.history_cap : 0, len = l.len < 0 ? 0 : (l.len > cap ? cap : l.len);
    const int drafts = p.draft ? j : 0;
    // fn(token within the slice, or a negative number; index in the list), by whole warps
    auto local = [&](int t) { return t >= base && t - base < n ? t - base : -1; };
    auto biases = [&](auto &&fn) {
        for (int i0 = first; i0 < p.num_bias; i0 += LG_THREADS) {
            const int i = i0 + lane;
            fn(local(i0 == first ? l.bias0 : (i < p.num_bias ? __ldg(p.bias_tokens + (int64_t)b * p.num_bias + i) : -1)), i);
        }
    };
    auto tokens = [&](auto &&fn) {
#pragma unroll
        for (int k = 0; k < LG_HELD; ++k) {
            if (first + k * LG_THREADS >= len) break;
            fn(tid + k * LG_THREADS < len ? local(l.hist0[k]) : -1, tid + k * LG_THREADS);
        }
        for (int i0 = first + LG_HELD * LG_THREADS; i0 < len; i0 += 4 * LG_THREADS) {
            int t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + lane + k * LG_THREADS;
                t[k] = i < len ? __ldg(p.history + b * p.history_stride + i) : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) fn(local(t[k]), i0 + lane + k * LG_THREADS);
        }
        for (int i0 = first; i0 < drafts; i0 += LG_THREADS) {
            const int i = i0 + lane;
            fn(local(i0 == first ? l.draft0 : (i < drafts ? __ldg(p.draft + b * (p.R - 1) + i) : -1)), 0x7fffffff);
        }
    };
    kept += (tid >> 5) * LG_KEPT;
    int count = 0;                                    // of this warp's entries
    auto keep = [&](int t) {
        const uint32_t all = __ballot_sync(0xffffffffu, t >= 0);
        const int at = count + __popc(all & ((1u << lane) - 1u));
        if (t >= 0 && at < LG_KEPT) kept[at] = (uint16_t)t;
        count += __popc(all);
    };
    if (p.num_bias > 0) {
        biases([&](int t, int i) {
            keep(t);
            if (t >= 0) atomicMax(table + t, (uint32_t)(i + 1) << LG_BIAS_SHIFT);
        });
        __syncthreads();                              // the bias field is final before counts are added below it
    }
    tokens([&](int t, int i) {
        keep(t);
        if (t < 0) return;
        if (i < l.prompt) atomicOr(table + t, LG_PROMPT);
        else atomicAdd(table + t, 1u);
    });
    __syncthreads();
    auto adjust = [&](int t) {
        if ((atomicOr(bits + (t >> 5), 1u << (t & 31)) >> (t & 31)) & 1u) return;   // another entry has it
        const uint32_t w = table[t], made = w & LG_COUNT;
        float x = load_logit(p, off + t);
        if (p.repetition && (w & (LG_COUNT | LG_PROMPT))) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        if (made) {
            if (p.frequency) x = __fsub_rn(x, __fmul_rn(freq, (float)made));
            if (p.presence) x = __fsub_rn(x, pres);
        }
        if (w >> LG_BIAS_SHIFT)
            x = __fadd_rn(x, __ldg(p.bias_values + (int64_t)b * p.num_bias + (w >> LG_BIAS_SHIFT) - 1));
        table[t] = __float_as_uint(x);
    };
    if (count <= LG_KEPT) {
        for (int i = lane; i < count; i += 32) adjust(kept[i]);
    } else {
        auto each = [&](int t, int) {
            if (t >= 0) adjust(t);
        };
        biases(each);
        tokens(each);
    }
    __syncthreads();
}

// The row's parts meet in shared memory: every warp of every block of the cluster sends its part to all of them.
__device__ __forceinline__ void send_part(RowPart (*parts)[LG_THREADS / 32], int rank, int warp, int to,
                                          const RowPart &x) {
    const uint32_t at = smem_u32(&parts[rank][warp]);
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(to));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(x.m) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there + 4), "f"(x.s) : "memory");
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there + 8), "r"(x.best) : "memory");
}

// NG groups of four values per thread. VEC: the four are consecutive (16- or 8-byte loads, 16-byte stores);
// else LG_THREADS apart, each access coalesced on its own (rows that start between vectors).
template <bool PROBS, bool VEC, int NG>
__global__ void __launch_bounds__(LG_THREADS, NG <= 8 ? 2 : 1) logits_kernel(const LogitsParams p, int slice,
                                                                            int slices) {
    extern __shared__ __align__(16) uint32_t lg_table[];
    __shared__ RowPart s_parts[LG_MAX_SLICES][LG_THREADS / 32];
    __shared__ uint32_t s_mask[NG * LG_GROUP / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / slices, rank = blockIdx.x - row * slices;
    const int b = row / p.R, j = row - b * p.R;
    const int base = rank * slice;
    const int n = p.V - base < slice ? (p.V - base > 0 ? p.V - base : 0) : slice;   // values of this block
    auto index = [&](int g, int e) { return VEC ? (g * LG_THREADS + tid) * 4 + e : (g * 4 + e) * LG_THREADS + tid; };
    if (PROBS && slices > 1) cluster_arrive();        // waited for below: every block's shared memory exists
    pdl_wait();
    const bool lists = p.history || p.draft || p.num_bias > 0;
    uint32_t *bits = lg_table + slice;                // slice / 32 words, then the kept tokens
    RowLists l;
    if (lists) {
        load_lists(p, b, j, tid, l);
        for (int i = tid * 4; i < slice + slice / 32; i += LG_THREADS * 4)
            *reinterpret_cast<uint4 *>(lg_table + i) = make_uint4(0u, 0u, 0u, 0u);
    }
    float T = 0.f;
    if constexpr (PROBS) T = __ldg(p.temperature + b);

    // the slice, raw: 32-bit words of four values (fp32), or two words of four 16-bit values, or one per word
    uint32_t raw[NG][4];
    const int64_t off = b * p.seq_stride + j * p.row_stride + base;
    if (p.dtype == PA_LOGITS_FP32) {
        const uint32_t *src = static_cast<const uint32_t *>(p.logits) + off;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if constexpr (VEC) {
                if (index(g, 0) < n) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(src + index(g, 0));
                    raw[g][0] = w.x, raw[g][1] = w.y, raw[g][2] = w.z, raw[g][3] = w.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (index(g, e) < n) raw[g][e] = src[index(g, e)];
            }
        }
    } else {
        const uint16_t *src = static_cast<const uint16_t *>(p.logits) + off;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if constexpr (VEC) {
                if (index(g, 0) < n) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src + index(g, 0));
                    raw[g][0] = w.x, raw[g][1] = w.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (index(g, e) < n) raw[g][e] = src[index(g, e)];
            }
        }
    }
    // the slice's mask, zero behind its end; without one, all ones up to there
    {
        const uint32_t *mask = reinterpret_cast<const uint32_t *>(p.mask) + (int64_t)row * ((p.V + 31) / 32) + base / 32;
        for (int i = tid; i < NG * LG_GROUP / 32; i += LG_THREADS) {
            const int left = n - 32 * i;
            uint32_t w = left <= 0 ? 0u : (p.mask ? __ldg(mask + i) : 0xFFFFFFFFu);
            if (left > 0 && left < 32) w &= (1u << left) - 1u;
            s_mask[i] = w;
        }
    }
    __syncthreads();
    if (lists)
        adjust_listed(p, l, b, j, base, n, off, lg_table, bits, reinterpret_cast<uint16_t *>(bits + slice / 32), tid);

    float x[NG][4];
    float m = -INFINITY;
    auto half = [&](int g, int e) { return VEC ? (raw[g][e >> 1] >> ((e & 1) * 16)) & 0xFFFFu : raw[g][e]; };
    if (p.dtype == PA_LOGITS_FP32) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[g][e] = __uint_as_float(raw[g][e]);
    } else if (p.dtype == PA_LOGITS_BF16) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[g][e] = __uint_as_float(half(g, e) << 16);
    } else {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[g][e] = __half2float(__ushort_as_half((unsigned short)half(g, e)));
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if constexpr (VEC) {
            const int i = index(g, 0);
            const uint32_t allowed = s_mask[i >> 5] >> (i & 31);
            if (lists) {
                const uint32_t listed = i < n ? (bits[i >> 5] >> (i & 31)) & 0xFu : 0u;
                if (listed) {
                    const float4 t = *reinterpret_cast<const float4 *>(lg_table + i);
                    x[g][0] = listed & 1u ? t.x : x[g][0];
                    x[g][1] = listed & 2u ? t.y : x[g][1];
                    x[g][2] = listed & 4u ? t.z : x[g][2];
                    x[g][3] = listed & 8u ? t.w : x[g][3];
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[g][e] = allowed & (1u << e) ? x[g][e] : -INFINITY;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = index(g, e);
                if (lists && i < n && ((bits[i >> 5] >> (i & 31)) & 1u)) x[g][e] = __uint_as_float(lg_table[i]);
                if (!((s_mask[i >> 5] >> (i & 31)) & 1u)) x[g][e] = -INFINITY;
            }
        }
        m = fmaxf(m, fmaxf(fmaxf(x[g][0], x[g][1]), fmaxf(x[g][2], x[g][3])));
    }

    float scale = 1.f;                                // of this warp's exponentials
    if constexpr (PROBS) {
        // the warp's maximum and its sum of exponentials relative to that; (max, sum) pairs of the row's warps
        // are then joined by their maxima
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool greedy = T == 0.f;
        // exp((x - m) / T) = 2^((x - m) k). A temperature so small that k overflows gets the largest float, one so
        // large that it vanishes the smallest normal one: 0 k stays 0 and -inf k stays -inf
        const float k = T > 0.f ? fminf(fmaxf(__fdiv_rn(1.4426950408889634f, T), 1.17549435e-38f), 3.402823466e38f)
                                : __int_as_float(0x7fc00000);
        float sum = 0.f;
        int best = 0x7fffffff;
        if (greedy) {
            // no exponentials: the first index of the maximum, and a NaN if there is one
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (x[g][e] == m && m > -INFINITY) best = min(best, base + index(g, e));
                    if (x[g][e] != x[g][e]) sum = x[g][e];
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        } else {
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[g][e] = ex2_approx((x[g][e] - ref) * k);
                sum += (x[g][0] + x[g][1]) + (x[g][2] + x[g][3]);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const RowPart mine = {m, sum, best};
        if (slices > 1) {
            cluster_wait();
            if (lane < slices) send_part(s_parts, rank, warp, lane, mine);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        } else {
            if (lane == 0) s_parts[0][warp] = mine;
            __syncthreads();
        }
        // the parts, in the same order in every warp of the row
        constexpr int W = LG_THREADS / 32;
        const RowPart *parts = &s_parts[0][0];
        float M = -INFINITY;
        for (int i = lane; i < slices * W; i += 32) M = fmaxf(M, parts[i].m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        auto weight = [&](float mc) { return mc == -INFINITY || greedy ? 1.f : ex2_approx((mc - M) * k); };
        float S = 0.f;
        best = 0x7fffffff;
        for (int i = lane; i < slices * W; i += 32) {
            const RowPart q = parts[i];
            S += q.s * weight(q.m);
            if (q.m == M) best = min(best, q.best);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            S += __shfl_xor_sync(0xffffffffu, S, o);
            best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        }
        if (greedy) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[g][e] = S != S ? S : (base + index(g, e) == best ? 1.f : 0.f);
        } else {
            scale = S == 0.f ? 0.f : weight(m) * __fdiv_rn(1.f, S);
        }
    }

    float *out = p.out + (int64_t)row * p.V + base;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = PROBS ? x[g][e] * scale : x[g][e];
        if constexpr (VEC) {
            if (index(g, 0) < n) *reinterpret_cast<float4 *>(out + index(g, 0)) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (index(g, e) < n) out[index(g, e)] = y[e];
        }
    }
}

template <bool PROBS, bool VEC, int NG>
static cudaError_t launch_ng(const LogitsParams &p, int slice, int slices, cudaStream_t stream) {
    const bool lists = p.history || p.draft || p.num_bias > 0;
    const size_t smem = lists ? (size_t)slice * 4 + slice / 8 + LG_KEPT_BYTES : 0;
    auto kernel = logits_kernel<PROBS, VEC, NG>;
    // from where it may pass 48 KB with the fixed part; set on every call: the attribute belongs to the current device,
    // and callers may use several
    if (smem > 32 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 NG * LG_GROUP * 4 + NG * LG_GROUP / 8 + LG_KEPT_BYTES);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.R * slices));
    cfg.blockDim = dim3(LG_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = PROBS ? slices : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, slice, slices);
}

template <bool PROBS>
static cudaError_t launch_logits_t(const LogitsParams &p, int sm_count, cudaStream_t stream) {
    // Slices per row: a power of two up to 8. Rows that fill the GPU take the fewest slices of at most
    // 8 groups (two blocks per SM); fewer rows are cut further, down to slices of one group.
    const int64_t rows = (int64_t)p.B * p.R;
    int slices = 1;
    while (slices < 8 && p.V > slices * 8 * LG_GROUP) slices *= 2;
    while (slices < 8 && rows * slices < 2 * sm_count && p.V > slices * LG_GROUP) slices *= 2;
    const int slice = ((p.V + slices - 1) / slices + 127) / 128 * 128;
    const int groups = (slice + LG_GROUP - 1) / LG_GROUP;
    const int esize = p.dtype == PA_LOGITS_FP32 ? 4 : 2;
    const bool vec = p.V % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.logits) % (4 * esize) == 0 && p.row_stride % 4 == 0 &&
                     p.seq_stride % 4 == 0;
#define PA_LG(NG_)                                                       \
    return vec ? launch_ng<PROBS, true, NG_>(p, slice, slices, stream)   \
               : launch_ng<PROBS, false, NG_>(p, slice, slices, stream)
    if (groups <= 2) PA_LG(2);
    if (groups <= 8) PA_LG(8);
    PA_LG(24);
#undef PA_LG
}

cudaError_t launch_logits(const LogitsParams &p, bool probs, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    return probs ? launch_logits_t<true>(p, sms, stream) : launch_logits_t<false>(p, sms, stream);
}

}  // namespace pa
