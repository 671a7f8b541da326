// selected.cu -- attention of new query rows over a list of blocks for each (sequence, KV head).
//
// out = sum_t softmax_t(scale q . K_t) V_t over the tokens t of the listed blocks that are at or before the row's
// position, by one pass with the running maximum and sum; rows that see none of them give zeros.
//
// What bounds it: the K and V rows of the listed blocks, read once. A unit (sequence, KV head; all its query rows together)
// is one cluster of CTAs. Its tiles of 16 tokens are dealt out to the warps of the whole cluster in turn, so a list that is
// short of its budget still spreads over all of them. Every warp looks its tiles up (list, then block table) before its
// first copy, keeps those that hold tokens, and runs a pipeline of its own over them: TMA tile loads, scores S^T = K Q^T
// and O^T += V^T P^T as warp-level products with the query rows as columns, softmax in fp32 between them. The states of a
// CTA's warps are joined in its shared memory, those of the cluster's CTAs through each other's, each CTA writing a share
// of the outputs: one launch, no workspace, a fixed order.
//
// Measured: 64 sequences of 128 blocks of 16 tokens, 64 / 8 heads of 128, bf16 (539 MB): 78 to 81 us, 6.7 to 6.9 TB/s, the copy
// rate; one sequence of 64 blocks 6.9 us (in a graph 5.9): launch 2, lookups 1.5, two tiles a warp 1, joins 2; 19 sequences of
// 50 blocks of 32 in an FP8 pool, 16 query rows, fp16: 20.4 us, bound by a warp's chain per tile at eight warps an SM (with
// weights in one part 17.2: scores 300 cycles, softmax 360, weights 90, values and the next copies 500).
#include <type_traits>

#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_sparse.h"

namespace pa {

namespace {

constexpr int ATT_WARPS = 4;
constexpr int ATT_THREADS = ATT_WARPS * 32;
constexpr int ATT_MAX_RANKS = 8;
constexpr int ATT_MAX_TILES = PA_SELECT_MAX_BUDGET * (32 / TILE_TOKENS);   // of a list, in blocks of 32 tokens
constexpr float ATT_RESCALE_LOG2 = 8.f;                // a row's reference maximum moves when it is passed by 2^8
// Many small weights beside a large one. fp16 and FP8 pools: weights (and the sums that they are divided by) are 2^7 as large, below 2^15,
// so that they keep bits down to 2^-32 of the large one instead of 2^-25. And a product's accumulator drops what lies below its
// own last bit, so a warp takes 256 tiles at most where a cluster can be made larger, as it can for every list: 4096 tokens below
// 2^-25 are 2^-13 of the output. (32768 to a warp: 2^-10; equal weights lost as much.) With the limit and without it: 608 lists of
// 4096 blocks of 32 tokens, shared by all, 2640 and 4340 us (FP8 2600 and 3230), 300 lists of 2048 blocks 757 and 1090 (739 and 658).
constexpr float ATT_LIFT_LOG2 = 7.f;
constexpr int ATT_WARP_TILES = 256;
// FP8: a weight goes into the product times its V scale, as fp16 (below 2^15), in a unit 2^vexp that follows the scales. The
// largest one of a tile sets it, with 2^2 of room above, and sets it anew where a scale passes it or lies below its 2^-6 (weights
// in one part of fp16) or 2^-14 (two parts); tokens that then still lie below are added apart, in fp32. So a weight is off by 2^-11
// of itself in one part and 2^-22 in two, or by 2^-26 and 2^-29 of the row's largest, and no token's scale costs another one its
// bits, whatever their weights are. The unit stays within 2^80 of the largest that it was, so that O stays in fp32's range. Of
// scales near each other, 8, 16, 32 rows of 64 sequences: bf16 44.9, 60.8, 86.3 -> 46.5, 61.4, 85.6 us, fp16 47.2, 70.9, 109 -> 47.5,
// 70.4, 107.
constexpr int ATT_ROOM_ABOVE = 2, ATT_ROOM_ONE = 6, ATT_ROOM_TWO = 14, ATT_MIN_UNIT = -110, ATT_MAX_UNIT = 119, ATT_UNIT_SPAN = 80;
static_assert(ATT_MAX_TILES <= ATT_WARP_TILES * ATT_WARPS * ATT_MAX_RANKS, "the longest list");

// Copies of a warp's pipeline in flight, and CTAs per SM. FP8 pools, tiles of 4 KB: two copies (three: 19 sequences of a verify
// 17.5 -> 17.7 us, 64 of 2048 tokens 44 -> 46), four CTAs with one column of eight rows, else two by registers (16 rows at
// three CTAs, with spills: 18.9 -> 23.0; as pairs of warps on a pipeline, eight rows each, 16 warps an SM: 17.6 -> 21.4). 16-bit
// pools, 8 KB: three copies, two CTAs. Three CTAs of two copies each keep as many bytes in flight: 64 sequences of 128 blocks 86
// us instead of 79.
__host__ __device__ constexpr int att_stages(bool kv8) { return kv8 ? 2 : 3; }
__host__ __device__ constexpr int att_ctas(bool kv8, int nt) { return kv8 && nt == 1 ? 4 : 2; }
__host__ __device__ constexpr int att_tile_bytes(int D, bool kv8) { return TILE_TOKENS * (kv8 ? 128 : 2 * D); }
__host__ __device__ constexpr int att_ring_bytes(int D, bool kv8) {
    return ATT_WARPS * att_stages(kv8) * 2 * att_tile_bytes(D, kv8);
}
// states of the warps [W][RP][D + 4] and (max, sum) [W][RP], the CTA's own [RP][D + 4] and (max, sum) [RP], factors [RP][W]
__host__ __device__ constexpr int att_join_bytes(int D, int nt) {
    return 4 * nt * 8 * ((ATT_WARPS + 1) * (D + 4) + (ATT_WARPS + 1) * 2 + ATT_WARPS);
}
__host__ __device__ constexpr int att_body_bytes(int D, bool kv8, int nt) {
    return (att_ring_bytes(D, kv8) > att_join_bytes(D, nt) ? att_ring_bytes(D, kv8) : att_join_bytes(D, nt)) + 15 & ~15;
}
// The query rows' fragments lie in shared memory from three columns of eight on, where they would not fit the registers: 64
// sequences of 2048 tokens, 32 rows, FP8 110 -> 86 us, bf16 102 -> 97; with two columns (16 rows) the loads lengthen the chain:
// 19 sequences of a verify, FP8, 17.5 -> 21.4.
__host__ __device__ constexpr bool att_q_shared(int nt) { return nt > 2; }
__host__ __device__ constexpr int att_q_bytes(int D, int nt) { return att_q_shared(nt) ? nt * (D / 16) * 32 * 8 : 0; }
// Ring or states, barriers, the flag of a lost copy, the query rows; the tile lists follow.
__host__ __device__ constexpr int att_flag_at(int D, bool kv8, int nt) {
    return att_body_bytes(D, kv8, nt) + ATT_WARPS * att_stages(kv8) * 8;
}
__host__ __device__ constexpr int att_q_at(int D, bool kv8, int nt) { return att_flag_at(D, kv8, nt) + 16; }
__host__ __device__ constexpr int att_lists_at(int D, bool kv8, int nt) { return att_q_at(D, kv8, nt) + att_q_bytes(D, nt); }

constexpr size_t att_smem(int D, bool kv8, int nt, int warp_tiles) {
    return 1024 + att_lists_at(D, kv8, nt) + (size_t)ATT_WARPS * warp_tiles * 8;
}

// Where 16 bytes (chunk c of a token's row r) of a tile lie: FP8 rows of 128 bytes; 16-bit ones in groups of eight rows, by
// halves of 64 dimensions; swizzled by the copy.
template <int D, bool KV8>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    if constexpr (KV8) return r * 128 + ((c ^ (r & 7)) << 4);
    return ((r >> 3) * (D / 64) + (c >> 3)) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// A tile of 16 rows as two groups of eight, the dimension halves and 64 dimensions: one copy, which a lane takes half as long
// to issue as two of 64 dimensions (a warp waits for its lane: 250 cycles a tile of K and V by four copies).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int32_t group, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(bar), "l"(policy)
        : "memory");
}

// Does a word of V hold a NaN or an infinity (E4M3 has NaN alone, all ones but for the sign)?
template <typename T, bool KV8>
__device__ __forceinline__ bool no_numbers(uint32_t x) {
    if constexpr (KV8) return (__vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0;
    constexpr uint32_t exp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    return (x & exp) == exp || ((x >> 16) & exp) == exp;
}

// Two 16-bit numbers of a register as floats (a bf16 is the top half of one).
template <typename M>
__device__ __forceinline__ float2 unpacked(uint32_t x) {
    if constexpr (std::is_same<M, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// Two fp16 numbers by 2^-11.
__device__ __forceinline__ uint32_t by_2_11(uint32_t x) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x1000)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float value16(uint16_t w, __half) { return __half2float(__ushort_as_half(w)); }
__device__ __forceinline__ float value16(uint16_t w, __nv_bfloat16) { return __bfloat162float(__ushort_as_bfloat16(w)); }

}  // namespace

template <typename T, int D, int NT, bool KV8>
__global__ void __launch_bounds__(ATT_THREADS, att_ctas(KV8, NT))
    selected_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                    const SelectedParams p) {
    static_assert(!KV8 || D == 128, "FP8 pools are built for head_dim 128");
    using M = typename std::conditional<KV8, __half, T>::type;   // E4M3 codes are exact in fp16
    constexpr int W = ATT_WARPS, STAGES = att_stages(KV8);
    constexpr int TILE = att_tile_bytes(D, KV8), STAGE = 2 * TILE;
    constexpr int KS = D / 16, MT = D / 16, RP = NT * 8, OS = D + 4;
    constexpr float LIFT = std::is_same<M, __half>::value ? ATT_LIFT_LOG2 : 0.f;
    constexpr bool TWO = !KV8 || std::is_same<T, __half>::value;   // weights in two parts in every tile

    extern __shared__ uint8_t smem_raw[];
    const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base_u32 - smem_u32(smem_raw));
    constexpr int BODY = att_body_bytes(D, KV8, NT);
    const uint32_t bars_u32 = base_u32 + BODY;
    int *failed = reinterpret_cast<int *>(smem + att_flag_at(D, KV8, NT));
    uint2 *q_sm = reinterpret_cast<uint2 *>(smem + att_q_at(D, KV8, NT));          // [NT][KS][32]
    int2 *lists = reinterpret_cast<int2 *>(smem + att_lists_at(D, KV8, NT));       // [W][warp_tiles]: pool row, position

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, tq = lane & 3;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int unit = (int)(blockIdx.x / ranks), g = unit % p.Hkv, b = unit / p.Hkv;
    if (lane == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        for (int s = 0; s < STAGES; ++s) mbar_init(bars_u32 + (warp * STAGES + s) * 8, 1);
        fence_barrier_init();
    }
    pdl_trigger();
    pdl_wait();

    // the length, the first listed blocks and the query rows: on their way together
    int L = p.context_lens[b];
    const int all = p.budget * (p.bs / TILE_TOKENS), step = ranks * W;
    int j = -1, id = -1;
    const auto look_up = [&](int i) {                  // the listed block of tile i and its id
        j = i < all ? p.selected[(int64_t)unit * p.budget + i * TILE_TOKENS / p.bs] : -1;
        id = j >= 0 && j < p.stride ? p.block_tables[b * p.stride + j] : -1;
    };
    look_up(rank * W + warp + lane * step);

    // ---- query rows as the B operand. FP8 pools: a lane's four codes are consecutive dimensions, the contraction's order
    // is theirs, and a bf16 row is taken into fp16's range by a power of two that its scores get back.
    uint32_t qf[NT][KS][2];
    float qscale[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + gq;
        qscale[nt][0] = qscale[nt][1] = p.scale_log2;
        if (r < p.rows) {
            const int qi = r / p.G, hh = r - qi * p.G;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(
                static_cast<const T *>(p.q) + (((int64_t)b * p.q_len + qi) * p.Hq + g * p.G + hh) * D);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qf[nt][ks][0] = q[ks * 8 + (KV8 ? 2 * tq : tq)];
                qf[nt][ks][1] = q[ks * 8 + (KV8 ? 2 * tq + 1 : 4 + tq)];
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[nt][ks][0] = qf[nt][ks][1] = 0u;
        }
    }
    if (L < 0 || L > p.max_len || (L > 0 && L < p.q_len)) {
        if (tid == 0 && rank == 0) set_status(p.status, STATUS_BOUNDS);
        L = L < 0 ? 0 : min(L, p.max_len);
    }

    // ---- this warp's tiles: those of the listed blocks that hold tokens
    int2 *list = lists + warp * p.warp_tiles;
    int tiles = 0;
    {
        const int blocks = (L + p.bs - 1) / p.bs;
        for (int i0 = rank * W + warp; i0 < all; i0 += 32 * step) {
            const int i = i0 + lane * step, off = i * TILE_TOKENS % p.bs;
            if (i0 >= 32 * step) look_up(i);
            int row = 0, pos = -1;
            if (j >= blocks) set_status(p.status, STATUS_BOUNDS);
            else if (j >= 0 && j * p.bs + off < L) {
                if (id < 0 || id >= p.num_blocks) set_status(p.status, STATUS_BOUNDS);
                else row = (id * p.Hkv + g) * p.bs + off, pos = j * p.bs + off;
            }
            const uint32_t have = __ballot_sync(0xffffffffu, pos >= 0);
            if (pos >= 0) list[tiles + __popc(have & ((1u << lane) - 1u))] = make_int2(row, pos);
            tiles += __popc(have);
        }
    }
    __syncwarp();

    const uint32_t ring_u32 = base_u32 + warp * STAGES * STAGE;
    const uint64_t policy = l2_policy_evict_first();
    int base = 0;                                      // copies before those of this look at the tiles: 0 in the first look
    auto issue = [&](int it) {
        const int s = (base + it) % STAGES, row = list[it].x;
        const uint32_t bar = bars_u32 + (warp * STAGES + s) * 8, dst = ring_u32 + s * STAGE;
        mbar_arrive_expect_tx(bar, STAGE);
        if constexpr (KV8) {
            tma_load_2d(dst, &tmk, 0, row, bar, policy);
            tma_load_2d(dst + TILE, &tmv, 0, row, bar, policy);
        } else {
            tma_load_4d(dst, &tmk, row / 8, bar, policy);
            tma_load_4d(dst + TILE, &tmv, row / 8, bar, policy);
        }
    };
    int issued = min(tiles, STAGES);
    if (lane == 0)
        for (int it = 0; it < issued; ++it) issue(it);

    if constexpr (KV8 && std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t top = 0;                          // bf16 without its sign, as an integer: the exponent on top
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t x = qf[nt][ks][e];
                    top = max(top, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // times 2^(141 - e): the largest magnitude between 2^14 and 2^15, so that small ones keep their bits too
            const int e = min(max((int)(top >> 7), 15), 254);
            const float down = __uint_as_float((uint32_t)(127 + 141 - e) << 23), up = __uint_as_float((uint32_t)(127 + e - 141) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qf[nt][ks][k]));
                    qf[nt][ks][k] = pack2<__half>(f.x * down, f.y * down);
                }
#pragma unroll
            for (int j = 0; j < 2; ++j) qscale[nt][j] *= __shfl_sync(0xffffffffu, up, (2 * tq + j) * 4);
        }
    }

    if constexpr (att_q_shared(NT)) {                  // every warp holds the same: one of them lays them down
        if (warp == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) q_sm[(nt * KS + ks) * 32 + lane] = make_uint2(qf[nt][ks][0], qf[nt][ks][1]);
        }
        __syncthreads();
    }
    const auto q_of = [&](int nt, int ks) {
        return att_q_shared(NT) ? q_sm[(nt * KS + ks) * 32 + lane] : make_uint2(qf[nt][ks][0], qf[nt][ks][1]);
    };

    int last[NT][2];                                   // positions of the columns' rows: the newest token that they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) last[nt][j] = L - p.q_len + min((nt * 8 + 2 * tq + j) / p.G, p.q_len - 1);
    const int seen_by_all = L - p.q_len + 1;           // tokens before this one

    float m[NT][2], l[NT][2], o[MT][NT][4];
    int vexp, vmost;                                   // FP8: O is in units of 2^vexp, at most 2^vmost
    uint32_t vlow;                                     // the smallest V scale in the unit's room, as bits; the sign's: no unit yet
    // FP8: a tile's scales are loaded while the tile before it is worked on
    const auto scales_of = [&](int i) {
        const int row = list[i].x + gq;
        return make_float4(p.k_scales[row], p.k_scales[row + 8], p.v_scales[row], p.v_scales[row + 8]);
    };
    float4 ahead = make_float4(0.f, 0.f, 0.f, 0.f);
    // A second look at the tiles where the first leaves an O that is no number. Infinities among V may have done it, whose
    // products with two parts of a weight (the second 0 or of either sign) need not be theirs with the weight: this time the
    // tokens that hold no numbers are added apart, in fp32. Looking for them in every tile would cost each call what this costs
    // none but those.
    bool ok = true;
    int it;
again:
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = -0.f;
#pragma unroll
        for (int md = 0; md < MT; ++md) o[md][nt][0] = o[md][nt][1] = o[md][nt][2] = o[md][nt][3] = 0.f;
    }
    vexp = 0, vmost = ATT_MIN_UNIT;
    vlow = 0x80000000u;
    if (KV8 && tiles > 0) ahead = scales_of(0);
    for (it = 0; it < tiles; ++it) {
        const int s = (base + it) % STAGES;
        // false: the copy did not land in time. A lane may see it land as another gives up, so the warp leaves by a vote (below).
        const bool landed = mbar_wait_bounded(bars_u32 + (warp * STAGES + s) * 8, (uint32_t)((base + it) / STAGES) & 1u, p.wait_ns);
        const int pos = list[it].y;
        const uint32_t kb = ring_u32 + s * STAGE, vb = kb + TILE;
        float4 scale = make_float4(1.f, 1.f, 1.f, 1.f);   // FP8: of K and V of the tokens gq and gq + 8
        if constexpr (KV8) {
            scale = ahead;
            if (it + 1 < tiles) ahead = scales_of(it + 1);
        }

        // S^T = K Q^T: 16 keys, 8 NT query rows
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
        if constexpr (KV8) {
#pragma unroll
            for (int kp = 0; kp < KS / 2; ++kp) {
                const int chunk = kp * 2 + (lane >> 4);
                uint32_t r0, r1, r2, r3;
                ldsm_x4(kb + tile_at<D, KV8>(krow, chunk), r0, r1, r2, r3);
                const uint32_t a0 = e4m3x2_to_f16x2((uint16_t)r0), a2 = e4m3x2_to_f16x2((uint16_t)(r0 >> 16));
                const uint32_t a1 = e4m3x2_to_f16x2((uint16_t)r1), a3 = e4m3x2_to_f16x2((uint16_t)(r1 >> 16));
                const uint32_t c0 = e4m3x2_to_f16x2((uint16_t)r2), c2 = e4m3x2_to_f16x2((uint16_t)(r2 >> 16));
                const uint32_t c1 = e4m3x2_to_f16x2((uint16_t)r3), c3 = e4m3x2_to_f16x2((uint16_t)(r3 >> 16));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 q0 = q_of(nt, 2 * kp), q1 = q_of(nt, 2 * kp + 1);
                    mma_16816<M>(sc[nt], a0, a1, a2, a3, q0.x, q0.y);
                    mma_16816<M>(sc[nt], c0, c1, c2, c3, q1.x, q1.y);
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int chunk = ks * 2 + (lane >> 4);
                uint32_t a0, a1, a2, a3;
                ldsm_x4(kb + tile_at<D, KV8>(krow, chunk), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 qv = q_of(nt, ks);
                    mma_16816<M>(sc[nt], a0, a1, a2, a3, qv.x, qv.y);
                }
            }
        }

        // softmax, in powers of two: weights are relative to a reference that moves only when it is passed by 2^8, which the
        // warp asks for all its columns (and the V scales) at once; the columns' maxima are looked for only then
        const int t0 = pos + gq, t1 = t0 + 8;
        const int whole = seen_by_all - pos;           // tokens of the tile that every row sees
        // FP8: does one of their V scales lie outside of the unit's room? Their order is that of their bits.
        constexpr uint32_t ROOM = (uint32_t)(TWO ? ATT_ROOM_TWO : ATT_ROOM_ONE) << 23;
        uint32_t v0 = __float_as_uint(scale.z) & 0x7FFFFFFFu, v1 = __float_as_uint(scale.w) & 0x7FFFFFFFu;
        if (whole < TILE_TOKENS) v0 = gq < whole ? v0 : vlow, v1 = gq + 8 < whole ? v1 : vlow;
        const bool outside = KV8 && max(v0 - vlow, v1 - vlow) >= ROOM && whole > 0;
        uint32_t apart = 0;                            // tokens to be added apart
        bool rest = TWO;                               // a second part of the weights
        bool passed = outside || !landed;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sc[nt][j] *= scale.x * qscale[nt][j];
                sc[nt][2 + j] *= scale.y * qscale[nt][j];
            }
        if (whole < TILE_TOKENS) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // what a masked place holds (a score, a scale) is selected away, not multiplied
                    sc[nt][j] = t0 <= last[nt][j] ? sc[nt][j] : -INFINITY;
                    sc[nt][2 + j] = t1 <= last[nt][j] ? sc[nt][2 + j] : -INFINITY;
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) passed |= fmaxf(sc[nt][j], sc[nt][2 + j]) > m[nt][j] + ATT_RESCALE_LOG2;
        if (__any_sync(0xffffffffu, passed)) {
            if (__any_sync(0xffffffffu, !landed)) {
                ok = false;
                break;
            }
            if (__any_sync(0xffffffffu, outside)) {
                v0 = gq < whole && v0 < 0x7F800000u ? v0 : 0u, v1 = gq + 8 < whole && v1 < 0x7F800000u ? v1 : 0u;
                const uint32_t top = __reduce_max_sync(0xffffffffu, max(v0, v1));
                int e = min(max((int)(top >> 23) - 126 + ATT_ROOM_ABOVE, ATT_MIN_UNIT), ATT_MAX_UNIT);
                e = max(e, vmost - ATT_UNIT_SPAN);
                if (top && (e < vexp || top - vlow >= ROOM)) {
                    const float f = ldexpf(1.f, vexp - e);
#pragma unroll
                    for (int md = 0; md < MT; ++md)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[md][nt][k] *= f;
                    vexp = e, vmost = max(vmost, e);
                    vlow = ((uint32_t)(127 + e) << 23) - ROOM;
                }
                // a scale of 0 has nothing to lose
                const uint32_t two = vlow + ROOM - ((uint32_t)ATT_ROOM_ONE << 23), none = vlow + ROOM - ((uint32_t)ATT_ROOM_TWO << 23);
                rest = TWO || __any_sync(0xffffffffu, v0 - 1 < two - 1 || v1 - 1 < two - 1);
                apart = __reduce_or_sync(0xffffffffu, (uint32_t)(v0 - 1 < none - 1) << gq | (uint32_t)(v1 - 1 < none - 1) << (gq + 8));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(sc[nt][j], sc[nt][2 + j]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    if (mx > m[nt][j] + ATT_RESCALE_LOG2) {   // also the first finite one (m = -inf)
                        const float alpha = ex2_approx(m[nt][j] - mx);
                        m[nt][j] = mx;
                        l[nt][j] *= alpha;
#pragma unroll
                        for (int md = 0; md < MT; ++md) o[md][nt][j] *= alpha, o[md][nt][2 + j] *= alpha;
                    }
                }
        }
        const float unit_v = KV8 ? __uint_as_float((uint32_t)(127 - vexp) << 23) : 1.f;   // 2^-vexp
        const float vs0 = scale.z * unit_v, vs1 = scale.w * unit_v;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float ref = (m[nt][j] == -INFINITY ? 0.f : m[nt][j]) - LIFT;
                // -0 for what is not seen: a sum of nothing keeps its sign, one of weights that are all 0 loses it
                float p0 = ex2_approx(sc[nt][j] - ref), p1 = ex2_approx(sc[nt][2 + j] - ref);
                if (whole < TILE_TOKENS) p0 = t0 <= last[nt][j] ? p0 : -0.f, p1 = t1 <= last[nt][j] ? p1 : -0.f;
                l[nt][j] = __fadd_rn(__fadd_rn(l[nt][j], p0), p1);
                sc[nt][j] = p0 * vs0;
                sc[nt][2 + j] = p1 * vs1;
            }

        // The tiles at the end of the context. What lies behind it may be anything: its words of V become 0, its weights are
        // 0 already. So may the value of a token that not every row sees be to the rows that do not: where it is no number
        // (or, FP8, has a scale outside of the unit's room), the token is added in fp32 to the rows that see it, and its weights
        // and words become 0 as well. On the second look that goes for every token.
        if (whole < TILE_TOKENS || base > 0 || apart) {
            const int w0 = whole < 0 || base > 0 ? 0 : whole, w1 = min(TILE_TOKENS, L - pos), some = w1 - w0;
            uint8_t *vs = smem + (vb - base_u32);
            uint32_t odd = apart;                      // such tokens
            for (int c = lane; c < some * (TILE / TILE_TOKENS / 16); c += 32) {
                const int row = w0 + c % some, chunk = c / some;
                const uint4 x = *reinterpret_cast<const uint4 *>(vs + tile_at<D, KV8>(row, chunk));
                const bool is = no_numbers<T, KV8>(x.x) || no_numbers<T, KV8>(x.y) || no_numbers<T, KV8>(x.z) || no_numbers<T, KV8>(x.w);
                odd |= (uint32_t)is << row;
            }
            if constexpr (KV8) {
                if (gq >= w0 && gq < w1) odd |= (uint32_t)((__float_as_uint(scale.z) & 0x7FFFFFFFu) - vlow >= ROOM) << gq;
                if (gq + 8 >= w0 && gq + 8 < w1) odd |= (uint32_t)((__float_as_uint(scale.w) & 0x7FFFFFFFu) - vlow >= ROOM) << (gq + 8);
            }
            odd = __reduce_or_sync(0xffffffffu, odd);
            for (uint32_t left = odd; left; left &= left - 1) {
                const int kk = __ffs(left) - 1, src = (kk & 7) * 4 + tq;   // the lane with this token's weights of the same columns
                float pv[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x = __shfl_sync(0xffffffffu, sc[nt][j], src), y = __shfl_sync(0xffffffffu, sc[nt][2 + j], src);
                        pv[nt][j] = kk < 8 ? x : y;
                    }
#pragma unroll
                for (int md = 0; md < MT; ++md)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v;
                        if constexpr (KV8) {
                            const int dim = md * 16 + 2 * gq + e;
                            const uint32_t h2 = e4m3x2_to_f16x2(vs[tile_at<D, KV8>(kk, dim >> 4) + (dim & 15)]);
                            v = __half2float(__ushort_as_half((uint16_t)(h2 & 0xFFFFu)));
                        } else {
                            const int dim = md * 16 + gq + 8 * e;
                            v = value16(*reinterpret_cast<const uint16_t *>(vs + tile_at<D, KV8>(kk, dim >> 3) + (dim & 7) * 2), T());
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (pos + kk <= last[nt][j]) o[md][nt][2 * e + j] += pv[nt][j] * v;
                    }
            }
            __syncwarp();
            const uint32_t gone = odd | (w1 < TILE_TOKENS ? 0xFFFFu << w1 : 0u);
            for (int c = lane; c < TILE / 16; c += 32) {
                const int row = c % TILE_TOKENS;
                if (gone >> row & 1u)
                    *reinterpret_cast<uint4 *>(vs + tile_at<D, KV8>(row, c / TILE_TOKENS)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();                  // before the copy that comes over these words
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (gone >> gq & 1u) sc[nt][j] = 0.f;
                    if (gone >> (gq + 8) & 1u) sc[nt][2 + j] = 0.f;
                }
        }

        // O^T += V^T P^T with P^T as the B operand, in V's type, as two parts: the nearest number and what is left of it. bf16's eight
        // bits would not do, and fp16's eleven alone made the error of fp16 outputs 1.3 to 1.4 times the last rounding's (16-bit
        // pools, 64 sequences of 2048 tokens: 84.5 -> 85.8 us for the second part; FP8, 8, 16, 32 rows: 44.2, 59.6, 86.4 -> 46.8,
        // 70.6, 100.5 us). The bf16 outputs of FP8 pools keep eight bits, 2^-8 beside the weights' 2^-11: one part, but in tiles
        // whose V scales lie far apart. FP8 pools take the second part 2^11 times as large, against V by 2^-11 (exact: codes are
        // multiples of 2^-9), so that it keeps its bits where the weight itself is near the end of fp16's range.
        // parts: 1 the nearest numbers, 2 what is left of the weights, 3 both
        const auto product = [&](auto parts) {
            constexpr bool NEAR = decltype(parts)::value & 1, REST = decltype(parts)::value & 2;
            constexpr float LARGER = KV8 ? 2048.f : 1.f;
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float x = sc[nt][2 * k], y = sc[nt][2 * k + 1];
                    const uint32_t hi = pack2<M>(x, y);
                    ph[nt][k] = NEAR ? movmatrix_trans(hi) : 0u;
                    const float2 near = unpacked<M>(hi);
                    pl[nt][k] = REST ? movmatrix_trans(pack2<M>((x - near.x) * LARGER, (y - near.y) * LARGER)) : 0u;
                }
            if constexpr (KV8) {
                // a lane gets two keys of two neighbouring dimensions: the even ones are rows 0-7 of the fragment, the odd 8-15
                const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int mp = 0; mp < MT / 2; ++mp) {
                    const int chunk = mp * 2 + (lane >> 4);
                    uint32_t r[4];
                    ldsm_x4_trans(vb + tile_at<D, KV8>(vrow, chunk), r[0], r[1], r[2], r[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t lo = r[2 * h], hi = r[2 * h + 1];
                        const uint32_t a0 = e4m3x2_to_f16x2((uint16_t)__byte_perm(lo, 0u, 0x4420));
                        const uint32_t a1 = e4m3x2_to_f16x2((uint16_t)__byte_perm(lo, 0u, 0x4431));
                        const uint32_t a2 = e4m3x2_to_f16x2((uint16_t)__byte_perm(hi, 0u, 0x4420));
                        const uint32_t a3 = e4m3x2_to_f16x2((uint16_t)__byte_perm(hi, 0u, 0x4431));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            if constexpr (NEAR) mma_16816<M>(o[2 * mp + h][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                        if constexpr (REST) {
                            const uint32_t b0 = by_2_11(a0), b1 = by_2_11(a1), b2 = by_2_11(a2), b3 = by_2_11(a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_16816<M>(o[2 * mp + h][nt], b0, b1, b2, b3, pl[nt][0], pl[nt][1]);
                        }
                    }
                }
            } else {
                const int vrow = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int md = 0; md < MT; ++md) {
                    const int chunk = md * 2 + ((lane >> 3) & 1);
                    uint32_t a0, a1, a2, a3;
                    ldsm_x4_trans(vb + tile_at<D, KV8>(vrow, chunk), a0, a1, a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_16816<M>(o[md][nt], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                        if constexpr (REST) mma_16816<M>(o[md][nt], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                    }
                }
            }
        };
        if constexpr (TWO) {
            product(std::integral_constant<int, 3>());
        } else {
            if (rest) product(std::integral_constant<int, 2>());
            product(std::integral_constant<int, 1>());
        }
        __syncwarp();
        if (it + STAGES < tiles) {
            if (lane == 0) issue(it + STAGES);
            ++issued;
        }
    }
    if (ok && base == 0) {
        float odd = 0.f;
#pragma unroll
        for (int md = 0; md < MT; ++md)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) odd = fmaf(o[md][nt][k], 0.f, odd);
        if (__any_sync(0xffffffffu, odd != 0.f)) {
            base = tiles;
            issued = min(tiles, STAGES);
            __syncwarp();
            if (lane == 0)
                for (int k = 0; k < issued; ++k) issue(k);
            goto again;
        }
    }
    if (!ok && lane == 0)                              // no copy lands behind the end of the pipeline
        for (int k = it; k < issued; ++k)
            mbar_wait_bounded(bars_u32 + (warp * STAGES + (base + k) % STAGES) * 8, (uint32_t)((base + k) / STAGES) & 1u, p.wait_ns);

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
        }
    const int lost = __syncthreads_or(!ok);            // the ring is free now
    if (tid == 0) {
        *failed = lost;
        if (lost) set_status(p.status, STATUS_TIMEOUT);
    }

    // ---- the warps' states
    const float unit_o = __uint_as_float((uint32_t)(127 + vexp) << 23);   // 2^vexp
    float *ow = reinterpret_cast<float *>(smem);       // [W][RP][OS]
    float *oc = ow + W * RP * OS;                      // [RP][OS]
    float2 *mw = reinterpret_cast<float2 *>(oc + RP * OS);   // [W][RP] (maximum, sum)
    float2 *mc = mw + W * RP;                          // [RP]
    float *fw = reinterpret_cast<float *>(mc + RP);    // [RP][W] factors
#pragma unroll
    for (int md = 0; md < MT; ++md)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dim = md * 16 + (KV8 ? 2 * gq + (e >> 1) : gq + (e >> 1) * 8);
                ow[(warp * RP + nt * 8 + 2 * tq + (e & 1)) * OS + dim] = KV8 ? o[md][nt][e] * unit_o : o[md][nt][e];
            }
    if (gq == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) mw[warp * RP + nt * 8 + 2 * tq + j] = make_float2(m[nt][j], l[nt][j]);
    }
    __syncthreads();
    for (int r = tid; r < p.rows; r += ATT_THREADS) {
        float top = -INFINITY, sum = -0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, mw[w * RP + r].x);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = exp2f(mw[w * RP + r].x - ref);
            fw[r * W + w] = f;
            sum = __fadd_rn(sum, __fmul_rn(f, mw[w * RP + r].y));
        }
        mc[r] = make_float2(top, sum);
    }
    __syncthreads();
    constexpr int D8 = D / 8;
    const auto store = [&](int r, int d0, const float (&a)[8], float sum) {
        const int qi = r / p.G, h = g * p.G + (r - qi * p.G);
        const float inv = __float_as_uint(sum) == 0x80000000u ? 0.f : 1.f / sum;   // a row that sees nothing: zeros
        uint4 v;
        v.x = pack2<T>(a[0] * inv, a[1] * inv);
        v.y = pack2<T>(a[2] * inv, a[3] * inv);
        v.z = pack2<T>(a[4] * inv, a[5] * inv);
        v.w = pack2<T>(a[6] * inv, a[7] * inv);
        *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (((int64_t)b * p.q_len + qi) * p.Hq + h) * D + d0) = v;
    };
    for (int idx = tid; idx < p.rows * D8; idx += ATT_THREADS) {
        const int r = idx / D8, d0 = (idx - r * D8) * 8;
        float a[8] = {};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = fw[r * W + w];
            const float4 x = *reinterpret_cast<const float4 *>(ow + (w * RP + r) * OS + d0);
            const float4 y = *reinterpret_cast<const float4 *>(ow + (w * RP + r) * OS + d0 + 4);
            a[0] += f * x.x, a[1] += f * x.y, a[2] += f * x.z, a[3] += f * x.w;
            a[4] += f * y.x, a[5] += f * y.y, a[6] += f * y.z, a[7] += f * y.w;
        }
        if (ranks == 1) {
            if (!lost) store(r, d0, a, mc[r].y);
        } else {
            float4 *dst = reinterpret_cast<float4 *>(oc + r * OS + d0);
            dst[0] = make_float4(a[0], a[1], a[2], a[3]);
            dst[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
    }
    if (ranks == 1) return;

    // ---- the CTAs' states, each CTA a share of the outputs
    cluster_sync();
    // every CTA's words on their way before the first is used
    const uint32_t at_failed = smem_u32(failed), at_mc = smem_u32(mc), at_oc = smem_u32(oc);
    const bool any_failed = __any_sync(0xffffffffu, lane < ranks && ld_cluster_int(map_rank(at_failed, lane < ranks ? lane : 0)));
    if (!any_failed) {
        for (int idx = rank * ATT_THREADS + tid; idx < p.rows * D8; idx += ranks * ATT_THREADS) {
            const int r = idx / D8, d0 = (idx - r * D8) * 8;
            float2 ms[ATT_MAX_RANKS];
            float4 x[ATT_MAX_RANKS], y[ATT_MAX_RANKS];
#pragma unroll
            for (int c = 0; c < ATT_MAX_RANKS; ++c) {
                ms[c] = make_float2(-INFINITY, -0.f);
                x[c] = y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < ranks) {
                    ms[c] = ld_cluster_float2(map_rank(at_mc + r * 8, c));
                    x[c] = ld_cluster_float4(map_rank(at_oc + (r * OS + d0) * 4, c));
                    y[c] = ld_cluster_float4(map_rank(at_oc + (r * OS + d0 + 4) * 4, c));
                }
            }
            float top = -INFINITY, sum = -0.f, a[8] = {};
#pragma unroll
            for (int c = 0; c < ATT_MAX_RANKS; ++c) top = fmaxf(top, ms[c].x);
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int c = 0; c < ATT_MAX_RANKS; ++c) {
                const float f = exp2f(ms[c].x - ref);
                sum = __fadd_rn(sum, __fmul_rn(f, ms[c].y));
                a[0] += f * x[c].x, a[1] += f * x[c].y, a[2] += f * x[c].z, a[3] += f * x[c].w;
                a[4] += f * y[c].x, a[5] += f * y[c].y, a[6] += f * y[c].z, a[7] += f * y[c].w;
            }
            store(r, d0, a, sum);
        }
    }
    cluster_sync();                                    // nobody reads this CTA's memory any more
}

template <typename T, int D, bool KV8>
static cudaError_t launch_selected_t(SelectedParams p, const CUtensorMap &tmk, const CUtensorMap &tmv, int sm_count,
                                     cudaStream_t stream) {
    const int64_t units = (int64_t)p.num_seqs * p.Hkv;
    const int tiles = p.budget * (p.bs / TILE_TOKENS), nt = (p.rows + 7) / 8;
    // CTAs of a cluster. A round of resident CTAs lasts as long as a warp's tiles and about three more for the start and the
    // joining of its warps, another three where a cluster joins. Of 130 shapes (1 to 2048 units, lists of 16 to 1024 blocks,
    // 4 to 32 rows, both formats) this picks the best of 1, 2, 4, 8 but for 0.8% on average, 20% at most; "at least two CTAs
    // per SM" lost 8.5% and up to 83% (128 units, 16 blocks: 6.1 us as single CTAs, 11.0 as clusters of four).
    const int64_t slots = (int64_t)att_ctas(KV8, nt) * sm_count;
    int ranks = 1;
    int64_t best = 0;
    for (int r = 1; r <= ATT_MAX_RANKS; r *= 2) {
        const int64_t cost = (units * r + slots - 1) / slots * ((r > 1 ? 6 : 3) + (tiles + r * ATT_WARPS - 1) / (r * ATT_WARPS));
        if (r == 1 || cost < best) best = cost, ranks = r;
    }
    while (tiles > ranks * ATT_WARPS * ATT_WARP_TILES) ranks *= 2;
    p.warp_tiles = (tiles + ranks * ATT_WARPS - 1) / (ranks * ATT_WARPS);
    const auto launch = [&](auto kernel, int n) {
        static_assert(att_smem(D, KV8, 4, ATT_WARP_TILES) <= MAX_SMEM_PER_CTA, "the most tiles of four warps");
        const size_t smem = att_smem(D, KV8, n, p.warp_tiles);
        // the most that any call takes: the attribute is the kernel's, and other threads' calls set it too
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)att_smem(D, KV8, n, ATT_WARP_TILES));
        return e != cudaSuccess
                   ? e
                   : launch_clusters(kernel, (unsigned)(units * ranks), ATT_THREADS, smem, ranks, stream, tmk, tmv, p);
    };
    switch (nt) {
        case 1: return launch(selected_kernel<T, D, 1, KV8>, 1);
        case 2: return launch(selected_kernel<T, D, 2, KV8>, 2);
        case 3: return launch(selected_kernel<T, D, 3, KV8>, 3);
        default: return launch(selected_kernel<T, D, 4, KV8>, 4);
    }
}

cudaError_t launch_selected(SelectedParams p, int dtype, int head_dim, const CUtensorMap &tmk, const CUtensorMap &tmv,
                            int sm_count, cudaStream_t stream) {
    if (p.k_scales)
        return dtype == PA_FP16 ? launch_selected_t<__half, 128, true>(p, tmk, tmv, sm_count, stream)
                                : launch_selected_t<__nv_bfloat16, 128, true>(p, tmk, tmv, sm_count, stream);
    if (dtype == PA_FP16)
        return head_dim == 128 ? launch_selected_t<__half, 128, false>(p, tmk, tmv, sm_count, stream)
                               : launch_selected_t<__half, 64, false>(p, tmk, tmv, sm_count, stream);
    return head_dim == 128 ? launch_selected_t<__nv_bfloat16, 128, false>(p, tmk, tmv, sm_count, stream)
                           : launch_selected_t<__nv_bfloat16, 64, false>(p, tmk, tmv, sm_count, stream);
}

}  // namespace pa
