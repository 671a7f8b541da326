// prompt.cu -- causal attention of packed prompts of different lengths through the block tables, on the
// 5th-generation tensor cores (tcgen05.mma, accumulators in tensor memory).
//
// Sequence b's new tokens are rows cu_q[b] .. cu_q[b+1] of q; row i of them sits at position
// p = context_lens[b] - n_b + i and attends to tokens 0..p:
//   out = sum_t softmax_t(scale q . K_t) V_t,
// one pass over the keys with the running maximum and sum of the softmax.
//
// Work. A query "row" is one (position, query head of the KV group) pair. A row tile holds the rows of
// P = 128 / G positions (G query heads per KV head), position-major, so that all heads of a group share
// one read of K and V; an item is two row tiles of one sequence and KV head. Items behind long contexts are cut
// along the keys into units where all items together are too few to fill the GPU (elsewhere a long context is not
// cut, however short the others are), and a second kernel joins the units' (O, max, sum). The lengths live on the
// device, so every block of the persistent grid computes the same plan from them (items by falling length, cut
// length) and takes every gridDim.x-th unit, the direction alternating from round to round so that falling lengths
// even out. A captured call follows lengths that change between replays.
//
// One block per SM, 384 threads:
//   warps 0-3, 4-7   softmax of row tile 0 and 1: one row per thread = one tensor-memory lane
//   warp 8, 11       K and V loads: one TMA copy per cache block, [8-key groups][64-dimension halves]
//                    [8 keys][128 bytes] in shared memory, so that a whole block of tokens is one copy and
//                    8-key groups stay a constant stride apart in the matrix descriptors
//   warp 9           one lane issues every MMA: per key tile and row tile O += P V (P from tensor
//                    memory, V MN-major), then S = Q K^T into the columns P came from, the row tiles in turn
//                    so that one's products run while the other's softmax does
//   warp 10          decodes units into a ring that all roles read, and loads their Q tiles (a TMA box of
//                    [P positions][G heads][64 dimensions])
// The MMA thread bounds a step: of about 3200 cycles (2048 of products), every wait and every commit it issues
// costs it 100 to 170, while the softmax is done 1000 cycles before its weights are asked for. So it waits for K
// and the weights alone: one thread of each row tile's softmax waits for V before it hands the weights over, and
// tells the loaders when a K tile (and the V tile before it) has been read. Measured: 4 x 4096 tokens, 64 / 8 heads
// of 128, bf16: 780 us, 1410 TFLOP/s (0.74 of cuBLAS; calls on end, at the power limit, 830 us, 1325 TFLOP/s, 0.77
// of what cuBLAS sustains), against 1003 us with the waits, divisions and descriptors in one thread of that warp.
// Not kept: an MMA warp per row tile, in turns or not (820, 940 us: their products interleave, or each turn costs
// two waits), two softmax threads per row (936 us and more), weights handed over in halves (840 us), barriers asked
// ahead of need (805 us), the whole warp on its way with one lane issuing (790 us with the lanes agreeing on every
// wait, which they must).
// 32 prompts of 1 to 2000 tokens, 32 / 8 heads: 108 us (46 at the product's rate), of which the prologue and plan
// take 5 and each of the up to 9 units per block about 3 at its end (masked tile, last product, stores). Heads of
// 64: 65 us; a step takes 2800 cycles with nothing at its limit (tensor pipe 18%, exponentials 22%, issue 34%): S,
// the softmax and P are a chain, as each row tile has one buffer for S and P. 30 rows behind 78000 cached tokens:
// 70 us, 4.6 TB/s; its key loop runs at 0.94 of the DRAM rate.
// The roles run across unit borders: the next unit's Q, K and V are on their way, and its first S may be
// issued, while the last softmax and the output of this one are still at work.
//
// Masks. Keys behind a row's position are excluded from its maximum and sum by selection, whatever the
// scores are. Their weight is 0 in P V, but 0 times a value that is no number is none either: V rows behind
// the unit's last position are zeroed, and the V tiles in which only some rows see a key are scanned; where
// one holds a NaN or infinity, those words are zeroed and the rows that do see them get them added to their
// outputs (each seen value has a weight > 0) in a slow path that real data never takes. The softmax threads do
// this, between their weights and the product: they have the time.
//
// Roundings. S, the softmax statistics and O are fp32. P is rounded once to the model's 16-bit type, as the
// product with V takes it (half a step per weight, averaged over the keys: of the size of the output's own
// rounding); the sum is of the unrounded weights. Keeping P in two 16-bit parts, as pa_prefill does for
// bf16, costs half of the P V rate.
#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_serving.h"

namespace pa {

constexpr int PR_BM = 128, PR_BN = 128;               // rows of a row tile, keys of a key tile
constexpr int PR_THREADS = 384;
constexpr int PR_K_WARP = 8, PR_SCHED_WARP = 10, PR_V_WARP = 11;    // warp 9: MMA
// Register split: 2 x 128 x 216 + 128 x 72 = 384 x 168, the launch's registers.
constexpr uint32_t PR_REGS_LAUNCH = 168, PR_REGS_SOFTMAX = 216, PR_REGS_OTHER = 72;
static_assert(2 * 128 * PR_REGS_SOFTMAX + 128 * PR_REGS_OTHER <= PR_THREADS * PR_REGS_LAUNCH, "register split");
constexpr int PR_UNITS = 4;                           // ring of decoded units
constexpr float PR_RESCALE_LOG2 = 8.f;                // stale-maximum headroom (P <= 2^8)
constexpr uint32_t PR_TMEM_COLS = 512;                // row tile t: S/P at 256 t, O at 256 t + 128

template <int D>
struct PromptShape {
    static constexpr int HALVES = D / 64;
    static constexpr int Q_BYTES = PR_BM * D * 2;     // HALVES x [128 rows x 128 B]
    static constexpr int KV_BYTES = PR_BN * D * 2;    // 16 groups x HALVES x [8 keys x 128 B]
    static constexpr int GROUP_BYTES = 1024 * HALVES;
    static constexpr int KST = D == 128 ? 2 : 4, VST = KST;
    static constexpr int OFF_K = 2 * Q_BYTES;
    static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
    static constexpr int OFF_STAGE = OFF_V + VST * KV_BYTES;          // 2 KB per softmax warp
    static constexpr int OFF_PREF = OFF_STAGE + 8 * 2048;
    static constexpr int OFF_KEYS = OFF_PREF + (PA_PACKED_MAX_SEQS + 4) * 4;
    static constexpr int OFF_UNITS = OFF_KEYS + 2 * 512 * 4;          // sort keys: 4 KB
    static constexpr int OFF_BAR = OFF_UNITS + PR_UNITS * 64;
    static constexpr int NBAR = 2 * KST + VST + 12 + 2 * PR_UNITS + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = 1024 + OFF_MISC + 32;
    static_assert(SMEM <= (int)MAX_SMEM_PER_CTA, "shared memory");
};

struct alignas(16) PromptUnit {
    int valid;                 // 0: no more units
    int b, g;
    int tok0;                  // row of q of the item's first position
    int npos;                  // the sequence's positions from there on
    int pos0;                  // that position
    int kt0;                   // first key tile
    int n0, n1;                // key tiles of row tile 0 and 1
    int slot;                  // where the unit's state goes; -1: the output itself
    int poison;                // V tiles of the unit held values that are no numbers
    int fold;                  // state slot that long sums are kept in meanwhile
    int pad[4];
};
static_assert(sizeof(PromptUnit) == 64, "unit ring");

// An item as the joining kernel needs it, written by the main kernel in the plan's order.
struct PromptItem {
    int tok0, npos;
    int first;                 // its first unit (of KV head 0)
    int splits0, splits1;      // units of row tile 0 and 1 (0: nothing to join)
};
static_assert(sizeof(PromptItem) <= PROMPT_ITEM_BYTES, "workspace items");

size_t prompt_slot_bytes(int head_dim) { return (size_t)256 * (head_dim + 2) * 4; }

// Sums over long contexts. An MMA aligns each product to the accumulator it is added to and drops what is below about
// 2^-26 of that, so a sum of N like terms comes out up to N 2^-26 too small (measured: N 2^-27, 2.6% at 2^22 keys). So
// where contexts may be longer, O leaves the accumulator every PROMPT_FOLD_TILES key tiles (2^14 keys: 2^-12 at most)
// for a state of the row in the workspace (as a unit's: [D / 4][256 rows] float4, then [256 rows] (max, sum)), is summed
// there in fp32 and starts anew; the row's sum of weights goes the same way. One thread per row does both, so
// nothing has to be waited for. A prompt of 32768 tokens, 32 / 8 heads of 128: 5.76 -> 5.90 ms (every 64 tiles 6.03).
constexpr int PR_FOLD = PROMPT_FOLD_TILES;
static_assert((PR_FOLD & (PR_FOLD - 1)) == 0, "a power of two");

template <int D>
struct RowState {
    float4 *o;                 // [D / 4], 256 apart
    float2 *ml;
    __device__ RowState(uint8_t *slot, int row)
        : o(reinterpret_cast<float4 *>(slot) + row), ml(reinterpret_cast<float2 *>(slot + (size_t)256 * D * 4) + row) {}
    // The weight of what is kept, relative to the maximum m; its sum is added to l.
    __device__ float weigh(float m, float &l) const {
        const float2 old = *ml;
        const float w = old.x == -INFINITY ? 0.f : ex2_approx(old.x - m);
        l += old.y * w;
        return w;
    }
};

template <typename T>
__device__ __forceinline__ uint32_t nonfinite_probe(uint32_t x, uint32_t acc) {
    // x * 0 + acc, two values at once: stays 0 while every x is finite
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
    return r;
}
template <typename T>
__device__ __forceinline__ bool is_nonfinite16(uint32_t x) {
    constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    return (x & E) == E;
}

__device__ __forceinline__ void mbar_arrive_count(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// Two fp32 operations at once (register pairs).
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// tcgen05.mma with descriptors as a constant upper word (128-byte swizzle, version, stride between 8-row groups)
// and a lower word (address / 16, leading offset / 16 << 16).
__host__ __device__ constexpr uint32_t desc_hi(int group_stride) { return (uint32_t)(group_stride >> 4) | 1u << 14 | 2u << 29; }

template <uint32_t HA, uint32_t HB>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(HA), "n"(HB));
}

// A in tensor memory.
template <uint32_t HB>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(HB));
}

template <int RANK>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar,
                                         uint64_t policy) {
    if constexpr (RANK == 3)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
            : "memory");
}

// New tokens and context of sequence b, clamped to what q and the tables hold (flagged where `status` is given).
__device__ __forceinline__ void sequence(const PromptParams &p, int b, int &first, int &n, int &L, int *status) {
    first = __ldg(p.cu_q + b);
    int end = __ldg(p.cu_q + b + 1);
    L = __ldg(p.context_lens + b);
    const bool bad = first < 0 || end < first || end > p.num_tokens || L > p.max_ctx || L < end - first;
    if (bad && status) set_status(status, STATUS_BOUNDS);
    first = first < 0 ? 0 : (first > p.num_tokens ? p.num_tokens : first);
    end = end > p.num_tokens ? p.num_tokens : end;
    n = end > first ? end - first : 0;
    L = L < 0 ? 0 : (L > p.max_ctx ? p.max_ctx : L);
}

// The plan, computed by every block alike. Up to PR_SORT items are sorted, the ones with most key tiles first, and
// cut into units of at most `chunk` key tiles. More items stay whole and in the caller's order of sequences, a sequence's
// last first: items of like lengths even out, but a long context that comes late in the batch ends late.
constexpr int PR_SORT = 512;
struct PromptPlan {
    int *pref;                 // items of the sequences before b; then, sorted: [512] items, [513] units, [512] tiles
    uint32_t *key, *pack;      // [PR_SORT] each, while sorting
    int *meta;                 // items, key tiles per unit, units (of one KV head)
    __device__ int *items() const { return pref; }                  // b << 16 | item within the sequence
    __device__ int *units() const { return pref + PR_SORT; }        // units of the items before
    __device__ int *tiles() const { return pref + 2 * PR_SORT + 4; }
};
static_assert(3 * PR_SORT + 4 <= PA_PACKED_MAX_SEQS, "the sorted plan takes the prefix's place");
constexpr int PR_WHOLE = 1 << 24;
static_assert(PA_PACKED_MAX_CONTEXT / PR_BN < PR_WHOLE && (PA_PACKED_MAX_CONTEXT / PR_BN + 1ull) * PR_SORT <= 1ull << 32,
              "an item's key tiles fit a sort key");

__device__ __forceinline__ int items_of(const PromptParams &p, int n) { return (n + 2 * p.P - 1) / (2 * p.P); }

// Key tiles of an item's row tiles, up to their last positions, and the units they are cut into.
__device__ __forceinline__ void cuts(const PromptParams &p, int pos0, int npos, int chunk, int &s0, int &s1,
                                     int *tiles0 = nullptr, int *tiles1 = nullptr) {
    const int end0 = pos0 + min(npos, p.P), end1 = npos > p.P ? pos0 + min(npos, 2 * p.P) : 0;
    const int e0 = end0 > 0 ? (end0 + PR_BN - 1) / PR_BN : 0, e1 = end1 > 0 ? (end1 + PR_BN - 1) / PR_BN : 0;
    s0 = max(1, (e0 + chunk - 1) / chunk);
    s1 = (e1 + chunk - 1) / chunk;
    if (tiles0) *tiles0 = e0, *tiles1 = e1;
}

// Costs are in key tiles of work: a unit costs PLAN_UNIT more than its tiles, joining PLAN_JOIN.
__device__ void make_plan(const PromptParams &p, const PromptPlan &pl, int tid, int lane) {
    constexpr int PLAN_UNIT = 3, PLAN_JOIN = 4, PLAN_MIN = 4;
    const int rows2 = 2 * p.P, grid = (int)gridDim.x;
    if (tid < 32) {
        int total = 0;
        // No more than non-decreasing cu_q can make: what else it holds (flagged) neither overflows the prefix nor makes
        // the sequences' work many times over.
        const int most = min(p.num_tokens, p.num_tokens / (2 * p.P) + min(p.num_tokens, p.num_seqs));
        for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
            const int b = b0 + lane;
            int first = 0, n = 0, L = 0;
            if (b < p.num_seqs) sequence(p, b, first, n, L, blockIdx.x == 0 ? p.status : nullptr);
            int x = items_of(p, n);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b < p.num_seqs) pl.pref[b + 1] = min(total + x, most);
            total = min(total + __shfl_sync(0xffffffffu, x, 31), most);
        }
        if (lane == 0) {
            pl.pref[0] = 0;
            pl.meta[0] = pl.meta[2] = total;
            pl.meta[1] = PR_WHOLE;
        }
    }
    __syncthreads();
    const int items = pl.meta[0];
    if (items > PR_SORT) return;
    for (int k = tid; k < items; k += PR_THREADS) {
        int lo = 0, hi = p.num_seqs;                  // pref[lo] <= k < pref[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pl.pref[mid] <= k) lo = mid;
            else hi = mid;
        }
        int first, n, L;
        sequence(p, lo, first, n, L, nullptr);
        const int i = k - pl.pref[lo], end = L - n + min(n, (i + 1) * rows2);
        const int e = end > PR_BN ? (end + PR_BN - 1) / PR_BN : 1;
        pl.key[k] = (uint32_t)e * PR_SORT + (PR_SORT - 1 - k);                      // all different
        pl.pack[k] = (uint32_t)lo << 16 | (uint32_t)i;
    }
    __syncthreads();
    for (int k = tid; k < items; k += PR_THREADS) {
        const uint32_t mine = pl.key[k];
        int rank = 0;
        for (int m = 0; m < items; ++m) rank += pl.key[m] > mine;
        pl.items()[rank] = (int)pl.pack[k];
        pl.tiles()[rank] = (int)(mine / PR_SORT);
    }
    __syncthreads();
    if (tid >= 32) return;
    int chunk = PR_WHOLE;
    const int *tiles = pl.tiles();
    if (p.max_units > 0 && items > 0 && (int64_t)items * p.Hkv < 2 * grid && tiles[0] > PLAN_MIN) {
        int64_t sum = 0;
        for (int k = lane; k < items; k += 32) sum += tiles[k];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum *= p.Hkv;
        // one candidate per lane, around an even share of the tiles; the last: whole items
        const int share = (int)((sum + grid - 1) / grid);
        int c = lane < 8 ? share * (lane + 2) / 10 : share + (lane - 8) * max(1, share / 12);
        c = lane == 31 ? PR_WHOLE : max(c, PLAN_MIN);
        int64_t units = 0;
        for (int k = 0; k < items; ++k) units += tiles[k] > c ? (tiles[k] + c - 1) / c : 1;
        units *= p.Hkv;
        const int64_t unit = min(c, tiles[0]);
        int64_t cost = units <= grid ? 2 * (unit + PLAN_UNIT) : 2 * ((sum + units * PLAN_UNIT) / grid) + unit;
        if (lane < 31) cost = units > p.max_units ? (int64_t)1 << 40 : cost + 2 * PLAN_JOIN;
        int64_t best = cost * 32 + (31 - lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        chunk = __shfl_sync(0xffffffffu, c, 31 - (int)(best & 31));
    }
    int total = 0;
    for (int k0 = 0; k0 < items; k0 += 32) {
        const int k = k0 + lane;
        int x = k < items ? (tiles[k] > chunk ? (tiles[k] + chunk - 1) / chunk : 1) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (k < items) pl.units()[k + 1] = total + x;
        total += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
        pl.units()[0] = 0;
        pl.meta[1] = chunk;
        pl.meta[2] = total;
    }
}

// LONG: contexts of more than PR_FOLD key tiles may come (elsewhere the code for them would cost 2 to 3%).
template <typename T, int D, bool LONG>
__global__ void __launch_bounds__(PR_THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptParams p) {
    using S = PromptShape<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base = (raw_u32 + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_u32);
    const uint32_t k_full = base + S::OFF_BAR, k_empty = k_full + S::KST * 8;
    const uint32_t v_full = k_empty + S::KST * 8, q_full = v_full + S::VST * 8, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, p_full = s_full + 16, o_done = p_full + 16, o_free = o_done + 16;
    const uint32_t u_full = o_free + 16, u_empty = u_full + PR_UNITS * 8;
    const uint32_t drain = u_empty + PR_UNITS * 8;
    PromptUnit *units = reinterpret_cast<PromptUnit *>(smem + S::OFF_UNITS);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const PromptPlan plan = {reinterpret_cast<int *>(smem + S::OFF_PREF), reinterpret_cast<uint32_t *>(smem + S::OFF_KEYS),
                             reinterpret_cast<uint32_t *>(smem + S::OFF_KEYS) + PR_SORT,
                             reinterpret_cast<int *>(tmem_slot + 2)};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), PR_TMEM_COLS);
    if (tid == 64) {
        for (int s = 0; s < S::KST; ++s) mbar_init(k_full + s * 8, 1), mbar_init(k_empty + s * 8, 2);
        for (int s = 0; s < S::VST; ++s) mbar_init(v_full + s * 8, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full + t * 8, 1);
            mbar_init(q_empty + t * 8, 1);
            mbar_init(s_full + t * 8, 1);
            mbar_init(p_full + t * 8, PR_BM);
            mbar_init(o_done + t * 8, 1);
            mbar_init(o_free + t * 8, PR_BM);
        }
        for (int s = 0; s < PR_UNITS; ++s) {
            mbar_init(u_full + s * 8, 1);
            mbar_init(u_empty + s * 8, 11);           // K, V and MMA warps, 8 softmax warps
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    make_plan(p, plan, tid, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int chunk = plan.meta[1];
    if (p.max_units > 0 && blockIdx.x == gridDim.x - 1) {             // a block that has no unit if any has none
        const int n_items = chunk == PR_WHOLE ? 0 : plan.meta[0], rows2 = 2 * p.P;
        if (tid == 0) *p.ws_total = n_items;
        for (int k = tid; k < n_items; k += PR_THREADS) {
            const int b = plan.items()[k] >> 16, i = plan.items()[k] & 0xFFFF;
            int first, n, L;
            sequence(p, b, first, n, L, nullptr);
            const int npos = n - i * rows2, pos0 = L - n + i * rows2;
            int s0, s1;
            cuts(p, pos0, npos, chunk, s0, s1);
            if (max(s0, s1) <= 1) s0 = s1 = 0;
            p.ws_items[k] = PromptItem{first + i * rows2, npos, plan.units()[k], s0, s1};
        }
    }

    // A bounded wait that also ends when another role gave up.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_timer_ns();
        for (uint32_t i = 1;; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((i & 63u) == 0) {
                if (*abort_flag) return false;
                if (global_timer_ns() - t0 > p.wait_ns) {
                    *abort_flag = 1;
                    return false;
                }
            }
        }
    };

    if (warp >= PR_K_WARP) {
        setmaxnreg_dec<PR_REGS_OTHER>();
        if (warp == PR_SCHED_WARP) {
            // ------------------------------------------------------------ units and their Q tiles
            if (lane == 0) {
                const int items = plan.meta[0], total = plan.meta[2] * p.Hkv, grid = (int)gridDim.x, rows2 = 2 * p.P;
                const uint64_t policy = l2_policy_evict_first();
                int published = 0, qn[2] = {0, 0};
                bool ok = true;
                for (int round = 0; ok; ++round) {
                    const int u = round * grid + ((round & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
                    PromptUnit un = {};
                    if ((int64_t)round * grid < total) {
                        if (u >= total) continue;     // the last, partial round: the next one ends the list
                        const int w = u / p.Hkv;
                        const int *pre = items > PR_SORT ? plan.pref : plan.units();
                        int lo = 0, hi = items > PR_SORT ? p.num_seqs : items;     // pre[lo] <= w < pre[hi]
                        while (hi - lo > 1) {
                            const int mid = (lo + hi) >> 1;
                            if (pre[mid] <= w) lo = mid;
                            else hi = mid;
                        }
                        int i = w - pre[lo], s = 0;
                        un.b = lo;
                        if (items <= PR_SORT) {
                            s = i;
                            i = plan.items()[lo] & 0xFFFF;
                            un.b = plan.items()[lo] >> 16;
                        }
                        int first, n, L;
                        sequence(p, un.b, first, n, L, nullptr);
                        if (items > PR_SORT) i = items_of(p, n) - 1 - i;
                        un.valid = 1;
                        un.g = u - w * p.Hkv;
                        un.tok0 = first + i * rows2;
                        un.npos = n - i * rows2;
                        un.pos0 = L - n + i * rows2;
                        int s0, s1, e0, e1;
                        cuts(p, un.pos0, un.npos, chunk, s0, s1, &e0, &e1);
                        un.kt0 = s * chunk;
                        un.n0 = max(0, min(e0 - un.kt0, chunk));
                        un.n1 = max(0, min(e1 - un.kt0, chunk));
                        const bool cut = max(s0, s1) > 1;
                        un.slot = cut ? u : -1;
                        un.fold = chunk == PR_WHOLE ? (int)blockIdx.x : u;
                    }
                    const int st = published % PR_UNITS;
                    if (published >= PR_UNITS && !(ok = wait(u_empty + st * 8, (uint32_t)(published / PR_UNITS - 1) & 1u)))
                        break;
                    units[st] = un;
                    mbar_arrive(u_full + st * 8);
                    ++published;
                    if (!un.valid) break;
                    for (int t = 0; t < 2 && ok; ++t) {
                        if ((t ? un.n1 : un.n0) == 0) continue;
                        if (qn[t] > 0 && !(ok = wait(q_empty + t * 8, (uint32_t)(qn[t] - 1) & 1u))) break;
                        mbar_arrive_expect_tx(q_full + t * 8, p.P * p.G * D * 2);
#pragma unroll
                        for (int h = 0; h < S::HALVES; ++h)
                            tma_load<3>(base + t * S::Q_BYTES + h * (PR_BM * 128), &tmq, h * 64, un.g * p.G,
                                        un.tok0 + t * p.P, 0, q_full + t * 8, policy);
                        ++qn[t];
                    }
                }
                // after a wait that ran out: no copy may land in shared memory that the block has given up
                if (!ok)
                    for (int t = 0; t < 2; ++t)
                        if (qn[t] > 0) mbar_wait_bounded(q_full + t * 8, (uint32_t)(qn[t] - 1) & 1u, p.wait_ns);
            }
        } else if (warp == PR_K_WARP || warp == PR_V_WARP) {
            // ------------------------------------------------------------ K or V tiles
            const bool is_v = warp == PR_V_WARP;
            const int nst = is_v ? S::VST : S::KST;
            const uint32_t full0 = is_v ? v_full : k_full;
            const uint32_t ring = base + (is_v ? S::OFF_V : S::OFF_K);
            const CUtensorMap *map = is_v ? &tmv : &tmk;
            const uint64_t policy = l2_policy_evict_last();   // other row tiles read it again
            const int per_tile = PR_BN / p.bs;                // cache blocks per key tile
            int issued = 0;
            bool ok = true;
            for (int c = 0; ok; ++c) {
                const int st_u = c % PR_UNITS;
                ok = __all_sync(0xffffffffu, wait(u_full + st_u * 8, (uint32_t)(c / PR_UNITS) & 1u));
                if (!ok) break;
                const PromptUnit &un = units[st_u];
                const int valid = un.valid, b = un.b, g = un.g, kt0 = un.kt0, nt = max(un.n0, un.n1);
                const int seen = un.pos0 + min(un.npos, 2 * p.P);             // keys that any row of the unit sees
                __syncwarp();
                if (!valid) break;
                const int32_t *table = p.block_tables + (int64_t)b * p.stride;
                auto lookup = [&](int j) -> int {
                    const int e = (kt0 + j) * per_tile + lane;
                    return lane < per_tile && e * p.bs < seen ? __ldg(table + e) : 0;
                };
                int id_next = nt > 0 ? lookup(0) : 0;
                for (int j = 0; j < nt; ++j) {
                    const int st = issued % nst;
                    if (issued >= nst) {
                        // K(i) takes the stage of K(i - nst), V(i) that of V(i - nst), which P V reads before the scores
                        // of tile i - nst + 1 are issued: one release per key tile frees both
                        const int free = issued - nst + (is_v ? 1 : 0);
                        ok = __all_sync(0xffffffffu, wait(k_empty + free % S::KST * 8, (uint32_t)(free / S::KST) & 1u));
                        if (!ok) break;
                    }
                    int id = id_next;
                    if (j + 1 < nt) id_next = lookup(j + 1);
                    const int t0 = (kt0 + j) * PR_BN, left = seen - t0;       // > 0
                    const int nblk = min(per_tile, (left + p.bs - 1) / p.bs);
                    const uint32_t bar = full0 + st * 8, dst = ring + st * S::KV_BYTES;
                    if (lane == 0) mbar_arrive_expect_tx(bar, nblk * p.bs * D * 2);
                    __syncwarp();
                    if (lane < nblk) {
                        if (id < 0 || id >= p.num_blocks) {
                            set_status(p.status, STATUS_BOUNDS);
                            id = 0;
                        }
                        tma_load<4>(dst + lane * (p.bs / 8) * S::GROUP_BYTES, map, 0, 0, 0,
                                    (id * p.Hkv + g) * (p.bs / 8), bar, policy);
                    }
                    ++issued;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(u_empty + st_u * 8);
            }
            if (!ok) {                                // copies still in flight land before the block ends
                for (int i = issued > nst ? issued - nst : 0; i < issued; ++i)
                    mbar_wait_bounded(full0 + (i % nst) * 8, (uint32_t)(i / nst) & 1u, p.wait_ns);
            }
        } else {
            // ------------------------------------------------------------ MMA issue (lane 0)
            // One thread feeds the tensor cores, so what it does besides counts: descriptors are a constant upper
            // word and a lower one (address and leading offset) to which constants are added.
            if (lane == 0) {
                constexpr uint32_t idesc_s = umma_idesc<T>(PR_BM, PR_BN, false);
                constexpr uint32_t idesc_o = umma_idesc<T>(PR_BM, D, true);
                constexpr uint32_t hi_q = desc_hi(1024), hi_kv = desc_hi(S::GROUP_BYTES);
                const uint32_t q_lo = base >> 4 | 1u << 16, k_lo = (base + S::OFF_K) >> 4 | 1u << 16;
                const uint32_t v_lo = (base + S::OFF_V) >> 4 | (1024u >> 4) << 16;
                int ks = 0, vs = 0, last_vs = 0;      // stages of the next K and V tile; the V stage not released yet
                uint32_t kph = 0;                     // and the K stage's phase
                uint32_t qph[2] = {0, 0}, pph[2] = {0, 0}, oph[2] = {1, 1};
                int pj = 0, pn0 = 0, pn1 = 0;         // the step before: its index, key tiles of its unit
                bool ok = true;
                // O_t += P_t V of the step before
                auto flush = [&](auto tc, int pn) -> bool {
                    constexpr int t = decltype(tc)::value;
                    if (pj >= pn) return true;
                    if (!wait(p_full + t * 8, pph[t])) return false;
                    pph[t] ^= 1u;
                    if (pj == 0) {                    // the output of the unit before has left tensor memory
                        if (!wait(o_free + t * 8, oph[t])) return false;
                        oph[t] ^= 1u;
                    }
                    tc_fence_after();
                    const uint32_t v = v_lo + last_vs * (S::KV_BYTES >> 4), pt = tmem + t * 256, ot = pt + 128;
                    umma_ts<hi_kv>(ot, pt, v, idesc_o, (LONG ? pj & (PR_FOLD - 1) : pj) > 0 ? 1u : 0u);
#pragma unroll
                    for (int k = 1; k < PR_BN / 16; ++k)
                        umma_ts<hi_kv>(ot, pt + k * 8, v + ((k * 2 * S::GROUP_BYTES) >> 4), idesc_o, 1u);
                    if (pj == pn - 1) umma_commit(o_done + t * 8);
                    return true;
                };
                // S_t = Q_t K^T
                auto issue_s = [&](auto tc, int j, int n) -> bool {
                    constexpr int t = decltype(tc)::value;
                    if (j >= n) return true;
                    if (j == 0) {
                        if (!wait(q_full + t * 8, qph[t])) return false;
                        qph[t] ^= 1u;
                    }
                    const uint32_t k = k_lo + ks * (S::KV_BYTES >> 4), q = q_lo + t * (S::Q_BYTES >> 4);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_ss<hi_q, hi_kv>(tmem + t * 256, q + (((i >> 2) * (PR_BM * 128) + (i & 3) * 32) >> 4),
                                             k + (((i >> 2) * 1024 + (i & 3) * 32) >> 4), idesc_s, i > 0 ? 1u : 0u);
                    umma_commit(s_full + t * 8);
                    if (j == n - 1) umma_commit(q_empty + t * 8);
                    return true;
                };
                constexpr std::integral_constant<int, 0> T0{};
                constexpr std::integral_constant<int, 1> T1{};
                for (int c = 0; ok; ++c) {
                    const int st_u = c % PR_UNITS;
                    if (!(ok = wait(u_full + st_u * 8, (uint32_t)(c / PR_UNITS) & 1u))) break;
                    const int valid = units[st_u].valid, n0 = units[st_u].n0, n1 = units[st_u].n1;
                    if (!valid) break;
                    mbar_arrive(u_empty + st_u * 8);
                    const int nt = max(n0, n1);
                    for (int j = 0; j < nt; ++j) {
                        if (!(ok = wait(k_full + ks * 8, kph) && flush(T0, pn0))) break;
                        // the scores of a step tell that all products with the V tile before are done: they are the
                        // last to be issued, so where row tile 1 has none, its product goes first
                        if (j < n1) {
                            if (!(ok = issue_s(T0, j, n0) && flush(T1, pn1) && issue_s(T1, j, n1))) break;
                        } else {
                            if (!(ok = flush(T1, pn1) && issue_s(T0, j, n0))) break;
                        }
                        if (++ks == S::KST) ks = 0, kph ^= 1u;
                        last_vs = vs;                 // the V tile that goes with this step's scores
                        if (++vs == S::VST) vs = 0;
                        pj = j;
                        pn0 = n0;
                        pn1 = n1;
                    }
                }
                if (ok) ok = flush(T0, pn0) && flush(T1, pn1);
                if (!ok) {
                    umma_commit(drain);
                    mbar_wait_bounded(drain, 0u, p.wait_ns);
                }
            }
        }
    } else {
        setmaxnreg_inc<PR_REGS_SOFTMAX>();
        // ---------------------------------------------------------------- softmax of row tile t
        const int t = tid >> 7, r = tid & (PR_BM - 1);
        const int rp = r / p.G, rh = r - rp * p.G;    // position and head of this thread's row
        const bool in_tile = r < p.P * p.G;
        const uint32_t tmem_s = tmem + t * 256 + ((uint32_t)((warp & 3) * 32) << 16), tmem_o = tmem_s + 128;
        uint8_t *stage = smem + S::OFF_STAGE + warp * 2048;
        // fp16 weights are kept 2^7 times larger (at most 2^15 with the stale maximum's headroom; sum and O with them), so
        // that small ones stay above the type's smallest number: off by 2^-32 of the largest weight at most, not 2^-25
        constexpr float SHIFT = std::is_same<T, __half>::value ? 7.f : 0.f;
        int sc = 0, oc = 0, tiles = 0;                // scores and outputs taken; key tiles of the units before
        bool ok = true;
        for (int c = 0; ok; ++c) {
            const int st_u = c % PR_UNITS;
            ok = __all_sync(0xffffffffu, wait(u_full + st_u * 8, (uint32_t)(c / PR_UNITS) & 1u));
            if (!ok || !units[st_u].valid) break;
            const PromptUnit &un = units[st_u];
            const int nt = t ? un.n1 : un.n0, key0 = un.kt0 * PR_BN;
            const bool live = in_tile && t * p.P + rp < un.npos;
            const int lim = live ? un.pos0 + t * p.P + rp : 0x7fffffff;      // last key this row sees
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < nt; ++j) {
                ok = __all_sync(0xffffffffu, wait(s_full + t * 8, (uint32_t)sc & 1u));
                if (!ok) break;
                ++sc;
                const int i_k = tiles + j;            // this key tile in the block's sequence of them
                // K (and the V of the step before, whose product comes before these scores) is read: the row tiles
                // that work on it release it
                if (r == 0) mbar_arrive_count(k_empty + i_k % S::KST * 8, j < min(un.n0, un.n1) ? 1u : 2u);
                tc_fence_after();
                if (LONG && j > 0 && (j & (PR_FOLD - 1)) == 0) {
                    // P(j-1) V was issued before S(j), so the commit of S(j) covers it; P(j) V overwrites O
                    const RowState<D> kept(p.ws_slots + (size_t)un.fold * 256 * (D + 2) * 4, t * PR_BM + r);
                    const bool more = j > PR_FOLD;
                    const float w = more ? kept.weigh(m_ref, l) : 0.f;
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float a[32];
                        tmem_ld32(tmem_o + c0, a);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 x = make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
                            float4 *at = kept.o + (c0 / 4 + i) * 256;
                            if (more) {
                                const float4 y = *at;
                                x.x += y.x * w, x.y += y.y * w, x.z += y.z * w, x.w += y.w * w;
                            }
                            *at = x;
                        }
                    }
                    *kept.ml = make_float2(m_ref, l);
                    l = 0.f;
                }
                float sv[PR_BN];
                tmem_ld_cols(tmem_s, sv);
                const int t0 = key0 + j * PR_BN;
                if (t0 + PR_BN - 1 > lim) {
#pragma unroll
                    for (int i = 0; i < PR_BN; ++i) sv[i] = t0 + i <= lim ? sv[i] : -INFINITY;
                }
                // raw-score maximum (the scale is positive, so it commutes with it)
                float m4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = max3(sv[3 * i], sv[3 * i + 1], sv[3 * i + 2]);
#pragma unroll
                for (int i = 12; i + 2 <= PR_BN; i += 2) m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], sv[i], sv[i + 1]);
                const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * p.scale_log2;
                float alpha = 1.f;
                bool rescale = false;
                if (mx > m_ref + PR_RESCALE_LOG2 || (m_ref == -INFINITY && mx > -INFINITY)) {
                    alpha = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mx);
                    m_ref = mx;
                    rescale = true;
                }
                // P(j-1) V was issued before S(j), so the commit of S(j) covers it: O is at rest
                if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float a[32];
                        tmem_ld32(tmem_o + c0, a);
#pragma unroll
                        for (int i = 0; i < 32; ++i) a[i] *= alpha;
                        tmem_st32(tmem_o + c0, a);
                    }
                }
                const float nm = (m_ref == -INFINITY ? 0.f : -m_ref) + SHIFT;
                const uint64_t sc2 = pair(p.scale_log2, p.scale_log2), nm2 = pair(nm, nm);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float &x = sv[64 * h + 2 * i], &y = sv[64 * h + 2 * i + 1];
                        unpair(fma_pair(pair(x, y), sc2, nm2), x, y);
                        x = ex2_approx(x);
                        y = ex2_approx(y);
                        w[i] = pack2<T>(x, y);
                    }
                    tmem_st32_raw(tmem_s + 32 * h, w);
                }
                tmem_wait_st();
                tc_fence_before();
                // the MMA thread asks for the weights alone: their V tile is waited for here
                const uint32_t v_bar = v_full + i_k % S::VST * 8, v_phase = (uint32_t)(i_k / S::VST) & 1u;
                if (t0 + PR_BN - 1 > un.pos0) {
                    // some row does not see some key: V is looked over, a half key (128-byte line, [group][half][key
                    // in group]) or two per thread
                    if (!wait(v_bar, v_phase)) *abort_flag = 1;
                    uint8_t *tile = smem + S::OFF_V + i_k % S::VST * S::KV_BYTES;
                    const int left = un.pos0 + min(un.npos, 2 * p.P) - t0;
                    uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int q = 0; q < S::HALVES; ++q) {
                        const int ln = q * PR_BM + r, key = ln / (8 * S::HALVES) * 8 + (ln & 7);
                        uint4 *line = reinterpret_cast<uint4 *>(tile + ln * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (key >= left) {
                                // behind the last position seen: other words of the pool, or what the stage held
                                line[(i + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);
                            } else {
                                const uint4 w = line[(i + lane) & 7];
                                acc[0] = nonfinite_probe<T>(w.x, acc[0]);
                                acc[1] = nonfinite_probe<T>(w.y, acc[1]);
                                acc[2] = nonfinite_probe<T>(w.z, acc[2]);
                                acc[3] = nonfinite_probe<T>(w.w, acc[3]);
                            }
                        }
                    }
                    if ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7FFF7FFFu) {
                        // told before the words change: the other row tile may find them changed
                        *reinterpret_cast<volatile int *>(&units[st_u].poison) = 1;
                        __threadfence_block();
                        for (int q = 0; q < S::HALVES; ++q) {
                            uint16_t *w = reinterpret_cast<uint16_t *>(tile + (q * PR_BM + r) * 128);
                            for (int i = 0; i < 64; ++i)
                                if (is_nonfinite16<T>(w[i])) w[i] = 0;
                        }
                    }
                    fence_proxy_async_smem();
                } else if (r == 0 && !wait(v_bar, v_phase)) {
                    *abort_flag = 1;
                }
                __syncwarp();
                mbar_arrive(p_full + t * 8);
                // the sum is nobody's to wait for
                uint64_t r4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int i = 0; i < PR_BN / 2; ++i) r4[i & 3] = add_pair(r4[i & 3], pair(sv[2 * i], sv[2 * i + 1]));
                float ra, rb;
                unpair(add_pair(add_pair(r4[0], r4[1]), add_pair(r4[2], r4[3])), ra, rb);
                l = l * alpha + (ra + rb);
            }
            if (!ok) break;
            float o[D];
            if (nt > 0) {
                ok = __all_sync(0xffffffffu, wait(o_done + t * 8, (uint32_t)oc & 1u));
                if (!ok) break;
                ++oc;
                tc_fence_after();
                tmem_ld_cols(tmem_o, o);
                tc_fence_before();
                mbar_arrive(o_free + t * 8);
                if (LONG && nt > PR_FOLD) {
                    const RowState<D> kept(p.ws_slots + (size_t)un.fold * 256 * (D + 2) * 4, t * PR_BM + r);
                    const float w = kept.weigh(m_ref, l);
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) {
                        const float4 y = kept.o[i * 256];
                        o[4 * i] += y.x * w, o[4 * i + 1] += y.y * w, o[4 * i + 2] += y.z * w, o[4 * i + 3] += y.w * w;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < D; ++i) o[i] = 0.f;
            }
            if (*reinterpret_cast<volatile int *>(&units[st_u].poison) && live) {                  // values that are no numbers, at keys this row sees
                const int end = min(lim + 1, key0 + nt * PR_BN);
                for (int k = max(key0, un.pos0 / PR_BN * PR_BN); k < end; ++k) {
                    int id = __ldg(p.block_tables + (int64_t)un.b * p.stride + k / p.bs);
                    if (id < 0 || id >= p.num_blocks) id = 0;
                    const uint4 *v = reinterpret_cast<const uint4 *>(
                        static_cast<const T *>(p.v_cache) + (((int64_t)id * p.Hkv + un.g) * p.bs + k % p.bs) * D);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 x = __ldg(v + i);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t bits = (w[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu;
                            if (is_nonfinite16<T>(bits)) {
                                if constexpr (std::is_same<T, __half>::value)
                                    o[8 * i + e] += __half2float(__ushort_as_half((unsigned short)bits));
                                else
                                    o[8 * i + e] += __uint_as_float(bits << 16);
                            }
                        }
                    }
                }
            }
            tiles += max(un.n0, un.n1);
            const int tok = un.tok0 + t * p.P + rp, slot = un.slot;
            const int64_t orow = live ? (int64_t)tok * p.Hq + un.g * p.G + rh : -1;
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty + st_u * 8);
            if (slot >= 0) {
                // unnormalised state, [D / 4][256 rows] float4, then [256 rows] (max, sum)
                uint8_t *ws = p.ws_slots + (size_t)slot * 256 * (D + 2) * 4;
                if (live && nt > 0) {
                    float4 *dst = reinterpret_cast<float4 *>(ws) + t * PR_BM + r;
#pragma unroll
                    for (int i = 0; i < D / 4; ++i)
                        dst[i * 256] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    reinterpret_cast<float2 *>(ws + (size_t)256 * D * 4)[t * PR_BM + r] = make_float2(m_ref, l);
                }
            } else {
                // the warp's 32 rows in rounds of 32 dimensions through 2 KB: 64 bytes of a row per four lanes
                const float inv = l == 0.f ? 0.f : 1.f / l;
                int64_t row4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) row4[k] = __shfl_sync(0xffffffffu, orow, 8 * k + (lane >> 2));
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *x = o + c0 + 8 * i;
                        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(pack2<T>(x[0] * inv, x[1] * inv), pack2<T>(x[2] * inv, x[3] * inv),
                                       pack2<T>(x[4] * inv, x[5] * inv), pack2<T>(x[6] * inv, x[7] * inv));
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = 8 * k + (lane >> 2), i = lane & 3;
                        const uint4 x =
                            *reinterpret_cast<const uint4 *>(stage + row * 64 + ((i ^ ((row >> 1) & 3)) << 4));
                        if (row4[k] >= 0)
                            *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row4[k] * D + c0 + 8 * i) = x;
                    }
                    __syncwarp();
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) set_status(p.status, STATUS_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, PR_TMEM_COLS);
    }
}

// Joins the units of the items that were cut: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s. One block
// per unit index and 32 rows; a lane is a row, so the states are read in whole lines; the rows leave through
// shared memory.
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptParams p) {
    __shared__ __align__(16) T rows[32][D + 8];
    pdl_wait();
    const int k = blockIdx.x / p.Hkv, g = blockIdx.x - k * p.Hkv;
    const int total = *p.ws_total;
    const PromptItem it = p.ws_items[k];              // (behind the last: whatever the workspace holds)
    if (k >= total || it.splits0 == 0) return;
    const int u = it.first * p.Hkv + g;
    const int r0 = blockIdx.y * 32, t = r0 / PR_BM, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int splits = t ? it.splits1 : it.splits0;
    auto row_of = [&](int i) -> int64_t {             // output row of row i of this block, or -1
        const int r = (r0 & (PR_BM - 1)) + i, rp = r / p.G, pos = t * p.P + rp;
        return r < p.P * p.G && pos < it.npos ? (int64_t)(it.tok0 + pos) * p.Hq + g * p.G + (r - rp * p.G) : -1;
    };
    const bool live = row_of(lane) >= 0;
    if (__syncthreads_or(live) == 0) return;
    const size_t slot_bytes = (size_t)256 * (D + 2) * 4, step = (size_t)p.Hkv * slot_bytes;
    const uint8_t *ws = p.ws_slots + (size_t)u * slot_bytes;
    float M = -INFINITY, sum = 0.f;
    float4 acc[D / 32] = {};
    if (live) {
        // the running maximum again, over units, four of them in flight
        constexpr int U = 4;
        for (int s0 = 0; s0 < splits; s0 += U) {
            float2 ml[U];
            float4 o[U][D / 32];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                if (s0 + k >= splits) continue;
                const uint8_t *at = ws + (s0 + k) * step;
                ml[k] = reinterpret_cast<const float2 *>(at + (size_t)256 * D * 4)[r0 + lane];
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    o[k][i] = reinterpret_cast<const float4 *>(at)[(warp * (D / 32) + i) * 256 + r0 + lane];
            }
            float m = M;
#pragma unroll
            for (int k = 0; k < U; ++k) m = fmaxf(m, ml[k].x);
            const float w0 = M == -INFINITY ? 0.f : ex2_approx(M - m);
            M = m;
            sum *= w0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i].x *= w0, acc[i].y *= w0, acc[i].z *= w0, acc[i].w *= w0;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (s0 + k >= splits) continue;
                const float w = ml[k].x == -INFINITY ? 0.f : ex2_approx(ml[k].x - m);
                sum += w * ml[k].y;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    acc[i].x += w * o[k][i].x;
                    acc[i].y += w * o[k][i].y;
                    acc[i].z += w * o[k][i].z;
                    acc[i].w += w * o[k][i].w;
                }
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        *reinterpret_cast<uint2 *>(&rows[lane][(warp * (D / 32) + i) * 4]) =
            make_uint2(pack2<T>(acc[i].x * inv, acc[i].y * inv), pack2<T>(acc[i].z * inv, acc[i].w * inv));
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * (D / 8); i += 256) {
        const int64_t row = row_of(i / (D / 8));
        if (row >= 0)
            *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * D + i % (D / 8) * 8) =
                *reinterpret_cast<const uint4 *>(&rows[i / (D / 8)][i % (D / 8) * 8]);
    }
}

template <typename T, int D>
static cudaError_t launch_prompt_t(const PromptParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                   const CUtensorMap &tmv, int sm_count, cudaStream_t stream) {
    const auto kernel = p.max_ctx > PR_FOLD * PR_BN ? prompt_kernel<T, D, true> : prompt_kernel<T, D, false>;
    const cudaError_t e =
        launch_pdl(kernel, dim3((unsigned)sm_count), dim3(PR_THREADS), (size_t)PromptShape<D>::SMEM, stream, tmq, tmk, tmv, p);
    if (e != cudaSuccess || p.max_units == 0) return e;
    // 32 rows of an item and KV head per block; what is cut has fewer than max_units items, and a call of few tokens
    // no more items and rows than they make
    const int64_t items = ((int64_t)p.num_tokens / (2 * p.P) + std::min(p.num_tokens, p.num_seqs)) * p.Hkv;
    const int64_t rows = (int64_t)p.num_tokens * p.G;
    const dim3 blocks((unsigned)std::min(items, (int64_t)p.max_units), p.num_tokens <= p.P ? (unsigned)((rows + 31) / 32) : 8u);
    return launch_pdl(prompt_join_kernel<T, D>, blocks, dim3(256), 0, stream, p);
}

// The kernels' shared memory on the current device: once per pool, not per call.
template <typename T, int D>
static cudaError_t setup_prompt_t() {
    const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T, D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               PromptShape<D>::SMEM);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(prompt_kernel<T, D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   PromptShape<D>::SMEM);
}

cudaError_t setup_prompt(int dtype, int head_dim) {
    if (dtype == PA_FP16) return head_dim == 64 ? setup_prompt_t<__half, 64>() : setup_prompt_t<__half, 128>();
    return head_dim == 64 ? setup_prompt_t<__nv_bfloat16, 64>() : setup_prompt_t<__nv_bfloat16, 128>();
}

cudaError_t launch_prompt(const PromptParams &p, int dtype, int head_dim, const CUtensorMap &tmq,
                          const CUtensorMap &tmk, const CUtensorMap &tmv, int sm_count, cudaStream_t stream) {
    if (dtype == PA_FP16)
        return head_dim == 64 ? launch_prompt_t<__half, 64>(p, tmq, tmk, tmv, sm_count, stream)
                              : launch_prompt_t<__half, 128>(p, tmq, tmk, tmv, sm_count, stream);
    return head_dim == 64 ? launch_prompt_t<__nv_bfloat16, 64>(p, tmq, tmk, tmv, sm_count, stream)
                          : launch_prompt_t<__nv_bfloat16, 128>(p, tmq, tmk, tmv, sm_count, stream);
}

}  // namespace pa
