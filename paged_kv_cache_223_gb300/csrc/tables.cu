// tables.cu -- the tables of a serving step on the device: sequences are cut back, given new tokens and the blocks
// that those need; positions and slots of the new tokens.
//
// With kept = min(length, keep), have = ceil(kept / bs), old = ceil(length / bs), want = max(have, ceil((kept + new) / bs)):
// blocks [have, old) of every sequence go back on the free stack, then every sequence takes want - have from its top, both
// in the order of (sequence, block), the returned ones so that the first of them ends on top. Exclusive sums B and T of
// old - have and want - have over the sequences place every move by itself: with n blocks free and F returned, returned
// block i lies at n + F - 1 - i, taken block i comes from n + F - 1 - i. Cutting back what a step took and taking it
// again therefore gives the same blocks.
//
// One cluster does all of it (the tokens of large calls apart): every CTA makes the sums of all sequences for itself (they are
// few words), checks them and comes to the same verdict, the CTAs share the returned blocks, meet at the cluster's barrier
// (twice, for a verdict on the returned ids), and share the taken blocks, the tokens and the new lengths. So the lengths,
// tables and the stack are changed in place by one launch without a workspace, and a call that is refused changes nothing of
// them.
//
// Bound by latency: one request 3.4 us (launch, two trips to memory); 257 sequences of a verify with cuts and ended requests 6.2
// us (four trips, two searches, the barriers); 2000 prompts of 292000 tokens, 40000 blocks moved: 16.1 us, two launches, 14.4 in
// a graph.
#include <algorithm>

#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_sparse.h"

namespace pa {

namespace {

constexpr int TAB_THREADS = 512;
constexpr int TOK_THREADS = 256;
// More tokens get a kernel of their own (65536: 10.3 us by the cluster's eight CTAs, 7.9 by two kernels; 32768: 6.8 and 7.1).
constexpr int TAB_MAX_TOKENS = 32768;

struct Sums {
    long long tokens, back, taken;
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
    return {a.tokens + b.tokens, a.back + b.back, a.taken + b.taken};
}

__device__ __forceinline__ Sums shfl_up(const Sums &v, int d) {
    return {__shfl_up_sync(0xffffffffu, v.tokens, d), __shfl_up_sync(0xffffffffu, v.back, d),
            __shfl_up_sync(0xffffffffu, v.taken, d)};
}

// The last index b < n with start[b] <= i, for i below start[n].
__device__ __forceinline__ int owner(const int *start, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Positions and slots of the call's tokens, N at a time: four share the search and, as a rule, the block; a call that has at most
// two rounds of threads for all its tokens one by one has the shorter chain (257 sequences of a few tokens in one CTA: 6.0 us,
// four at a time 7.0; 8192 tokens in eight: 6.3, and 8.0 with four rounds one by one).
// block_of(b, kept, j): the id of the sequence's block j; kept_of(b): its tokens before the new ones.
template <int N, typename Kept, typename Block>
__device__ __forceinline__ void write_tokens(const TablesParams &p, const int *cu, int tokens, int first, int step, Kept kept_of,
                                             Block block_of) {
    const int bs = 1 << p.bs_shift;
    for (int in = first; in < (p.num_tokens + N - 1) / N; in += step) {
        int pos[N];
        long long slot[N];
        int b = N * in < tokens ? owner(cu, p.num_seqs, N * in) : 0, was = -1, id = -1, kept = N * in < tokens ? kept_of(b) : 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = N * in + e;
            pos[e] = 0;
            slot[e] = -1;
            if (i >= tokens) continue;
            if (cu[b + 1] <= i) {
                do ++b;
                while (cu[b + 1] <= i);
                kept = kept_of(b);
                was = -1;
            }
            pos[e] = kept + i - cu[b];
            const int j = pos[e] >> p.bs_shift;
            if (j != was) {
                id = block_of(b, kept, j);
                was = j;
                if (id < 0 || id >= p.num_blocks) {
                    set_status(p.status, STATUS_BOUNDS);
                    id = -1;
                }
            }
            if (id >= 0) slot[e] = ((long long)id << p.bs_shift) + (pos[e] & (bs - 1));
        }
        if constexpr (N == 4) {
            if (p.vectors && 4 * in + 4 <= p.num_tokens) {
                reinterpret_cast<int4 *>(p.positions)[in] = make_int4(pos[0], pos[1], pos[2], pos[3]);
                reinterpret_cast<longlong2 *>(p.slots)[2 * in] = make_longlong2(slot[0], slot[1]);
                reinterpret_cast<longlong2 *>(p.slots)[2 * in + 1] = make_longlong2(slot[2], slot[3]);
                continue;
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (N * in + e < p.num_tokens) p.positions[N * in + e] = pos[e], p.slots[N * in + e] = slot[e];
    }
}

}  // namespace

__global__ void __launch_bounds__(TAB_THREADS) tables_kernel(const TablesParams p) {
    extern __shared__ int tsm[];
    const int B = p.num_seqs;
    int *cu = tsm, *back = cu + B + 1, *taken = back + B + 1, *kept = taken + B + 1;   // sums of B + 1, then [B]
    __shared__ Sums wsum[TAB_THREADS / 32];
    __shared__ int bad;
    __shared__ uint32_t bad_id;                        // set by any CTA of the cluster
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int all = threads * ranks, gid = rank * threads + tid;
    pdl_trigger();
    pdl_wait();

    if (tid == 0) bad = 0, bad_id = 0;
    __syncthreads();
    const int bs = 1 << p.bs_shift;
    const int n_free = __ldcg(p.num_free);
    for (int b = tid; b < B; b += threads) {
        const int len = __ldcg(p.context_lens + b), add = __ldcg(p.new_lens + b);
        const int keep = p.keep_lens ? __ldcg(p.keep_lens + b) : 0x7FFFFFFF;
        const int k = keep < len ? keep : len;
        cu[b] = back[b] = taken[b] = 0;
        if (len < 0 || len > p.max_len || add < 0 || keep < 0 || (long long)k + add > p.max_len) {
            bad = 1;                                   // every writer writes the same
        } else {
            const int have = (k + bs - 1) >> p.bs_shift, old = (len + bs - 1) >> p.bs_shift;
            const int want = (k + add + bs - 1) >> p.bs_shift;
            kept[b] = k;
            cu[b] = add;
            back[b] = old - have;
            taken[b] = max(want - have, 0);
        }
    }
    // exclusive sums: a stretch of sequences per thread (its own ones where there are as many threads), whose totals are
    // summed over the block
    if (B > threads) __syncthreads();
    const int per = (B + threads - 1) / threads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    Sums own = {0, 0, 0};
    for (int b = b0; b < b1; ++b) own = own + Sums{cu[b], back[b], taken[b]};
    Sums s = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums u = shfl_up(s, d);
        if (lane >= d) s = s + u;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    Sums run = {s.tokens - own.tokens, s.back - own.back, s.taken - own.taken}, carry = {0, 0, 0};
    for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) run = run + wsum[w];
        carry = carry + wsum[w];
    }
    for (int b = b0; b < b1; ++b) {
        const Sums v = {cu[b], back[b], taken[b]};
        cu[b] = (int)run.tokens;
        back[b] = (int)run.back;
        taken[b] = (int)run.taken;
        run = run + v;
    }
    const bool wrong = bad || n_free < 0 || n_free > p.num_blocks || n_free + carry.back > p.num_blocks ||
                       carry.tokens > p.num_tokens;
    const bool none_left = !wrong && carry.taken > n_free + carry.back;
    const auto refuse = [&] {                          // by the same verdict in every CTA: no table, length or block is touched
        for (int b = gid; b <= B; b += all) p.cu_q[b] = 0;
        for (int i = gid; i < p.num_tokens && !p.tokens_apart; i += all) {
            p.positions[i] = 0;
            p.slots[i] = -1;
        }
    };
    if (wrong || none_left) {
        if (gid == 0) set_status(p.status, wrong ? STATUS_BOUNDS : STATUS_NO_BLOCKS);
        return refuse();
    }
    cluster_arrive();                                  // this CTA has read the lengths and set its word
    const int tokens = (int)carry.tokens, F = (int)carry.back, T = (int)carry.taken, top = n_free + F - 1;
    if (tid == 0) {
        cu[B] = tokens;
        back[B] = F;
        taken[B] = T;
    }
    __syncthreads();

    // returned blocks onto the stack, above *num_free, where nothing is lost if the step is refused after all: an id outside the
    // pool would go from one sequence to the next. Whoever finds one tells every CTA, which takes a barrier more (257 sequences
    // of a verify 5.6 -> 6.2 us; a step that returns nothing has one barrier as before).
    if (F > 0) {
        bool odd = false;
        for (int i = gid; i < F; i += all) {
            const int b = owner(back, B, i);
            const int j = ((kept[b] + bs - 1) >> p.bs_shift) + i - back[b];
            const int id = __ldcg(p.block_tables + b * p.stride + j);
            odd |= id < 0 || id >= p.num_blocks;
            __stcg(p.free_blocks + top - i, id);
        }
        cluster_wait();
        if (odd) {
            set_status(p.status, STATUS_BOUNDS);
            for (int r = 0; r < ranks; ++r) red_cluster_max(map_rank(smem_u32(&bad_id), r), 1u);
        }
        __syncwarp();
        cluster_arrive();
    }
    cluster_wait();                                    // every CTA has read the lengths; the stack is whole
    if (bad_id) return refuse();

    for (int i = gid; i < T; i += all) {
        const int b = owner(taken, B, i);
        const int j = ((kept[b] + bs - 1) >> p.bs_shift) + i - taken[b];
        const int id = __ldcg(p.free_blocks + top - i);
        if (id < 0 || id >= p.num_blocks) set_status(p.status, STATUS_BOUNDS);
        p.block_tables[b * p.stride + j] = id;
    }
    const auto kept_of = [&](int b) { return kept[b]; };
    // a block that this call takes is read where it comes from, not from the table that it is written to
    const auto block_of = [&](int b, int k, int j) {
        const int have = (k + bs - 1) >> p.bs_shift;
        return j < have ? __ldcg(p.block_tables + b * p.stride + j) : __ldcg(p.free_blocks + top - (taken[b] + j - have));
    };
    if (!p.tokens_apart && p.num_tokens <= 2 * all) write_tokens<1>(p, cu, tokens, gid, all, kept_of, block_of);
    else if (!p.tokens_apart) write_tokens<4>(p, cu, tokens, gid, all, kept_of, block_of);
    for (int b = gid; b <= B; b += all) {
        p.cu_q[b] = cu[b];
        if (b < B) p.context_lens[b] = kept[b] + cu[b + 1] - cu[b];
    }
    if (gid == 0) *p.num_free = n_free + F - T;
}

// The tokens of a large call, behind tables_kernel, on all SMs: from the tables as they are then.
__global__ void __launch_bounds__(TOK_THREADS) tokens_kernel(const TablesParams p) {
    extern __shared__ int cu_sm[];
    pdl_trigger();
    pdl_wait();
    for (int b = threadIdx.x; b <= p.num_seqs; b += TOK_THREADS) cu_sm[b] = __ldcg(p.cu_q + b);
    __syncthreads();
    write_tokens<4>(p, cu_sm, cu_sm[p.num_seqs], blockIdx.x * TOK_THREADS + threadIdx.x, gridDim.x * TOK_THREADS,
                 [&](int b) { return __ldcg(p.context_lens + b) - (cu_sm[b + 1] - cu_sm[b]); },
                 [&](int b, int, int j) { return __ldcg(p.block_tables + b * p.stride + j); });
}

cudaError_t launch_tables(TablesParams p, int sm_count, cudaStream_t stream) {
    const size_t smem = (size_t)(4 * p.num_seqs + 3) * sizeof(int);
    // The attribute belongs to the kernel on this device, not to a call: always the most that any call takes, so that a call of
    // another thread between here and the launch cannot lower it.
    cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (4 * PA_TABLES_MAX_SEQS + 3) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    p.vectors = (reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) % 16 == 0;
    p.tokens_apart = p.num_tokens > TAB_MAX_TOKENS;
    // CTAs of the cluster: eight even for small steps, whose lengths are known on the device only (257 sequences, before the
    // barrier for returned ids: 5.6 us, a single CTA 6.5; one request 3.3 and 3.9), 16 in front of the tokens' kernel (2000
    // prompts in a graph: 14.4 us, eight 16.0; in a stream 16.1 and 16.2)
    const int ranks = p.tokens_apart ? 16 : 8;
    if (ranks > 8) e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = launch_clusters(tables_kernel, ranks, TAB_THREADS, smem, ranks, stream, p);
    if (e != cudaSuccess || !p.tokens_apart) return e;
    const int ctas = std::min((p.num_tokens + 4 * TOK_THREADS - 1) / (4 * TOK_THREADS), 4 * sm_count);
    return launch_pdl(tokens_kernel, dim3(ctas), dim3(TOK_THREADS), (size_t)(p.num_seqs + 1) * sizeof(int), stream, p);
}

}  // namespace pa
