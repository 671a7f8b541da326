// pa_pool.h -- the pool object and what the entry points share (not part of the C ABI).
#pragma once

#include <cudaTypedefs.h>

#include <mutex>
#include <new>
#include <unordered_map>

#include "pa_internal.h"

struct pa_pool {
    pa_pool_config cfg;
    void *k_cache = nullptr;
    void *v_cache = nullptr;
    bool owns_caches = false;
    uint64_t cache_bytes = 0;
    float *part_o = nullptr;
    float2 *part_ml = nullptr;
    int64_t ws_slots = 0;        // (output row, partition) pairs the workspace holds
    int *status = nullptr;
    int *work = nullptr;         // tensor-core decode's item counters (in the status allocation; reset by each launch)
    int sm_count = 0;
    int part_tokens = 512;
    uint64_t wait_ns = 2000000000ull;
    // shared-prefix decode: the prefix kernel runs on this stream beside the caller's decode
    cudaStream_t side = nullptr;
    cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
    std::mutex mu;
    std::unordered_map<const void *, CUtensorMap> maps;
    std::unordered_map<const void *, CUtensorMap> group_maps;   // the same caches by groups of eight rows
};

namespace pa {

struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) return;
        ok = (prev == dev) || cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cuTensorMapEncodeTiled, looked up once (nullptr: the driver has none).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Keeps a map for the next call. Without memory for that it is made anew then: no exception leaves a C entry.
inline void keep_map(std::unordered_map<const void *, CUtensorMap> &maps, const void *cache, const CUtensorMap &m) {
    if (maps.size() > 4096) maps.clear();
    try {
        maps.emplace(cache, m);
    } catch (const std::bad_alloc &) {
    }
}

// The map of one of the pool's caches for copies of 16 token rows, kept per cache address.
pa_status tensor_map(pa_pool *pool, const void *cache, CUtensorMap *out);
// One of a 16-bit pool's caches for copies of 16 token rows at once, as two groups of eight rows by halves of 64 dimensions.
pa_status group_map(pa_pool *pool, const void *cache, CUtensorMap *out);

}  // namespace pa
