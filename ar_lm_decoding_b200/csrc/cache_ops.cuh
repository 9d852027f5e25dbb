// Parameters of the shared-prefix attention, the attention mass and the cache eviction.
#pragma once

#include <atomic>

#include "common.cuh"

namespace tidar {

constexpr long long kCacheWaitCycles = 4000000000LL;  // bound of the on-chip waits of a normal launch (about 2 s)
constexpr int kMaxBatchShared = 1024;     // longest batch the shared-prefix attention and the mass accept
constexpr int kMaxSharedPages = 4096;     // longest shared page table (262144 shared tokens)
constexpr int kMaxCausalRows = 4096;      // most rows per sequence of the causal shared-prefix attention
constexpr int kMaxMassRows = 1 << 22;     // longest cache the mass accepts
constexpr int kMaxEvictRows = 65536;      // longest cache the eviction accepts (16-bit row lists)

struct SharedAttnParams {
    const bf16 *q, *k_new, *v_new;
    const bf16 *k_shared, *v_shared;  // [Hkv, S_max, D] (contiguous), or the pools
    const bf16 *k_cache, *v_cache;    // [B, Hkv, P_max, D] (contiguous), or the pools
    const int32_t *shared_len, *prefix_len;
    const int32_t *shared_table, *block_table;  // paged (block_table not null): page ids of the shared / own rows
    int max_pages, num_pages;
    int B, Hq, Hkv, D, k, R, G, S_max, P_max;
    float scale_log2;  // softmax_scale * log2(e)
    int mask_mode;
    bf16 *out;   // [B, R, Hq, D]
    float *lse;  // [B, R, Hq] or null
    uint8_t *ws;
    int32_t *dev_status;
    long long wait_cycles;  // bound of every on-chip wait, in SM clock cycles
    int stall_test;         // 1: the MMA issuers first wait on a barrier nothing arrives on (timeout test)
};

// Whether the cost of the call's key tiles counts in 32 bits.
bool shared_attn_fits(int B, int R, int Hkv, int G, int S_max, int P_max);
size_t shared_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int R, int S_max, int P_max);
cudaError_t shared_attn_launch(const SharedAttnParams &p, cudaStream_t s);

struct MassParams {
    const void *const *qs;
    const float *const *lses;
    const void *const *k_caches;
    float *const *masses;
    const int32_t *block_table;  // null: contiguous
    int max_pages, num_pages;
    const int32_t *prefix_len, *row_count;  // row_count null: R
    int L, B, Hq, Hkv, D, R, G, P_max;
    float scale_log2, decay;
    int32_t *dev_status;
    long long wait_cycles;  // as in SharedAttnParams
    int stall_test;
};

cudaError_t mass_launch(const MassParams &p, cudaStream_t s);

struct EvictParams {
    void *const *k_caches;
    void *const *v_caches;
    float *const *masses;
    const int32_t *block_table;  // null: contiguous
    int max_pages, num_pages;
    int32_t *prefix_len;
    int L, B, Hkv, D, P_max, budget, sink, recent;
    int32_t *dev_status;
};

cudaError_t evict_launch(const EvictParams &p, cudaStream_t s);

// Lets kernel K take `bytes` of dynamic shared memory, once per device (the call costs a launch's tenth).
template <auto K>
cudaError_t allow_shared_memory(int bytes) {
    static std::atomic<unsigned long long> done{0};  // bit = device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ULL << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Whether one of the pages holding rows [0, n) of a table row is outside [0, num_pages); every thread of the block
// calls it and gets the answer.
__device__ __forceinline__ bool block_bad_page(const int32_t *pages, int n, int num_pages) {
    int bad = 0;
    for (int i = threadIdx.x; i < ceil_div(n, kPageRows); i += blockDim.x) {
        const int pg = pages[i];
        bad |= pg < 0 || pg >= num_pages;
    }
    return __syncthreads_or(bad) != 0;
}

}  // namespace tidar
