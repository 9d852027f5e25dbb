// Eviction from the KV caches by accumulated attention mass, in place.
//
// A cluster of C CTAs takes one (layer, sequence, KV head).  Every CTA finds the rows to give up by itself (the masses
// are read from L2), then moves its share of the columns of K and V; CTA 0 also moves the masses.
//
// Selection: the keepth-greatest mass among the candidates, by histograms over a shrinking range of keys (a monotone
// 32-bit image of the float).  The first pass takes the exact range of the keys, so its 2048 bins are spread over the
// values that occur; a range of 2^32 needs at most three passes, ties of equal masses none beyond.  Ties at the
// threshold go to the lower rows.
//
// Moves: rows that survive behind the final heavy zone fill the holes inside it pairwise (sources all behind the zone,
// destinations all inside: no order among the copies).  Then the newest rows slide down by N - budget, tile by tile in
// ascending order: a tile is loaded before any of it is stored, and a later tile's sources lie behind an earlier
// tile's destinations.
#include "cache_ops.cuh"
#include "tc.cuh"

namespace tidar {

namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int MAXC = 8;
static_assert(BINS == 4 * THREADS, "four bins a thread in the bin search");

struct EvictSmem {
    uint32_t hist[BINS];
    uint32_t warp_sum[WARPS];
    uint32_t lo, hi;        // key range under search
    uint32_t bin, above;    // the bin that holds the keepth-greatest key, keys above it
};

__device__ __forceinline__ uint32_t key_of(float m) {
    if (m != m) return 0xffffffffu;
    const uint32_t u = __float_as_uint(m + 0.f);  // (-0 + 0 = 0)
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of v, in thread order (every thread calls it); *total the block's sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sum, uint32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const uint32_t s = warp_sum[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return before + x - v;
}

// Byte offset of cache row n of (b, kvh).
__device__ __forceinline__ size_t row_bytes(const EvictParams &p, int b, int kvh, int n) {
    size_t row = ((size_t)b * p.Hkv + kvh) * p.P_max + n;
    if (p.block_table)
        row = ((size_t)p.block_table[(size_t)b * p.max_pages + n / kPageRows] * p.Hkv + kvh) * kPageRows + n % kPageRows;
    return row * p.D * 2;
}

__global__ void __launch_bounds__(THREADS, 2) evict_kernel(const EvictParams p, int C) {
    extern __shared__ uint16_t lists[];  // holes (from the sink), then the survivors behind the zone (from its end)
    __shared__ EvictSmem sm;
    const int tid = threadIdx.x, part = blockIdx.x % C, head = blockIdx.x / C;
    const int kvh = head % p.Hkv, b = head / p.Hkv % p.B, l = head / p.Hkv / p.B;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int N = p.prefix_len[b];
    const bool bad = N < 0 || N > p.P_max;
    if (bad || N <= p.budget) {  // (uniform over the cluster)
        if (bad && tid == 0) atomicOr(p.dev_status, TIDAR_DEV_BAD_PREFIX);
        return;
    }
    if (p.block_table && block_bad_page(p.block_table + (size_t)b * p.max_pages, N, p.num_pages)) {
        if (tid == 0) atomicOr(p.dev_status, TIDAR_DEV_BAD_PAGE);
        return;
    }
    float *mass = p.masses[l] + ((size_t)b * p.Hkv + kvh) * p.P_max;
    const int zone = p.budget - p.recent;      // [sink, zone): the heaviest rows
    const int lo = p.sink, hi = N - p.recent;  // candidates
    const int keep = zone - p.sink;            // of them stay

    // ---- the keepth-greatest key T; of the keys equal to T the first need_eq rows stay ----
    uint32_t T = 0xffffffffu, need_eq = 0;
    bool ties = false;
    if (keep > 0) {
        uint32_t kmin = 0xffffffffu, kmax = 0;
        for (int i = lo + tid; i < hi; i += THREADS) {
            const uint32_t k = key_of(mass[i]);
            kmin = min(kmin, k);
            kmax = max(kmax, k);
        }
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        if (tid == 0) {
            sm.lo = 0xffffffffu;
            sm.hi = 0;
        }
        __syncthreads();
        if ((tid & 31) == 0) {
            atomicMin(&sm.lo, kmin);
            atomicMax(&sm.hi, kmax);
        }
        __syncthreads();
        uint32_t rlo = sm.lo, rhi = sm.hi, want = keep, equal = hi - lo;
        while (rlo < rhi) {  // (each pass divides the range by up to 2048: at most three)
            const int bits = 32 - __clz(rhi - rlo);
            const int shift = max(0, bits - 11);
#pragma unroll
            for (int i = 0; i < 4; ++i) sm.hist[i * THREADS + tid] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += THREADS) {
                const uint32_t k = key_of(mass[i]);
                if (k >= rlo && k <= rhi) atomicAdd(&sm.hist[(k - rlo) >> shift], 1u);
            }
            __syncthreads();
            // bins from the top: thread t has bins 2047 - 4t .. 2044 - 4t
            uint32_t c[4], mine = 0, all;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = sm.hist[BINS - 1 - (4 * tid + i)];
                mine += c[i];
            }
            uint32_t before = block_scan(mine, sm.warp_sum, &all);
            if (before < want && want <= before + mine) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (before < want && want <= before + c[i]) {
                        sm.bin = BINS - 1 - (4 * tid + i);
                        sm.above = before;
                    }
                    before += c[i];
                }
            }
            __syncthreads();
            const uint32_t bin = sm.bin;
            want -= sm.above;
            equal = sm.hist[bin];
            rlo += bin << shift;
            rhi = rlo + min(rhi - rlo, (1u << shift) - 1u);
            __syncthreads();
        }
        T = rlo;
        need_eq = want;
        ties = want < equal;
    }

    // ---- holes and the survivors that fill them: a contiguous run of candidates per thread, in row order ----
    const int per = ceil_div(hi - lo, THREADS);
    const int i0 = min(hi, lo + tid * per), i1 = min(hi, i0 + per);
    uint32_t eq_before = 0;
    if (ties) {
        uint32_t eq = 0, all;
        for (int i = i0; i < i1; ++i) eq += key_of(mass[i]) == T;
        eq_before = block_scan(eq, sm.warp_sum, &all);
    }
    auto stays = [&](int i, uint32_t &eq) {
        const uint32_t k = key_of(mass[i]);
        bool s = keep > 0 && k >= T;
        if (k == T && ties) s = keep > 0 && eq++ < need_eq;
        return s;
    };
    uint32_t count = 0, eq = eq_before, total;  // holes in the upper half word, survivors in the lower
    for (int i = i0; i < i1; ++i) {
        const bool s = stays(i, eq);
        if (i < zone && !s) count += 1u << 16;
        if (i >= zone && s) count += 1;
    }
    const uint32_t base = block_scan(count, sm.warp_sum, &total);
    const int moves = total & 0xffffu;
    uint16_t *holes = lists, *tails = lists + moves;
    uint32_t h = base >> 16, t = base & 0xffffu;
    eq = eq_before;
    for (int i = i0; i < i1; ++i) {
        const bool s = stays(i, eq);
        if (i < zone && !s) holes[h++] = (uint16_t)(i - p.sink);
        if (i >= zone && s) tails[t++] = (uint16_t)(i - zone);
    }
    __syncthreads();
    if (C > 1) tc::cluster_sync();  // every CTA has read the masses
    if (part == 0) {
        for (int i = tid; i < moves; i += THREADS) mass[p.sink + holes[i]] = mass[zone + tails[i]];
        for (int i = 0; i < p.recent; i += THREADS) {
            const float m = i + tid < p.recent ? mass[N - p.recent + i + tid] : 0.f;
            __syncthreads();  // (before the first tile is stored the survivors behind the zone have left it, too)
            if (i + tid < p.recent) mass[zone + i + tid] = m;
        }
    }

    // ---- this CTA's columns of K and V: vectors [v0, v0 + vn) of a row of D/8, of K (x = 0) or V (x = 1) ----
    const int vec = p.D / 8;
    const int x0 = C == 1 ? 0 : part & 1, x1 = C == 1 ? 2 : x0 + 1;
    const int vn = C <= 2 ? vec : vec / (C / 2), v0 = C <= 2 ? 0 : (part >> 1) * vn;
    for (int x = x0; x < x1; ++x) {
        uint8_t *cache = static_cast<uint8_t *>(x ? p.v_caches[l] : p.k_caches[l]);
        constexpr int U = 4;
        for (int i = tid; i < moves * vn; i += U * THREADS) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int it = i + u * THREADS;
                if (it < moves * vn)
                    v[u] = *reinterpret_cast<const uint4 *>(cache + row_bytes(p, b, kvh, zone + tails[it / vn]) +
                                                            (v0 + it % vn) * 16);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int it = i + u * THREADS;
                if (it < moves * vn)
                    *reinterpret_cast<uint4 *>(cache + row_bytes(p, b, kvh, p.sink + holes[it / vn]) +
                                               (v0 + it % vn) * 16) = v[u];
            }
        }
        __syncthreads();
        for (int i0 = 0; i0 < p.recent * vn; i0 += U * THREADS) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int it = i0 + u * THREADS + tid;
                if (it < p.recent * vn)
                    v[u] = *reinterpret_cast<const uint4 *>(cache + row_bytes(p, b, kvh, N - p.recent + it / vn) +
                                                            (v0 + it % vn) * 16);
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int it = i0 + u * THREADS + tid;
                if (it < p.recent * vn)
                    *reinterpret_cast<uint4 *>(cache + row_bytes(p, b, kvh, zone + it / vn) + (v0 + it % vn) * 16) = v[u];
            }
        }
    }
}

// The new lengths, once every layer has been trimmed.
__global__ void evict_lengths_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int b = blockIdx.x;
    const int N = p.prefix_len[b];
    if (N <= p.budget || N > p.P_max) return;
    if (p.block_table && block_bad_page(p.block_table + (size_t)b * p.max_pages, N, p.num_pages)) return;
    if (threadIdx.x == 0) p.prefix_len[b] = p.budget;
}

}  // namespace

cudaError_t evict_launch(const EvictParams &p, cudaStream_t s) {
    // At most this many rows fill holes: no more than leave, and no more than the heavy zone holds.
    const int cap = max(0, min(p.P_max - p.budget, p.budget - p.recent - p.sink));
    const int heads = p.L * p.B * p.Hkv;
    // Few heads: a cluster per head, so that the moves use more SMs (and more loads in flight).
    int C = 1;
    while (C < MAXC && heads * C * 2 <= 2 * kNumSMs) C *= 2;
    const int smem = 2 * 2 * cap;
    cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(heads * C, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_kernel, p, C);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.B, 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_lengths_kernel, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace tidar
