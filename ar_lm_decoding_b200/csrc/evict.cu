// Eviction from the KV caches by accumulated attention mass, in place.
//
// A cluster of C CTAs takes one (layer, sequence, KV head).  Every CTA finds the rows to give up by itself (the masses
// are read from L2), then moves its share of the columns of K and V; CTA 0 also moves the masses.
//
// Selection: the last row to stay, by a histogram of the masses' monotone 32-bit images over their upper 11 bits; the
// rows of the bin that holds it (256 at most) are ranked against each other by (mass, row), a fuller bin is divided by
// another histogram, and equal masses by a count over the rows in order.
//
// Moves: rows that survive behind the final heavy zone fill the holes inside it pairwise (sources all behind the zone,
// destinations all inside: no order among the copies).  Then the newest rows slide down by N - budget, in ascending
// order.  Both are one list, taken in tiles: a tile is loaded before any of it is stored, a later tile's sources lie
// behind an earlier tile's destinations, and a slide's destination is loaded, if it survives, by an earlier item.
//
// Bound by the moves' bytes for a long cut, by latency for a step's trim (a few rows of holes and the newest rows).
#include "cache_ops.cuh"
#include "tc.cuh"

namespace tidar {

namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int MAXC = 8;
constexpr int RANKED = 256;         // rows ranked against each other at most
constexpr int kSmemBytes = 227 * 1024 - 14 * 1024;  // dynamic shared memory at most (EvictSmem is static)
static_assert(4 * (kMaxEvictRows / 2 + 8192) <= kSmemBytes, "lists and images beyond the shared memory");
static_assert(BINS == 4 * THREADS, "four bins a thread in the bin search");

struct EvictSmem {
    union {
        uint32_t hist[BINS];
        uint2 ranked[RANKED];  // (image, row)
    };
    uint32_t warp_sum[WARPS];
    uint32_t bin, above;  // the bin that holds the last row to stay, rows above it
    uint32_t count;
    uint32_t T;           // the last row to stay: its image,
    int row;              // its place
    int pages[kMaxPagesPerSeq];  // of the sequence (paged caches)
};
static_assert(sizeof(EvictSmem) <= 14 * 1024 - 512, "static shared memory beyond its part");

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

__global__ void __launch_bounds__(THREADS, 2) evict_kernel(const EvictParams p, int C, int cap, int keys_held) {
    extern __shared__ uint32_t dyn[];  // lists of 16-bit rows (holes from the sink, survivors from the zone's end), images
    __shared__ EvictSmem sm;
    const int tid = threadIdx.x, part = blockIdx.x % C, head = blockIdx.x / C;
    const int kvh = head % p.Hkv, b = head / p.Hkv % p.B, l = head / p.Hkv / p.B;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // (evict_lengths_kernel waits for this grid's end)
#pragma unroll
    for (int i = 0; i < 4; ++i) sm.hist[i * THREADS + tid] = 0;
    if (tid == 0) sm.count = 0;
    const int N = p.prefix_len[b];
    const bool bad = N < 0 || N > p.P_max;
    if (bad || N <= p.budget) {  // (uniform over the cluster)
        if (bad && tid == 0) atomicOr(p.dev_status, TIDAR_DEV_BAD_PREFIX);
        return;
    }
    if (p.block_table) {
        bool bad_page = false;
        for (int i = tid; i < ceil_div(N, kPageRows); i += THREADS) {
            const int pg = p.block_table[(size_t)b * p.max_pages + i];
            bad_page |= pg < 0 || pg >= p.num_pages;
            sm.pages[i] = pg;
        }
        if (__syncthreads_or(bad_page)) {
            if (tid == 0) atomicOr(p.dev_status, TIDAR_DEV_BAD_PAGE);
            return;
        }
    }
    __syncthreads();
    float *mass = p.masses[l] + ((size_t)b * p.Hkv + kvh) * p.P_max;
    const int zone = p.budget - p.recent;            // [sink, zone): the heaviest rows
    const int lo = p.sink, n = N - p.recent - lo;    // candidates: rows lo .. lo + n - 1
    const int keep = zone - p.sink;                  // of them stay
    uint16_t *lists = reinterpret_cast<uint16_t *>(dyn);
    uint32_t *keys = dyn + cap;
    const bool held = n <= keys_held;  // the images, in shared memory
    // f(candidate, image) for the candidates from, from + step, .. below to
    auto each = [&](int from, int step, int to, auto &&f) {
        if (held) {
            for (int i = from; i < to; i += step) f(i, keys[i]);
            return;
        }
        constexpr int U = 8;  // loads under way
        for (int i = from; i < to; i += U * step) {
            uint32_t k[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                k[u] = i + u * step < to ? key_of(mass[lo + i + u * step]) : 0u;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * step < to) f(i + u * step, k[u]);
        }
    };

    // ---- the last candidate to stay: image T, place `last` among the candidates ----
    uint32_t T = 0xffffffffu;
    int last = -1;
    if (keep > 0) {
        constexpr int U = 8;  // loads under way
        for (int i0 = tid; i0 < n; i0 += U * THREADS) {
            float m[U];
#pragma unroll
            for (int u = 0; u < U; ++u) m[u] = i0 + u * THREADS < n ? mass[lo + i0 + u * THREADS] : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + u * THREADS >= n) break;
                const uint32_t k = key_of(m[u]);
                if (held) keys[i0 + u * THREADS] = k;
                atomicAdd(&sm.hist[k >> 21], 1u);
            }
        }
        uint32_t base = 0, want = keep;  // images from base on, of which the want-th greatest is sought
        for (int shift = 21;; shift = shift == 21 ? 10 : 0) {
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
            const uint32_t inside = sm.hist[sm.bin], span = (1u << shift) - 1u;
            base += sm.bin << shift;
            want -= sm.above;
            __syncthreads();
            if (inside <= RANKED) {
                each(tid, THREADS, n, [&](int i, uint32_t k) {
                    if (k >= base && k - base <= span) sm.ranked[atomicAdd(&sm.count, 1u)] = make_uint2(k, i);
                });
                __syncthreads();
                if (tid < (int)inside) {
                    const uint2 me = sm.ranked[tid];
                    uint32_t first = 0;
                    for (int i = 0; i < (int)inside; ++i) {
                        const uint2 o = sm.ranked[i];
                        first += o.x > me.x || (o.x == me.x && o.y < me.y);
                    }
                    if (first == want - 1) {
                        sm.T = me.x;
                        sm.row = (int)me.y;
                    }
                }
                __syncthreads();
                T = sm.T;
                last = sm.row;
                break;
            }
            if (shift == 0) {  // more equal images than can be ranked: the want-th of them in the order of the rows
                const int per = ceil_div(n, THREADS), i0 = min(n, tid * per), i1 = min(n, i0 + per);
                uint32_t eq = 0, all_eq;
                each(i0, 1, i1, [&](int, uint32_t k) { eq += k == base; });
                uint32_t seen = block_scan(eq, sm.warp_sum, &all_eq);
                if (seen < want && want <= seen + eq)
                    each(i0, 1, i1, [&](int i, uint32_t k) {
                        if (k == base && ++seen == want) sm.row = i;
                    });
                __syncthreads();
                T = base;
                last = sm.row;
                break;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sm.hist[i * THREADS + tid] = 0;
            __syncthreads();
            const int sub = shift == 21 ? 10 : 0;
            each(tid, THREADS, n, [&](int, uint32_t k) {
                if (k >= base && k - base <= span) atomicAdd(&sm.hist[(k - base) >> sub], 1u);
            });
        }
    } else if (held) {
        for (int i = tid; i < n; i += THREADS) keys[i] = 0;
        __syncthreads();
    }

    // ---- holes and the survivors that fill them: a contiguous run of candidates per thread, in row order ----
    const int per = ceil_div(n, THREADS), i0 = min(n, tid * per), i1 = min(n, i0 + per);
    auto stays = [&](int i, uint32_t k) { return keep > 0 && (k > T || (k == T && i <= last)); };
    uint32_t count = 0, total;  // holes in the upper half word, survivors in the lower
    each(i0, 1, i1, [&](int i, uint32_t k) {
        const bool s = stays(i, k);
        if (i < keep && !s) count += 1u << 16;
        if (i >= keep && s) count += 1;
    });
    const uint32_t before = block_scan(count, sm.warp_sum, &total);
    const int moves = total & 0xffffu;
    uint16_t *holes = lists, *tails = lists + moves;
    uint32_t h = before >> 16, t = before & 0xffffu;
    if (count) {
        each(i0, 1, i1, [&](int i, uint32_t k) {
            const bool s = stays(i, k);
            if (i < keep && !s) holes[h++] = (uint16_t)i;
            if (i >= keep && s) tails[t++] = (uint16_t)(i - keep);
        });
    }
    __syncthreads();
    if (C > 1) tc::cluster_sync();  // every CTA has read the masses

    // ---- the list of moves: item i < moves fills a hole, the others slide ----
    const int rows = moves + p.recent;
    auto source = [&](int i) { return i < moves ? zone + tails[i] : N - p.recent + (i - moves); };
    auto target = [&](int i) { return i < moves ? p.sink + holes[i] : zone + (i - moves); };
    if (part == 0) {
        constexpr int U = 4;
        for (int i0 = 0; i0 < rows; i0 += U * THREADS) {
            float m[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * THREADS + tid;
                m[u] = i < rows ? mass[source(i)] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * THREADS + tid;
                if (i < rows) mass[target(i)] = m[u];
            }
        }
    }
    // This CTA's columns of K and V: vectors [v0, v0 + vn) of a row of D/8, of K (x = 0) and V (x = 1) or of one of them.
    const int vec = p.D / 8, nx = C == 1 ? 2 : 1;
    const int vn = C <= 2 ? vec : vec / (C / 2), v0 = C <= 2 ? 0 : (part >> 1) * vn;
    uint8_t *cache[2] = {static_cast<uint8_t *>(C > 1 && (part & 1) ? p.v_caches[l] : p.k_caches[l]),
                         static_cast<uint8_t *>(p.v_caches[l])};
    const size_t first = ((size_t)b * p.Hkv + kvh) * p.P_max;
    auto row_bytes = [&](int i) {  // byte offset of cache row i
        const size_t row = p.block_table ? ((size_t)sm.pages[i / kPageRows] * p.Hkv + kvh) * kPageRows + i % kPageRows : first + i;
        return row * (p.D * 2);
    };
    const int per_row = vn * nx, bits = 31 - __clz(per_row);  // (powers of two)
    constexpr int U = 8;
    for (int i0 = 0; i0 < rows * per_row; i0 += U * THREADS) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int it = i0 + u * THREADS + tid;
            if (it < rows * per_row) {
                const int c = it & (per_row - 1);
                v[u] = *reinterpret_cast<const uint4 *>(cache[c >= vn] + row_bytes(source(it >> bits)) +
                                                        (v0 + (c & (vn - 1))) * 16);
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int it = i0 + u * THREADS + tid;
            if (it < rows * per_row) {
                const int c = it & (per_row - 1);
                *reinterpret_cast<uint4 *>(cache[c >= vn] + row_bytes(target(it >> bits)) +
                                           (v0 + (c & (vn - 1))) * 16) = v[u];
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
    // The images of a head's masses are held in shared memory where the longest sequence's fit: in a CTA's part, if few
    // CTAs run, in half an SM's elsewhere, so that two CTAs share one.  Otherwise those of sequences of up to 8192
    // candidates are, and longer ones read the masses again in every pass, from the L1 that is left.  The capacity decides,
    // as the lengths are on the device.  Measured with the masses' copy beside it, held in a whole SM's part and not held:
    // one head of capacity 20032, 20000 -> 12000 rows: 34 and 46 us; of 40064, 40000 -> 39992 rows: 34 and 95; 8 heads of
    // it: 35 and 96; but also 9 heads of it, which are not held: 35 and 98, and 128 heads: 75 and 133.  Where caches are
    // short against their capacity it is the other way round: 288 heads of capacity 32768, 4104 -> 4096 rows: 32.6 and 27.1;
    // 32768 -> 4096 rows: 348 and 302; 20000 -> 19992 rows: 48 and 65.
    constexpr int kPairBytes = 100 * 1024;  // with EvictSmem and the reserved KB less than half of 228 KB
    const int most = max(0, p.P_max - p.recent - p.sink);
    const int room = (heads * C <= 64 ? kSmemBytes : kPairBytes) / 4 - cap;
    const int keys_held = most <= room ? most : 8192;
    const int smem = 4 * cap + 4 * keys_held;
    cudaError_t e = allow_shared_memory<evict_kernel>(kSmemBytes);
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
    e = cudaLaunchKernelEx(&cfg, evict_kernel, p, C, cap, keys_held);
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
