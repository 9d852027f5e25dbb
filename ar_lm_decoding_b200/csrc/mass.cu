// Attention mass of the cache rows (sm_100a, tcgen05): w(n) = sum over the newest rows' queries q of 2^(q k_n scale' -
// lse'), the column sums of the softmax, for all layers in one launch.
//
// The products are taken as S^T = K Q^T: 128 keys are the rows of a tile (the lanes of TMEM) and up to 128 queries its
// columns, so that a key's weights are summed by one thread in a fixed order and written by it alone: no atomics, no
// exchange.  A key tile feeds all its queries from one read of K: up to 128 queries stay in shared memory while a CTA's
// run of key tiles streams by; more take turns against four key tiles that stay there meanwhile (so that the next turn's
// queries arrive while this turn's weights are summed: by estimate 1.5 us of latency against 2 us of work).
//
// Work: the key tiles of all (layer, sequence, KV head) form one line, cut into equal shares of cost, one per CTA (every
// SM the same work, whatever the lengths).  The pointers of the layers are on the device, so K comes by cp.async into the
// swizzled layout, not through tensor maps.
//
// A CTA (13 warps): warps 0-3 and 4-7 take the sums of every other key tile, warps 8-11 copy (K tiles through a ring of 4
// to 8, Q through two buffers), warp 12 issues the MMAs into two TMEM buffers for each half of the summing warps.
//
// Bound by the bytes of K up to about 175 queries per key at D = 128 (a tile's 32 KB take an SM's share of HBM as long as
// 128 x 175 exponentials its MUFU) and 88 at D = 64, by the exponentials above.
#include "cache_ops.cuh"
#include "tc.cuh"

namespace tidar {

namespace {

constexpr int TM = 128;       // keys of a tile
constexpr int TQ = 128;       // queries of a turn
constexpr int THREADS = 416;
constexpr int COPIERS = 128;  // threads of warps 8-11
constexpr int GROUP = 4;      // key tiles that stay for several turns (at most the ring)
constexpr int kBytesCost = 176;  // cost of a tile that is bound by its bytes, in queries (at D = 64 too, where 88 would be it)
constexpr int kSkip = 1 << 30;                   // in rows[b]: a page out of range

template <int D>
struct Smem {
    static constexpr int K_TILE = TM * D * 2;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int Q_BUF = TQ * D * 2;
    static constexpr int K_OFF = 2 * Q_BUF;
    static constexpr int LSE_OFF = K_OFF + STAGES * K_TILE;  // float[4 turns][TQ]: -lse in log2 units
    static constexpr int BAR_OFF = LSE_OFF + 4 * TQ * 4;
    // k_full[STAGES], k_empty[STAGES], q_full[2], q_empty[2], d_full[4], d_empty[4], l_full[4], l_empty[4], fin, stall
    static constexpr int NBARS = 2 * STAGES + 22;
    static constexpr int MISC_OFF = BAR_OFF + (NBARS * 8 + 15) / 16 * 16;
    static constexpr int SEQ_OFF = MISC_OFF + 16;  // long long cum[B + 1], int tiles[B], int rows[B]
    static int alloc(int B) { return SEQ_OFF + (B + 1) * 8 + B * 8 + 1024; }
};
static_assert(Smem<128>::SEQ_OFF + (kMaxBatchShared + 1) * 16 + 1024 <= 227 * 1024 &&
                  Smem<64>::SEQ_OFF + (kMaxBatchShared + 1) * 16 + 1024 <= 227 * 1024,
              "shared memory beyond 227 KB");

__device__ __forceinline__ int tile_cost(int queries) { return min(max(queries, kBytesCost), 1 << 16); }

// A run of key tiles [t0, t1) of one head, as a CTA works on it.
struct Run {
    int l, b, h, t0, t1;
};

// Walks a CTA's runs.  cum[b]: cost of one KV head's tiles of the sequences before b; the line goes layer by layer,
// sequence by sequence, head by head.
struct Walker {
    const long long *cum;
    const int *tiles, *rows;
    int L, B, Hkv, G;
    __device__ int cost_of(int seq) const { return tile_cost((rows[seq] & ~kSkip) * G); }
    int l, b, h;
    int t;             // first tile of the next run
    long long pos, x1; // position of that tile, end of the share
    __device__ void start(const MassParams &p, const long long *c, const int *ti, const int *ro, int cta, int n) {
        cum = c;
        tiles = ti;
        rows = ro;
        L = p.L;
        B = p.B;
        Hkv = p.Hkv;
        G = p.G;
        const long long layer = cum[B] * Hkv, total = layer * L;
        auto cut = [&](int i) { return total / n * i + (total % n * i + n - 1) / n; };
        pos = cut(cta);
        x1 = cut(cta + 1);
        l = b = h = t = 0;
        if (pos >= x1) return;
        l = (int)(pos / layer);
        const long long in = pos - l * layer;
        int lo = 0, hi = B;  // the sequence that holds the position
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] * Hkv <= in) lo = mid;
            else hi = mid;
        }
        b = lo;
        const long long rest = in - cum[b] * Hkv, head = cum[b + 1] - cum[b];
        const int cost = cost_of(b);
        h = (int)(rest / head);
        t = (int)((rest - h * head + cost - 1) / cost);  // the first tile that begins at or behind the cut
        pos = l * layer + cum[b] * Hkv + h * head + (long long)t * cost;
    }
    __device__ bool next(Run &r) {
        while (pos < x1) {
            const int n = tiles[b], cost = cost_of(b);
            const long long left = (x1 - pos + cost - 1) / cost;
            r = Run{l, b, h, t, (int)min((long long)n, t + left)};
            pos += (long long)(n - t) * cost;
            t = 0;
            if (++h == Hkv) {
                h = 0;
                do {
                    if (++b == B) {
                        b = 0;
                        ++l;
                    }
                } while (l < L && tiles[b] == 0);
            }
            if (r.t0 < r.t1) return true;
        }
        return false;
    }
};

__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Whether the phase has completed, without the wait of a try (which may hold the thread for microseconds).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P1;\n\tmbarrier.test_wait.parity.shared::cta.b64 P1, [%1], %2;\n\tselp.b32 %0, 1, 0, P1;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool read) {  // zeros where it does not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) mass_kernel(const MassParams p) {
    using L = Smem<D>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem), sK = sbase + L::K_OFF, bar0 = sbase + L::BAR_OFF;
    auto k_full = [&](int s) { return bar0 + 8u * s; };
    auto k_empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto q_full = [&](int i) { return bar0 + 8u * (2 * STAGES + i); };
    auto q_empty = [&](int i) { return bar0 + 8u * (2 * STAGES + 2 + i); };
    auto d_full = [&](int i) { return bar0 + 8u * (2 * STAGES + 4 + i); };
    auto d_empty = [&](int i) { return bar0 + 8u * (2 * STAGES + 8 + i); };
    auto l_full = [&](int i) { return bar0 + 8u * (2 * STAGES + 12 + i); };
    auto l_empty = [&](int i) { return bar0 + 8u * (2 * STAGES + 16 + i); };
    const uint32_t fin = bar0 + 8u * (2 * STAGES + 20), stall = fin + 8u;  // (nothing arrives on stall: timeout test)
    float *nlse = reinterpret_cast<float *>(smem + L::LSE_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::MISC_OFF + 4);
    long long *cum = reinterpret_cast<long long *>(smem + L::SEQ_OFF);
    int *tiles = reinterpret_cast<int *>(cum + p.B + 1), *rows = tiles + p.B;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long wl = p.wait_cycles;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(k_full(s), COPIERS);
            tc::mbar_init(k_empty(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full(i), COPIERS);
            tc::mbar_init(q_empty(i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(d_full(i), 1);
            tc::mbar_init(d_empty(i), 128);
            tc::mbar_init(l_full(i), COPIERS);
            tc::mbar_init(l_empty(i), 8);  // the summing warps
        }
        tc::mbar_init(fin, 1);
        tc::mbar_init(stall, 1);
        *abort_flag = 0;
        tc::mbar_fence_init();
    }
    if (warp == 12) tc::tmem_alloc(smem_u32(tmem_slot), 512);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // the line; a sequence whose length or row count is out of range has no tiles
    if (warp == 0) {
        long long sum = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int x = 0, a = 0;
            if (b < p.B) {
                const int N = p.prefix_len[b];
                a = p.row_count ? p.row_count[b] : p.R;
                int bits = 0;
                if (N < 0 || N > p.P_max) bits = TIDAR_DEV_BAD_PREFIX;
                else if (a < 0 || a > p.R || a > N) bits = TIDAR_DEV_BAD_ACCEPT;
                if (bits && blockIdx.x == 0) atomicOr(p.dev_status, bits);
                // (no rows: the sums only decay, below)
                x = bits || a == 0 ? 0 : ceil_div(N, TM);
                if (bits) a = 0;
                tiles[b] = x;
                rows[b] = a;
            }
            long long inc = (long long)x * tile_cost(a * p.G);
            const long long own = inc;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (b < p.B) cum[b] = sum + inc - own;
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) cum[p.B] = sum;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tmem_slot;
    const int cta = blockIdx.x, ncta = gridDim.x;
    Walker walk;
    walk.start(p, cum, tiles, rows, cta, ncta);
    // Paged caches: the CTA looks over the pages of the sequences of its share; one with a page out of range is skipped.
    if (p.block_table && walk.pos < walk.x1) {
        Walker end = walk;
        Run r;
        int b0 = p.B, b1 = -1, first = walk.l;
        while (end.next(r)) {
            if (r.l != first || b1 - b0 >= p.B) {  // (into another layer: every sequence, perhaps)
                b0 = 0;
                b1 = p.B - 1;
                break;
            }
            b0 = min(b0, r.b);
            b1 = max(b1, r.b);
        }
        for (int b = b0; b <= b1; ++b) {
            if (tiles[b] == 0) continue;  // (uniform over the block)
            if (block_bad_page(p.block_table + (size_t)b * p.max_pages, p.prefix_len[b], p.num_pages) && tid == 0) {
                rows[b] |= kSkip;
                atomicOr(p.dev_status, TIDAR_DEV_BAD_PAGE);
            }
        }
        __syncthreads();
    }
    auto skipped = [&](const Run &r) { return (rows[r.b] & kSkip) != 0; };
    // Queries take `turns` of TQ; with more than one, each against a group of key tiles.
    auto turns = [&](int a) { return ceil_div(a * p.G, TQ); };
    auto group = [&](const Run &r, int nturn) { return nturn == 1 ? r.t1 - r.t0 : GROUP; };

    if (warp < 8) {
        // ================= sums: warpgroup w takes every other tile; thread = key =================
        const int w = warp >> 2, q4 = warp & 3, row = q4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint64_t sl2 = pair(p.scale_log2, p.scale_log2);
        int turn = 0, run = 0, taken = 0;  // turns, runs, this warpgroup's products
        bool ok = true;
        Run r;
        while (ok && walk.next(r)) {
            if (skipped(r)) continue;
            const int flip = (run++ ^ w) & 1;
            const int N = p.prefix_len[r.b], a = rows[r.b], nturn = turns(a), gs = group(r, nturn);
            float *mass = p.masses[r.l] + ((size_t)r.b * p.Hkv + r.h) * p.P_max;
            for (int g0 = r.t0; g0 < r.t1 && ok; g0 += gs) {
                const int g1 = min(g0 + gs, r.t1);
                uint64_t sums[GROUP / 2][4];  // of this warpgroup's tiles of the group, over the turns
#pragma unroll
                for (int j = 0; j < GROUP / 2 * 4; ++j) sums[j / 4][j % 4] = 0;
                for (int c = 0; c < nturn && ok; ++c, ++turn) {
                    const int ls = turn & 3, nq = min(TQ, a * p.G - c * TQ), chunks = ceil_div(nq, 32);
                    const float *nl = nlse + ls * TQ;
                    // (also without a tile: the arrival below is for this turn)
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(l_full(ls), (turn >> 2) & 1, abort_flag, wl));
                    auto tile = [&](int t, uint64_t(&sum)[4]) {
                        const int key = t * TM + row, buf = 2 * w + (taken & 1);
                        const uint32_t d_col = tbase + lane_off + buf * TQ;
                        const bool mine = key < N, last = c == nturn - 1;
                        float old = 0.f;
                        if (mine && last && key < N - a) old = mass[key];
                        ok = __all_sync(0xffffffffu, tc::mbar_wait(d_full(buf), (taken >> 1) & 1, abort_flag, wl));
                        if (!ok) return;  // (TMEM accesses are warp-wide)
                        ++taken;
                        tc::fence_after_sync();
                        // a newest row n sees only itself and what follows: queries of rows j >= n - (N - a)
                        const int cmin = max(0, (key - (N - a)) * p.G - c * TQ);
                        const bool cut = t * TM + TM > N - a;
                        for (int x = 0; x < chunks; ++x) {
                            uint32_t u[32];
                            tc::tmem_ld32(d_col + x * 32, u);
                            uint64_t nl2[16];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const ulonglong2 v = reinterpret_cast<const ulonglong2 *>(nl + x * 32)[j];
                                nl2[2 * j] = v.x;
                                nl2[2 * j + 1] = v.y;
                            }
                            tc::tmem_wait_ld();
                            if (x == chunks - 1) {
                                tc::fence_before_sync();
                                tc::mbar_arrive(d_empty(buf));
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float e, f;
                                unpair(fma2(pair(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), sl2, nl2[j]), e, f);
                                e = fast_exp2(e);
                                f = fast_exp2(f);
                                if (cut) {  // by select: a masked weight may be anything
                                    e = x * 32 + 2 * j >= cmin ? e : 0.f;
                                    f = x * 32 + 2 * j + 1 >= cmin ? f : 0.f;
                                }
                                sum[j & 3] = add2(sum[j & 3], pair(e, f));
                            }
                        }
                        if (last) {
                            float e, f;
                            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), e, f);
                            if (mine) mass[key] = key < N - a ? fmaf(p.decay, old, e + f) : e + f;
#pragma unroll
                            for (int j = 0; j < 4; ++j) sum[j] = 0;
                        }
                    };
                    if (nturn == 1) {
                        for (int t = g0 + flip; t < g1 && ok; t += 2) tile(t, sums[0]);
                    } else {
#pragma unroll
                        for (int j = 0; j < GROUP / 2; ++j)
                            if (g0 + flip + 2 * j < g1 && ok) tile(g0 + flip + 2 * j, sums[j]);
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(l_empty(ls));
                }
            }
        }
        // sequences without new rows: their sums decay
        if (p.decay != 1.f) {
            const long heads = (long)p.L * p.B * p.Hkv;
            for (long hd = cta; hd < heads; hd += ncta) {
                const int h = (int)(hd % p.Hkv), b = (int)(hd / p.Hkv % p.B), l = (int)(hd / p.Hkv / p.B);
                const int N = p.prefix_len[b];
                if (N <= 0 || N > p.P_max || !p.row_count || p.row_count[b] != 0) continue;
                float *mass = p.masses[l] + ((size_t)b * p.Hkv + h) * p.P_max;
                for (int i = tid; i < N; i += 256) mass[i] *= p.decay;
            }
        }
    } else if (warp < 12) {
        // ================= copies =================
        const int ct = tid - 256;
        constexpr int CH = D / 8, RW = COPIERS / CH;  // 16-byte chunks of a row; rows of one sweep (a multiple of 8)
        const int c16 = ct % CH, r0 = ct / CH;
        const uint32_t dst0 = (c16 >> 3) * TM * 128 + r0 * 128 + (((c16 & 7) ^ (r0 & 7)) << 4);
        int it = 0, turn = 0;  // K tiles, turns
        // Every K tile and every Q is one copy group; it is announced once at most LAG younger ones are under way.
        constexpr int LAG = STAGES - 2;
        uint32_t codes = 0;  // the groups under way, youngest in the low four bits: a K stage, or 8 + turn % 4
        int under_way = 0;
        uint32_t has_lse = 0;  // bit turn % 4: this thread copies an LSE of the turn
        auto announce = [&](int keep) {
            tc::fence_proxy_async_smem();
            for (; under_way > keep; --under_way) {
                const int code = codes >> (4 * (under_way - 1)) & 15;
                if (code >= 8) {  // the LSE that this thread copied
                    float *x = nlse + (code - 8) * TQ + ct;
                    *x = has_lse >> (code - 8) & 1 ? -*x * kLog2e : -INFINITY;
                    tc::mbar_arrive(l_full(code - 8));
                }
                tc::mbar_arrive(code < 8 ? k_full(code) : q_full(code & 1));
            }
        };
        auto close = [&](int code) {
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            codes = codes << 4 | code;
            if (++under_way > LAG) {
                asm volatile("cp.async.wait_group %0;\n" ::"n"(LAG) : "memory");
                announce(LAG);
            }
        };
        // a place that is not free yet may wait for what is under way
        auto wait_free = [&](uint32_t bar, uint32_t ph) {
            while (!mbar_test(bar, ph)) {
                if (under_way == 0) return tc::mbar_wait(bar, ph, abort_flag, wl);
                switch (under_way - 1) {  // the oldest of them
                    case 0: asm volatile("cp.async.wait_group 0;\n" ::: "memory"); break;
                    case 1: asm volatile("cp.async.wait_group 1;\n" ::: "memory"); break;
                    case 2: asm volatile("cp.async.wait_group 2;\n" ::: "memory"); break;
                    case 3: asm volatile("cp.async.wait_group 3;\n" ::: "memory"); break;
                    case 4: asm volatile("cp.async.wait_group 4;\n" ::: "memory"); break;
                    default: asm volatile("cp.async.wait_group 5;\n" ::: "memory"); break;
                }
                announce(under_way - 1);
            }
            return true;
        };
        bool ok = true;
        Run r;
        while (ok && walk.next(r)) {
            if (skipped(r)) continue;
            const int N = p.prefix_len[r.b], a = rows[r.b], nturn = turns(a), gs = group(r, nturn);
            const uint8_t *kc = static_cast<const uint8_t *>(p.k_caches[r.l]);
            const uint8_t *q = static_cast<const uint8_t *>(p.qs[r.l]) + ((size_t)r.b * p.R * p.Hq + r.h * p.G) * D * 2;
            const float *lse = p.lses[r.l] + (size_t)r.b * p.R * p.Hq + r.h * p.G;
            for (int g0 = r.t0; g0 < r.t1 && ok; g0 += gs) {
                const int g1 = min(g0 + gs, r.t1);
                for (int c = 0; c < nturn && ok; ++c, ++turn) {
                    const int qb = turn & 1, nq = min(TQ, a * p.G - c * TQ);
                    const int ls = turn & 3;
                    if (turn >= 2) ok = wait_free(q_empty(qb), ((turn >> 1) - 1) & 1);
                    if (ok && turn >= 4) ok = wait_free(l_empty(ls), ((turn >> 2) - 1) & 1);
                    if (!ok) break;
                    {  // query c TQ + x is row j, head gq; places past the last query repeat it (with -inf for its LSE: a
                       // zero row would make a NaN of an infinity in K, and the last query sees every key that one does)
                        const int e = c * TQ + nq - 1, je = e / p.G;
                        const uint8_t *end = q + ((size_t)je * p.Hq + e - je * p.G) * (D * 2) + c16 * 16;
                        int j = (c * TQ + r0) / p.G, gq = c * TQ + r0 - j * p.G;
                        const uint8_t *at = q + ((size_t)j * p.Hq + gq) * (D * 2) + c16 * 16;
                        const uint32_t dst = sbase + qb * L::Q_BUF + dst0 - r0 * 128;
                        for (int x = r0; x < (nq + 31) / 32 * 32; x += RW) {
                            copy16(dst + x * 128, x < nq ? at : end);
                            at += RW * D * 2;
                            for (gq += RW; gq >= p.G; gq -= p.G) at += (size_t)(p.Hq - p.G) * (D * 2);
                        }
                    }
                    {
                        const int i = c * TQ + ct, j = i / p.G, gq = i - j * p.G;
                        if (ct < nq)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(
                                             sbase + L::LSE_OFF + (ls * TQ + ct) * 4),
                                         "l"(lse + (size_t)j * p.Hq + gq)
                                         : "memory");
                        has_lse = (has_lse & ~(1u << ls)) | (uint32_t)(ct < nq) << ls;
                    }
                    close(8 + ls);
                    if (c > 0) continue;
                    for (int t = g0; t < g1; ++t, ++it) {
                        const int st = it % STAGES;
                        if (it >= STAGES) ok = wait_free(k_empty(st), (it / STAGES - 1) & 1);
                        if (!ok) break;
                        const uint32_t dst = sK + st * L::K_TILE + dst0;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int n0 = t * TM + half * kPageRows;
                            size_t first = ((size_t)r.b * p.Hkv + r.h) * p.P_max + n0;
                            if (p.block_table)  // (a page of rows past the end is not read)
                                first = ((size_t)(n0 < N ? p.block_table[(size_t)r.b * p.max_pages + n0 / kPageRows] : 0) *
                                             p.Hkv + r.h) * kPageRows;
                            const uint8_t *src = kc + first * (D * 2) + c16 * 16;
                            const uint8_t *at = src + r0 * (D * 2);
                            if (n0 + kPageRows <= N) {  // (constant offsets: one instruction a copy)
#pragma unroll
                                for (int x = 0; x < kPageRows; x += RW)
                                    copy16(dst + (half * kPageRows + x) * 128, at + x * (D * 2));
                            } else {
#pragma unroll 1
                                for (int x = 0; x < kPageRows; x += RW) {
                                    const bool read = n0 + x + r0 < N;
                                    copy16(dst + (half * kPageRows + x) * 128, read ? at + x * (D * 2) : kc, read);
                                }
                            }
                        }
                        close(st);
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");  // (nothing may land after the CTA exits)
        if (ok) announce(0);
    } else {
        // ================= MMA issue =================
        const bool one = lane == 0;
        const uint64_t dk = tc::smem_desc_sw128(sK, 16, 1024), dq = tc::smem_desc_sw128(sbase, 16, 1024);
        int it = 0, turn = 0, run = 0, used[2] = {0, 0};  // K tiles, turns, runs, products of each summing half
        bool ok = !one || !p.stall_test || tc::mbar_wait(stall, 0, abort_flag, wl);
        Run r;
        while (one && ok && walk.next(r)) {
            if (skipped(r)) continue;
            const int a = rows[r.b], nturn = turns(a), gs = group(r, nturn), flip = run++ & 1;
            for (int g0 = r.t0; g0 < r.t1 && ok; g0 += gs) {
                const int g1 = min(g0 + gs, r.t1);
                for (int c = 0; c < nturn && ok; ++c, ++turn) {
                    const int qb = turn & 1, nq = min(TQ, a * p.G - c * TQ);
                    const uint32_t id = tc::idesc_bf16_f32(TM, ceil_div(nq, 32) * 32, 0, 0);
                    ok = tc::mbar_wait(q_full(qb), (turn >> 1) & 1, abort_flag, wl);
                    for (int t = g0; t < g1 && ok; ++t) {
                        const int i = it + t - g0, st = i % STAGES, w = (t - g0 + flip) & 1;
                        const int nu = w ? used[1]++ : used[0]++, buf = 2 * w + (nu & 1);
                        if (nu >= 2) ok = tc::mbar_wait(d_empty(buf), ((nu >> 1) - 1) & 1, abort_flag, wl);
                        if (ok && c == 0) ok = tc::mbar_wait(k_full(st), (i / STAGES) & 1, abort_flag, wl);
                        if (!ok) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t ka = (uint64_t)(kk >> 2) * ((TM * 128) >> 4) + (kk & 3) * 2;
                            const uint64_t qa = (uint64_t)(kk >> 2) * ((TQ * 128) >> 4) + (kk & 3) * 2;
                            tc::mma_ss(tbase + buf * TQ, dk + (uint64_t)st * (L::K_TILE >> 4) + ka,
                                       dq + (uint64_t)qb * (L::Q_BUF >> 4) + qa, id, kk > 0 ? 1u : 0u);
                        }
                        tc::mma_commit(d_full(buf));
                        if (c == nturn - 1) tc::mma_commit(k_empty(st));
                    }
                    if (ok) tc::mma_commit(q_empty(qb));
                }
                it += g1 - g0;
            }
        }
        if (one) {
            tc::mma_commit(fin);  // every MMA completes before TMEM is freed
            tc::mbar_wait_drain(fin, 0, kCacheWaitCycles);
        }
        __syncwarp();
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 12) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, 512);
    }
    if (tid == 0 && *abort_flag) atomicOr(p.dev_status, TIDAR_DEV_TIMEOUT);
}

template <int D>
cudaError_t launch(const MassParams &p, cudaStream_t s) {
    const int smem = Smem<D>::alloc(p.B);
    cudaError_t e = allow_shared_memory<mass_kernel<D>>(Smem<D>::alloc(kMaxBatchShared));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kNumSMs, 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, mass_kernel<D>, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t mass_launch(const MassParams &p, cudaStream_t s) {
    return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

}  // namespace tidar
