// Attention of a batch behind one shared prefix (sm_100a: TMA + tcgen05, TMEM accumulators).
//
// out = softmax(scale q [K_shared | K_own | K_new]^T) [V_shared | V_own | V_new] is a sum over disjoint key sets, so it
// is computed per set and joined by the sets' log-sum-exps: with (O_s, lse_s) a normalised partial row,
// O = sum_s w_s O_s, w_s = exp(lse_s - lse), lse = log sum_s exp(lse_s).
//
// Work: a row tile is RT = floor(128 / G) rows (b, r) times the G query heads of one KV head.  Against the shared keys
// the rows of all sequences are packed into row tiles together (that is what sharing buys: B R G rows multiply each
// shared K/V byte); against its own cache and the new keys each sequence has row tiles of its own.  A block is two row
// tiles (the last may be one) with all their key tiles of 128.  The blocks' key tiles form one line (per KV head: the
// shared blocks, then each sequence's own), which is cut into equal shares of cost, one per CTA: every SM gets the same
// work whatever the lengths, and a CTA's share is a few segments (block, run of key tiles).  Each segment leaves one
// partial record; combine_kernel joins a row's records in a fixed order.  The line and its cuts follow from the lengths
// alone, which every CTA reads on the device, so nothing waits on the host and nothing on timing.
//
// A CTA (12 warps): warp 0 streams K and V tiles by TMA through one ring; warp 2 walks the line, hands out the segments
// and loads Q; warps 1 and 3 issue the MMAs of row tile 0 and 1; warps 4-7 and 8-11 are the softmax of row tile 0 and 1
// (thread = row = TMEM lane).  The two row tiles share each K/V tile and are independent otherwise, so the tensor cores
// multiply for one while the other exponentiates.
// A key tile is taken in halves of 64 keys.  TMEM: S of row tile t in two buffers [128t, 128t + 64) and [128t + 64,
// 128t + 128), O at [256 + D t, 256 + D t + D); P (bf16) overwrites the first 32 columns of its S.  S of half u + 2 is
// issued once the PV of half u, the last reader of that buffer, has completed, while the softmax works on half u + 1:
// the round trip P -> PV -> next S is off its path.  (Whole tiles of 128 keys in one buffer each, as TMEM holds no more
// at D = 128, left the softmax waiting 2,240 of 4,395 cycles per tile on that round trip.)
//
// Scaling and sums use the packed fp32 pair instructions (64 values per thread, two warps per sub-partition, measured
// alone: 1,224 cycles scalar, 1,126 packed, of which the MUFU's ex2 are about 1,000).
#include "cache_ops.cuh"
#include "tc.cuh"

namespace tidar {

namespace {

constexpr int TM = 128;
constexpr int TN = 128;
constexpr int TH = 64;  // keys of half a tile
constexpr int THREADS = 384;
constexpr int BOXR = kPageRows;
// Cost of one key tile for a block of two row tiles and of one, and of a block's start and end (Q, the record), where
// every CTA has a few tiles (see Line): measured ~3,300, ~2,900 and ~4,200 cycles, the ratio then tuned on the whole call
// (8 x Qwen3-8B k 8: 69.5 us with 3 : 2 : 2, 62.3 with 8 : 7 : 10, 62.6 with 8 : 6 : 12; 16 single-token rows: 22.3, 21.5,
// 21.5 us; 32 of them with 100 to 2000 rows of their own: 42.8, 41.6, 47.8; 16 x k 8, G 6, D 64: 41.3, 38.0, 37.1).
constexpr int kLongBlock = 6;  // key tiles from which a block of a short line has two tiles a CTA
constexpr int kCostPair = 8, kCostSingle = 6, kCostBlock = 12;

// The line of key tiles (cum[b], beside it: key tiles of the sequences before b, nseq[b]: sequences before b that have
// any).  Every CTA's share is at least the cost of one tile, so the CTAs from a block's first tile to its last all have
// a part of it: where there are too few tiles for that every tile costs 1 and as many CTAs work as there are tiles, or
// half as many where a block has many of them, so that its rows have fewer records to join (8 x Qwen2.5-1.5B k 4: blocks of
// 5 tiles take 15.0 us with a CTA per tile and 16.8 with one per two, of 6 tiles 16.7 and 14.2, of 9 tiles 20.4 and 18.6; two
// single-token rows of Qwen3-8B, 5 tiles: 11.9 and 13.6, 6 tiles: 12.5 and 12.0, 8 tiles: 15.7 and 12.3).
struct Line {
    int total;               // cost of all KV heads
    int head;                // cost of one KV head
    int shared;              // of its shared blocks
    int shared_tiles;        // key tiles of the shared prefix
    int pair, single, block; // cost of a key tile for two row tiles, for one, and of a block beside its tiles
    int ncta;                // CTAs that work
};

__host__ __device__ __forceinline__ int rows_per_tile(int G) { return TM / G; }
// The workspace: (first, last) CTA of every block, whether a sequence's pages (and, last, the shared ones) are all in
// range, then the records.
__host__ __device__ __forceinline__ size_t info_bytes(size_t blocks, int B) { return align256(blocks * 8 + (size_t)B * 4 + 4); }
// One record: two row tiles, each [D/8 chunks][128 rows] 16-byte chunks of 8 fp16 and a header [128 rows] (log2 of the
// row's sum, scale of its values).
__host__ __device__ __forceinline__ size_t tile_record_bytes(int D) { return (size_t)TM * (D * 2 + 8); }

struct Geometry {
    int RT, shared_rt, shared_blocks, own_rt, own_blocks, blocks;  // (rt: row tiles; per KV head)
};
__host__ __device__ __forceinline__ Geometry geometry(int B, int R, int G) {
    Geometry g;
    g.RT = rows_per_tile(G);
    g.shared_rt = ceil_div(B * R, g.RT);
    g.shared_blocks = ceil_div(g.shared_rt, 2);
    g.own_rt = ceil_div(R, g.RT);
    g.own_blocks = ceil_div(g.own_rt, 2);
    g.blocks = g.shared_blocks + B * g.own_blocks;
    return g;
}

// First position of CTA c of n on a line of length total: the position s belongs to CTA floor(s n / total).
__device__ __forceinline__ int cut(int total, int c, int n) {
    const int q = total / n, r = total - q * n;
    return q * c + (r * c + n - 1) / n;
}

// A block of the line: `tiles` key tiles of cost `w` each from position `start`, the first of cost block + w.
struct Block {
    int start, tiles, w;
};
// Cost of n row tiles' blocks against `tiles` key tiles.
__device__ __forceinline__ int blocks_cost(const Line &ln, int n, int tiles) {
    return (n / 2) * (ln.block + tiles * ln.pair) + (n & 1) * (ln.block + tiles * ln.single);
}
// Tiles [i0, i1) of a block whose positions fall in [x0, x1).
__device__ __forceinline__ int first_tile(const Line &ln, const Block &bl, int x) {
    const int a = x - bl.start;
    return a <= 0 ? 0 : min(max(1, (a - ln.block + bl.w - 1) / bl.w), bl.tiles);
}

// One run of key tiles of one block, as a CTA works on it.
struct __align__(16) Segment {
    int kvh, b;      // b = -1: shared
    int i0, i1;      // key tiles
    int row0;        // first row (of the sequence, or of the batch) of the block's first row tile
    int nt;          // row tiles (1 or 2; 0: no more segments)
    int id;          // block
    int len;         // cached keys (the shared or the sequence's own length)
};

// Walks the segments of a CTA's share [x0, x1).
struct Walker {
    const Line &ln;
    const Geometry &g;
    const int *cum, *nseq;
    int B, cta, x0, x1, pos;
    bool last;  // the segment ends its block
    __device__ Walker(const Line &l, const Geometry &ge, const int *c, const int *ns, int B_, int cta_)
        : ln(l), g(ge), cum(c), nseq(ns), B(B_), cta(cta_) {
        x0 = pos = cta < l.ncta ? cut(l.total, cta_, l.ncta) : 0;
        x1 = cta < l.ncta ? cut(l.total, cta_ + 1, l.ncta) : 0;
    }
    // cost of the own blocks of the sequences before b
    __device__ int own_before(int b) const {
        return cum[b] * ((g.own_rt / 2) * ln.pair + (g.own_rt & 1) * ln.single) + nseq[b] * g.own_blocks * ln.block;
    }
    __device__ bool next(Segment &s) {
        while (pos < x1) {
            const int kvh = pos / ln.head, rem = pos - kvh * ln.head;
            Block bl;
            int rt, j;
            s.kvh = kvh;
            if (rem < ln.shared) {
                rt = g.shared_rt;
                bl.tiles = ln.shared_tiles;
                const int per = ln.block + bl.tiles * ln.pair;
                j = rem / per;
                bl.start = kvh * ln.head + j * per;
                s.b = -1;
                s.id = kvh * g.blocks + j;
            } else {
                int lo = 0, hi = B;  // the sequence whose blocks hold the position
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (own_before(mid) <= rem - ln.shared) lo = mid;
                    else hi = mid;
                }
                rt = g.own_rt;
                bl.tiles = cum[lo + 1] - cum[lo];
                const int per = ln.block + bl.tiles * ln.pair, at = own_before(lo);
                j = (rem - ln.shared - at) / per;
                bl.start = kvh * ln.head + ln.shared + at + j * per;
                s.b = lo;
                s.id = kvh * g.blocks + g.shared_blocks + lo * g.own_blocks + j;
            }
            s.nt = 2 * j + 1 < rt ? 2 : 1;
            s.row0 = 2 * j * g.RT;
            bl.w = s.nt == 2 ? ln.pair : ln.single;
            s.i0 = first_tile(ln, bl, x0);
            s.i1 = first_tile(ln, bl, x1);
            last = s.i1 == bl.tiles;
            pos = bl.start + ln.block + bl.tiles * bl.w;
            if (s.i0 < s.i1) return true;
        }
        s.nt = 0;
        return false;
    }
};
constexpr int SEGS = 4;                // segments the scheduler keeps ahead
constexpr int kSegReaders = 3 + 8;     // the K/V and MMA warps and the softmax warps

template <int D>
struct Smem {
    static constexpr int Q_TILE = TM * D * 2;
    static constexpr int KV_TILE = TN * D * 2;
    static constexpr int STAGES = D == 128 ? 4 : 8;  // one K or V tile each
    static constexpr int KV_OFF = 2 * Q_TILE;
    static constexpr int BAR_OFF = KV_OFF + STAGES * KV_TILE;
    // full[STAGES], empty[STAGES], q_full, q_empty, per row tile and S buffer s_full, p_full, pv_done, per row tile
    // o_full, o_free, fin; stall, seg_full[SEGS], seg_empty[SEGS]
    static constexpr int NBARS = 2 * STAGES + 2 + 12 + 6 + 2 + 2 * SEGS;
    static constexpr int SEG_OFF = (BAR_OFF + NBARS * 8 + 63) / 64 * 64;
    static constexpr int LINE_OFF = SEG_OFF + SEGS * (int)sizeof(Segment);
    static constexpr int MISC_OFF = LINE_OFF + 64;
    static constexpr int CUM_OFF = MISC_OFF + 16;  // int[B + 1] three times
    static int alloc(int B) { return CUM_OFF + 3 * (B + 1) * 4 + 1024; }
};
static_assert(sizeof(Line) <= 64, "the line's place in shared memory");
static_assert(Smem<128>::CUM_OFF + 3 * (kMaxBatchShared + 1) * 4 + 1024 <= 227 * 1024 &&
                  Smem<64>::CUM_OFF + 3 * (kMaxBatchShared + 1) * 4 + 1024 <= 227 * 1024,
              "shared memory beyond 227 KB");

// One lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(one));
    return one != 0;
}

// Bit i set iff key base + i lies in [a, b) (i = 0..31).
__device__ __forceinline__ uint32_t range_bits(int a, int b, int base) {
    const int lo = max(a - base, 0), hi = min(b - base, 32);
    if (hi <= lo) return 0u;
    const uint32_t below_hi = hi >= 32 ? 0xffffffffu : ((1u << hi) - 1u);
    return below_hi & ~((1u << lo) - 1u);
}

// S = Q K^T over 64 keys (both K-major, 128-byte swizzle, blocks of 64 columns).
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_s, uint64_t dq, uint64_t dk, uint32_t id) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(kk >> 2) * ((TM * 128) >> 4) + (kk & 3) * 2;
        tc::mma_ss(d_s, dq + off, dk + off, id, kk > 0 ? 1u : 0u);
    }
}
// O (+)= P V over 64 keys: P in TMEM (two bf16 per column), V MN-major.
__device__ __forceinline__ void issue_pv(uint32_t d_o, uint32_t a_p, uint64_t dv, uint32_t id, bool acc) {
#pragma unroll
    for (int kk = 0; kk < TH / 16; ++kk) tc::mma_ts(d_o, a_p + kk * 8, dv + kk * 128, id, (acc || kk > 0) ? 1u : 0u);
}

// Pairs of fp32 in one 64-bit register (the packed instructions round each half as the scalar ones do).
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// The greatest of three; NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The greatest of 64 scores (NaN if one is).
__device__ __forceinline__ float half_max(const uint32_t (&u)[2][32]) {
    float m4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m4[j] = __uint_as_float(u[0][j]);
#pragma unroll
    for (int j = 4; j < 64; j += 2)
        m4[(j >> 1) & 3] = max3_nan(m4[(j >> 1) & 3], __uint_as_float(u[j >> 5][j & 31]),
                                    __uint_as_float(u[j >> 5][(j + 1) & 31]));
    return max3_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]);
}

// 64 scores of this thread's row; those of the keys k0 + j outside [0, lo) and [glo, ghi) become -inf (by select, so that
// they may hold anything).
__device__ __forceinline__ void load_scores(uint32_t sc, uint32_t (&u)[2][32]) {
    tc::fence_after_sync();
    tc::tmem_ld32(sc, u[0]);
    tc::tmem_ld32(sc + 32, u[1]);
    tc::tmem_wait_ld();
}
__device__ __forceinline__ void mask_scores(uint32_t (&u)[2][32], int k0, int lo, int glo, int ghi) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t bits = range_bits(0, lo, k0 + c * 32) | range_bits(glo, ghi, k0 + c * 32);
#pragma unroll
        for (int j = 0; j < 32; ++j) u[c][j] = (bits >> j) & 1u ? u[c][j] : 0xff800000u;
    }
}

// P = 2^(x sl2 + neg_m) of 64 scores as bf16 pairs; returns the sum of the unrounded values.
__device__ __forceinline__ float half_exp(const uint32_t (&u)[2][32], float sl2, float neg_m, uint32_t (&pk)[32]) {
    const uint64_t sc = pair(sl2, sl2), nm = pair(neg_m, neg_m);
    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint64_t x =
            fma2(pair(__uint_as_float(u[j >> 4][(2 * j) & 31]), __uint_as_float(u[j >> 4][(2 * j + 1) & 31])), sc, nm);
        float a, b;
        unpair(x, a, b);
        a = fast_exp2(a);
        b = fast_exp2(b);
        sum[j & 3] = add2(sum[j & 3], pair(a, b));
        pk[j] = pack_bf16x2(a, b);
    }
    float a, b;
    unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
    return a + b;
}

// The weights are 2^(x - m) with m the row's running maximum plus kHeadroom: a maximum that is behind by up to 2^kHeadroom
// leaves a half's weights below 1 in sum, and O below the number of halves times the largest |v|, as weights against the
// true maximum would.  (With weights of up to 2^16, values of 1e33 overflowed.)
constexpr float kHeadroom = 16.f;
constexpr float kMaxHalfSum = 1.f;

// The running max m of a row is raised to the maximum of the half at sc, where the row has none yet or its weights
// against m sum to lt >= kMaxHalfSum (or are not finite), and O and the row's sum l are scaled to it.  (A call of its own: it is
// rare, and inlined it would spread the loop over the instruction cache.)
struct RowState {
    float m, l;
    int ok;
};
template <int D>
__device__ __noinline__ RowState raise_max(uint32_t sc, int k0, int lo, int glo, int ghi, float sl2, float lt, float m, float l,
                                           uint32_t o_col, uint32_t pv_bar, uint32_t pv_phase, volatile int *abort_flag) {
    uint32_t u[2][32];
    load_scores(sc, u);
    mask_scores(u, k0, lo, glo, ghi);
    const float mx = half_max(u) * sl2 + kHeadroom;
    RowState st{m, l, 1};
    if (!(mx < INFINITY)) st.l = __int_as_float(0x7fffffff);  // a score of NaN or infinity: no softmax
    const bool grow = mx > m && mx < INFINITY && (m == -INFINITY || !(lt < kMaxHalfSum));
    const float f = grow && m > -INFINITY ? fast_exp2(m - mx) : 1.f;
    if (__any_sync(0xffffffffu, f < 1.f)) {
        // O is at rest once the last half's PV has completed: the next one awaits this half's P
        st.ok = __all_sync(0xffffffffu, tc::mbar_wait(pv_bar, pv_phase, abort_flag, kCacheWaitCycles));
        if (!st.ok) return st;
        tc::fence_after_sync();
        st.l *= f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tc::tmem_ld32(o_col + c * 32, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
            tc::tmem_st32(o_col + c * 32, v);
        }
    }
    if (grow) st.m = mx;
    return st;
}

// The scale of a record whose largest magnitude is amax, and its reciprocal: the power of two that brings amax to [2^13,
// 2^14), 2^126 at most, so that both are normal numbers whatever amax is (zero and subnormal ones included).
__device__ __forceinline__ float2 record_scale(float amax) {
    const int e = min(267 - (__float_as_int(amax) >> 23), 253);
    return make_float2(__int_as_float(e << 23), __int_as_float((254 - e) << 23));
}

// The record of a row whose O holds an infinity (V does): over its largest finite magnitude, so that the other columns keep
// their values.  (A call of its own: inlined it took 22.2 -> 23.1 us of 16 single-token rows, so 22.2 -> 22.4.)
template <int D>
__device__ __noinline__ void record_beside_infinities(uint32_t o_col, uint8_t *rec, int row, float m, float l) {
    uint32_t v[32];
    float amax = 0.f;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        tc::tmem_ld32(o_col + c * 32, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float x = fabsf(__uint_as_float(v[j]));
            if (x < INFINITY) amax = fmaxf(amax, x);
        }
    }
    const float2 scale = record_scale(amax);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        tc::tmem_ld32(o_col + c * 32, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = pack_half2(__uint_as_float(v[j + 2 * e]) * scale.x, __uint_as_float(v[j + 2 * e + 1]) * scale.x);
            if (rec) reinterpret_cast<uint4 *>(rec)[(c * 4 + j / 8) * TM + row] = make_uint4(h[0], h[1], h[2], h[3]);
        }
        __syncwarp();  // (the next load is the whole warp's)
    }
    if (rec)
        reinterpret_cast<float2 *>(rec + TM * D * 2)[row] =
            make_float2(l == 0.f ? -INFINITY : m + __log2f(l), l == 0.f ? 0.f : scale.y / l);
}

// Keys of key tile kt: P cached keys in TP tiles, then R new ones.
__device__ __forceinline__ int tile_keys(int kt, int P, int TP, int R) {
    return kt < TP ? min(TN, P - kt * TN) : min(TN, R - (kt - TP) * TN);
}

struct Maps {
    CUtensorMap ks, vs, kc, vc, kn, vn, q;
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    shared_attn_kernel(const SharedAttnParams p, const __grid_constant__ Maps maps) {
    using L = Smem<D>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem), sKV = sbase + L::KV_OFF, bar0 = sbase + L::BAR_OFF;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t q_full = bar0 + 8u * (2 * STAGES), q_empty = q_full + 8;
    auto s_full = [&](int t, int b) { return q_full + 16u + 8u * (2 * t + b); };
    auto p_full = [&](int t, int b) { return q_full + 48u + 8u * (2 * t + b); };
    auto pv_done = [&](int t, int b) { return q_full + 80u + 8u * (2 * t + b); };
    auto o_full = [&](int t) { return q_full + 112u + 8u * t; };
    auto o_free = [&](int t) { return q_full + 128u + 8u * t; };
    auto fin = [&](int i) { return q_full + 144u + 8u * i; };
    const uint32_t stall = q_full + 160u;  // nothing arrives here (timeout test)
    auto seg_full = [&](int i) { return q_full + 176u + 8u * i; };
    auto seg_empty = [&](int i) { return q_full + 176u + 8u * (SEGS + i); };
    Segment *segs = reinterpret_cast<Segment *>(smem + L::SEG_OFF);
    Line *line = reinterpret_cast<Line *>(smem + L::LINE_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::MISC_OFF + 4);
    int *cum = reinterpret_cast<int *>(smem + L::CUM_OFF), *nseq = cum + p.B + 1, *lens = nseq + p.B + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Geometry g = geometry(p.B, p.R, p.G);

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(empty(s), 2);  // both MMA issuers
        }
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_empty, 2);
        for (int t = 0; t < 2; ++t) {
            for (int b = 0; b < 2; ++b) {
                tc::mbar_init(s_full(t, b), 1);
                tc::mbar_init(p_full(t, b), 128);
                tc::mbar_init(pv_done(t, b), 1);
            }
            tc::mbar_init(o_full(t), 1);
            tc::mbar_init(o_free(t), 128);
        }
        for (int i = 0; i < 2; ++i) tc::mbar_init(fin(i), 1);
        tc::mbar_init(stall, 1);
        for (int i = 0; i < SEGS; ++i) {
            tc::mbar_init(seg_full(i), 1);
            tc::mbar_init(seg_empty(i), kSegReaders);
        }
        *abort_flag = 0;
        tc::mbar_fence_init();
        tc::tma_prefetch_desc(&maps.ks);
        tc::tma_prefetch_desc(&maps.vs);
        tc::tma_prefetch_desc(&maps.kc);
        tc::tma_prefetch_desc(&maps.vc);
        tc::tma_prefetch_desc(&maps.kn);
        tc::tma_prefetch_desc(&maps.vn);
        tc::tma_prefetch_desc(&maps.q);
    }
    if (warp == 1) tc::tmem_alloc(smem_u32(tmem_slot), 512);
    // The rows of a Q tile past its G RT queries, which no copy fills, are zeros.  (What earlier launches left there could
    // score NaN, so that the row never got a maximum and every half of its row tile was looked at twice: 4 sequences of k 8
    // with 14 heads on 2 KV heads over 8000 shared keys took 54 to 67 us, 41 so.)
    const int queries = g.RT * p.G, spare = (TM - queries) * (D / 8);
    for (int i = tid; i < 2 * spare; i += THREADS) {
        const int t = i >= spare, e = i - t * spare, row = queries + e / (D / 8), c = e % (D / 8);
        *reinterpret_cast<uint4 *>(smem + t * L::Q_TILE + (c >> 3) * TM * 128 + row * 128 + ((c & 7) << 4)) =
            make_uint4(0, 0, 0, 0);
    }
    if (spare > 0) tc::fence_proxy_async_smem();
    // every global read below waits for the previous kernel in the stream
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    int S = p.shared_len[0];
    if (S < 0 || S > p.S_max) S = 0;  // (combine_kernel reports it and writes nothing)
    if (warp == 3) {  // the line: key tiles of every sequence (none where the length is out of range)
        int sum = 0, seqs = 0, longest = ceil_div(S, TN);
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int x = 0;
            if (b < p.B) {
                const int P = p.prefix_len[b];
                lens[b] = P;
                if (P >= 0 && P <= p.P_max) x = ceil_div(P, TN) + ceil_div(p.R, TN);
            }
            int inc = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const uint32_t any = __ballot_sync(0xffffffffu, x > 0);
            if (b < p.B) {
                cum[b] = sum + inc - x;
                nseq[b] = seqs + __popc(any & ((1u << lane) - 1u));
            }
            sum += __shfl_sync(0xffffffffu, inc, 31);
            seqs += __popc(any);
            longest = max(longest, (int)__reduce_max_sync(0xffffffffu, (unsigned)x));
        }
        if (lane == 0) {
            cum[p.B] = sum;
            nseq[p.B] = seqs;
            const int st = ceil_div(S, TN), n = gridDim.x;
            Line l;
            l.shared_tiles = st;
            auto lay = [&](int pair, int single, int block) {
                l.pair = pair;
                l.single = single;
                l.block = block;
                l.shared = st > 0 ? blocks_cost(l, g.shared_rt, st) : 0;
                l.head = l.shared + (g.own_rt / 2) * (seqs * block + sum * pair) + (g.own_rt & 1) * (seqs * block + sum * single);
                l.total = l.head * p.Hkv;
            };
            lay(kCostPair, kCostSingle, kCostBlock);
            l.ncta = n;
            if (l.total < n * (kCostPair + kCostBlock)) {
                lay(1, 1, 0);
                l.ncta = min(n, longest < kLongBlock ? l.total : (l.total + 1) / 2);
            }
            *line = l;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tmem_slot;
    const int cta = blockIdx.x;
    const size_t info = info_bytes((size_t)p.Hkv * g.blocks, p.B);
    const long long wl = p.wait_cycles;

    // The next segment for the calling thread (`all`: for its whole warp, which calls it together).
    int seg_at = 0;
    auto next = [&](Segment &sg, bool all) {
        const int i = seg_at % SEGS;
        bool got = tc::mbar_wait(seg_full(i), (seg_at / SEGS) & 1, abort_flag, wl);
        if (all) got = __all_sync(0xffffffffu, got);
        if (!got) return false;
        sg = segs[i];
        if (all) {
            int *f = reinterpret_cast<int *>(&sg);
#pragma unroll
            for (int e = 0; e < (int)(sizeof(Segment) / 4); ++e) f[e] = __shfl_sync(0xffffffffu, f[e], 0);
        }
        if (!all || lane == 0) tc::mbar_arrive(seg_empty(i));
        ++seg_at;
        return sg.nt > 0;
    };

    if (p.block_table && warp == 3) {  // every CTA looks over some of the page tables, for combine_kernel
        int *bad_pages = reinterpret_cast<int *>(reinterpret_cast<int2 *>(p.ws) + (size_t)p.Hkv * g.blocks);
        for (int b = (int)gridDim.x - 1 - cta; b <= p.B; b += gridDim.x) {
            const int n = b < p.B ? p.prefix_len[b] : S;
            const int32_t *pages = b < p.B ? p.block_table + (size_t)b * p.max_pages : p.shared_table;
            bool bad = false;
            for (int i = lane; i < ceil_div(min(max(n, 0), b < p.B ? p.P_max : p.S_max), kPageRows); i += 32)
                bad |= pages[i] < 0 || pages[i] >= p.num_pages;
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) bad_pages[b] = bad;
        }
    }
    if (warp < 4) {
        Segment sg;
        if (warp == 2 && lane == 0) {
            // ================= scheduler and Q producer =================
            const uint32_t bytes = (uint32_t)D * p.G * g.RT * 2;
            Walker walk(*line, g, cum, nseq, p.B, cta);
            bool more = true;
            int n = 0;
            for (; more; ++n) {
                if (n >= SEGS && !tc::mbar_wait(seg_empty(n % SEGS), (n / SEGS - 1) & 1, abort_flag, wl)) break;
                more = walk.next(sg);
                sg.len = !more ? 0 : sg.b < 0 ? S : lens[sg.b];
                segs[n % SEGS] = sg;
                tc::mbar_arrive(seg_full(n % SEGS));
                if (!more) break;
                // for combine_kernel: the CTAs of the block
                if (sg.i0 == 0) reinterpret_cast<int2 *>(p.ws)[sg.id].x = cta;
                if (walk.last) reinterpret_cast<int2 *>(p.ws)[sg.id].y = cta;
                if (n > 0 && !tc::mbar_wait(q_empty, (n - 1) & 1, abort_flag, wl)) break;
                tc::mbar_arrive_expect_tx(q_full, sg.nt * bytes);
                for (int t = 0; t < sg.nt; ++t) {
                    const int z = (sg.b < 0 ? 0 : sg.b * p.R) + sg.row0 + t * g.RT;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        tc::tma_load_3d(sbase + t * L::Q_TILE + h * TM * 128, &maps.q, h * 64, sg.kvh * p.G, z, q_full);
                }
            }
            if (n > 0) tc::mbar_wait_drain(q_full, (n - 1) & 1, kCacheWaitCycles);
        } else if (warp == 0 && lane == 0) {
            // ================= K/V producer =================
            int it = 0;
            bool ok = true;
            while (ok && next(sg, false)) {
                const int P = sg.len, TP = ceil_div(P, TN), np = ceil_div(P, BOXR);
                const int32_t *pages = sg.b < 0 ? p.shared_table : p.block_table + (size_t)sg.b * p.max_pages;
                for (int i = sg.i0; i < sg.i1 && ok; ++i) {
#pragma unroll 1
                    for (int v = 0; v < 2; ++v, ++it) {
                        const int st = it % STAGES;
                        if (it >= STAGES && !tc::mbar_wait(empty(st), (it / STAGES - 1) & 1, abort_flag, wl)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = full(st), dst = sKV + st * L::KV_TILE;
                        tc::mbar_arrive_expect_tx(bar, L::KV_TILE);
                        if (i >= TP) {  // new keys
                            const int z = sg.b * p.R + (i - TP) * TN;
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tc::tma_load_3d(dst + h * TN * 128, v ? &maps.vn : &maps.kn, h * 64, sg.kvh, z, bar);
                        } else if (p.block_table) {  // two pages
                            // (the second box of a tile that ends within its first page re-reads that page: rows past
                            // the end are excluded below; a page id out of range reads page 0 and is reported, and its
                            // rows dropped, by combine_kernel)
                            for (int h2 = 0; h2 < 2; ++h2) {
                                const int pi = min(2 * i + h2, np - 1);
                                int pg = __ldg(pages + pi);
                                if (pg < 0 || pg >= p.num_pages) pg = 0;
                                const int y = (pg * p.Hkv + sg.kvh) * BOXR;
#pragma unroll
                                for (int h = 0; h < D / 64; ++h)
                                    tc::tma_load_2d(dst + h * TN * 128 + h2 * BOXR * 128, v ? &maps.vc : &maps.kc,
                                                    h * 64, y, bar);
                            }
                        } else {
                            const int y = (sg.b < 0 ? sg.kvh * p.S_max : (sg.b * p.Hkv + sg.kvh) * p.P_max) + i * TN;
                            const CUtensorMap *m = sg.b < 0 ? (v ? &maps.vs : &maps.ks) : (v ? &maps.vc : &maps.kc);
#pragma unroll
                            for (int h = 0; h < D / 64; ++h) tc::tma_load_2d(dst + h * TN * 128, m, h * 64, y, bar);
                        }
                    }
                }
            }
            // nothing may land after the CTA exits: only the last copy of each stage can still be in flight
            for (int i = max(0, it - STAGES); i < it; ++i)
                tc::mbar_wait_drain(full(i % STAGES), (i / STAGES) & 1, kCacheWaitCycles);
        } else if (warp & 1) {
            // ================= MMA issue: warp 1 for row tile 0, warp 3 for row tile 1 =================
            // (The whole warp runs the loop, so that descriptors stay in uniform registers; one elected lane issues.)
            // S of half tile u + 2 overwrites the P that the PV of half tile u reads, so it is issued once that PV has
            // completed.  (Right behind it, on the order of issue alone: 61.3 against 63.0 us for 8 x Qwen3-8B k 8, the
            // same elsewhere; that order is promised for MMAs of one shape and accumulator only.)  S runs ahead of PV
            // across segments too, so that the next segment's first scores are there when the softmax has written the
            // last record.
            const int t = __shfl_sync(0xffffffffu, warp >> 1, 0);
            constexpr uint32_t id_qk = tc::idesc_bf16_f32(TM, TH, 0, 0), id_pv = tc::idesc_bf16_f32(TM, D, 0, 1);
            const uint64_t dq = tc::smem_desc_sw128(sbase + t * L::Q_TILE, 16, 1024);
            const uint64_t dk = tc::smem_desc_sw128(sKV, 16, 1024);
            const uint64_t dv = tc::smem_desc_sw128(sKV, TN * 128, 1024);
            constexpr uint64_t kS = L::KV_TILE >> 4, kHalf = (TH * 128) >> 4;
            const uint32_t s_col = tbase + t * 128, o_col = tbase + 256 + t * D;
            const bool one = elect_one();
            auto commit = [&](uint32_t bar) {
                if (one) tc::mma_commit(bar);
            };
            auto arrive = [&](uint32_t bar) {
                if (one) tc::mbar_arrive(bar);
            };
            auto wait = [&](uint32_t bar, uint32_t ph) {
                return __all_sync(0xffffffffu, tc::mbar_wait(bar, ph, abort_flag, wl)) != 0;
            };
            auto wait_full = [&](int i) { return wait(full(i % STAGES), (i / STAGES) & 1); };
            // A place on the segments: half h of key tile i of [first, last), whose K is tile `ring` of the ring.
            struct Cursor {
                int seg;         // segments taken
                int i, h, first, last, ring;
                int one0, one1;  // key tiles of 64 keys or fewer: the cached tail, the new keys' tail (-1: none)
                bool in;         // inside a segment
            };
            Cursor q{0, 0, 0, 0, 0, 0, -1, -1, false}, v{0, 0, 0, 0, 0, 0, -1, -1, false};
            int ns = 0;                  // segments of the PV
            uint32_t pph = 0, busy = 0;  // phases of p_full; S buffers (h of the half) whose PV is not issued yet
            uint32_t read_ph = 0, reading = 0;  // phases of pv_done; S buffers whose PV is not known to have completed
            bool ok = true, more = true;
            auto read = [&](Cursor &c, Segment &sg) {  // segment c.seg
                if (!wait(seg_full(c.seg % SEGS), (c.seg / SEGS) & 1)) return false;
                sg = segs[c.seg % SEGS];
                int *f = reinterpret_cast<int *>(&sg);
#pragma unroll
                for (int e = 0; e < (int)(sizeof(Segment) / 4); ++e) f[e] = __shfl_sync(0xffffffffu, f[e], 0);
                return true;
            };
            auto enter = [&](Cursor &c, const Segment &sg) {
                const int P = sg.len, TP = ceil_div(P, TN);
                c.i = c.first = sg.i0;
                c.last = sg.i1;
                c.h = 0;
                const int new_last = TP + ceil_div(p.R, TN) - 1;
                c.one0 = TP > 0 && tile_keys(TP - 1, P, TP, p.R) <= TH ? TP - 1 : -1;
                c.one1 = tile_keys(new_last, P, TP, p.R) <= TH ? new_last : -1;
                c.in = true;
                ++c.seg;
            };
            auto halves = [&](const Cursor &c) { return c.i == c.one0 || c.i == c.one1 ? 1 : 2; };
            if (p.stall_test) ok = wait(stall, 0);
            while (ok) {
                while (busy != 3 && more) {  // S
                    if (!q.in) {
                        Segment sg;
                        ok = read(q, sg);
                        if (!ok) break;
                        if (sg.nt == 0) {
                            more = false;
                            break;
                        }
                        if (t >= sg.nt) {  // nothing to multiply here: the tiles are freed as they come, once no PV is due
                            if (busy) break;
                            ok = wait(q_full, q.seg & 1);
                            if (!ok) break;
                            arrive(q_empty);
                            for (int i = 0; i < 2 * (sg.i1 - sg.i0) && ok; ++i, ++q.ring) {
                                ok = wait_full(q.ring);
                                if (ok) arrive(empty(q.ring % STAGES));
                            }
                            arrive(seg_empty(q.seg % SEGS));
                            ++q.seg;
                            v.seg = q.seg;
                            v.ring = q.ring;
                            if (!ok) break;
                            continue;
                        }
                        enter(q, sg);
                        ok = wait(q_full, (q.seg - 1) & 1);
                        if (!ok) break;
                    }
                    if (busy >> q.h & 1) break;  // (a tile of one half, and the next one's first)
                    const int st = q.ring % STAGES;
                    if (q.h == 0) {
                        ok = wait_full(q.ring);
                        if (!ok) break;
                    }
                    if (reading >> q.h & 1) {
                        ok = wait(pv_done(t, q.h), read_ph >> q.h & 1);
                        if (!ok) break;
                        read_ph ^= 1u << q.h;
                        reading &= ~(1u << q.h);
                        tc::fence_after_sync();
                    }
                    if (one) issue_qk<D>(s_col + q.h * TH, dq, dk + st * kS + q.h * kHalf, id_qk);
                    commit(s_full(t, q.h));
                    busy |= 1u << q.h;
                    if (++q.h == halves(q)) {
                        commit(empty(st));
                        q.h = 0;
                        q.ring += 2;
                        if (++q.i == q.last) {
                            commit(q_empty);
                            q.in = false;
                        }
                    }
                }
                if (!ok || !busy) break;
                // PV of the oldest half whose S is out
                if (!v.in) {
                    Segment sg;
                    ok = read(v, sg);
                    if (!ok) break;
                    arrive(seg_empty(v.seg % SEGS));
                    enter(v, sg);
                    if (ns++ > 0) ok = wait(o_free(t), ns & 1);  // (the record before has been read)
                }
                const int vi = v.ring + 1, st = vi % STAGES, h = v.h;
                if (ok && h == 0) ok = wait_full(vi);
                ok = ok && wait(p_full(t, h), pph >> h & 1);
                if (!ok) break;
                pph ^= 1u << h;
                tc::fence_after_sync();
                if (one) issue_pv(o_col, s_col + h * TH, dv + st * kS + h * kHalf, id_pv, v.i > v.first || h > 0);
                commit(pv_done(t, h));
                reading |= 1u << h;
                busy &= ~(1u << h);
                if (++v.h == halves(v)) {
                    commit(empty(st));
                    v.h = 0;
                    v.ring += 2;
                    if (++v.i == v.last) {
                        commit(o_full(t));
                        v.in = false;
                    }
                }
            }
            commit(fin(t));  // every MMA completes before TMEM is freed
            if (one) tc::mbar_wait_drain(fin(t), 0, kCacheWaitCycles);
            __syncwarp();
        }
        __syncwarp();
    } else {
        // ================= softmax: warpgroup t has row tile t =================
        const int t = (warp - 4) >> 2, q4 = warp & 3, row = q4 * 32 + lane;
        const int rr = row / p.G;  // row (b, r) within the tile
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint32_t s_col = tbase + lane_off + t * 128, o_col = tbase + lane_off + 256 + t * D;
        const float sl2 = p.scale_log2;
        Segment sg;
        int ring = 0, n_seg = 0;
        uint32_t ph = 0;  // phases of s_full (bits 0, 1: S buffers) and of pv_done (bits 2, 3)
        bool ok = true;
        while (next(sg, true)) {
            const int nk = sg.i1 - sg.i0, ring0 = ring;
            ring += 2 * nk;
            if (t >= sg.nt) continue;
            const int P = sg.len, TP = ceil_div(P, TN);
            const int r = sg.row0 + t * g.RT + rr;  // row of the sequence, or of the batch (shared)
            const bool valid = rr < g.RT && r < (sg.b < 0 ? p.B * p.R : p.R);
            const bool work = __any_sync(0xffffffffu, valid);
            // visible new keys of row r: [0, vis_lim) and [vis_glo, vis_ghi)
            int vis_lim = r + 1, vis_glo = 0, vis_ghi = 0;
            if (p.mask_mode == TIDAR_MASK_HYBRID && r >= p.k) {
                const int grp = (r - p.k) / p.k;
                vis_lim = grp;
                vis_glo = p.k + grp * p.k;
                vis_ghi = vis_glo + p.k;
            }
            // (A row whose sum is NaN asks for no maximum: one that has met a score of NaN or infinity, and from the start one
            // that holds no query of this segment, whatever its scores.  Otherwise it did so for every half: one sequence of
            // NaN queries in 8 of Qwen3-8B k 8 took 133 us, 61 so.)
            float m_run = -INFINITY, l_run = valid ? 0.f : __int_as_float(0x7fffffff);
            int prev = -1;      // S buffer of the half before (-1: none in this segment)
            bool fresh = true;  // some row of the warp has seen no key yet
            auto wait_s = [&](int h) {
                const uint32_t sp = ph >> h & 1;
                if (!__all_sync(0xffffffffu, tc::mbar_try_wait(s_full(t, h), sp)))  // (TMEM accesses are warp-wide)
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(s_full(t, h), sp, abort_flag, wl));
                ph ^= 1u << h;
                if (prev >= 0) ph ^= 4u << prev;  // (counts the PV of the half before: the phase that half's P began)
                return ok;
            };
            // Exponentials of a half against the running max as it stands: a stale one is exact as long as the weights
            // fit, whatever their size, so no maximum is taken while their sum stays below kMaxHalfSum.
            auto softmax = [&](int h, bool masked, int lo, int glo, int ghi) {
                const uint32_t sc = s_col + h * TH;
                float lt = 0.f;
                bool again = fresh;
                for (int tries = 0;; again = true) {
                    if (again) {
                        const RowState st = raise_max<D>(sc, h * TH, lo, glo, ghi, sl2, lt, m_run, l_run, o_col,
                                                         pv_done(t, max(prev, 0)), (ph >> (2 + max(prev, 0)) & 1) ^ 1u, abort_flag);
                        m_run = st.m;
                        l_run = st.l;
                        ok = st.ok;
                        if (!ok) return;
                        fresh = __any_sync(0xffffffffu, m_run == -INFINITY && l_run == l_run);
                    }
                    uint32_t u[2][32], pk[32];
                    load_scores(sc, u);
                    if (masked) mask_scores(u, h * TH, lo, glo, ghi);
                    lt = half_exp(u, sl2, m_run == -INFINITY ? 0.f : -m_run, pk);
                    if (__all_sync(0xffffffffu, lt < kMaxHalfSum || l_run != l_run) || tries++ > 0) {
                        tc::tmem_st32(sc, pk);
                        break;
                    }
                }
                l_run += lt;
            };
            auto hand_over = [&](int h) {
                prev = h;
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(p_full(t, h));
            };
            // whole tiles of cached keys: nothing masked.  (A loop of its own, its halves unrolled: 462 k cycles against
            // 537 k for the largest shapes below.)
            const int whole = work ? min(sg.i1, P / TN) - sg.i0 : 0;
            int i = 0;
            for (; i < whole && ok; ++i) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait_s(h)) break;
                    softmax(h, false, TN, 0, 0);
                    if (!ok) break;
                    hand_over(h);
                }
            }
            // the others
            for (; i < nk && ok; ++i) {
                const int kt = sg.i0 + i, keys = tile_keys(kt, P, TP, p.R);
                const int nh = keys > TH ? 2 : 1;
                int lo = keys, glo = 0, ghi = 0;
                if (kt >= TP) {
                    const int nn0 = (kt - TP) * TN;
                    lo = min(vis_lim - nn0, keys);
                    glo = vis_glo - nn0;
                    ghi = min(vis_ghi - nn0, keys);
                }
#pragma unroll 1
                for (int h = 0; h < nh; ++h) {
                    if (!wait_s(h)) break;
                    if (work) softmax(h, true, lo, glo, ghi);
                    if (!ok) break;
                    if (h == nh - 1 && keys < TH * nh) {
                        // keys past the end: zero their V rows (0 * garbage could be NaN) before this row tile's PV
                        // reads them (with two row tiles both do)
                        const int vi = ring0 + 2 * i + 1, st = vi % STAGES;
                        const bool got = tc::mbar_wait(full(st), (vi / STAGES) & 1, abort_flag, wl);
                        ok = __all_sync(0xffffffffu, got);
                        if (!ok) break;
                        uint8_t *vrow = smem + L::KV_OFF + st * L::KV_TILE;
                        for (int idx = row; idx < (TH * nh - keys) * (D / 8); idx += 128) {
                            const int j = keys + idx / (D / 8), c = idx % (D / 8);
                            *reinterpret_cast<uint4 *>(vrow + (c >> 3) * TN * 128 + j * 128 + ((c & 7) << 4)) =
                                make_uint4(0, 0, 0, 0);
                        }
                        tc::fence_proxy_async_smem();
                    }
                    hand_over(h);
                }
            }
            tc::tmem_wait_st();
            // ---- the record: the row over a power of two as fp16 (a value of 2^-27 of the largest magnitude or more is
            // off by 2^-11 of itself at most, a smaller one by 2^-38 of that magnitude) and an fp32 scale ----
            bool got = ok && tc::mbar_wait(o_full(t), n_seg & 1, abort_flag, wl);
            ok = __all_sync(0xffffffffu, got);
            if (!ok) break;
            ++n_seg;
            if (prev >= 0) ph ^= 4u << prev;
            if (work) {
                tc::fence_after_sync();
                uint32_t v[D / 32][32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tc::tmem_ld32(o_col + c * 32, v[c]);
                tc::tmem_wait_ld();
                float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < D; j += 2)
                    a4[(j >> 1) & 3] = max3(a4[(j >> 1) & 3], fabsf(__uint_as_float(v[j >> 5][j & 31])),
                                            fabsf(__uint_as_float(v[j >> 5][(j + 1) & 31])));
                const float amax = fmaxf(fmaxf(a4[0], a4[1]), fmaxf(a4[2], a4[3]));
                const float2 scale = record_scale(amax);
                uint8_t *rec = p.ws + info + ((size_t)(cta + sg.id) * 2 + t) * tile_record_bytes(D);
                if (__any_sync(0xffffffffu, valid && amax == INFINITY)) {
                    record_beside_infinities<D>(o_col, valid ? rec : nullptr, row, m_run, l_run);
                } else if (valid) {
                    uint4 *vals = reinterpret_cast<uint4 *>(rec) + row;
                    const uint64_t rs2 = pair(scale.x, scale.x);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = (c & 3) * 8 + 2 * e;
                            float x, y;
                            unpair(mul2(pair(__uint_as_float(v[c >> 2][j]), __uint_as_float(v[c >> 2][j + 1])), rs2), x, y);
                            h[e] = pack_half2(x, y);
                        }
                        vals[c * TM] = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    reinterpret_cast<float2 *>(rec + TM * D * 2)[row] =
                        make_float2(l_run == 0.f ? -INFINITY : m_run + __log2f(l_run),  // (a NaN sum stays one)
                                    l_run == 0.f ? 0.f : scale.y / l_run);
                }
            }
            tc::fence_before_sync();
            tc::mbar_arrive(o_free(t));
        }
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, 512);
    }
    if (tid == 0 && *abort_flag) atomicOr(p.dev_status, TIDAR_DEV_TIMEOUT);
}

// Joins the records of kJoin rows of one KV head; a thread has 16 columns of one row.  A row has as many
// records as CTAs worked on its two blocks; their headers are read all at once (a group of threads per record), their values U at
// a time (the first U beside the headers), in the order of the line: eight where there are fewer blocks than CTAs, so that
// a block is split over several, four elsewhere, for more threads on an SM (eight everywhere: 22.5 -> 22.1 us for 16
// single-token rows, but 62.2 -> 65.8 us for 8 x Qwen3-8B k 8).  Also reports lengths and pages out of range and
// leaves those rows alone.
constexpr int kHeads = 64;  // records whose headers are held at a time
constexpr int kJoin = 16;   // rows of a CTA
template <int D, int U>
__global__ void __launch_bounds__(D / 16 * kJoin) combine_kernel(const SharedAttnParams p) {
    constexpr int GROUPS = D / 16;
    __shared__ float2 heads[kHeads][kJoin];
    const int lane = threadIdx.x % kJoin, chunk = threadIdx.x / kJoin;
    const int kvh = blockIdx.y;
    const long rows = (long)p.B * p.R * p.G;
    const long m = (long)blockIdx.x * kJoin + lane;
    const Geometry g = geometry(p.B, p.R, p.G);
    const int per_seq = p.R * p.G;
    const int b = (int)min(m / per_seq, (long)p.B - 1);
    const int mr = (int)(m - (long)b * per_seq), r = mr / p.G, gq = mr - r * p.G;
    // the two blocks that hold this row: shared (x = 0) and own (x = 1)
    const int sr = b * p.R + r, st = sr / g.RT, ot = r / g.RT;
    const int id[2] = {kvh * g.blocks + st / 2, kvh * g.blocks + g.shared_blocks + b * g.own_blocks + ot / 2};
    const int row[2] = {(sr - st * g.RT) * p.G + gq, (r - ot * g.RT) * p.G + gq};
    const bool in = m < rows;
    const int2 *ctas = reinterpret_cast<const int2 *>(p.ws);
    const int *bad_pages = reinterpret_cast<const int *>(ctas + (size_t)p.Hkv * g.blocks);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int S = p.shared_len[0], P = p.prefix_len[b];
    int2 c[2] = {make_int2(0, -1), make_int2(0, -1)};
    int pages = 0;
    if (in) {
        c[0] = ctas[id[0]];
        c[1] = ctas[id[1]];
        if (p.block_table) pages = bad_pages[b] | bad_pages[p.B];
    }
    int bits = (S < 0 || S > p.S_max || P < 0 || P > p.P_max) ? TIDAR_DEV_BAD_PREFIX : 0;
    if (pages) bits |= TIDAR_DEV_BAD_PAGE;
    if (bits && in && chunk == 0) atomicOr(p.dev_status, bits);
    if (S == 0) c[0] = make_int2(0, -1);
    // (a launch whose waits ran out may have left these unset: it has reported that)
    auto sound = [](int2 v) { return v.x >= 0 && v.y < kNumSMs && v.x <= v.y + 1; };
    const bool go = in && !bits && sound(c[0]) && sound(c[1]);
    const int n0 = go ? c[0].y - c[0].x + 1 : 0;          // records: shared ones,
    const int n = go ? n0 + c[1].y - c[1].x + 1 : 0;      // all
    const size_t rec_bytes = tile_record_bytes(D);
    const uint8_t *recs = p.ws + info_bytes((size_t)p.Hkv * g.blocks, p.B);
    const uint8_t *rec0 = recs + ((size_t)(c[0].x + id[0]) * 2 + (st & 1)) * rec_bytes;
    const uint8_t *rec1 = recs + ((size_t)(c[1].x + id[1]) * 2 + (ot & 1)) * rec_bytes - (size_t)n0 * 2 * rec_bytes;
    auto values = [&](int i, uint4 (&v)[2]) {
        const bool sh = i < n0;
        const uint4 *x = reinterpret_cast<const uint4 *>((sh ? rec0 : rec1) + (size_t)i * 2 * rec_bytes) + 2 * chunk * TM +
                         (sh ? row[0] : row[1]);
        v[0] = x[0];
        v[1] = x[TM];
    };
    auto head = [&](int i) {
        const bool sh = i < n0;
        return reinterpret_cast<const float2 *>((sh ? rec0 : rec1) + (size_t)i * 2 * rec_bytes + TM * D * 2)[sh ? row[0] : row[1]];
    };
    const int nmax = __reduce_max_sync(0xffffffffu, n);  // (every warp has the same rows once or twice)
    float mx = -INFINITY, wsum = 0.f, acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    for (int h0 = 0; h0 < nmax; h0 += kHeads) {
        const int nh = min(kHeads, nmax - h0);
        uint4 raw[U][2];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (h0 + i < n) values(h0 + i, raw[i]);
        if (h0 > 0) __syncthreads();
#pragma unroll 4
        for (int i = chunk; i < nh; i += GROUPS) heads[i][lane] = h0 + i < n ? head(h0 + i) : make_float2(-INFINITY, 0.f);
        __syncthreads();
        float top = mx;
#pragma unroll 8
        for (int i = 0; i < nh; ++i) top = fmaxf(top, heads[i][lane].x);
        const float keep = mx == -INFINITY ? 0.f : fast_exp2(mx - top);
        wsum *= keep;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= keep;
        mx = top;
        for (int i0 = 0; i0 < nh; i0 += U) {
            if (i0 > 0) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (i0 + i < nh && h0 + i0 + i < n) values(h0 + i0 + i, raw[i]);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (!(i0 + i < nh && h0 + i0 + i < n)) continue;
                const float2 hd = heads[i0 + i][lane];
                const float w = hd.x == -INFINITY ? 0.f : fast_exp2(hd.x - mx);
                wsum += w;
                const float f = w * hd.y;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t u[4] = {raw[i][x].x, raw[i][x].y, raw[i][x].z, raw[i][x].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = unpack_half2(u[e]);
                        acc[8 * x + 2 * e] = fmaf(f, v.x, acc[8 * x + 2 * e]);
                        acc[8 * x + 2 * e + 1] = fmaf(f, v.y, acc[8 * x + 2 * e + 1]);
                    }
                }
            }
        }
    }
    if (n == 0) return;
    const float inv = 1.f / wsum;
    const size_t orow = ((size_t)b * p.R + r) * p.Hq + kvh * p.G + gq;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const float *a = acc + 8 * x;
        reinterpret_cast<uint4 *>(p.out + orow * D)[2 * chunk + x] =
            make_uint4(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv),
                       pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
    }
    if (chunk == 0 && p.lse) p.lse[orow] = (mx + __log2f(wsum)) * kLn2;
}

// ---- host side ---------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiledFn) nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// bf16, 128-byte swizzle; dims and box innermost first, rows packed.
bool map_2d(CUtensorMap *m, const void *base, int D, long long rows, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_3d(CUtensorMap *m, const void *base, int D, int heads, long long rows, int box_heads, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * heads};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const SharedAttnParams &p, cudaStream_t s) {
    Maps mp;
    if (!encode_fn()) return cudaErrorNotSupported;
    const bool paged = p.block_table != nullptr;
    // (an empty part has no map of its own: no tile of it is ever loaded)
    const bool no_shared = p.S_max == 0, no_own = p.P_max == 0;
    const long long pool_rows = (long long)p.num_pages * p.Hkv * kPageRows;
    const long long s_rows = no_shared ? 1 : (long long)p.Hkv * p.S_max;
    const long long o_rows = no_own ? 1 : (long long)p.B * p.Hkv * p.P_max;
    const int box = paged ? BOXR : TN;
    if (!paged && (!map_2d(&mp.ks, no_shared ? p.q : p.k_shared, D, s_rows, box) ||
                   !map_2d(&mp.vs, no_shared ? p.q : p.v_shared, D, s_rows, box)))
        return cudaErrorInvalidValue;
    if (!map_2d(&mp.kc, paged || !no_own ? p.k_cache : p.q, D, paged ? pool_rows : o_rows, box) ||
        !map_2d(&mp.vc, paged || !no_own ? p.v_cache : p.q, D, paged ? pool_rows : o_rows, box) ||
        !map_3d(&mp.kn, p.k_new, D, p.Hkv, (long long)p.B * p.R, 1, TN) ||
        !map_3d(&mp.vn, p.v_new, D, p.Hkv, (long long)p.B * p.R, 1, TN) ||
        !map_3d(&mp.q, p.q, D, p.Hq, (long long)p.B * p.R, p.G, rows_per_tile(p.G)))
        return cudaErrorInvalidValue;
    if (paged) {  // (the shared rows lie in the same pools)
        mp.ks = mp.kc;
        mp.vs = mp.vc;
    }
    const int smem = Smem<D>::alloc(p.B);
    cudaError_t e = allow_shared_memory<shared_attn_kernel<D>>(Smem<D>::alloc(kMaxBatchShared));
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
    e = cudaLaunchKernelEx(&cfg, shared_attn_kernel<D>, p, mp);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(((long long)p.B * p.R * p.G + kJoin - 1) / kJoin), p.Hkv, 1);
    cfg.blockDim = dim3(D / 16 * kJoin, 1, 1);
    cfg.dynamicSmemBytes = 0;
    const long long blocks = (long long)p.Hkv * geometry(p.B, p.R, p.G).blocks;
    e = cudaLaunchKernelEx(&cfg, blocks < kNumSMs ? combine_kernel<D, 8> : combine_kernel<D, 4>, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

bool shared_attn_fits(int B, int R, int Hkv, int G, int S_max, int P_max) {
    const Geometry g = geometry(B, R, G);
    const long long own = (long long)ceil_div(P_max, TN) + ceil_div(R, TN);
    const long long cost = (long long)g.shared_blocks * (kCostBlock + (long long)ceil_div(S_max, TN) * kCostPair) +
                           (long long)B * g.own_blocks * (kCostBlock + own * kCostPair);
    return cost * Hkv < (1LL << 31);
}

size_t shared_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int R, int, int) {
    const Geometry g = geometry(B, R, Hq / Hkv);
    // a segment's record is at cta + block: along the line both only grow, and one of them from segment to segment
    return info_bytes((size_t)Hkv * g.blocks, B) + ((size_t)kNumSMs + (size_t)Hkv * g.blocks) * 2 * tile_record_bytes(D);
}

cudaError_t shared_attn_launch(const SharedAttnParams &p, cudaStream_t s) {
    return p.D == 64 ? launch<64>(p, s) : launch<128>(p, s);
}

}  // namespace tidar
