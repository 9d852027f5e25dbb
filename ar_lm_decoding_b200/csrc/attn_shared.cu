// Attention of a batch behind one shared prefix: one warp per query row, online softmax over all its keys.
#include "cache_ops.cuh"

namespace tidar {

namespace {

__global__ void __launch_bounds__(256) shared_attn_rows_kernel(const SharedAttnParams p) {
    const int lane = threadIdx.x & 31;
    const long row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long rows = (long)p.B * p.R * p.Hq;
    if (row >= rows) return;
    const int h = (int)(row % p.Hq), r = (int)(row / p.Hq % p.R), b = (int)(row / p.Hq / p.R);
    const int kvh = h / p.G, per = p.D / 32;
    const int S = p.shared_len[0], P = p.prefix_len[b];
    if (S < 0 || S > p.S_max || P < 0 || P > p.P_max) {
        if (lane == 0) atomicOr(p.dev_status, TIDAR_DEV_BAD_PREFIX);
        return;
    }
    if (p.block_table) {
        bool bad = false;
        for (int i = lane; i < ceil_div(S, kPageRows); i += 32)
            bad |= p.shared_table[i] < 0 || p.shared_table[i] >= p.num_pages;
        for (int i = lane; i < ceil_div(P, kPageRows); i += 32) {
            const int pg = p.block_table[(size_t)b * p.max_pages + i];
            bad |= pg < 0 || pg >= p.num_pages;
        }
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0) atomicOr(p.dev_status, TIDAR_DEV_BAD_PAGE);
            return;
        }
    }
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < per; ++e) q[e] = __bfloat162float(p.q[row * p.D + lane * per + e]);
    for (int n = 0; n < S + P + p.R; ++n) {
        const bf16 *kr, *vr;
        if (n >= S + P) {
            const int nn = n - S - P;
            if (!new_key_visible(p.mask_mode, p.k, r, nn)) continue;
            const size_t at = ((size_t)(b * p.R + nn) * p.Hkv + kvh) * p.D;
            kr = p.k_new + at;
            vr = p.v_new + at;
        } else if (p.block_table) {
            const int i = n < S ? n : n - S;
            const int pg = n < S ? p.shared_table[i / kPageRows] : p.block_table[(size_t)b * p.max_pages + i / kPageRows];
            const size_t at = (((size_t)pg * p.Hkv + kvh) * kPageRows + i % kPageRows) * p.D;
            kr = p.k_cache + at;
            vr = p.v_cache + at;
        } else if (n < S) {
            const size_t at = ((size_t)kvh * p.S_max + n) * p.D;
            kr = p.k_shared + at;
            vr = p.v_shared + at;
        } else {
            const size_t at = (((size_t)b * p.Hkv + kvh) * p.P_max + (n - S)) * p.D;
            kr = p.k_cache + at;
            vr = p.v_cache + at;
        }
        float s = 0.f;
        for (int e = 0; e < per; ++e) s = fmaf(q[e], __bfloat162float(kr[lane * per + e]), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        l = l * f + w;
        for (int e = 0; e < per; ++e) o[e] = o[e] * f + w * __bfloat162float(vr[lane * per + e]);
        m = mn;
    }
    for (int e = 0; e < per; ++e) p.out[row * p.D + lane * per + e] = __float2bfloat16_rn(o[e] / l);
    if (lane == 0 && p.lse) p.lse[row] = (m + log2f(l)) * kLn2;
}

}  // namespace

size_t shared_attn_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

cudaError_t shared_attn_launch(const SharedAttnParams &p, cudaStream_t s) {
    const long rows = (long)p.B * p.R * p.Hq;
    shared_attn_rows_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace tidar
