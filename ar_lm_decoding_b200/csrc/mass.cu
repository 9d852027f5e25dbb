// Attention mass of the cache rows: one warp per (layer, sequence, KV head, row), its weights summed over the queries.
#include "cache_ops.cuh"

namespace tidar {

namespace {

__global__ void __launch_bounds__(256) mass_rows_kernel(const MassParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = p.D / 32;
    const int b = blockIdx.y, l = blockIdx.z / p.Hkv, kvh = blockIdx.z % p.Hkv;
    const int N = p.prefix_len[b], a = p.row_count ? p.row_count[b] : p.R;
    int bits = 0;
    if (N < 0 || N > p.P_max) bits = TIDAR_DEV_BAD_PREFIX;
    else if (a < 0 || a > p.R || a > N) bits = TIDAR_DEV_BAD_ACCEPT;
    else if (p.block_table && block_bad_page(p.block_table + (size_t)b * p.max_pages, N, p.num_pages))
        bits = TIDAR_DEV_BAD_PAGE;
    if (bits) {
        if (threadIdx.x == 0) atomicOr(p.dev_status, bits);
        return;
    }
    const bf16 *q = reinterpret_cast<const bf16 *>(p.qs[l]);
    const bf16 *kc = reinterpret_cast<const bf16 *>(p.k_caches[l]);
    const float *lse = p.lses[l];
    float *mass = p.masses[l] + ((size_t)b * p.Hkv + kvh) * p.P_max;
    for (int n = blockIdx.x * 8 + warp; n < N; n += gridDim.x * 8) {
        size_t at = (((size_t)b * p.Hkv + kvh) * p.P_max + n) * p.D;
        if (p.block_table)
            at = (((size_t)p.block_table[(size_t)b * p.max_pages + n / kPageRows] * p.Hkv + kvh) * kPageRows +
                  n % kPageRows) * p.D;
        float k[4], w = 0.f;
        for (int e = 0; e < per; ++e) k[e] = __bfloat162float(kc[at + lane * per + e]);
        for (int j = max(0, n - (N - a)); j < a; ++j)
            for (int g = 0; g < p.G; ++g) {
                const size_t row = ((size_t)b * p.R + j) * p.Hq + kvh * p.G + g;
                float s = 0.f;
                for (int e = 0; e < per; ++e) s = fmaf(k[e], __bfloat162float(q[row * p.D + lane * per + e]), s);
                for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                w += exp2f(fmaf(s, p.scale_log2, -lse[row] * kLog2e));
            }
        if (lane == 0) mass[n] = n < N - a ? p.decay * mass[n] + w : w;
    }
}

}  // namespace

cudaError_t mass_launch(const MassParams &p, cudaStream_t s) {
    const dim3 grid(32, p.B, p.L * p.Hkv);
    mass_rows_kernel<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace tidar
