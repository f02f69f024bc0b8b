// Attention of new tokens over the 4-bit paged cache.
#pragma once

#include "kvcache.cuh"

namespace akv {

struct CacheAttendIo {
    const void *q;
    void *out;          // [B][N][H][D], or null
    float *lse;         // [B][N][H], or null
    long long qs;       // token stride of q in elements
    int H, G;
    float scale_log2;   // scale * log2(e)
};

// One warp per (sequence, token, query head), CUDA cores.
template <typename T, int D>
__global__ void __launch_bounds__(128) cache_attend_simple_kernel(const CacheParams c, const CacheAttendIo io)
{
    constexpr int PER = D / 32;
    using B = Blk<D>;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)c.B * c.N * io.H) return;
    const int h = (int)(row % io.H);
    const long long tok = row / io.H;
    const int b = (int)(tok / c.N), n = (int)(tok - (long long)b * c.N);
    const Seq s = load_seq(c, b);
    if (n >= s.q) return;
    const int last = s.kv - s.q + n, hkv = h / io.G;
    const T *q = reinterpret_cast<const T *>(io.q) + tok * io.qs + (size_t)h * D + lane * PER;
    float qv[PER], acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        qv[i] = elem_f32(q[i]);
        acc[i] = 0.f;
    }
    const int ch = lane * PER, g = ch / 32, r = ch / (D / 8);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i <= last; ++i) {
        const uint8_t *blk = block_at<D>(c, c.table[(size_t)b * c.max_pages + i / c.page_size], hkv, i);
        if (!blk) continue;
        const int t = i & 15;
        const __nv_bfloat162 kp = *reinterpret_cast<const __nv_bfloat162 *>(blk + B::k_pair(t, g));
        const __nv_bfloat16 *vp = reinterpret_cast<const __nv_bfloat16 *>(blk + B::v_scale(t, g));
        const uint8_t *kc = blk + B::k_codes(t) + ch / 2;
        const uint8_t *vc = blk + B::v_codes(t, r) + (ch % (D / 8)) / 2;
        float dot = 0.f, v[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int sh = 4 * (e & 1);
            const float k = __bfloat162float(__hfma(__float2bfloat16((float)((kc[e / 2] >> sh) & 15)), kp.x, kp.y));
            v[e] = __bfloat162float(__hfma(__float2bfloat16((float)((vc[e / 2] >> sh) & 15)), vp[0], vp[2]));
            dot = fmaf(qv[e], k, dot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float x = dot * io.scale_log2, mn = fmaxf(m, x), f = exp2f(m - mn), w = exp2f(x - mn);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, v[e], acc[e] * f);
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T *out = reinterpret_cast<T *>(io.out) + (size_t)row * D + ch;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        if constexpr (sizeof(T) == 4) out[e] = acc[e] * inv;
        else out[e] = __float2bfloat16(acc[e] * inv);
    }
    if (io.lse && lane == 0) io.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace akv
