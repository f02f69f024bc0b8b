// Rotary positions.
//
// Pair i of a head's first rot channels is a complex number turned by
// position * freq[i] and scaled by the amplitude a:
//     y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin);
// the backward direction is the transpose (sin -> -sin), which maps dL/dy to
// dL/dx.  Angles are kept in turns and reduced in float64 (position * turns
// per position, minus its nearest integer: exact to 2^-53 of the product), so
// cos and sin are float32-accurate at any int32 position.
//
// HBM bounds it for many tokens, latency for few.  A CTA takes whole tokens
// (one, or several when their heads are few): it starts the loads, computes
// each token's rot / 2 angles once into shared memory, then turns the rows.  A
// lane owns 8 consecutive channels of a row ("chunk"), D / 8 lanes per row,
// 2 or 4 rows per warp; the partner channels of the half layout live in
// another lane of the row and come by shuffle.
#pragma once

#include "common.cuh"

namespace akv {

constexpr int kRopeMaxPairs = 64;

struct RopeParams {
    int on;             // 0: no rotation
    int interleaved;
    int rot;            // rotated channels, a multiple of 16
    double amp;
    double turns[kRopeMaxPairs];   // turns per position
};

// 8 channels in registers <-> memory, 16-byte accesses.
template <typename T> __device__ __forceinline__ void load8(const T *p, float *x);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float *x)
{
    Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(p), x);
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float *x)
{
    Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(p), x);
    Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(p + 4), x + 4);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float *x);
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float *x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8<float>(float *p, const float *x)
{
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// cos and sin of `t` turns, |t| <= 1/2, times amp, each rounded once to
// float32: the Taylor series on an eighth of a turn around the nearest quarter
// (|x| <= pi / 4: the first terms left out are below 4e-13).  float32
// functions lose another unit in the last place, and a key that is off by that
// is stored under the neighbouring code more often.
__device__ __forceinline__ void turn(int pos, double turns, double amp, float &c, float &s)
{
    double t = (double)pos * turns;
    t -= rint(t);
    const double quarter = rint(4.0 * t);
    const double x = (t - 0.25 * quarter) * 6.283185307179586, y = x * x;
    double a = 1.0 / 6227020800.0, e = 1.0 / 479001600.0;
    a = fma(a, y, -1.0 / 39916800.0);
    e = fma(e, y, -1.0 / 3628800.0);
    a = fma(a, y, 1.0 / 362880.0);
    e = fma(e, y, 1.0 / 40320.0);
    a = fma(a, y, -1.0 / 5040.0);
    e = fma(e, y, -1.0 / 720.0);
    a = fma(a, y, 1.0 / 120.0);
    e = fma(e, y, 1.0 / 24.0);
    a = fma(a, y, -1.0 / 6.0);
    e = fma(e, y, -0.5);
    const double sn = fma(a * y, x, x) * amp, cs = fma(e, y, 1.0) * amp;
    const int q = (int)quarter & 3;
    const float fs = (float)sn, fc = (float)cs;
    c = q == 0 ? fc : q == 1 ? -fs : q == 2 ? -fc : fs;
    s = q == 0 ? fs : q == 1 ? fc : q == 2 ? -fs : -fc;
}

constexpr int kTokThreads = 256;   // of the kernels below and of the cache's append
constexpr int kTokMax = 32;        // tokens per CTA at most

// The cosines and sines of `n` tokens' pairs: pos(i) is token i's position.
struct RopeTable {
    float c[kTokMax * kRopeMaxPairs], s[kTokMax * kRopeMaxPairs];
};
template <typename F>
__device__ __forceinline__ void rope_fill(const RopeParams &p, RopeTable &t, int n, float sign, F &&pos)
{
    const int pairs = p.rot / 2;   // 8 .. 64
    for (int i = threadIdx.x; i < n * pairs; i += kTokThreads) {
        const int tok = i / pairs, e = i - tok * pairs;
        float c, s;
        turn(pos(tok), p.turns[e], p.amp, c, s);
        t.c[tok * kRopeMaxPairs + e] = c;
        t.s[tok * kRopeMaxPairs + e] = sign * s;
    }
}

// Rotate a lane's 8 channels (chunk j of a row of token slot tok) in place.
// All 32 lanes call it (shuffles); row0: the row's first lane.
__device__ __forceinline__ void rope_apply(const RopeParams &p, const RopeTable &t, int tok, int j, int row0, float *x)
{
    const bool active = 8 * j < p.rot;
    if (p.interleaved) {
        if (!active) return;
        const float4 c = *reinterpret_cast<const float4 *>(&t.c[tok * kRopeMaxPairs + 4 * j]);
        const float4 s = *reinterpret_cast<const float4 *>(&t.s[tok * kRopeMaxPairs + 4 * j]);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = fmaf(u, cc[e], -v * ss[e]);
            x[2 * e + 1] = fmaf(v, cc[e], u * ss[e]);
        }
        return;
    }
    const int hc = p.rot / 16;   // chunks of one half
    const bool first = j < hc;
    const int partner = !active ? j : first ? j + hc : j - hc, at = tok * kRopeMaxPairs + 8 * (first ? j : j - hc);
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (active) {
            c = *reinterpret_cast<const float4 *>(&t.c[at + e]);
            s = *reinterpret_cast<const float4 *>(&t.s[at + e]);
        }
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_sync(0xffffffffu, x[e + i], row0 + partner);
            if (active) x[e + i] = fmaf(x[e + i], cc[i], first ? -o * ss[i] : o * ss[i]);
        }
    }
}

struct RopeIo {
    const void *x;
    void *y;
    const int32_t *pos;
    long long tokens, xs, ys;   // strides in elements
    int H, per_cta, backward;   // heads; tokens per CTA
};

// Row slots (token, head) of the CTA's tokens, kRowBatch passes of loads at a time.
constexpr int kRowBatch = 2;

template <typename T, int D>
__global__ void __launch_bounds__(kTokThreads) rope_kernel(const __grid_constant__ RopeParams p, const RopeIo io)
{
    constexpr int L = D / 8, R = kTokThreads / L;   // lanes per row, rows per pass
    __shared__ RopeTable table;
    const int row = threadIdx.x / L, j = threadIdx.x % L, row0 = (threadIdx.x & 31) / L * L;
    const long long t0 = (long long)blockIdx.x * io.per_cta;
    const int n = (int)min((long long)io.per_cta, io.tokens - t0), slots = n * io.H;
    griddep_wait();
    for (int base = 0; base < slots; base += kRowBatch * R) {   // CTA-uniform
        float x[kRowBatch][8];
        int tok[kRowBatch], h[kRowBatch];
#pragma unroll
        for (int k = 0; k < kRowBatch; ++k) {
            const int i = base + k * R + row;
            tok[k] = i < slots ? i / io.H : 0;
            h[k] = i < slots ? i - tok[k] * io.H : -1;
            if (h[k] >= 0)
                load8<T>(reinterpret_cast<const T *>(io.x) + (t0 + tok[k]) * io.xs + (size_t)h[k] * D + 8 * j, x[k]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
        }
        if (base == 0) {
            rope_fill(p, table, n, io.backward ? -1.f : 1.f, [&](int i) { return io.pos[t0 + i]; });
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kRowBatch; ++k) {
            rope_apply(p, table, tok[k], j, row0, x[k]);
            if (h[k] >= 0)
                store8<T>(reinterpret_cast<T *>(io.y) + (t0 + tok[k]) * io.ys + (size_t)h[k] * D + 8 * j, x[k]);
        }
    }
}

}  // namespace akv
