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
// lane owns two chunks of 8 consecutive channels of a row (D / 16 lanes per
// row): in the half layout the two whose channels are partners.  8188 tokens of
// 32 heads of 128 bfloat16 (134 MB): 24.8 us, 5.4 TB/s, 83 % of a copy's rate;
// 64 tokens: 2 us on the device, less than the call takes on the host.
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

// 8 channels in registers <-> memory, 16-byte accesses: as stored, and widened.
template <typename T> struct Raw8 {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void widen(float *x) const
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) Vec16<T>::unpack(v[i], x + i * Vec16<T>::E);
    }
};
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

// cos and sin of pos * turns turns, times amp, in float64: the Taylor series on an
// eighth of a turn around the nearest quarter (|x| <= pi / 4: the first terms
// left out are below 4e-13).
__device__ __forceinline__ void turn(int pos, double turns, double amp, double &c, double &s)
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
    c = q == 0 ? cs : q == 1 ? -sn : q == 2 ? -cs : sn;
    s = q == 0 ? sn : q == 1 ? cs : q == 2 ? -sn : -cs;
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
        // a load through the generic address: as constant-bank reads the lanes' different addresses would take turns
        double turns;
        asm("ld.f64 %0, [%1];" : "=d"(turns) : "l"(p.turns + e));
        double c, s;
        turn(pos(tok), turns, p.amp, c, s);
        t.c[tok * kRopeMaxPairs + e] = (float)c;
        t.s[tok * kRopeMaxPairs + e] = sign * (float)s;
    }
}

// The two chunks of lane l of a row's D / 16 lanes.
__device__ __forceinline__ void rope_chunks(const RopeParams &p, int l, int &a, int &b)
{
    const int hc = p.rot / 16;   // chunks of one half
    if (p.interleaved || l >= hc) {   // behind the halves: two that pass through
        a = 2 * l;
        b = a + 1;
    } else {
        a = l;
        b = l + hc;
    }
}

// Rotate a lane's two chunks in place.
__device__ __forceinline__ void rope_apply(const RopeParams &p, const RopeTable &t, int tok, int l, float *a, float *b)
{
    const float *tc = t.c + tok * kRopeMaxPairs, *ts = t.s + tok * kRopeMaxPairs;
    if (16 * l >= p.rot) return;   // in either layout the first rot / 16 lanes rotate
    // half: pairs 8 l + e of (a[e], b[e]); interleaved: pairs 8 l + i of (a[2 i], a[2 i + 1]), 8 l + 4 + i of b's
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4 *>(c + e) = *reinterpret_cast<const float4 *>(tc + 8 * l + e);
        *reinterpret_cast<float4 *>(s + e) = *reinterpret_cast<const float4 *>(ts + 8 * l + e);
    }
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = a[2 * i], v = a[2 * i + 1], x = b[2 * i], y = b[2 * i + 1];
            a[2 * i] = fmaf(u, c[i], -v * s[i]);
            a[2 * i + 1] = fmaf(v, c[i], u * s[i]);
            b[2 * i] = fmaf(x, c[4 + i], -y * s[4 + i]);
            b[2 * i + 1] = fmaf(y, c[4 + i], x * s[4 + i]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = a[e], v = b[e];
            a[e] = fmaf(u, c[e], -v * s[e]);
            b[e] = fmaf(v, c[e], u * s[e]);
        }
    }
}

// Rows (token, head) of n tokens from x to y, Batch passes of loads at a time
// (kept as stored: widened they would halve the rows in flight).  begin() runs
// once, after the first loads have been started, and fills the table; a token's
// rows are not written where use(token) is false.
constexpr int kRowBatch = 2;

template <typename T, int D, int Batch, typename Begin, typename Use>
__device__ __forceinline__ void rope_rows(const RopeParams &p, const RopeTable &table, const T *x, long long xs, T *y,
                                          long long ys, int n, int H, Begin &&begin, Use &&use)
{
    constexpr int L = D / 16, R = kTokThreads / L;   // lanes per row, rows per pass
    const int l = threadIdx.x % L;
    int ca, cb;
    rope_chunks(p, l, ca, cb);
    int tok = 0, h = threadIdx.x / L;   // this lane's row
    auto wrap = [&](int &t, int &hh) {
        while (hh >= H) {
            hh -= H;
            ++t;
        }
    };
    wrap(tok, h);
    bool started = false;
    for (int base = 0; base < n * H; base += Batch * R) {   // CTA-uniform
        Raw8<T> ra[Batch], rb[Batch];
        int t2 = tok, h2 = h;
#pragma unroll
        for (int k = 0; k < Batch; ++k) {
            if (t2 < n) {
                const T *src = x + t2 * xs + h2 * D;
                ra[k].load(src + 8 * ca);
                rb[k].load(src + 8 * cb);
            }
            h2 += R;
            wrap(t2, h2);
        }
        if (!started) {
            begin();
            started = true;
        }
#pragma unroll
        for (int k = 0; k < Batch; ++k) {
            if (tok < n && use(tok)) {
                float a[8], b[8];
                ra[k].widen(a);
                rb[k].widen(b);
                if (p.on) rope_apply(p, table, tok, l, a, b);
                T *dst = y + tok * ys + h * D;
                store8<T>(dst + 8 * ca, a);
                store8<T>(dst + 8 * cb, b);
            }
            h += R;
            wrap(tok, h);
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

template <typename T, int D>
__global__ void __launch_bounds__(kTokThreads, 4) rope_kernel(const __grid_constant__ RopeParams p, const RopeIo io)
{
    __shared__ RopeTable table;
    const long long t0 = (long long)blockIdx.x * io.per_cta;
    const int n = (int)min((long long)io.per_cta, io.tokens - t0);
    griddep_wait();
    rope_rows<T, D, kRowBatch>(
        p, table, reinterpret_cast<const T *>(io.x) + t0 * io.xs, io.xs, reinterpret_cast<T *>(io.y) + t0 * io.ys, io.ys, n,
        io.H,
        [&] {
            rope_fill(p, table, n, io.backward ? -1.f : 1.f, [&](int i) { return io.pos[t0 + i]; });
            __syncthreads();
        },
        [](int) { return true; });
}

}  // namespace akv
