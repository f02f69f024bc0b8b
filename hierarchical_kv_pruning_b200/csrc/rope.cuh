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
// A lane owns 8 consecutive channels of a row ("chunk"), D / 8 lanes per row,
// 2 or 4 rows per warp; the partner channels of the half layout live in
// another lane of the row and come by shuffle.  The lane's 8 (half) or 4
// (interleaved) cosines serve every head that its warp visits.
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

// A lane's cosines and sines (times the amplitude) for chunk j of a row at
// `pos`: entry e belongs to channel 8 j + e (half) or to channels 8 j + 2 e,
// 8 j + 2 e + 1 (interleaved, e < 4).
struct RopeLane {
    float c[8], s[8];
    int partner;       // half layout: lane offset within the row of the partner chunk
    bool first, active;
};

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

__device__ __forceinline__ RopeLane rope_lane(const RopeParams &p, const double *turns, int j, int pos, bool backward)
{
    RopeLane r;
    r.active = p.on && 8 * j < p.rot;
    r.partner = j;
    r.first = true;
    if (!r.active) return r;
    const int hc = p.rot / 16;   // chunks of one half
    r.first = j < hc;
    r.partner = p.interleaved ? j : r.first ? j + hc : j - hc;
    const int base = p.interleaved ? 4 * j : 8 * (r.first ? j : j - hc);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e >= 4 && p.interleaved) break;
        turn(pos, turns[base + e], p.amp, r.c[e], r.s[e]);
        if (backward) r.s[e] = -r.s[e];
    }
    return r;
}

// Rotate the lane's 8 channels in place.  All 32 lanes call it (shuffles);
// row0: the row's first lane.
__device__ __forceinline__ void rope_apply(const RopeParams &p, const RopeLane &r, int row0, float *x)
{
    if (!p.on) return;
    if (p.interleaved) {
        if (!r.active) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = fmaf(u, r.c[e], -v * r.s[e]);
            x[2 * e + 1] = fmaf(v, r.c[e], u * r.s[e]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, x[e], row0 + r.partner);
        if (r.active) x[e] = fmaf(x[e], r.c[e], r.first ? -o * r.s[e] : o * r.s[e]);
    }
}

// The spec's turns in shared memory (a lane's index into them is its own).
__device__ __forceinline__ void rope_turns(const RopeParams &p, double *sm)
{
    if (p.on && threadIdx.x < kRopeMaxPairs) sm[threadIdx.x] = p.turns[threadIdx.x];
    __syncthreads();
}

struct RopeIo {
    const void *x;
    void *y;
    const int32_t *pos;
    long long tokens, xs, ys;   // strides in elements
    int H, heads_per_warp, backward;
};

constexpr int kRopeThreads = 256;

// A warp takes one token's heads_per_warp heads (a multiple of the rows per
// warp, the last group ragged).
template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, const RopeIo io)
{
    constexpr int L = D / 8, R = 32 / L;   // lanes per row, rows per warp
    __shared__ double turns[kRopeMaxPairs];
    rope_turns(p, turns);
    const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
    const int parts = (io.H + io.heads_per_warp - 1) / io.heads_per_warp;
    const long long w = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (w >= io.tokens * parts) return;
    const long long tok = w / parts;
    const int h0 = (int)(w - tok * parts) * io.heads_per_warp, h1 = min(io.H, h0 + io.heads_per_warp);
    const T *x = reinterpret_cast<const T *>(io.x) + tok * io.xs + 8 * j;
    T *y = reinterpret_cast<T *>(io.y) + tok * io.ys + 8 * j;
    const RopeLane r = rope_lane(p, turns, j, io.pos[tok], io.backward != 0);
    for (int h = h0; h < h1; h += R) {   // warp-uniform
        const bool ok = h + sub < h1;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (ok) load8<T>(x + (size_t)(h + sub) * D, v);
        rope_apply(p, r, sub * L, v);
        if (ok) store8<T>(y + (size_t)(h + sub) * D, v);
    }
}

}  // namespace akv
