// The 4-bit paged cache of sequence keys and values: storing and reading.
//
// A group of 32 channels x is stored as codes c in 0 .. 15 with
//     m = bf16_down(min x),  s = bf16_up((max x - m) / 15),  c = rne((x - m) / s),
// and stands for bf16(m + c s).  Rounding m down and s up keeps every x inside
// the code range, so an x is off by at most s / 2 before the last rounding.
// That last rounding makes a stored number a bfloat16, which is what the
// tensor cores multiply: attention over the cache and attention over the read
// back keys and values are the same sums.
//
// The block layout (16 tokens of one KV head, 20 D bytes) is in the header.
// It is chosen for the matrix instructions of the attention: a lane of a 16 x 8
// x 16 product wants, of the keys, 32 (D = 128) or 16 channels of two tokens,
// and of the values, 16 or 8 channels of two token pairs; each is one 16- or
// 8-byte piece, and the pieces of a warp are consecutive.
#pragma once

#include "rope.cuh"

namespace akv {

enum : int { kDevBadPage = 4, kDevNonFinite = 5 };   // cache status words (common.cuh has the others)

template <int D>
struct Blk {
    static constexpr int kGroups = D / 32;
    static constexpr int kKS = 8 * D, kVC = 10 * D, kVS = 18 * D, kBytes = 20 * D;
    static constexpr int kSliceBytes = D / 16;
    // byte offsets inside a block
    __device__ static __forceinline__ int k_codes(int tok) { return tok * (D / 2); }
    __device__ static __forceinline__ int k_pair(int tok, int g) { return kKS + (tok * kGroups + g) * 4; }
    // value codes of slice r (D / 8 channels)
    __device__ static __forceinline__ int v_codes(int tok, int r)
    {
        return kVC + ((((tok >> 3) * 8 + r) * 4 + ((tok & 7) >> 1)) * 2 + (tok & 1)) * kSliceBytes;
    }
    // value scale of group g; the minimum is 4 bytes later
    __device__ static __forceinline__ int v_scale(int tok, int g)
    {
        return kVS + (((tok >> 3) * kGroups + g) * 4 + ((tok & 7) >> 1)) * 8 + (tok & 1) * 2;
    }
};

struct CacheParams {
    uint8_t *pages;
    long long n_pages;
    int H_kv, page_size;
    int B, N, max_pages;
    const int32_t *table, *kv_len, *q_len;
    int *status;
};

// One sequence as the kernels use it: lengths checked against the table.
struct Seq {
    int kv, q;   // stored tokens; new tokens
};

__device__ __forceinline__ Seq load_seq(const CacheParams &c, int b)
{
    Seq s;
    s.kv = c.kv_len[b];
    s.q = c.q_len ? c.q_len[b] : c.N;
    const long long cap = (long long)c.max_pages * c.page_size;
    if (s.kv < 0 || s.kv > cap || s.q < 0 || s.q > c.N) {
        set_status(c.status, kDevBadPage);
        s.kv = s.kv < 0 ? 0 : (int)min((long long)s.kv, cap);
        s.q = max(0, min(s.q, c.N));
    }
    return s;
}

// The block of (page, KV head) that holds a slot; null for a page id outside the pool.
template <int D>
__device__ __forceinline__ uint8_t *block_at(const CacheParams &c, int page, int hkv, int slot)
{
    if ((unsigned)page >= (unsigned long long)c.n_pages) {
        set_status(c.status, kDevBadPage);
        return nullptr;
    }
    const int bpp = c.page_size >> 4;
    const long long blk = ((long long)page * c.H_kv + hkv) * bpp + ((slot & (c.page_size - 1)) >> 4);
    return c.pages + blk * Blk<D>::kBytes;
}

constexpr float kMaxStored = 1.329227995784916e36f;     // 2^120
constexpr float kMinScale = 7.888609052210118e-31f;     // 2^-100

// bfloat16 numbers as float32: the largest one not above x, ...
__device__ __forceinline__ float bf16_floor(float x)
{
    const uint32_t u = __float_as_uint(x);
    return __uint_as_float((u + (x < 0.f ? 0xffffu : 0u)) & 0xffff0000u);
}
// ... and the smallest one not below x / 15 (x >= 0).  The product is below the
// quotient by 2^-21 of it at most, so what it rounds up to is one step short at
// most; 15 times a bfloat16 is a float32, which shows it.
__device__ __forceinline__ float bf16_ceil15(float x)
{
    const uint32_t u = (__float_as_uint(x * (0x1.fffff8p-1f / 15.f)) + 0xffffu) & 0xffff0000u;
    return __uint_as_float(15.f * __uint_as_float(u) < x ? u + 0x10000u : u);
}
__device__ __forceinline__ __nv_bfloat16 upper_half(float x) { return __ushort_as_bfloat16(__float_as_uint(x) >> 16); }

// Quantise the lane's 16 channels; the 32-channel group is 2 neighbouring lanes
// (all lanes of the warp call it).  The codes of channels 0 .. 7 and 8 .. 15 as
// two words, channel e at bits 4 e.  doubt says whether float32's roundings could
// have changed the minimum, the scale or a code.  The scale of exact x is exact
// (the range, rounded up, passes 15 times a bfloat16 only if the exact one does).
// Rounding can then only change a code where x - m has more bits than a float32.
//   kExact    x are bfloat16: a difference has more bits only if one number is
//             2^-14 of the other, and decides a code only if the larger alone lies
//             in the middle of two.
//   kFloat    x are float32: the distances of the quotients (below 15.1, two
//             roundings: 2^-19) from the middle of two codes say so.
//   kRotated  x are rotated, some of the group's (turned: the lane's): a rotation
//             by float32 cosines is off by at most 3.3 2^-24 of the pair's radius,
//             that is 4.6 2^-24 of the larger of its two results.  pair0 and pair1
//             are the lanes with the partners of the lane's two chunks; err = 6
//             2^-24 of the largest result there and here covers the sums lo +- err, too.
// The latter two need Doubt, whose lanes may be of any kind.
enum Exactness { kExact, kFloat, kRotated };

template <bool Doubt>
__device__ __forceinline__ uint2 quantise16(float *x, __nv_bfloat16 &scale, __nv_bfloat16 &low, bool &bad, Exactness kind,
                                            bool turned, int pair0, int pair1, bool &doubt)
{
    // 0 x is NaN for an infinity or NaN and 0 else
    float2 z = make_float2(0.f, 0.f);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        z = fma2(make_float2(x[e], x[e + 1]), make_float2(0.f, 0.f), z);
        lo = min3(lo, x[e], x[e + 1]);
        hi = max3(hi, x[e], x[e + 1]);
    }
    if (!(z.x + z.y == 0.f && lo >= -kMaxStored && hi <= kMaxStored)) {   // hardly ever
        lo = INFINITY;
        hi = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            bad |= !(fabsf(x[e]) <= 3.402823466e38f);   // infinity or NaN
            x[e] = isnan(x[e]) ? 0.f : fminf(fmaxf(x[e], -kMaxStored), kMaxStored);
            lo = fminf(lo, x[e]);
            hi = fmaxf(hi, x[e]);
        }
    }
    const float own = lo;
    float err = 0.f;
    if constexpr (Doubt) {
        const float most = fmaxf(fabsf(lo), fabsf(hi));
        float r = max3(most, __shfl_sync(0xffffffffu, most, pair0), __shfl_sync(0xffffffffu, most, pair1));
        r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 1));
        err = kind == kRotated ? 0x1.8p-22f * r : 0.f;
    }
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
    const float m = bf16_floor(lo), range = __fsub_ru(hi, m), s = bf16_ceil15(range);
    low = upper_half(m);
    scale = upper_half(s);
    doubt = false;
    if constexpr (Doubt) {
        // whether the minimum's neighbourhood holds a bfloat16 (an exact minimum, of a lane that is not turned, stands), or
        // the range's, with what its own rounding added, 15 times one
        const float e = fmaf(range, 0x1p-22f, err), below = __uint_as_float(__float_as_uint(s) - 0x10000u);
        doubt = kind == kRotated && ((turned && own <= lo + 2.f * err && bf16_floor(lo - err) != bf16_floor(lo + err)) ||
                                     15.f * s < range + e || 15.f * below >= range - e);
    }
    if (s < kMinScale) {
        scale = __float2bfloat16(0.f);
        return make_uint2(0u, 0u);
    }
    // The nearest code of (x - m) / s without a division or a conversion.  The quotient times the rounded reciprocal,
    // corrected by its remainder, is the correctly rounded quotient (Markstein); adding 1.5 2^23 rounds that to
    // an integer in the low bits, borders (frequent in bfloat16 input) to the even code.
    const float inv = __frcp_rn(s);
    const float2 inv2 = make_float2(inv, inv), ns2 = make_float2(-s, -s), nm2 = make_float2(-m, -m),
                 magic = make_float2(12582912.f, 12582912.f);
    uint32_t w[2] = {0u, 0u};
    float off = 0.f;   // largest distance of a quotient from its code
#pragma unroll
    for (int e = 14; e >= 0; e -= 2) {
        const float2 d = add2(make_float2(x[e], x[e + 1]), nm2);
        float2 q = mul2(d, inv2);
        const float2 y = fma2(fma2(ns2, q, d), inv2, q);
        q = add2(y, magic);
        if constexpr (Doubt) {
            const float2 away = add2(y, add2(make_float2(-q.x, -q.y), magic));   // exact
            off = max3(off, fabsf(away.x), fabsf(away.y));
        }
        // the bits of 1.5 2^23 are taken off at the end, modulo 2^32
        w[e >> 3] = 16u * w[e >> 3] + __float_as_uint(q.y);
        w[e >> 3] = 16u * w[e >> 3] + __float_as_uint(q.x);
    }
    if (Doubt && kind != kExact) {
        doubt |= off > 0.5f - 0x1p-19f - err * inv;
    } else {
        const float q = -m * inv, zero = fmaf(fmaf(-s, q, -m), inv, q);   // the quotient of a 0, corrected as above
        doubt = m != 0.f && fabsf(m) < 0x1p-14f * range;
        if (fabsf(zero - ((zero + 12582912.f) - 12582912.f)) == 0.5f) {   // hardly ever
#pragma unroll
            for (int e = 0; e < 16; ++e) doubt |= x[e] != 0.f && fabsf(x[e]) < 0x1p-14f * fabsf(m);
        }
    }
    return make_uint2(w[0] - 0x4b400000u * 0x11111111u, w[1] - 0x4b400000u * 0x11111111u);
}

// Channel ch of a row in float64, rotated or as it is.
template <typename T>
__device__ __forceinline__ double rotated64(const RopeParams &p, const T *row, int ch, int pos, bool rotate)
{
    const double x = elem_f32(row[ch]);
    if (!rotate || ch >= p.rot) return x;
    const int half = p.rot / 2;
    const bool first = p.interleaved ? ch % 2 == 0 : ch < half;
    const int pair = p.interleaved ? ch / 2 : first ? ch : ch - half;
    const double o = elem_f32(row[p.interleaved ? ch ^ 1 : first ? ch + half : ch - half]);
    double c, s;
    turn(pos, p.turns[pair], p.amp, c, s);
    return first ? x * c - o * s : x * c + o * s;
}

// The groups that float32 leaves in doubt (of normal numbers one in 1100 where they
// are rotated, one in 10000 of float32 rows as they are, and hardly any of bfloat16
// rows as they are), decided in float64 from the rows
// themselves, a channel per lane: what is stored does not depend on float32's
// roundings, nor on float64's: the scale rounds up at each step, and a tie is broken
// by what x - m lost.  5.3k tokens take 1 us more, half of that with queries beside
// them.  All lanes of a warp call it, with
// what quantise16 gave them: lane l of a row holds channels 16 l .. 16 l + 15.
template <typename T>
__device__ __forceinline__ void settle(const RopeParams &p, bool doubt, const T *row, int l, int pos, bool rotate,
                                       uint2 &code, __nv_bfloat16 &scale, __nv_bfloat16 &low)
{
    const int lane = threadIdx.x & 31;
    for (unsigned todo = __ballot_sync(0xffffffffu, doubt); todo;) {   // warp-uniform
        const int owner = (__ffs(todo) - 1) & ~1;                      // the group's first lane
        todo &= ~(3u << owner);
        const T *r = reinterpret_cast<const T *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), owner));
        const int first = 16 * __shfl_sync(0xffffffffu, l, owner), at = __shfl_sync(0xffffffffu, pos, owner);
        const bool turned = __shfl_sync(0xffffffffu, rotate ? 1 : 0, owner) != 0;
        double x = rotated64(p, r, first + lane, at, turned);
        x = isnan(x) ? 0.0 : fmin(fmax(x, -(double)kMaxStored), (double)kMaxStored);
        double lo = x, hi = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const __nv_bfloat16 m = __float2bfloat16_rd(__double2float_rd(lo));
        const double md = __bfloat162float(m);
        __nv_bfloat16 s = __float2bfloat16_ru(__double2float_ru(__ddiv_ru(__dsub_ru(hi, md), 15.0)));
        const double d = x - md, back = d - x, lost = (x - (d - back)) - (md + back);   // d + lost = x - md
        const double y = d / (double)__bfloat162float(s), floor_y = floor(y);
        double t = rint(y);
        if (y - floor_y == 0.5 && lost != 0.0) t = lost > 0.0 ? floor_y + 1.0 : floor_y;
        if (__bfloat162float(s) < kMinScale) {
            s = __float2bfloat16(0.f);
            t = 0.0;
        }
        const uint32_t c = (uint32_t)(int)fmin(fmax(t, 0.0), 15.0) << (4 * (lane & 7));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __reduce_or_sync(0xffffffffu, lane >> 3 == i ? c : 0u);
        if ((lane & ~1) == owner) {
            code = lane & 1 ? make_uint2(w[2], w[3]) : make_uint2(w[0], w[1]);
            scale = s;
            low = m;
        }
    }
}

// Codes to numbers, two at a time (bfloat16 pairs).  A nibble alone in the low 8
// bits of a 16-bit lane is the tiny bfloat16 c 2^-133 (bits 0..3) or c 2^-129
// (bits 4..7: the exponent's last bit continues the subnormals linearly).  Times
// 2^127 it is c 2^-6 or c 2^-2, exactly, and one fused multiply-add with the scale
// times 2^6 or 2^2 (at most 2^123) and the minimum rounds m + c s once.  So a
// word of 8 codes needs one shift, 4 ANDs, 4 products and 4 fused operations.
struct Scale2 {
    uint32_t lo, hi, low;   // scale 2^6, scale 2^2, minimum
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ Scale2 scale2(uint32_t s2, uint32_t m2)
{
    return {mul_bf16x2(s2, 0x42804280u), mul_bf16x2(s2, 0x40804080u), m2};
}

__device__ __forceinline__ uint32_t stored2(uint32_t masked, uint32_t scale, uint32_t low)
{
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(mul_bf16x2(masked, 0x7f007f00u)), "r"(scale), "r"(low));
    return r;
}

// Pairs (nibble i, nibble i + 4) of a word, i = 0 .. 3.
__device__ __forceinline__ void stored8(uint32_t w, const Scale2 &s, uint32_t *out)
{
    const uint32_t v = w >> 8;
    out[0] = stored2(w & 0x000f000fu, s.lo, s.low);
    out[1] = stored2(w & 0x00f000f0u, s.hi, s.low);
    out[2] = stored2(v & 0x000f000fu, s.lo, s.low);
    out[3] = stored2(v & 0x00f000f0u, s.hi, s.low);
}

struct AppendIo {
    const void *k, *v, *q;
    void *q_out;
    long long ks, vs, qs;       // token strides in elements
    const int32_t *pos;         // rotary positions or null
    int H;                      // query heads (0: none)
    int kv_ctas, kv_per, q_per; // CTAs of the keys and values; tokens per CTA of either kind
};

// kv_ctas of the CTAs store keys and values, the others turn queries; both
// take whole tokens, like rope_kernel, start their loads, find the tokens'
// slots, fill the table and go through the rows.  Most of the bytes are the
// queries', but the rounding to codes, about 15 instructions a number, takes
// as long: side by side the one's memory time hides the other's issue slots
// (the same CTA doing one after the other measured 51 us where this took 34,
// 5.3k tokens of 32 + 2 x 8 heads; with settle and exact scales it takes 37.6, 2.5
// TB/s: the issue slots, 2.6 instructions a cycle, bound it, not HBM).
template <typename T, int D>
__global__ void __launch_bounds__(kTokThreads, 4)
    cache_append_kernel(const __grid_constant__ RopeParams p, const CacheParams c, const AppendIo io)
{
    constexpr int L = D / 16, R = kTokThreads / L;   // lanes per row (16 consecutive channels each), rows per pass
    using B = Blk<D>;
    __shared__ RopeTable table;
    __shared__ int s_slot[kTokMax], s_page[kTokMax];   // a token's slot (-1: not there) and page
    // the two kinds of CTAs evenly mixed over the grid
    const int kv_at = (int)((long long)blockIdx.x * io.kv_ctas / gridDim.x);
    const bool is_q = kv_at == (int)((blockIdx.x + 1LL) * io.kv_ctas / gridDim.x);
    const int per = is_q ? io.q_per : io.kv_per;
    const long long t0 = (long long)(is_q ? (int)blockIdx.x - kv_at : kv_at) * per;
    const int n = (int)min((long long)per, (long long)c.B * c.N - t0);
    griddep_wait();
    // slots and table, while the first loads are on their way
    auto begin = [&] {
        if (threadIdx.x < n) {
            const long long x = t0 + threadIdx.x;
            const int b = (int)(x / c.N), i = (int)(x - (long long)b * c.N);
            const Seq s = load_seq(c, b);
            int slot = -1, page = 0;
            if (i < s.q) {
                slot = s.kv - s.q + i;
                if (slot < 0) {
                    set_status(c.status, kDevBadPage);
                    slot = -1;
                } else if (!is_q) {
                    page = c.table[(size_t)b * c.max_pages + slot / c.page_size];
                }
            }
            s_slot[threadIdx.x] = slot;
            s_page[threadIdx.x] = page;
        }
        __syncthreads();
        if (p.on) {
            rope_fill(p, table, n, 1.f, [&](int i) { return io.pos ? io.pos[t0 + i] : s_slot[i]; });
            __syncthreads();
        }
    };
    if (is_q) {
        rope_rows<T, D, kRowBatch>(
            p, table, reinterpret_cast<const T *>(io.q) + t0 * io.qs, io.qs,
            reinterpret_cast<T *>(io.q_out) + t0 * io.H * D, (long long)io.H * D, n, io.H, begin,
            [&](int t) { return s_slot[t] >= 0; });
        return;
    }
    const int l = threadIdx.x % L, row0 = (threadIdx.x & 31) / L * L, rows = 2 * c.H_kv;
    bool bad = false;
    int tok = 0, h = threadIdx.x / L;
    auto wrap = [&](int &t, int &hh) {
        while (hh >= rows) {
            hh -= rows;
            ++t;
        }
    };
    auto load = [&](int t, int hh, Raw8<T> *raw) {
        if (t >= n) return;
        const T *src = (hh < c.H_kv ? reinterpret_cast<const T *>(io.k) + (t0 + t) * io.ks + hh * D
                                    : reinterpret_cast<const T *>(io.v) + (t0 + t) * io.vs + (hh - c.H_kv) * D) +
                       16 * l;
        raw[0].load(src);
        raw[1].load(src + 8);
    };
    wrap(tok, h);
    Raw8<T> raw[2];
    load(tok, h, raw);
    begin();
    const int hc = p.rot / 16;                    // chunks of 8 channels in a half
    // half layout: the lanes that hold the partners of this lane's two chunks
    const auto partner = [&](int ch) { return ch >= 2 * hc || p.interleaved ? ch : ch < hc ? ch + hc : ch - hc; };
    const int pair0 = row0 + (partner(2 * l) >> 1), pair1 = row0 + (partner(2 * l + 1) >> 1);
    for (int base = 0; base < n * rows; base += R) {   // CTA-uniform
        const int slot = tok < n ? s_slot[tok] : -1;
        const bool is_k = slot >= 0 && h < c.H_kv, ok = slot >= 0;
        float x[16];
        raw[0].widen(x);
        raw[1].widen(x + 8);
        const int tok1 = tok, h1 = h;
        h += R;
        wrap(tok, h);
        if (base + R < n * rows) load(tok, h, raw);
        if (p.on && __any_sync(0xffffffffu, is_k)) {
            const float *tc = table.c + (ok ? tok1 : 0) * kRopeMaxPairs, *ts = table.s + (ok ? tok1 : 0) * kRopeMaxPairs;
            if (p.interleaved) {
                if (is_k && 16 * l < p.rot) rope_apply(p, table, tok1, l, x, x + 8);
            } else {   // a chunk's partner is in another lane, in the other of its two chunks when hc is odd
                const bool swap = hc & 1;
                float o[16];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[8 * k + e] = __shfl_sync(0xffffffffu, swap ? x[8 * (1 - k) + e] : x[8 * k + e], k ? pair1 : pair0);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int ch = 2 * l + k;
                    const bool first = ch < hc;
                    if (is_k && ch < 2 * hc) {
                        const int at = 8 * (first ? ch : ch - hc);
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const float4 cc = *reinterpret_cast<const float4 *>(tc + at + e);
                            const float4 ss = *reinterpret_cast<const float4 *>(ts + at + e);
                            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float q = o[8 * k + e + i] * sv[i];
                                x[8 * k + e + i] = fmaf(x[8 * k + e + i], cv[i], first ? -q : q);
                            }
                        }
                    }
                }
            }
        }
        __nv_bfloat16 scale, low;
        bool nf = false, doubt = false;
        uint2 code;
        const Exactness kind = p.on && is_k && 32 * (l / 2) < p.rot ? kRotated : sizeof(T) == 4 ? kFloat : kExact;
        if (__any_sync(0xffffffffu, kind != kExact))
            code = quantise16<true>(x, scale, low, nf, kind, p.on && is_k && 16 * l < p.rot, pair0, pair1, doubt);
        else
            code = quantise16<false>(x, scale, low, nf, kind, false, pair0, pair1, doubt);
        if (__any_sync(0xffffffffu, doubt && ok)) {
            const T *src = is_k ? reinterpret_cast<const T *>(io.k) + (t0 + tok1) * io.ks + h1 * D
                                : reinterpret_cast<const T *>(io.v) + (t0 + tok1) * io.vs + (h1 - c.H_kv) * D;
            settle<T>(p, doubt && ok, src, l, ok && io.pos ? io.pos[t0 + tok1] : slot, p.on && is_k, code, scale, low);
        }
        if (!ok) continue;
        bad |= nf;
        const int t = slot & 15;
        uint8_t *blk = block_at<D>(c, s_page[tok1], is_k ? h1 : h1 - c.H_kv, slot);
        if (!blk) continue;
        if (is_k) {
            *reinterpret_cast<uint2 *>(blk + B::k_codes(t) + 8 * l) = code;
            if (l % 2 == 0) *reinterpret_cast<__nv_bfloat162 *>(blk + B::k_pair(t, l / 2)) = __nv_bfloat162(scale, low);
        } else {
            if constexpr (D == 128) {
                *reinterpret_cast<uint2 *>(blk + B::v_codes(t, l)) = code;
            } else {
                *reinterpret_cast<uint32_t *>(blk + B::v_codes(t, 2 * l)) = code.x;
                *reinterpret_cast<uint32_t *>(blk + B::v_codes(t, 2 * l + 1)) = code.y;
            }
            // the pair's two lanes write one number each
            *reinterpret_cast<__nv_bfloat16 *>(blk + B::v_scale(t, l / 2) + 4 * (l & 1)) = l & 1 ? low : scale;
        }
    }
    if (bad) set_status(c.status, kDevNonFinite);
}

// 32 bytes of an output row: one store when the tensors allow it (wide: 32-byte aligned).
__device__ __forceinline__ void store32(void *p, const uint32_t *w, bool wide)
{
    if (!wide) {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// bf16 pairs (channel 2 i, 2 i + 1) of the 8 codes of a word.
__device__ __forceinline__ void stored8_in_order(uint32_t w, const Scale2 &s, uint32_t *out)
{
    uint32_t v[4];
    stored8(w, s, v);
    out[0] = __byte_perm(v[0], v[1], 0x5410);
    out[1] = __byte_perm(v[2], v[3], 0x5410);
    out[2] = __byte_perm(v[0], v[1], 0x7632);
    out[3] = __byte_perm(v[2], v[3], 0x7632);
}

// 16 channels given as 8 bf16 pairs into an output row.
template <typename T>
__device__ __forceinline__ void store16(T *p, const uint32_t *w, bool wide)
{
    if constexpr (sizeof(T) == 2) {
        store32(p, w, wide);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = w[4 * k + i] << 16;
                f[2 * i + 1] = w[4 * k + i] & 0xffff0000u;
            }
            store32(p + 8 * k, f, wide);
        }
    }
}

// A warp reads one block (16 slots of a KV head) of a sequence: HBM bounds it,
// so all of the block's loads are started before the first code is turned into
// a number, and a lane writes whole 32-byte sectors.  Slots that the call does
// not read are skipped at the stores.  4 histories of 9k .. 16k tokens, 8 KV heads, D = 128, into
// bfloat16 (300 MB): 50.8 us, 5.9 TB/s, 90 % of a copy's rate.
constexpr int kReadWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kReadWarps) cache_read_kernel(const CacheParams c, T *k_out, T *v_out, int blocks, int wide)
{
    constexpr int L = D / 16, R = 32 / L, P = 16 / R;   // lanes per row (16 channels each), rows per step, steps
    using B = Blk<D>;
    griddep_wait();
    const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
    const long long w = (long long)blockIdx.x * kReadWarps + (threadIdx.x >> 5);   // (sequence, block, KV head)
    if (w >= (long long)c.B * blocks * c.H_kv) return;
    const int h = (int)(w % c.H_kv);
    const long long x = w / c.H_kv;
    const int b = (int)(x / blocks), i = (int)(x - (long long)b * blocks);
    const Seq s = load_seq(c, b);
    if (s.kv < s.q) set_status(c.status, kDevBadPage);   // tokens below slot 0
    const int first = s.kv - s.q, slot0 = (max(first, 0) & ~15) + 16 * i;
    if (slot0 >= s.kv || s.q == 0) return;
    const uint8_t *blk = block_at<D>(c, c.table[(size_t)b * c.max_pages + slot0 / c.page_size], h, slot0);
    if (!blk) return;
    const int g = j / 2;   // 16 channels lie in one group of 32
    uint2 kc[P], vc[P];
    uint32_t kp[P], vs[P], vm[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int t = k * R + sub;
        if (k_out) {
            kc[k] = *reinterpret_cast<const uint2 *>(blk + B::k_codes(t) + 8 * j);
            kp[k] = *reinterpret_cast<const uint32_t *>(blk + B::k_pair(t, g));
        }
        if (v_out) {
            if constexpr (D == 128) {
                vc[k] = *reinterpret_cast<const uint2 *>(blk + B::v_codes(t, j));
            } else {
                vc[k].x = *reinterpret_cast<const uint32_t *>(blk + B::v_codes(t, 2 * j));
                vc[k].y = *reinterpret_cast<const uint32_t *>(blk + B::v_codes(t, 2 * j + 1));
            }
            vs[k] = *reinterpret_cast<const uint16_t *>(blk + B::v_scale(t, g));
            vm[k] = *reinterpret_cast<const uint16_t *>(blk + B::v_scale(t, g) + 4);
        }
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int slot = slot0 + k * R + sub;
        if (slot < first || slot >= s.kv) continue;
        const size_t at = (((size_t)b * c.N + slot - first) * c.H_kv + h) * D + 16 * j;
        uint32_t out[8];
        if (k_out) {
            const Scale2 s2 = scale2(__byte_perm(kp[k], kp[k], 0x1010), __byte_perm(kp[k], kp[k], 0x3232));
            stored8_in_order(kc[k].x, s2, out);
            stored8_in_order(kc[k].y, s2, out + 4);
            store16<T>(k_out + at, out, wide);
        }
        if (v_out) {
            const Scale2 s2 = scale2(vs[k] | vs[k] << 16, vm[k] | vm[k] << 16);
            stored8_in_order(vc[k].x, s2, out);
            stored8_in_order(vc[k].y, s2, out + 4);
            store16<T>(v_out + at, out, wide);
        }
    }
}

}  // namespace akv
