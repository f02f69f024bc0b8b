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

// Quantise the lane's 8 channels; the 32-channel group is 4 consecutive lanes
// (all lanes of the warp call it).  Returns the 8 codes, channel e at bits 4 e.
__device__ __forceinline__ uint32_t quantise8(float *x, __nv_bfloat16 &scale, __nv_bfloat16 &low, bool &bad)
{
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (!(fabsf(x[e]) <= 3.402823466e38f)) bad = true;   // infinity or NaN
        x[e] = isnan(x[e]) ? 0.f : fminf(fmaxf(x[e], -kMaxStored), kMaxStored);
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    low = __float2bfloat16_rd(lo);
    const float m = __bfloat162float(low);
    scale = __float2bfloat16_ru(__fdiv_rn(hi - m, 15.f));
    float s = __bfloat162float(scale);
    if (s < kMinScale) {
        s = 0.f;
        scale = __float2bfloat16(0.f);
    }
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = s > 0.f ? rintf(__fdiv_rn(x[e] - m, s)) : 0.f;
        w |= (uint32_t)(int)fminf(fmaxf(t, 0.f), 15.f) << (4 * e);
    }
    return w;
}

// bf16(low + c scale) of the 8 codes of a word.
__device__ __forceinline__ void stored8(uint32_t w, __nv_bfloat16 scale, __nv_bfloat16 low, float *x)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = __bfloat162float(__hfma(__float2bfloat16((float)((w >> (4 * e)) & 15u)), scale, low));
}

struct AppendIo {
    const void *k, *v, *q;
    void *q_out;
    long long ks, vs, qs;       // token strides in elements
    const int32_t *pos;         // rotary positions or null
    int H, rows_per_warp;       // query heads (0: none); rows of a token per warp
};

constexpr int kAppendThreads = 256;

// A token's rows are its H_kv keys, its H_kv values and its H queries; a warp
// takes rows_per_warp of them.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads)
    cache_append_kernel(const __grid_constant__ RopeParams p, const CacheParams c, const AppendIo io)
{
    constexpr int L = D / 8, R = 32 / L;
    using B = Blk<D>;
    __shared__ double turns[kRopeMaxPairs];
    rope_turns(p, turns);
    const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
    const int rows = 2 * c.H_kv + io.H, parts = (rows + io.rows_per_warp - 1) / io.rows_per_warp;
    const long long w = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (w >= (long long)c.B * c.N * parts) return;
    const long long tok = w / parts;
    const int b = (int)(tok / c.N), n = (int)(tok - (long long)b * c.N);
    const Seq s = load_seq(c, b);
    if (n >= s.q) return;
    const int slot = s.kv - s.q + n;
    if (slot < 0) {
        set_status(c.status, kDevBadPage);
        return;
    }
    const int page = c.table[(size_t)b * c.max_pages + slot / c.page_size];
    const RopeLane r = rope_lane(p, turns, j, io.pos ? io.pos[tok] : slot, false);
    const int r0 = (int)(w - tok * parts) * io.rows_per_warp, r1 = min(rows, r0 + io.rows_per_warp);
    bool bad = false;
    for (int i = r0; i < r1; i += R) {
        const int row = i + sub;
        const bool ok = row < r1, is_k = row < c.H_kv, is_q = row >= 2 * c.H_kv;
        const int h = is_k ? row : is_q ? row - 2 * c.H_kv : row - c.H_kv;
        const T *src = is_k   ? reinterpret_cast<const T *>(io.k) + tok * io.ks
                       : is_q ? reinterpret_cast<const T *>(io.q) + tok * io.qs
                              : reinterpret_cast<const T *>(io.v) + tok * io.vs;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, y[8];
        if (ok) load8<T>(src + (size_t)h * D + 8 * j, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e];
        rope_apply(p, r, sub * L, y);
        if (is_k || is_q) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[e];
        }
        if (ok && is_q) store8<T>(reinterpret_cast<T *>(io.q_out) + ((size_t)tok * io.H + h) * D + 8 * j, x);
        if (__any_sync(0xffffffffu, ok && !is_q)) {   // keys or values among the warp's rows
            __nv_bfloat16 scale, low;
            bool nf = false;
            const uint32_t code = quantise8(x, scale, low, nf);
            if (ok && !is_q) {
                bad |= nf;
                uint8_t *blk = block_at<D>(c, page, h, slot);
                const int t = slot & 15;
                if (blk && is_k) {
                    *reinterpret_cast<uint32_t *>(blk + B::k_codes(t) + 4 * j) = code;
                    if (j % 4 == 0)
                        *reinterpret_cast<__nv_bfloat162 *>(blk + B::k_pair(t, j / 4)) = __nv_bfloat162(scale, low);
                } else if (blk) {
                    *reinterpret_cast<uint32_t *>(blk + B::v_codes(t, 64 * j / D) + (D == 128 ? (j & 1) * 4 : 0)) = code;
                    if (j % 4 == 0) {
                        *reinterpret_cast<__nv_bfloat16 *>(blk + B::v_scale(t, j / 4)) = scale;
                        *reinterpret_cast<__nv_bfloat16 *>(blk + B::v_scale(t, j / 4) + 4) = low;
                    }
                }
            }
        }
    }
    if (bad) set_status(c.status, kDevNonFinite);
}

// A warp reads the key and the value rows of one (token, KV head) per row slot.
template <typename T, int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheParams c, T *k_out, T *v_out)
{
    constexpr int L = D / 8, R = 32 / L;
    using B = Blk<D>;
    const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
    const long long row = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * R + sub;
    if (row >= (long long)c.B * c.N * c.H_kv) return;
    const int h = (int)(row % c.H_kv);
    const long long tok = row / c.H_kv;
    const int b = (int)(tok / c.N), n = (int)(tok - (long long)b * c.N);
    const Seq s = load_seq(c, b);
    if (n >= s.q) return;
    const int slot = s.kv - s.q + n;
    if (slot < 0) {
        set_status(c.status, kDevBadPage);
        return;
    }
    const uint8_t *blk = block_at<D>(c, c.table[(size_t)b * c.max_pages + slot / c.page_size], h, slot);
    if (!blk) return;
    const int t = slot & 15;
    float x[8];
    if (k_out) {
        const __nv_bfloat162 pr = *reinterpret_cast<const __nv_bfloat162 *>(blk + B::k_pair(t, j / 4));
        stored8(*reinterpret_cast<const uint32_t *>(blk + B::k_codes(t) + 4 * j), pr.x, pr.y, x);
        store8<T>(k_out + (size_t)row * D + 8 * j, x);
    }
    if (v_out) {
        const __nv_bfloat16 *pr = reinterpret_cast<const __nv_bfloat16 *>(blk + B::v_scale(t, j / 4));
        stored8(*reinterpret_cast<const uint32_t *>(blk + B::v_codes(t, 64 * j / D) + (D == 128 ? (j & 1) * 4 : 0)),
                pr[0], pr[2], x);
        store8<T>(v_out + (size_t)row * D + 8 * j, x);
    }
}

}  // namespace akv
