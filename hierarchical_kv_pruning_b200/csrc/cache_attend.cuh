// Attention of new tokens over the 4-bit paged cache.
#pragma once

#include "kvcache.cuh"
#include "tcgen05.cuh"

namespace akv {

struct CacheAttendIo {
    const void *q;
    void *out;          // [B][N][H][D]
    float *lse;         // [B][N][H], or null
    float *oseq;        // not null: the result goes here and to lse_seq, float32, row (b, KV head, g N + n)
    float *lse_seq;
    long long qs;       // token stride of q in elements
    int H, G;
    float scale_log2;   // scale * log2(e)
    uint8_t *ws;        // workspace
};

// Four channels of one row's result: O / L, and the log-sum-exp with the first.
template <typename T, int D>
__device__ __forceinline__ void ca_write(const CacheParams &c, const CacheAttendIo &io, int b, int hkv, int row, int d4,
                                         float4 o, float M, float L)
{
    const int n = row / io.G, g = row - n * io.G;
    const size_t at = ((size_t)b * c.N + n) * io.H + hkv * io.G + g;
    const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;   // nothing visible: 0; NaN stays
    if (io.oseq) {
        const size_t r = (((size_t)b * c.H_kv + hkv) * io.G + g) * c.N + n;
        *reinterpret_cast<float4 *>(io.oseq + r * D + d4) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (d4 == 0) io.lse_seq[r] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
        return;
    }
    T *dst = reinterpret_cast<T *>(io.out) + at * D + d4;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), e = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&e));
    }
    if (io.lse && d4 == 0) io.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

// ---- few query rows per KV head: decode and short drafts -------------------------
//
// For one KV head the query rows are (token n, head g of the group), row
// n G + g; a unit of work is 32 stored tokens against a block of 8 NT rows.
// Per row the online softmax keeps a running maximum m, sum l and output O:
//     S = q k;  p = 2^(S scale log2 e - m);  l += sum p;  O += p v.
// What bounds it: the codes are read once and every code becomes a bfloat16,
// exactly the stored number, at 13 instructions a word of 8.  A unit (D = 128,
// 8 rows) takes 760 warp instructions for 5120 bytes, 270 of them the 8192 codes'
// and 64 products; at 2.6 issued a cycle the issue slots are nearer their limit
// than HBM.  64 sequences of 700 .. 8192 tokens, 8 KV heads, one token of 32 heads
// (374 MB): 97 us, 3.9 TB/s.  Two of 131k .. 262k tokens, one KV head, 32 rows (76 MB):
// 51 us; there the products of 4 x 8 rows (38 % of the tensor pipe) and 253
// registers a thread, so two CTAs an SM, bound it.  One sequence of 513 tokens: 10 us,
// a chain of the plan, the table, a copy and five rounds of units (1 us each).
//
// Rounding: logits, maxima, sums and O are float32.  A bfloat16 call's
// probabilities are rounded to bfloat16 for their product with V (2^-9 each, as in
// the dense sequence attention; O is rounded as much at the end, and a second
// part would double that product), the sum l takes them unrounded; a float32
// call's are three bfloat16 parts, exact to 2^-24.  The matrix unit's sums are cut,
// not rounded, which a bfloat16 call does not feel; a float32 call's sums over a
// step of 32 channels or of 16 tokens are taken from 0 and added to the running
// ones by rounded additions.  With one running sum all the way, outputs over 16000
// tokens were 9e-6 too small; now they are 1.6e-7 too small and off by 4e-7 of their
// norm, for 2 to 9 % more time (512 x 16 rows of 128 or 64 channels over 16000
// tokens: 616 -> 628, 363 -> 395 us).
//
// The products run on m16n8k16 with the cache as the 16-row operand, S^T = K
// Q^T and O^T = V^T P^T: a decode step has few rows, so they take the 8-wide
// side (tcgen05 has 128-row operands only, and its operands go through shared
// memory or TMEM, while here a lane's codes become its own fragment in
// registers).  The order of channels in the contraction and of output channels
// is free, which lets a lane read its codes in 16-byte pieces.  P^T comes from
// S^T by transposing 8 x 8 tiles between lanes (movmatrix).
//
// Work is split over sequences, KV heads and tokens alike: the units of all
// (sequence, KV head, row block) items in order are cut into equal runs, one per
// CTA, from the lengths on the device.  An item inside a run is finished there;
// an item that a cut divides leaves partial (O, m, l) in the workspace, which
// cache_combine_kernel joins.  Four warps of a CTA take units in turn, each
// with a ring of bulk copies (a unit of a page is contiguous) of its own, and
// join their rows in shared memory at the end of an item.

constexpr int kCaWarps = 4;
constexpr int kCaThreads = 32 * kCaWarps;
constexpr int kCaUnit = 32;   // stored tokens of a unit: two blocks

template <typename T, int D, int NT>
struct Ca {
    static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;   // bfloat16 parts of a query element and of a probability
    static constexpr int kRB = 8 * NT;                      // rows of a row block
    static constexpr bool kQRegs = NT * kParts <= 2;        // query fragments in registers, else in shared memory
    static constexpr int kCtas = NT * kParts == 1 ? 4 : NT * kParts == 2 ? 3 : 2;   // per SM
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kUnitBytes = 2 * Blk<D>::kBytes;
    static constexpr int kRing = kCaWarps * kStages * kUnitBytes;
    static constexpr int kMergeRow = D + 4;                 // floats
    static constexpr int kMerge = kCaWarps * 8 * (kMergeRow + 2) * 4;   // overlays the ring
    static_assert(kMerge <= kRing, "the merge buffer overlays the ring");
    static constexpr int kOffQ = kRing;
    static constexpr int kQBytes = kQRegs ? 0 : kParts * NT * (D / 16) * 32 * 8;
    static constexpr int kOffBar = kOffQ + kQBytes;
    static constexpr int kSmem = kOffBar + kCaWarps * kStages * 8;
    static constexpr int kSlot = kRB * (D + 2);             // floats of a partial: O, m, l
};

// A divided item costs about as much as this many units more on every CTA: the
// join takes about 4 us, four units (one a warp) about 1.1 us where a warp is alone.
constexpr int kCaPartialUnits = 20;

// Whether whole items, round-robin over the CTAs, end about as early as equal
// runs of units would.
__host__ __device__ __forceinline__ bool ca_whole(long long items, long long ctas, long long longest, long long total,
                                                  int partial_units)
{
    // ceil(items / ctas) longest <= ceil(total / ctas) + partial_units, without 64-bit divisions where they fit 32 bits
    const bool small = ((items | total | ctas) >> 31) == 0;
    const long long rounds = small ? (uint32_t)(items + ctas - 1) / (uint32_t)ctas : (items + ctas - 1) / ctas;
    const long long run = small ? (uint32_t)(total + ctas - 1) / (uint32_t)ctas : (total + ctas - 1) / ctas;
    return rounds * longest <= run + partial_units;
}

// What CTA c left for the join: its first item, where in it the CTA began.
struct CaDesc {
    long long total;        // units of the call
    int active;             // CTAs with units
    int k0, units;          // first unit within the item (0: not divided before it); the item's units
    int b, hkv, rb;
};

// A CTA's walk over its runs of units, kept in shared memory by one thread.
struct CaWalk {
    long long total, u, end, off;   // units of the call; next unit (item) and the end; its offset within sequence b
    int active, whole, b;           // CTAs with units; whole items?
};

// One stretch of an item's units.
struct CaSeg {
    Seq s;
    int b, hkv, rb, k0, cnt, units;   // cnt = 0: no more
};

// a / b of numbers >= 0: a 64-bit division takes some 100 instructions, and the
// plans of small calls are a chain of them.
__device__ __forceinline__ long long ca_div(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ long long ca_start(long long total, int active, int c) { return ca_div(total * c, active); }

__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, const uint32_t *b)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ void add4(float *d, const float *a)
{
    const float2 x = add2(make_float2(d[0], d[1]), make_float2(a[0], a[1])), y = add2(make_float2(d[2], d[3]), make_float2(a[2], a[3]));
    d[0] = x.x;
    d[1] = x.y;
    d[2] = y.x;
    d[3] = y.y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(mbar)
                 : "memory");
}

// 8 query channels as kParts x 4 bf16 pairs (channel i, channel i + 4): the
// float32 value is the exact sum of three bfloat16 parts.
template <typename T>
__device__ __forceinline__ void query_pairs(const float *x, uint32_t (*out)[4])
{
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rest[e] = x[e];
#pragma unroll
    for (int p = 0; p < (sizeof(T) == 4 ? 3 : 1); ++p) {
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = __bfloat162float(__float2bfloat16(rest[e]));
            rest[e] -= h[e];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) out[p][i] = pack_bf16(h[i], h[i + 4]);
    }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kCaThreads, Ca<T, D, NT>::kCtas)
    cache_attend_kernel(const CacheParams c, const CacheAttendIo io)
{
    using C = Ca<T, D, NT>;
    using B = Blk<D>;
    constexpr int P = C::kParts, KS = D / 16, S = C::kStages;
    extern __shared__ __align__(128) uint8_t ca_smem[];
    __shared__ long long s_sum[kCaWarps], s_items[kCaWarps];
    __shared__ int s_top[kCaWarps];
    __shared__ CaWalk walk;
    __shared__ CaSeg segs[2];
    __shared__ long long s_first[kCaThreads + 1];   // items before thread t's sequences
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
    const uint32_t sb = tc::smem_addr(ca_smem);
    const uint32_t ring = sb + warp * S * C::kUnitBytes, bars = sb + C::kOffBar + warp * S * 8;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) tc::mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    griddep_launch();
    griddep_wait();

    // ---- this CTA's run of units ----
    auto n_blocks = [&](const Seq &s) { return (io.G * s.q + C::kRB - 1) / C::kRB; };
    auto n_units = [&](const Seq &s) { return max(1, (s.kv + kCaUnit - 1) / kCaUnit); };
    auto total_of = [&](int b) -> long long {
        const Seq s = load_seq(c, b);
        return (long long)c.H_kv * n_blocks(s) * n_units(s);
    };
    const int per = (c.B + kCaThreads - 1) / kCaThreads, b_lo = min(c.B, tid * per), b_hi = min(c.B, b_lo + per);
    long long mine = 0, items = 0;
    int top = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const Seq s = load_seq(c, b);
        const long long n = (long long)c.H_kv * n_blocks(s);
        items += n;
        mine += n * n_units(s);
        top = max(top, n > 0 ? n_units(s) : 0);
    }
    long long scan = mine, iscan = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, scan, o), x = __shfl_up_sync(0xffffffffu, iscan, o);
        if (lane >= o) {
            scan += v;
            iscan += x;
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (lane == 31) {
        s_sum[warp] = scan;
        s_items[warp] = iscan;
        s_top[warp] = top;
    }
    __syncthreads();
    long long total = 0, before = scan - mine, all = 0, ibefore = iscan - items;
    int longest = 0;
#pragma unroll
    for (int w = 0; w < kCaWarps; ++w) {
        if (w < warp) {
            before += s_sum[w];
            ibefore += s_items[w];
        }
        total += s_sum[w];
        all += s_items[w];
        longest = max(longest, s_top[w]);
    }
    s_first[tid] = ibefore;
    if (tid == 0) s_first[kCaThreads] = all;
    CaDesc *desc = reinterpret_cast<CaDesc *>(io.ws) + blockIdx.x;
    if (tid == 0) desc->k0 = 0;   // until the CTA begins inside an item
    {
        const bool whole = ca_whole(all, gridDim.x, longest, total, kCaPartialUnits);
        const int active = (int)max(1LL, min((long long)gridDim.x, (total + kCaWarps - 1) / kCaWarps));
        if (blockIdx.x >= (whole ? all : min((long long)active, total))) return;   // CTA-uniform
        const long long u = whole ? 0 : ca_start(total, active, blockIdx.x);
        if (u >= before && u < before + mine) {   // the thread whose sequences hold the CTA's first unit
            long long off = u - before;
            int b = b_lo;
            for (; !whole; ++b) {
                const long long n = total_of(b);
                if (off < n) break;
                off -= n;
            }
            walk = CaWalk{total, whole ? blockIdx.x : u, whole ? all : ca_start(total, active, blockIdx.x + 1), off, active,
                          whole, b};
        }
    }
    // the next stretch, by one thread: while the CTA is busy with the one before
    auto advance = [&](CaSeg &g) {
        CaWalk w = walk;
        g.cnt = 0;
        if (w.whole) {   // item w.u: the thread whose sequences hold it, then its place among them
            if (w.u >= s_first[kCaThreads]) return;
            int lo = 0, hi = kCaThreads;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                (s_first[mid] <= w.u ? lo : hi) = mid;
            }
            w.b = lo * per;
            w.off = w.u - s_first[lo];
        }
        while (w.b < c.B && w.u < w.end) {
            const Seq s = load_seq(c, w.b);
            const int nb = n_blocks(s), units = n_units(s);
            const long long n = (long long)c.H_kv * nb * (w.whole ? 1 : units);
            if (w.off >= n) {
                w.off -= n;
                ++w.b;
                continue;
            }
            const int item = (int)(w.whole ? w.off : ca_div(w.off, units));
            g.s = s;
            g.b = w.b;
            g.hkv = item / nb;
            g.rb = item - g.hkv * nb;
            g.units = units;
            g.k0 = w.whole ? 0 : (int)(w.off - (long long)item * units);
            g.cnt = w.whole ? units : (int)min((long long)(units - g.k0), w.end - w.u);
            w.u += w.whole ? gridDim.x : g.cnt;
            w.off += g.cnt;
            break;
        }
        walk = w;
    };
    __syncthreads();
    if (tid == 0) {
        advance(segs[0]);
        if (segs[0].k0 > 0)
            *desc = CaDesc{walk.total, walk.active, segs[0].k0, segs[0].units, segs[0].b, segs[0].hkv, segs[0].rb};
    }
    __syncthreads();

    int T_ = 0;   // units this warp has taken from its ring
    bool failed = false;
    for (int si = 0;; si ^= 1) {
        const CaSeg &seg = segs[si];
        if (seg.cnt == 0) break;   // CTA-uniform
        const Seq s = seg.s;
        const int b = seg.b, hkv = seg.hkv, rb = seg.rb, k0 = seg.k0, cnt = seg.cnt;
        const int R = io.G * s.q, row0 = rb * C::kRB;
        // last visible slot of this lane's rows (row 2 t, 2 t + 1 of each 8), and of the block's first row
        int lim[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                lim[j][e] = s.kv - s.q + min(row0 + 8 * j + 2 * t + e, R - 1) / io.G;
        const int lim_first = s.kv - s.q + row0 / io.G;
        const int lim_last = s.kv - s.q + (min(row0 + C::kRB, R) - 1) / io.G;   // and of its last row

        // ---- copies ----
        const int mine_n = cnt > warp ? (cnt - warp + kCaWarps - 1) / kCaWarps : 0;
        const int32_t *tab = c.table + (size_t)b * c.max_pages;
        const int pshift = 31 - __clz(c.page_size);
        // lane j looks the blocks of this warp's units j, j + 32, .. up in the table: block indices in the pool
        auto find = [&](int i, uint32_t &x, uint32_t &y) {
            const int slot = (k0 + warp + kCaWarps * i) * kCaUnit;
            x = y = 0u;
            if (i >= mine_n || slot >= s.kv) return;
            auto at = [&](int sl) -> uint32_t {
                int page = tab[sl >> pshift];
                if ((unsigned)page >= (unsigned long long)c.n_pages) {   // reported; another page's bytes stand in
                    set_status(c.status, kDevBadPage);
                    page = 0;
                }
                return (uint32_t)((((long long)page * c.H_kv + hkv) << (pshift - 4)) + ((sl & (c.page_size - 1)) >> 4));
            };
            x = at(slot);
            y = slot + 16 >= s.kv ? 0u : c.page_size > 16 ? x + 1 : at(slot + 16);
        };
        uint32_t at0, at1, nx0 = 0, nx1 = 0;
        find(lane, at0, at1);
        if (mine_n > 32) find(32 + lane, nx0, nx1);
        auto issue = [&](int i) {   // warp-uniform i
            const int j = i & 31;
            if (j == 0 && i > 0) {
                at0 = nx0;
                at1 = nx1;
                find(i + 32 + lane, nx0, nx1);
            }
            const uint32_t x = __shfl_sync(0xffffffffu, at0, j), y = __shfl_sync(0xffffffffu, at1, j);
            if (lane == 0) {
                const int st = (T_ + i) % S;
                const uint32_t bar = bars + 8 * st, dst = ring + st * C::kUnitBytes;
                const uint8_t *src = c.pages + (unsigned long long)x * B::kBytes;
                if (y == x + 1) {
                    tc::mbar_arrive_expect_tx(bar, 2 * B::kBytes);
                    bulk_load(dst, src, 2 * B::kBytes, bar);
                } else if ((k0 + warp + kCaWarps * i) * kCaUnit + 16 < s.kv) {
                    tc::mbar_arrive_expect_tx(bar, 2 * B::kBytes);
                    bulk_load(dst, src, B::kBytes, bar);
                    bulk_load(dst + B::kBytes, c.pages + (unsigned long long)y * B::kBytes, B::kBytes, bar);
                } else {
                    tc::mbar_arrive_expect_tx(bar, B::kBytes);
                    bulk_load(dst, src, B::kBytes, bar);
                }
            }
        };
        const int n_run = s.kv > 0 && !failed ? mine_n : 0;
        for (int i = 0; i < min(S - 1, n_run); ++i) issue(i);
        if (tid == 0) advance(segs[si ^ 1]);

        // ---- queries ----
        uint32_t qf[C::kQRegs ? P : 1][C::kQRegs ? NT : 1][KS][2];
        auto load_queries = [&](int j, auto &&store) {
            const int row = row0 + 8 * j + r;
            const bool ok = row < R;
            const int tok = ok ? row / io.G : 0, g = ok ? row - tok * io.G : 0;
            const T *q = reinterpret_cast<const T *>(io.q) + ((size_t)b * c.N + tok) * io.qs +
                         (size_t)(hkv * io.G + g) * D + t * (D / 4);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (ok) load8<T>(q + 8 * w, x);
                uint32_t pr[P][4];
                query_pairs<T>(x, pr);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    store(p, 2 * w, pr[p][0], pr[p][1]);
                    store(p, 2 * w + 1, pr[p][2], pr[p][3]);
                }
            }
        };
        uint2 *q_sm = reinterpret_cast<uint2 *>(ca_smem + C::kOffQ);
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                load_queries(j, [&](int p, int ks, uint32_t x, uint32_t y) {
                    qf[p][j][ks][0] = x;
                    qf[p][j][ks][1] = y;
                });
        } else {
            for (int j = warp; j < NT; j += kCaWarps)
                load_queries(j, [&](int p, int ks, uint32_t x, uint32_t y) {
                    q_sm[((p * NT + j) * KS + ks) * 32 + lane] = make_uint2(x, y);
                });
            __syncthreads();
        }

        float acc[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][k][e] = 0.f;
            m[j][0] = m[j][1] = -INFINITY;
            l[j][0] = l[j][1] = 0.f;
        }

        for (int i = 0; i < n_run; ++i) {
            if (i + S - 1 < n_run) issue(i + S - 1);
            const int st = (T_ + i) % S;
            if (__any_sync(0xffffffffu, !tc::mbar_wait(bars + 8 * st, ((T_ + i) / S) & 1))) {
                failed = true;   // the copies still in flight must land before the CTA ends
                for (int x = i; x < min(i + S, n_run); ++x) tc::mbar_wait(bars + 8 * ((T_ + x) % S), ((T_ + x) / S) & 1);
                break;
            }
            const int key0 = (k0 + warp + kCaWarps * i) * kCaUnit;
            if (key0 > lim_last) {   // past every row of the block
                __syncwarp();
                continue;
            }
            const uint8_t *ub = ca_smem + (ring - sb) + st * C::kUnitBytes;
            float sc[2][NT][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[k][j][e] = 0.f;
            // ---- S^T = K Q^T: a lane holds tokens r, r + 8, channels t D / 4 .. ----
            // (a second block past the sequence was not copied: what lies there is masked below)
            uint32_t w[2][2][D / 32];
            Scale2 ks[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *blk = ub + k * B::kBytes;
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(blk + B::k_codes(r + 8 * h) + t * 16);
                        w[k][h][0] = v.x;
                        w[k][h][1] = v.y;
                        w[k][h][2] = v.z;
                        w[k][h][3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(blk + B::k_codes(r + 8 * h) + t * 8);
                        w[k][h][0] = v.x;
                        w[k][h][1] = v.y;
                    }
                    const uint32_t pr =
                        *reinterpret_cast<const uint32_t *>(blk + B::k_pair(r + 8 * h, t * (D / 4) / 32));
                    ks[k][h] = scale2(prmt(pr, pr, 0x1010), prmt(pr, pr, 0x3232));
                }
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                uint32_t n[2][2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) stored8(w[k][h][x], ks[k][h], n[k][h]);
                float part[2][NT][4];   // this step's, of float32 queries
                if constexpr (P > 1) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) part[k][j][e] = 0.f;
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)   // contraction step 2 x + y
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            uint32_t bq[2];
                            if constexpr (C::kQRegs) {
                                bq[0] = qf[p][j][2 * x + y][0];
                                bq[1] = qf[p][j][2 * x + y][1];
                            } else {
                                const uint2 v = q_sm[((p * NT + j) * KS + 2 * x + y) * 32 + lane];
                                bq[0] = v.x;
                                bq[1] = v.y;
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t a[4] = {n[k][0][2 * y], n[k][1][2 * y], n[k][0][2 * y + 1],
                                                       n[k][1][2 * y + 1]};
                                mma16816(P > 1 ? part[k][j] : sc[k][j], a, bq);
                            }
                        }
                if constexpr (P > 1) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < NT; ++j) add4(sc[k][j], part[k][j]);
                }
            }

            // ---- softmax: element (token r + 8 (e / 2), row 2 t + (e & 1)) ----
            const bool edge = key0 + kCaUnit - 1 > min(lim_first, s.kv - 1);
            uint32_t pf[P][NT][2][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float v[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[k][e] = sc[k][j][e];
                if (edge) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + 16 * k + r + 8 * (e >> 1) > lim[j][e & 1]) v[k][e] = -INFINITY;
                }
                float x0 = fmaxf(max3(v[0][0], v[0][2], v[1][0]), v[1][2]) * io.scale_log2;
                float x1 = fmaxf(max3(v[0][1], v[0][3], v[1][1]), v[1][3]) * io.scale_log2;
                // the maximum moves only when a logit exceeds it by 2^8: any m gives the same quotient O / l
                if (__any_sync(0xffffffffu, x0 > m[j][0] + 8.f || x1 > m[j][1] + 8.f)) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
                        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
                    }
                    const float n0 = fmaxf(m[j][0], x0), n1 = fmaxf(m[j][1], x1);
                    const float f0 = n0 == -INFINITY ? 1.f : tc::fast_exp2(m[j][0] - n0);
                    const float f1 = n1 == -INFINITY ? 1.f : tc::fast_exp2(m[j][1] - n1);
                    m[j][0] = n0;
                    m[j][1] = n1;
                    l[j][0] *= f0;
                    l[j][1] *= f1;
#pragma unroll
                    for (int d = 0; d < KS; ++d) {
                        acc[j][d][0] *= f0;
                        acc[j][d][2] *= f0;
                        acc[j][d][1] *= f1;
                        acc[j][d][3] *= f1;
                    }
                }
                const float z0 = m[j][0] == -INFINITY ? 0.f : -m[j][0], z1 = m[j][1] == -INFINITY ? 0.f : -m[j][1];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[k][e] = tc::fast_exp2(fmaf(v[k][e], io.scale_log2, (e & 1) ? z1 : z0));
                    l[j][0] += v[k][0] + v[k][2];
                    l[j][1] += v[k][1] + v[k][3];
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint32_t lo = pack_bf16(v[k][0], v[k][1]), hi = pack_bf16(v[k][2], v[k][3]);
                        pf[p][j][k][0] = transpose8x8(lo);
                        pf[p][j][k][1] = transpose8x8(hi);
                        if (p + 1 < P) {   // what this part left
                            v[k][0] -= __uint_as_float(lo << 16);
                            v[k][1] -= __uint_as_float(lo & 0xffff0000u);
                            v[k][2] -= __uint_as_float(hi << 16);
                            v[k][3] -= __uint_as_float(hi & 0xffff0000u);
                        }
                    }
                }
            }

            // ---- O^T += V^T P^T: a lane holds channels r D / 8 .., tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9 ----
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint8_t *blk = ub + k * B::kBytes;
                uint32_t x[2][D / 32];   // 4 channels of a token pair each
                Scale2 s2[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(blk + B::kVC + h * 512 + lane * 16);
                        x[h][0] = prmt(v.x, v.z, 0x5410);
                        x[h][1] = prmt(v.x, v.z, 0x7632);
                        x[h][2] = prmt(v.y, v.w, 0x5410);
                        x[h][3] = prmt(v.y, v.w, 0x7632);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(blk + B::kVC + h * 256 + lane * 8);
                        x[h][0] = prmt(v.x, v.y, 0x5410);
                        x[h][1] = prmt(v.x, v.y, 0x7632);
                    }
                    const uint2 pr = *reinterpret_cast<const uint2 *>(
                        blk + B::kVS + ((h * B::kGroups + r * (D / 8) / 32) * 4 + t) * 8);
                    uint32_t keep = 0xffffffffu;
                    if (edge) {   // tokens past the sequence may hold anything, NaN too
                        const int a = key0 + 16 * k + 8 * h + 2 * t;
                        keep = (a < s.kv ? 0xffffu : 0u) | (a + 1 < s.kv ? 0xffff0000u : 0u);
                    }
                    s2[h] = scale2(pr.x & keep, pr.y & keep);
                }
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {   // channels 4 y .. 4 y + 3 of the slice
                    uint32_t n0[4], n1[4];
                    stored8(x[0][y], s2[0], n0);
                    stored8(x[1][y], s2[1], n1);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {    // channels 2 d, 2 d + 1
                        const int d = 2 * y + e;
                        const uint32_t a[4] = {n0[2 * e], n0[2 * e + 1], n1[2 * e], n1[2 * e + 1]};
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int p = 0; p < P; ++p) mma16816(P > 1 ? part : acc[j][d], a, pf[p][j][k]);
                            if constexpr (P > 1) add4(acc[j][d], part);
                        }
                    }
                }
            }
            __syncwarp();   // the stage may be refilled
        }
        T_ += n_run;

        // ---- join the warps' rows, 8 at a time, and write them ----
        const bool whole = k0 == 0 && cnt == seg.units;
        // cut before: slot 0; only after: slot 1
        float *slot = reinterpret_cast<float *>(io.ws + gridDim.x * sizeof(CaDesc)) +
                      ((size_t)blockIdx.x * 2 + (k0 > 0 ? 0 : 1)) * C::kSlot;
        float *mg = reinterpret_cast<float *>(ca_smem);
        float *mg_m = mg + kCaWarps * 8 * C::kMergeRow, *mg_l = mg_m + kCaWarps * 8;
        __syncthreads();   // every ring has been read
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (row0 + 8 * j >= R) break;   // CTA-uniform
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[j][0] += __shfl_xor_sync(0xffffffffu, l[j][0], o);
                l[j][1] += __shfl_xor_sync(0xffffffffu, l[j][1], o);
            }
            if (lane < 4) {
                mg_m[warp * 8 + 2 * t] = m[j][0];
                mg_m[warp * 8 + 2 * t + 1] = m[j][1];
                mg_l[warp * 8 + 2 * t] = l[j][0];
                mg_l[warp * 8 + 2 * t + 1] = l[j][1];
            }
#pragma unroll
            for (int d = 0; d < KS; ++d) {
                float *o = mg + (warp * 8 + 2 * t) * C::kMergeRow + r * (D / 8) + 2 * d;
                *reinterpret_cast<float2 *>(o) = make_float2(acc[j][d][0], acc[j][d][2]);
                *reinterpret_cast<float2 *>(o + C::kMergeRow) = make_float2(acc[j][d][1], acc[j][d][3]);
            }
            __syncthreads();
            for (int e = tid; e < 8 * D / 4; e += kCaThreads) {
                const int rr = e / (D / 4), d4 = (e % (D / 4)) * 4, row = row0 + 8 * j + rr;
                if (row < R) {
                    float M = -INFINITY, L = 0.f;
#pragma unroll
                    for (int w = 0; w < kCaWarps; ++w) M = fmaxf(M, mg_m[w * 8 + rr]);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kCaWarps; ++w) {
                        const float f = M == -INFINITY ? 0.f : tc::fast_exp2(mg_m[w * 8 + rr] - M);
                        const float4 v = *reinterpret_cast<const float4 *>(mg + (w * 8 + rr) * C::kMergeRow + d4);
                        L = fmaf(f, mg_l[w * 8 + rr], L);
                        o.x = fmaf(f, v.x, o.x);
                        o.y = fmaf(f, v.y, o.y);
                        o.z = fmaf(f, v.z, o.z);
                        o.w = fmaf(f, v.w, o.w);
                    }
                    if (whole) {
                        ca_write<T, D>(c, io, b, hkv, row, d4, o, M, L);
                    } else {
                        *reinterpret_cast<float4 *>(slot + (8 * j + rr) * D + d4) = o;
                        if (d4 == 0) {
                            slot[C::kRB * D + 8 * j + rr] = M;
                            slot[C::kRB * D + C::kRB + 8 * j + rr] = L;
                        }
                    }
                }
            }
            __syncthreads();   // the buffer is reused, by the next rows or as the ring
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // plain writes above, copies next
        __syncthreads();
    }
    if (failed && lane == 0) set_status(c.status, kDevTimeout);
}

// Joins the items that the cuts between CTAs divided: block (x, y) the x-th of
// them (every gridDim.x-th), rows y, y + gridDim.y, ... of its RB.  An item is
// found at its first cut: the cut before CTA c is one if the item that CTA c
// begins inside of began in CTA c - 1's run.  The parts lie in the CTAs' slots:
// slot 1 of CTA c - 1, where the item began, and slot 0 of c, c + 1, ...  Latency
// bounds it: all cuts are looked at at once, and a row's parts are loaded at once,
// by a warp where they are few (items cut once or twice, as most are) and by the
// block where they are many (one long sequence).
constexpr int kJoinThreads = 256, kMaxCtas = 2048;

template <typename T, int D, int RB>
__global__ void __launch_bounds__(kJoinThreads) cache_combine_kernel(const CacheParams c, const CacheAttendIo io, int ctas)
{
    constexpr int V = D / 32, W = kJoinThreads / 32;   // channels per lane; warps
    constexpr int kSlot = RB * (D + 2);
    __shared__ float part_o[W][D], s_m[W], s_l[W];
    __shared__ float weight[kJoinThreads];
    __shared__ int16_t firsts[kMaxCtas];               // the first cuts, in order
    __shared__ int counts[W];
    griddep_wait();
    const CaDesc *descs = reinterpret_cast<const CaDesc *>(io.ws);
    const float *slots = reinterpret_cast<const float *>(io.ws + ctas * sizeof(CaDesc));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int n_first = 0;
    for (int base = 1; base < ctas; base += kJoinThreads) {
        const int x = base + tid;
        bool first = false;
        if (x < ctas) {
            const CaDesc d = descs[x];
            first = d.k0 > 0 && ca_start(d.total, d.active, x) - d.k0 >= ca_start(d.total, d.active, x - 1);
        }
        const unsigned vote = __ballot_sync(0xffffffffu, first);
        if (lane == 0) counts[warp] = __popc(vote);
        __syncthreads();
        int at = n_first + __popc(vote & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) at += counts[w];
            n_first += counts[w];
        }
        if (first) firsts[at] = (int16_t)x;
        __syncthreads();
    }
    for (int fi = blockIdx.x; fi < n_first; fi += gridDim.x) {   // block-uniform
        const int cta = firsts[fi];
        const CaDesc d = descs[cta];
        const long long item = ca_start(d.total, d.active, cta) - d.k0;
        const int last = (int)ca_div((item + d.units) * d.active - 1, d.total);   // CTA of the item's last unit
        const int parts = last - cta + 2;
        const Seq s = load_seq(c, d.b);
        auto part = [&](int p) { return slots + ((size_t)(cta - 1 + p) * 2 + (p == 0 ? 1 : 0)) * kSlot; };
        if (parts <= 32) {   // a warp a row: a lane a part's weight
            for (int rr = blockIdx.y * W + warp; rr < RB; rr += gridDim.y * W) {
                const int row = d.rb * RB + rr;
                if (row >= io.G * s.q) break;
                const float m = lane < parts ? part(lane)[RB * D + rr] : -INFINITY;
                const float l = lane < parts ? part(lane)[RB * D + RB + rr] : 0.f;
                float M = m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                const float wt = tc::fast_exp2(m - (M == -INFINITY ? 0.f : M));
                float L = wt * l, acc[4] = {0.f, 0.f, 0.f, 0.f};   // V of them are a lane's channels
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll 4
                for (int p = 0; p < parts; ++p) {
                    const float *q = part(p) + rr * D + lane * V, w = __shfl_sync(0xffffffffu, wt, p);
                    float v[V];
                    if constexpr (V == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(q);
                    else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(q);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(w, v[e], acc[e]);
                }
                if constexpr (V == 2) {   // four channels to the even lanes
                    acc[2] = __shfl_down_sync(0xffffffffu, acc[0], 1);
                    acc[3] = __shfl_down_sync(0xffffffffu, acc[1], 1);
                }
                if (V == 4 || lane % 2 == 0)
                    ca_write<T, D>(c, io, d.b, d.hkv, row, lane * V, make_float4(acc[0], acc[1], acc[2], acc[3]), M, L);
            }
            continue;
        }
        for (int rr = blockIdx.y; rr < RB; rr += gridDim.y) {   // block-uniform; a row at a time
            const int row = d.rb * RB + rr;
            if (row >= io.G * s.q) break;
            float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = 0.f;
            // online over batches of parts, one per thread (a device has fewer CTAs than a few batches)
            for (int p0 = 0; p0 < parts; p0 += kJoinThreads) {
                const int p = p0 + tid;
                const float m = p < parts ? part(p)[RB * D + rr] : -INFINITY, l = p < parts ? part(p)[RB * D + RB + rr] : 0.f;
                float x = m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                if (lane == 0) s_m[warp] = x;
                __syncthreads();
                float top = M;
#pragma unroll
                for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w]);
                const float z = top == -INFINITY ? 0.f : top, f = tc::fast_exp2(m - z), g = tc::fast_exp2(M - z);
                weight[tid] = f;
                float y = f * l;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (lane == 0) s_l[warp] = y;
                __syncthreads();
                L *= g;
#pragma unroll
                for (int w = 0; w < W; ++w) L += s_l[w];
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] *= g;
                M = top;
#pragma unroll 8
                for (int i = warp; i < min(kJoinThreads, parts - p0); i += W) {
                    const float *q = part(p0 + i) + rr * D + lane * V;
                    const float wt = weight[i];
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(wt, q[e], acc[e]);
                }
                __syncthreads();
            }
#pragma unroll
            for (int e = 0; e < V; ++e) part_o[warp][lane * V + e] = acc[e];
            __syncthreads();
            if (tid < D / 4) {
                float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] += part_o[w][4 * tid + e];
                ca_write<T, D>(c, io, d.b, d.hkv, row, 4 * tid, make_float4(o[0], o[1], o[2], o[3]), M, L);
            }
            __syncthreads();
        }
    }
}

}  // namespace akv
