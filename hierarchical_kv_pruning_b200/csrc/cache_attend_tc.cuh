// Attention over the 4-bit cache for many query rows (prompts, query blocks):
// bfloat16 queries on tcgen05.
//
// An item is a block of 256 query rows of one KV head (row n G + g: token n,
// head g of the group), as two tiles of 128; its units are the 64-token key
// tiles up to the last row's causal limit.  One persistent CTA per SM, 20
// warps:
//   copy warp       the codes of a key tile into a ring (bulk copies; a page's
//                   blocks of one KV head are contiguous);
//   8 warps         turn them into bfloat16 K and V tiles in the 128-byte
//                   swizzled operand layout (three stages each); tokens past
//                   the sequence become zeros.  Within 8 channels a pair of a
//                   register is (channel i, i + 4), as the nibbles come out; Q
//                   is stored in the same order, O is put back in the epilogue;
//   2 MMA warps     S = Q K^T (M 128, N 64) of the next key tile for both row
//                   tiles, and O += P V, P read from TMEM where it overlays S;
//   2 x 4 warps     softmax, one thread per row, roundings as in the few-rows
//                   kernel: P is bfloat16, because the product takes its two
//                   operands in one type and V is; everything else float32.
// TMEM: S / P 2 x 2 x 64 and O 2 x D columns.  Shared memory (D = 128): Q 64, K
// 48, V 48, codes 40 KB.
// What bounds it: per key tile and both row tiles (D = 128) the products take
// 1280 cycles of the tensor cores and, with their commits and the changes
// between them, 1900 in a loop that does nothing else; the exponentials 1024 of
// the MUFU pipe; shared memory about 1400.  A tile takes 2500: the warps that
// issue pay for their waits.  Measured on the way, cycles per 128 tokens: one
// S buffer of 128 tokens and one issuing warp 6800 (each softmax waits for two
// products), 64-token tiles with two S buffers and one issuing warp 7400, products
// issued under elect.sync instead of one lane's branch 6200, S and P V issued by a
// warp each 5200, the maximum searched only where it must grow 5000.  2 x 2048 tokens over
// 6k .. 8k, 32 heads on 8 (390 GFLOP): 515 us with the join, 0.76 PFLOP/s.  96
// registers a thread at launch leave 308 bytes of spills, 324 at D = 64.
//
// The runs of units per CTA are as in the few-rows kernel, unless whole items
// balance about as well (a partial of 256 rows costs as much as several tiles).
//
// Every wait is bounded, by a number of tries within which key tiles have to go
// on; one that gives up sets ETIMEOUT in the status word.
#pragma once

#include <type_traits>

#include "cache_attend.cuh"

namespace akv {
namespace ctc {

using namespace tc;

constexpr int kRows = 128, kBlockRows = 256, kKeys = 64;
constexpr int kKV = 3, kRaw = 4;    // stages of the K and V tiles, of the codes
constexpr int kThreads = 640;
constexpr int kDequantWarp = 8, kDequantWarps = 8, kSWarp = 16, kCopyWarp = 17, kPvWarp = 18;
constexpr int kSoftmaxRegs = 152, kOtherRegs = 56;   // 256 x 152 + 384 x 56, within the 640 x 96 of the launch
constexpr float kMaxSum = 1024.f;   // a tile's sum of a row's probabilities that calls for a larger maximum
// A partial costs about this many units to write, read and join.
constexpr int kPartialUnits = 12;

// [2] x 2: row tile, parity of its running tile count
constexpr int kBarRawFull = 0, kBarRawEmpty = kBarRawFull + kRaw, kBarKFull = kBarRawEmpty + kRaw,
              kBarKEmpty = kBarKFull + kKV, kBarVFull = kBarKEmpty + kKV, kBarVEmpty = kBarVFull + kKV,
              kBarS = kBarVEmpty + kKV, kBarP = kBarS + 4, kBarO = kBarP + 4, kBarQ = kBarO + 4,
              kBarDrained = kBarQ + 2, kBarEnd = kBarDrained + 2, kNumBars = kBarEnd + 2;

template <int D>
struct Smem {
    static constexpr int kQ = kRows * D * 2, kT = kKeys * D * 2, kR = 4 * Blk<D>::kBytes;
    static constexpr int kOffQ = 0, kOffK = 2 * kQ, kOffV = kOffK + kKV * kT, kOffR = kOffV + kKV * kT,
                         kOffBar = kOffR + kRaw * kR, kOffSlot = kOffBar + kNumBars * 8, kOffSched = kOffSlot + 16, kBytes = kOffSched + 64;
    static constexpr int kColS = 0, kColO = 4 * kKeys;
    static constexpr int kSlot = kBlockRows * (D + 2);   // floats of a partial: O, m, l
    // at D = 64 a tile has 128 groups of 32 channels: half of the warps convert keys, half values
    static constexpr int kSideWarps = D == 128 ? kDequantWarps : kDequantWarps / 2;
};

template <int R> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// tcgen05.mma with the operand descriptors as their low words (start address in
// 16-byte units, lbo) plus a constant step: the steps of a tile then need two
// registers and no 64-bit sums, which the compiler would keep 32 of.
template <int StepA, int StepB>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "add.u32 x, %1, %6;\n\tadd.u32 y, %2, %7;\n\t"
        "mov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc), "n"(StepA), "n"(StepB));
}

template <int StepA, int StepB>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "add.u32 x, %1, %6;\n\tadd.u32 y, %2, %7;\n\t"
        "mov.b64 b, {y, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, {%8, %8, %8, %8}, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc), "n"(StepA), "n"(StepB), "r"(0u));
}

// One lane of a converged warp.  The products are issued under this and not
// under a comparison of the lane number: the compiler then takes their
// operands for uniform and needs 5 instructions a product instead of 12.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}\n" : "=r"(p));
    return p != 0;
}

// f(integral constant 0 .. N - 1)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void steps(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        steps<N, I + 1>(f);
    }
}

// An entry: 256-row block rb of sequence b (for every KV head).
struct Entry {
    Seq s;
    int b, rb, rows, units;   // rows of the block; key tiles (0: no rows)
};

// A stretch of units of one item that a CTA runs.
struct Seg {
    Entry e;
    int hkv, k0, cnt;
};

// The CTA's share of the call, in shared memory.
struct Sched {
    long long total, off0, u0, u1;   // units of the call; start within entry e0; the CTA's units
    int whole_items, active, e0, nb; // whole items round-robin?; CTAs with units; first entry; row blocks per sequence
    int copied;                      // key tiles asked for so far (the copy warp's count)
};

__device__ __forceinline__ Entry entry_at(const CacheParams &c, const CacheAttendIo &io, int nb, int e)
{
    Entry x;
    x.b = e / nb;
    x.rb = e - x.b * nb;
    x.s = load_seq(c, x.b);
    const int R = io.G * x.s.q, row0 = x.rb * kBlockRows;
    x.rows = max(0, min(kBlockRows, R - row0));
    const int last = x.s.kv - x.s.q + (row0 + x.rows - 1) / io.G;
    x.units = x.rows > 0 ? max(1, (last + kKeys) / kKeys) : 0;
    return x;
}

// Walks the CTA's stretches; every role walks its own copy.
struct Walk {
    int e, item;
    long long off, u;
    __device__ __forceinline__ void begin(const Sched &s)
    {
        e = s.e0;
        off = s.off0;
        u = s.u0;
        item = blockIdx.x;
    }
    __device__ __forceinline__ bool next(const CacheParams &c, const CacheAttendIo &io, const Sched &s, Seg &g)
    {
        const int nb = s.nb, entries = c.B * nb;
        if (s.whole_items) {   // items round-robin, the long ones (late row blocks) first
            for (; item < entries * c.H_kv; item += gridDim.x) {
                const int x = item / c.H_kv;
                g.e = entry_at(c, io, nb, entries - 1 - x);
                if (g.e.units == 0) continue;
                g.hkv = item - x * c.H_kv;
                g.k0 = 0;
                g.cnt = g.e.units;
                item += gridDim.x;
                return true;
            }
            return false;
        }
        while (u < s.u1) {
            g.e = entry_at(c, io, nb, e);
            const long long n = (long long)c.H_kv * g.e.units;
            if (off >= n) {
                off -= n;
                ++e;
                continue;
            }
            g.hkv = (int)ca_div(off, g.e.units);
            g.k0 = (int)(off - (long long)g.hkv * g.e.units);
            g.cnt = (int)min((long long)(g.e.units - g.k0), s.u1 - u);
            u += g.cnt;
            off += g.cnt;
            return true;
        }
        return false;
    }
};

}  // namespace ctc

template <int D>
__global__ void __launch_bounds__(ctc::kThreads, 1)
    cache_attend_tc_kernel(const CacheParams c, const CacheAttendIo io, int nb)
{
    using namespace ctc;
    using SM = Smem<D>;
    using B = Blk<D>;
    extern __shared__ __align__(1024) uint8_t ctc_smem[];
    const uint32_t sb = smem_addr(ctc_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return sb + SM::kOffBar + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctc_smem + SM::kOffSlot);
    // scratch of the share's scan, in the ring before its first copy (static
    // shared memory would move the dynamic base off its 1024-byte alignment)
    long long *s_sum = reinterpret_cast<long long *>(ctc_smem + SM::kOffR);
    int *s_max = reinterpret_cast<int *>(s_sum + kThreads / 32), *s_items = s_max + kThreads / 32;
    griddep_launch();
    griddep_wait();
    CaDesc *desc = reinterpret_cast<CaDesc *>(io.ws) + blockIdx.x;
    if (tid == 0) desc->k0 = 0;   // until a stretch begins inside an item
    if (sb & 1023u) {             // the swizzle atoms need a 1024-byte aligned base (CTA-uniform exit)
        if (tid == 0) set_status(c.status, kDevBadSmem);
        return;
    }

    // ---- the CTA's share ----
    Sched &sch = *reinterpret_cast<Sched *>(ctc_smem + SM::kOffSched);
    const int entries = c.B * nb, per = (entries + kThreads - 1) / kThreads;
    {
        const int lo = min(entries, tid * per), hi = min(entries, lo + per);
        long long mine = 0;
        int big = 0, items = 0;
        for (int e = lo; e < hi; ++e) {
            const int n = entry_at(c, io, nb, e).units;
            mine += (long long)c.H_kv * n;
            big = max(big, n);
            items += n > 0 ? c.H_kv : 0;
        }
        long long scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
            big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
            items += __shfl_xor_sync(0xffffffffu, items, o);
        }
        if (lane == 31) {
            s_sum[warp] = scan;
            s_max[warp] = big;
            s_items[warp] = items;
        }
        __syncthreads();
        long long total = 0, before = scan - mine, all_items = 0;
        int top = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_sum[w];
            total += s_sum[w];
            top = max(top, s_max[w]);
            all_items += s_items[w];
        }
        const long long ctas = gridDim.x;
        const bool whole = ca_whole(all_items, ctas, top, total, kPartialUnits);
        const int active = (int)max(1LL, min(ctas, total));
        if (!whole && (total == 0 || blockIdx.x >= active)) return;   // CTA-uniform
        if (tid == 0) {
            sch.total = total;
            sch.active = active;
            sch.whole_items = whole;
            sch.nb = nb;
            sch.copied = 0;
        }
        if (!whole) {
            const long long u0 = ca_start(total, active, blockIdx.x);
            if (u0 >= before && u0 < before + mine) {   // one thread
                long long off = u0 - before;
                int e = lo;
                for (;; ++e) {
                    const long long n = (long long)c.H_kv * entry_at(c, io, nb, e).units;
                    if (off < n) break;
                    off -= n;
                }
                sch.e0 = e;
                sch.off0 = off;
                sch.u0 = u0;
                sch.u1 = ca_start(total, active, blockIdx.x + 1);
            }
        }
    }
    if (tid == 0) {
        fence_async_smem();   // the scratch was plainly written, copies come next
        for (int i = 0; i < kNumBars; ++i) {
            const auto in = [&](int from, int n) { return i >= from && i < from + n; };
            int count = 1;
            if (in(kBarRawEmpty, kRaw)) count = kDequantWarps;
            if (in(kBarKFull, kKV) || in(kBarVFull, kKV)) count = SM::kSideWarps;
            if (in(kBarP, 4) || in(kBarQ, 2) || in(kBarDrained, 2)) count = 4;
            mbar_init(bar(i), count);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kSWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Walk walk;
    walk.begin(sch);
    Seg g;

    if (warp < 8) {
        // ================= softmax: one thread per query row =================
        regs_up<kSoftmaxRegs>();
        const int grp = warp >> 2, lrow = tid & 127, w4 = warp & 3;
        const uint32_t lane_off = (uint32_t)(w4 * 32) << 16;
        const uint32_t tS0 = tmem + SM::kColS + 2 * grp * kKeys + lane_off, tO = tmem + SM::kColO + grp * D + lane_off;
        uint8_t *q_tile = ctc_smem + SM::kOffQ + grp * SM::kQ;
        bool failed = false;
        // The second group sits out the stretches of up to 128 rows, so its next S may be many tiles away: the wait's
        // limit begins anew while tiles are being copied, and still ends when they stop.
        auto wait_s = [&](uint32_t b, int parity) -> bool {
            for (int seen = -1;;) {
                if (mbar_wait(b, parity)) return true;
                const int now = *const_cast<volatile int *>(&sch.copied);
                if (now == seen) return false;
                seen = now;
            }
        };
        auto next_own = [&](Seg &x) -> bool {
            while (walk.next(c, io, sch, x))
                if (x.e.rows > grp * kRows) return true;
            return false;
        };
        // this group's 128 rows of a stretch into the swizzled A tile, zeros past its rows
        auto load_q = [&](const Seg &x) {
            constexpr int CPR = D / 8, RPI = 128 / CPR;   // chunks of a row; rows per step of the 128 threads
            const int cc = lrow % CPR;
            const int row0 = x.e.rb * kBlockRows + grp * kRows, rows = x.e.rows - grp * kRows;
#pragma unroll 8
            for (int i = 0; i < kRows / RPI; ++i) {
                const int rl = i * RPI + lrow / CPR;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (rl < rows) {
                    const int row = row0 + rl, n = row / io.G, h = row - n * io.G;
                    v = ldg16(reinterpret_cast<const __nv_bfloat16 *>(io.q) + ((size_t)x.e.b * c.N + n) * io.qs +
                              (size_t)(x.hkv * io.G + h) * D + cc * 8);
                }
                *reinterpret_cast<uint4 *>(q_tile + (cc >> 3) * (kRows * 128) + sw128(rl, cc & 7)) =
                    make_uint4(prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632), prmt(v.y, v.w, 0x5410),
                               prmt(v.y, v.w, 0x7632));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarQ + grp));
        };
        int T = 0;   // this group's tiles so far
        bool more = next_own(g);
        if (more) load_q(g);
        bool first_seg = true;
        while (more && !failed) {
            const Seg cur = g;
            const int row = cur.e.rb * kBlockRows + grp * kRows + lrow;
            const bool row_ok = grp * kRows + lrow < cur.e.rows;
            const int lim = row_ok ? cur.e.s.kv - cur.e.s.q + row / io.G : -1;   // last visible slot
            // the tiles up to here need no mask
            const int lim_first = cur.e.s.kv - cur.e.s.q + (cur.e.rb * kBlockRows + grp * kRows) / io.G;
            const bool all_rows = cur.e.rows >= (grp + 1) * kRows;
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int t = 0; t < cur.cnt; ++t, ++T) {
                const int bs = T & 1;
                const uint32_t tS = tS0 + bs * kKeys;
                failed = __any_sync(0xffffffffu, !wait_s(bar(kBarS + 2 * grp + bs), (T >> 1) & 1));
                if (failed) break;
                fence_after_sync();
                const int key0 = (cur.k0 + t) * kKeys;
                float sc[kKeys];
                tmem_ld32(tS, sc);
                tmem_ld32(tS + 32, sc + 32);
                tmem_wait_ld();
                if (!all_rows || key0 + kKeys - 1 > lim_first) {   // warp-uniform
                    const int hi = lim - key0;
#pragma unroll
                    for (int j = 0; j < kKeys; ++j) sc[j] = j <= hi ? sc[j] : -INFINITY;
                }
                // P over the first 32 columns of S, with the maximum as it is; the row's sum of P
                auto probabilities = [&]() -> float {
                    float2 ps[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) ps[j] = make_float2(0.f, 0.f);
                    const float neg = m == -INFINITY ? 0.f : -m;
                    const float2 sc2 = make_float2(io.scale_log2, io.scale_log2), neg2 = make_float2(neg, neg);
#pragma unroll
                    for (int k = 0; k < kKeys; k += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float2 x = fma2(make_float2(sc[k + j], sc[k + j + 1]), sc2, neg2);
                            x.x = fast_exp2(x.x);
                            x.y = fast_exp2(x.y);
                            ps[(j >> 1) & 3] = add2(ps[(j >> 1) & 3], x);
                            pk[j / 2] = pack_bf16(x.x, x.y);
                        }
                        tmem_st16(tS + k / 2, pk);
                    }
                    const float2 p = add2(add2(ps[0], ps[1]), add2(ps[2], ps[3]));
                    return p.x + p.y;
                };
                // The maximum is only looked for in a stretch's first tile and where a row's sum of probabilities shows that
                // it has become much too small (or that the row sees its first key): any m gives the same O / l,
                // and 32 comparisons a tile take a fifth of the softmax's time.
                float psum = 0.f;
                bool search = t == 0;
                if (!search) {
                    psum = probabilities();
                    search = __any_sync(0xffffffffu, !(psum <= kMaxSum) || (m == -INFINITY && psum > 0.f));
                }
                if (search) {   // warp-uniform
                    float top = sc[0];
#pragma unroll
                    for (int j = 1; j < kKeys - 1; j += 2) top = max3(top, sc[j], sc[j + 1]);
                    const float m_new = fmaxf(m, fmaxf(top, sc[kKeys - 1]) * io.scale_log2);
                    if (t > 0) {
                        // O may be rescaled only once the previous P V has landed in it
                        failed = __any_sync(0xffffffffu,
                                            !mbar_wait(bar(kBarO + 2 * grp + ((T - 1) & 1)), ((T - 1) >> 1) & 1));
                        if (failed) break;
                        fence_after_sync();
                        const float f = m_new == -INFINITY ? 1.f : fast_exp2(m - m_new);
#pragma unroll
                        for (int d = 0; d < D; d += 32) {
                            float o[32];
                            tmem_ld32(tO + d, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= f;
                            tmem_st32(tO + d, o);
                        }
                        l *= f;
                    }
                    m = m_new;
                    if (t > 0) tmem_wait_st();   // P is stored over the first attempt's
                    psum = probabilities();
                }
                l += psum;
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarP + 2 * grp + bs));
            }
            if (failed) break;
            // the stretch's last S is done: Q is free
            more = next_own(g);
            if (more) load_q(g);
            failed = __any_sync(0xffffffffu, !mbar_wait(bar(kBarO + 2 * grp + ((T - 1) & 1)), ((T - 1) >> 1) & 1));
            if (failed) break;
            fence_after_sync();
            // ---- out: O / l with its log-sum-exp, or a partial ----
            const bool whole = cur.k0 == 0 && cur.cnt == cur.e.units;
            const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
            const int n = row / io.G, h = row - n * io.G;
            const size_t at = ((size_t)cur.e.b * c.N + n) * io.H + cur.hkv * io.G + h;
            float *slot = reinterpret_cast<float *>(io.ws + gridDim.x * sizeof(CaDesc)) +
                          ((size_t)blockIdx.x * 2 + (cur.k0 > 0 ? 0 : 1)) * SM::kSlot;
            const int sr = grp * kRows + lrow;
            const size_t part = (((size_t)cur.e.b * c.H_kv + cur.hkv) * io.G + h) * c.N + n;   // row of oseq
#pragma unroll
            for (int d = 0; d < D; d += 32) {
                float o[32];
                tmem_ld32(tO + d, o);
                tmem_wait_ld();
                if (d == D - 32) {   // O has been read: the next stretch may start it afresh
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarDrained + grp));
                }
                if (!row_ok) continue;
                // position p of 8 holds channel (p >> 1) + 4 (p & 1)
                if (whole && io.oseq) {
                    float *dst = io.oseq + part * D + d;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        *reinterpret_cast<float4 *>(dst + i) =
                            make_float4(o[i] * inv, o[i + 2] * inv, o[i + 4] * inv, o[i + 6] * inv);
                        *reinterpret_cast<float4 *>(dst + i + 4) =
                            make_float4(o[i + 1] * inv, o[i + 3] * inv, o[i + 5] * inv, o[i + 7] * inv);
                    }
                } else if (whole) {
                    __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(io.out) + at * D + d;
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4 *>(dst + i) =
                            make_uint4(pack_bf16(o[i] * inv, o[i + 2] * inv), pack_bf16(o[i + 4] * inv, o[i + 6] * inv),
                                       pack_bf16(o[i + 1] * inv, o[i + 3] * inv), pack_bf16(o[i + 5] * inv, o[i + 7] * inv));
                } else {
                    float *dst = slot + sr * D + d;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        *reinterpret_cast<float4 *>(dst + i) = make_float4(o[i], o[i + 2], o[i + 4], o[i + 6]);
                        *reinterpret_cast<float4 *>(dst + i + 4) = make_float4(o[i + 1], o[i + 3], o[i + 5], o[i + 7]);
                    }
                }
            }
            if (row_ok) {
                const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
                if (whole && io.oseq) {
                    io.lse_seq[part] = lse;
                } else if (whole) {
                    if (io.lse) io.lse[at] = lse;
                } else {
                    slot[kBlockRows * D + sr] = m;
                    slot[kBlockRows * D + kBlockRows + sr] = l;
                }
            }
            // the join needs to know where the CTA's first stretch began (group 0 has rows in every stretch)
            if (grp == 0 && lrow == 0 && first_seg)
                *desc = CaDesc{sch.total, sch.active, cur.k0, cur.e.units, cur.e.b, cur.hkv, cur.e.rb};
            first_seg = false;
        }
        if (failed && lane == 0) set_status(c.status, kDevTimeout);
    } else if (warp < kSWarp) {
        // ================= codes to bfloat16 tiles =================
        regs_down<kOtherRegs>();
        // One group of 32 channels of a token per thread, keys and values apart.  Keys: the lanes of a quad take a token's
        // groups, so that a warp reads consecutive 16-byte codes; values: consecutive lanes take consecutive
        // tokens, whose 8-byte pieces are.  Either way the 16-byte stores of 8 lanes fall into
        // distinct banks.
        const int w8 = warp - kDequantWarp;
        const bool does_k = D == 128 || w8 < 4, does_v = D == 128 || w8 >= 4;
        const int side = D == 128 ? w8 * 32 + lane : (w8 & 3) * 32 + lane;   // 0 .. 64 kGroups - 1
        const int k_key = side / B::kGroups, k_gr = side % B::kGroups, v_key = side % kKeys, v_gr = side / kKeys;
        const int k_src = (k_key >> 4) * B::kBytes, v_src = (v_key >> 4) * B::kBytes, k_tok = k_key & 15, v_tok = v_key & 15;
        const int k_codes = k_src + B::k_codes(k_tok) + 16 * k_gr, k_pair = k_src + B::k_pair(k_tok, k_gr);
        const int v_codes = v_src + B::v_codes(v_tok, D == 128 ? 2 * v_gr : 4 * v_gr), v_pair = v_src + B::v_scale(v_tok, v_gr);
        constexpr int kSlice = 64 * B::kSliceBytes / 8;   // bytes from a slice's piece to the next slice's
        const int k_dst = (k_gr >> 1) * (kKeys * 128) + k_key * 128, v_dst = (v_gr >> 1) * (kKeys * 128) + v_key * 128;
        const int k_first = (k_gr >> 1) * 2;   // chunk order: the two 64-channel blocks start two chunks apart
        bool failed = false;
        int T = 0;
        while (!failed && walk.next(c, io, sch, g)) {
#pragma unroll 1
            for (int t = 0; t < g.cnt; ++t, ++T) {
                const int st = T % kKV, rs = T % kRaw, key0 = (g.k0 + t) * kKeys;
                const uint8_t *raw = ctc_smem + SM::kOffR + rs * SM::kR;
                const bool tail = key0 + kKeys > g.e.s.kv;   // tokens past the sequence become zeros
                failed = __any_sync(0xffffffffu, !mbar_wait(bar(kBarRawFull + rs), (T / kRaw) & 1));
                if (failed) break;
                uint4 kc;
                uint32_t kp, vc[4], vs, vm;
                if (does_k) {
                    kc = *reinterpret_cast<const uint4 *>(raw + k_codes);
                    kp = *reinterpret_cast<const uint32_t *>(raw + k_pair);
                }
                if (does_v) {
                    if constexpr (D == 128) {
                        const uint2 a = *reinterpret_cast<const uint2 *>(raw + v_codes);
                        const uint2 e = *reinterpret_cast<const uint2 *>(raw + v_codes + kSlice);
                        vc[0] = a.x;
                        vc[1] = a.y;
                        vc[2] = e.x;
                        vc[3] = e.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) vc[i] = *reinterpret_cast<const uint32_t *>(raw + v_codes + i * kSlice);
                    }
                    vs = *reinterpret_cast<const uint16_t *>(raw + v_pair);
                    vm = *reinterpret_cast<const uint16_t *>(raw + v_pair + 4);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarRawEmpty + rs));   // the codes are in registers
                if (does_k) {
                    if (T >= kKV) failed = __any_sync(0xffffffffu, !mbar_wait(bar(kBarKEmpty + st), ((T / kKV) + 1) & 1));
                    if (failed) break;
                    uint8_t *dst = ctc_smem + SM::kOffK + st * SM::kT + k_dst;
                    const Scale2 s = scale2(prmt(kp, kp, 0x1010), prmt(kp, kp, 0x3232));
                    const bool zero = tail && key0 + k_key >= g.e.s.kv;
                    const uint32_t w[4] = {k_first ? kc.z : kc.x, k_first ? kc.w : kc.y, k_first ? kc.x : kc.z,
                                           k_first ? kc.y : kc.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o[4];
                        stored8(w[i], s, o);
                        uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                        if (zero) v = make_uint4(0u, 0u, 0u, 0u);
                        const int ch = (k_gr & 1) * 4 + ((i + k_first) & 3);
                        *reinterpret_cast<uint4 *>(dst + ((ch ^ (k_key & 7)) << 4)) = v;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarKFull + st));
                }
                if (does_v) {
                    if (T >= kKV) failed = __any_sync(0xffffffffu, !mbar_wait(bar(kBarVEmpty + st), ((T / kKV) + 1) & 1));
                    if (failed) break;
                    uint8_t *dst = ctc_smem + SM::kOffV + st * SM::kT + v_dst;
                    const Scale2 s = scale2(vs | vs << 16, vm | vm << 16);
                    const bool zero = tail && key0 + v_key >= g.e.s.kv;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t o[4];
                        stored8(vc[i], s, o);
                        uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                        if (zero) v = make_uint4(0u, 0u, 0u, 0u);
                        const int ch = (v_gr & 1) * 4 + i;
                        *reinterpret_cast<uint4 *>(dst + ((ch ^ (v_key & 7)) << 4)) = v;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarVFull + st));
                }
            }
        }
        if (failed && lane == 0) set_status(c.status, kDevTimeout);
    } else {
        regs_down<kOtherRegs>();
        if (warp == kCopyWarp) {
            // ================= copies of the codes, 64 tokens each =================
            bool failed = false;
            int raw = 0;
            const int pshift = 31 - __clz(c.page_size);
            while (!failed && walk.next(c, io, sch, g)) {
                const int32_t *tab = c.table + (size_t)g.e.b * c.max_pages;
#pragma unroll 1
                for (int i = 0; i < g.cnt; ++i, ++raw) {
                    const int rs = raw % kRaw, key = (g.k0 + i) * kKeys;
                    const int blocks = max(0, min(4, (g.e.s.kv - key + 15) >> 4));
                    // lane j: the block of tokens key + 16 j
                    const uint8_t *src = nullptr;
                    if (lane < blocks) {
                        src = block_at<D>(c, tab[(key + 16 * lane) >> pshift], g.hkv, key + 16 * lane);
                        if (!src) src = c.pages;   // reported; any page's bytes stand in
                    }
                    if (raw >= kRaw)
                        failed = __any_sync(0xffffffffu, !mbar_wait(bar(kBarRawEmpty + rs), ((raw / kRaw) + 1) & 1));
                    if (failed) break;
                    if (lane == 0) {
                        if (blocks > 0) mbar_arrive_expect_tx(bar(kBarRawFull + rs), blocks * B::kBytes);
                        else mbar_arrive(bar(kBarRawFull + rs));
                    }
                    if (lane == 0) *const_cast<volatile int *>(&sch.copied) = raw + 1;
                    __syncwarp();
                    const uint32_t dst = sb + SM::kOffR + rs * SM::kR;
                    if (c.page_size >= kKeys) {   // 64 tokens of a page are contiguous
                        if (lane == 0 && blocks > 0) bulk_load(dst, src, blocks * B::kBytes, bar(kBarRawFull + rs));
                    } else if (lane < blocks) {
                        bulk_load(dst + lane * B::kBytes, src, B::kBytes, bar(kBarRawFull + rs));
                    }
                }
            }
            // the CTA must not end with copies in flight
            bool landed = true;
            for (int x = max(0, raw - kRaw); x < raw; ++x) landed &= mbar_wait(bar(kBarRawFull + x % kRaw), (x / kRaw) & 1);
            if ((failed || !landed) && lane == 0) set_status(c.status, kDevTimeout);
        } else if (warp == kSWarp || warp == kPvWarp) {
            // ================= MMA issue: one lane of a converged warp; S and P V by a warp each =================
            // Such a warp pays its instructions' latency (one that waited for all the barriers took 3700 cycles a key
            // tile), so there are two, and the bookkeeping is kept to counters.
            auto wait = [&](int b, int parity) -> bool { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity)); };
            int st = 0, ph = 0, n0 = 0, n1 = 0, seg0 = 0, seg1 = 0;   // ring stage and phase; key tiles and stretches
            bool ok = true;                                           // of each row tile so far
            if (warp == kSWarp) {
                const uint32_t idesc = make_idesc(kRows, kKeys, 0, 0);
                const uint64_t dq = make_desc(sb + SM::kOffQ, 16, 1024), dk = make_desc(sb + SM::kOffK, 16, 1024);
                const uint32_t hi = (uint32_t)(dq >> 32), dq0 = (uint32_t)dq, dk0 = (uint32_t)dk;
                auto s_of = [&](int grp, int n, bool last) -> bool {   // S of a row tile's n-th key tile
                    // its buffer holds the P of two tiles before until its P V is done
                    const int bs = 2 * grp + (n & 1);
                    if (n >= 2 && !wait(kBarO + bs, ((n - 2) >> 1) & 1)) return false;
                    // that product read P, and the softmax S and P, in the columns that this one writes
                    fence_after_sync();
                    const uint32_t d = tmem + SM::kColS + bs * kKeys, q = dq0 + grp * (SM::kQ >> 4), k = dk0 + st * (SM::kT >> 4);
                    if (elect_one()) {
                        steps<D / 16>([&](auto i) {
                            constexpr int x = i, a = ((x >> 2) * (kRows * 128) + (x & 3) * 32) / 16,
                                          b = ((x >> 2) * (kKeys * 128) + (x & 3) * 32) / 16;
                            mma_ss<a, b>(d, q, k, hi, idesc, x > 0 ? 1u : 0u);
                        });
                        mma_commit(bar(kBarS + bs));
                        if (last) mma_commit(bar(kBarKEmpty + st));
                    }
                    __syncwarp();
                    return true;
                };
                while (ok && __any_sync(0xffffffffu, walk.next(c, io, sch, g))) {
                    const int cnt = g.cnt;
                    const bool two = g.e.rows > kRows;
                    ok = wait(kBarQ, seg0 & 1) && (!two || wait(kBarQ + 1, seg1 & 1));
#pragma unroll 1
                    for (int r = 0; ok && r < cnt; ++r) {
                        ok = wait(kBarKFull + st, ph) && s_of(0, n0, !two) && (!two || s_of(1, n1, true));
                        ++n0;
                        n1 += two;
                        if (++st == kKV) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                    ++seg0;
                    seg1 += two;
                }
            } else {
                const uint32_t idesc = make_idesc(kRows, D, 0, 1);
                const uint64_t dv = make_desc(sb + SM::kOffV, kKeys * 128, 1024);
                const uint32_t hi = (uint32_t)(dv >> 32), dv0 = (uint32_t)dv;
                auto pv_of = [&](int grp, int n, bool first, int seg, bool last) -> bool {   // O += P V of its n-th key tile
                    const int bs = 2 * grp + (n & 1);
                    if (!wait(kBarP + bs, (n >> 1) & 1)) return false;
                    // a stretch's first P V starts O afresh once the previous O has been read out
                    if (first && seg > 0 && !wait(kBarDrained + grp, (seg - 1) & 1)) return false;
                    fence_after_sync();
                    const uint32_t p = tmem + SM::kColS + bs * kKeys, d = tmem + SM::kColO + grp * D, v = dv0 + st * (SM::kT >> 4);
                    if (elect_one()) {
                        steps<kKeys / 16>([&](auto i) {
                            constexpr int x = i;
                            mma_ts<8 * x, x * 128>(d, p, v, hi, idesc, (!first || x > 0) ? 1u : 0u);
                        });
                        mma_commit(bar(kBarO + bs));
                        if (last) mma_commit(bar(kBarVEmpty + st));
                    }
                    __syncwarp();
                    return true;
                };
                while (ok && __any_sync(0xffffffffu, walk.next(c, io, sch, g))) {
                    const int cnt = g.cnt;
                    const bool two = g.e.rows > kRows;
#pragma unroll 1
                    for (int r = 0; ok && r < cnt; ++r) {
                        ok = wait(kBarVFull + st, ph) && pv_of(0, n0, r == 0, seg0, !two) &&
                             (!two || pv_of(1, n1, r == 0, seg1, true));
                        ++n0;
                        n1 += two;
                        if (++st == kKV) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                    ++seg0;
                    seg1 += two;
                }
            }
            // before TMEM is released every MMA must have completed, on the failure path too
            const int end = kBarEnd + (warp == kSWarp ? 0 : 1);
            if (elect_one()) mma_commit(bar(end));
            if (!wait(end, 0) || !ok) set_status(c.status, kDevTimeout);
        }
        __syncwarp();
    }

    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == kSWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace akv
