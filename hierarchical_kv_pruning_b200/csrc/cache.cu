// C ABI of the rotary positions and of the 4-bit paged cache (include/atlaskv.h):
// argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "atlaskv.h"
#include "cache_attend.cuh"
#include "cache_attend_tc.cuh"
#include "internal.h"
#include "kvcache.cuh"
#include "rope.cuh"

struct atlaskv_cache {
    atlaskv_cache_desc d;
    int device;
    int num_sms;
    int *status;   // device sticky status word
};

namespace {

atlaskv_status fail(atlaskv_status st, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return akv_report(st, buf);
}

#define AKV_CUDA(call)                                                                                 \
    do {                                                                                               \
        cudaError_t e_ = (call);                                                                       \
        if (e_ != cudaSuccess) {                                                                       \
            cudaGetLastError();                                                                        \
            return fail(ATLASKV_ECUDA, "%s: %s", #call, cudaGetErrorString(e_));                       \
        }                                                                                              \
    } while (0)
#define AKV_RET(x)                                 \
    do {                                           \
        const atlaskv_status st_ = (x);            \
        if (st_ != ATLASKV_OK) return st_;         \
    } while (0)

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
int esize(int dtype) { return dtype == ATLASKV_F32 ? 4 : 2; }

atlaskv_status check_dtype(int dtype)
{
    if (dtype != ATLASKV_F32 && dtype != ATLASKV_BF16) return fail(ATLASKV_EINVAL, "dtype %d", dtype);
    return ATLASKV_OK;
}

atlaskv_status check_head_dim(int D)
{
    if (D != 64 && D != 128) return fail(ATLASKV_EUNSUPPORTED, "head_dim %d (64 or 128)", D);
    return ATLASKV_OK;
}

// A token tensor: base aligned, stride 0 (dense) or at least a row and keeping
// every row 16-byte aligned.  *stride becomes the stride in elements.
atlaskv_status check_rows(const char *name, const void *p, int64_t row, int dtype, int64_t given, int64_t *stride)
{
    if (!p) return fail(ATLASKV_EINVAL, "null %s", name);
    if (!aligned16(p)) return fail(ATLASKV_EINVAL, "%s must be 16-byte aligned", name);
    if (given == 0) given = row;
    if (given < row) return fail(ATLASKV_EINVAL, "%s: a token stride of %lld is below a row's %lld elements", name,
                                 (long long)given, (long long)row);
    if (given * esize(dtype) % 16) return fail(ATLASKV_EINVAL, "%s: its token stride must be a multiple of 16 bytes", name);
    *stride = given;
    return ATLASKV_OK;
}

atlaskv_status rope_params(const atlaskv_rope_spec *spec, int head_dim, akv::RopeParams *p)
{
    *p = akv::RopeParams{};
    if (!spec) return ATLASKV_OK;
    if (spec->layout != ATLASKV_ROPE_HALF && spec->layout != ATLASKV_ROPE_INTERLEAVED)
        return fail(ATLASKV_EINVAL, "rotary layout %d", spec->layout);
    if (spec->rotary_dim < 16 || spec->rotary_dim > head_dim || spec->rotary_dim % 16)
        return fail(ATLASKV_EINVAL, "rotary_dim %d is not a multiple of 16 in [16, head_dim = %d]", spec->rotary_dim,
                    head_dim);
    if (!std::isfinite(spec->amplitude)) return fail(ATLASKV_EINVAL, "rotary amplitude is not finite");
    p->on = 1;
    p->interleaved = spec->layout == ATLASKV_ROPE_INTERLEAVED;
    p->rot = spec->rotary_dim;
    p->amp = spec->amplitude;
    for (int i = 0; i < spec->rotary_dim / 2; ++i) {
        if (!std::isfinite(spec->freq[i])) return fail(ATLASKV_EINVAL, "rotary frequency %d is not finite", i);
        p->turns[i] = spec->freq[i] / (2.0 * 3.14159265358979323846);
    }
    return ATLASKV_OK;
}

atlaskv_status check_grid(long long blocks)
{
    if (blocks > 0x7fffffffLL) return fail(ATLASKV_EUNSUPPORTED, "too many tokens and heads for one launch");
    return ATLASKV_OK;
}

int num_sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        n <= 0) {
        cudaGetLastError();
        n = 148;
    }
    return n;
}

// Launch with programmatic stream serialization (the kernel begins while the
// one before it drains, and waits before it reads or writes).
template <typename... KArgs, typename... Args>
atlaskv_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    AKV_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
    return ATLASKV_OK;
}

// Tokens per CTA: whole tokens up to one batch of row slots, so that a CTA's
// loads are all started at once; fewer in calls too small to fill the device.
int tokens_per_cta(long long tokens, int rows, int D, int sms)
{
    const int slots = akv::kRowBatch * akv::kTokThreads / (D / 16);
    const long long spread = (tokens + 4LL * sms - 1) / (4LL * sms);
    return (int)std::max(1LL, std::min({(long long)akv::kTokMax, (long long)slots / rows, spread}));
}

atlaskv_status check_cache(const atlaskv_cache *c)
{
    if (!c) return fail(ATLASKV_EINVAL, "null cache");
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(ATLASKV_ECUDA, "no current CUDA device");
    }
    if (dev != c->device)
        return fail(ATLASKV_EINVAL, "the cache lives on device %d and the current device is %d", c->device, dev);
    return ATLASKV_OK;
}

atlaskv_status cache_params(const atlaskv_cache *c, const atlaskv_seqs *s, akv::CacheParams *p)
{
    if (!s) return fail(ATLASKV_EINVAL, "null seqs");
    if (s->B < 0) return fail(ATLASKV_EINVAL, "B = %d < 0", s->B);
    if (s->N < 1) return fail(ATLASKV_EINVAL, "N = %d < 1", s->N);
    if (s->max_pages < 1) return fail(ATLASKV_EINVAL, "max_pages = %d < 1", s->max_pages);
    if ((long long)s->max_pages * c->d.page_size > 0x7fffffffLL - 256)
        return fail(ATLASKV_EUNSUPPORTED, "a block table of more than 2^31 slots");
    *p = akv::CacheParams{};
    p->pages = static_cast<uint8_t *>(c->d.pages);
    p->n_pages = c->d.n_pages;
    p->H_kv = c->d.n_kv_heads;
    p->page_size = c->d.page_size;
    p->B = s->B;
    p->N = s->N;
    p->max_pages = s->max_pages;
    p->table = s->block_table;
    p->kv_len = s->kv_len;
    p->q_len = s->q_len;
    p->status = c->status;
    if (s->B == 0) return ATLASKV_OK;
    if (!s->block_table || !s->kv_len) return fail(ATLASKV_EINVAL, "null block_table or kv_len");
    if (!aligned4(s->block_table) || !aligned4(s->kv_len) || (s->q_len && !aligned4(s->q_len)))
        return fail(ATLASKV_EINVAL, "block_table, kv_len and q_len must be 4-byte aligned");
    return ATLASKV_OK;
}

// Row blocks of 8, 16 or 32 rows: the fewest that hold a KV head's rows (a
// unit's codes are turned into bfloat16 once per row block).  float32 queries
// are three bfloat16 parts: 16 rows at most, 32 would not fit the registers.
int row_tiles(int dtype, long long rows) { return rows <= 8 ? 1 : rows <= 16 || dtype == ATLASKV_F32 ? 2 : 4; }

// Slots that the block table can name, an upper bound of every length.
long long slots_of(const akv::CacheParams &p) { return (long long)p.max_pages * p.page_size; }

template <typename T, int D, int NT>
int ca_ctas(const atlaskv_cache *c)
{
    return akv::Ca<T, D, NT>::kCtas * c->num_sms;
}

template <typename T, int D, int NT>
size_t ca_workspace(const atlaskv_cache *c)
{
    const size_t n = ca_ctas<T, D, NT>(c);
    return n * sizeof(akv::CaDesc) + n * 2 * akv::Ca<T, D, NT>::kSlot * sizeof(float);
}

// Blocks of the join: as many divided items as there can be, each by as many
// blocks as make about one wave (blocks that find nothing to do cost, too).
dim3 join_grid(long long items, int ctas, int rows)
{
    const int x = (int)std::min<long long>(items, ctas - 1);
    return dim3(std::max(1, x), std::max(1, std::min(rows, 592 / std::max(1, x))));
}

template <typename T, int D, int NT>
atlaskv_status launch_ca(const atlaskv_cache *c, const akv::CacheParams &p, const akv::CacheAttendIo &a, cudaStream_t s)
{
    using C = akv::Ca<T, D, NT>;
    AKV_RET(akv_smem_limit(reinterpret_cast<const void *>(akv::cache_attend_kernel<T, D, NT>), C::kSmem));
    const int n = ca_ctas<T, D, NT>(c);
    AKV_RET(launch_pdl(akv::cache_attend_kernel<T, D, NT>, dim3(n), akv::kCaThreads, C::kSmem, s, p, a));
    // no cuts whatever the lengths are: no join
    const long long items = (long long)p.B * p.H_kv * (((long long)p.N * a.G + C::kRB - 1) / C::kRB);
    if (akv::ca_whole(items, n, slots_of(p) / akv::kCaUnit + 1, 0, akv::kCaPartialUnits)) return ATLASKV_OK;
    return launch_pdl(akv::cache_combine_kernel<T, D, C::kRB>, join_grid(items, n, C::kRB), akv::kJoinThreads, 0, s, p, a,
                      n);
}

// Many rows of bfloat16 queries: tcgen05 (the few-rows kernel would turn the
// codes into bfloat16 again for every 32 rows).  Measured on either side, few-rows
// against tcgen05, us: 64 sequences of 4096 tokens, 8 KV heads, with 32 rows 157
// against 311, with 64 290 against 326, with 96 422 against 342, with 128 537
// against 310; 4 such sequences 29 / 37, 38 / 41, 47 / 46, 55 / 47; 2 of 200k, one KV
// head, 41 / 68, 62 / 70, 89 / 72, 106 / 66; one of 600 20 / 20 from 40 rows on.
// (Two blocks of 32 rows are up to 12 % faster than one padded tile.)
bool use_tc(int dtype, long long rows) { return dtype == ATLASKV_BF16 && rows > 32; }

long long tc_blocks(long long rows) { return (rows + akv::ctc::kBlockRows - 1) / akv::ctc::kBlockRows; }

template <int D>
size_t tc_workspace(const atlaskv_cache *c)
{
    return (size_t)c->num_sms * (sizeof(akv::CaDesc) + 2 * akv::ctc::Smem<D>::kSlot * sizeof(float));
}

template <int D>
atlaskv_status launch_tc(const atlaskv_cache *c, const akv::CacheParams &p, const akv::CacheAttendIo &a, cudaStream_t s)
{
    constexpr int RB = akv::ctc::kBlockRows;
    const long long nb = tc_blocks((long long)p.N * a.G);
    AKV_RET(akv_smem_limit(reinterpret_cast<const void *>(akv::cache_attend_tc_kernel<D>), akv::ctc::Smem<D>::kBytes));
    const int n = c->num_sms;
    AKV_RET(launch_pdl(akv::cache_attend_tc_kernel<D>, dim3(n), akv::ctc::kThreads, akv::ctc::Smem<D>::kBytes, s, p, a,
                       (int)nb));
    const long long items = nb * p.B * p.H_kv;
    if (akv::ca_whole(items, n, slots_of(p) / akv::ctc::kKeys + 1, 0, akv::ctc::kPartialUnits)) return ATLASKV_OK;
    return launch_pdl(akv::cache_combine_kernel<__nv_bfloat16, D, RB>, join_grid(items, n, RB), akv::kJoinThreads, 0, s, p,
                      a, n);
}

// f<T, D, NT>(args...) for the call's type, head dimension and rows
#define AKV_CA(dtype, D, NT, f, ...)                                                                              \
    ((dtype) == ATLASKV_F32                                                                                       \
         ? ((D) == 64 ? ((NT) == 1 ? f<float, 64, 1>(__VA_ARGS__) : f<float, 64, 2>(__VA_ARGS__))                 \
                      : ((NT) == 1 ? f<float, 128, 1>(__VA_ARGS__) : f<float, 128, 2>(__VA_ARGS__)))              \
         : ((D) == 64 ? ((NT) == 1   ? f<__nv_bfloat16, 64, 1>(__VA_ARGS__)                                       \
                         : (NT) == 2 ? f<__nv_bfloat16, 64, 2>(__VA_ARGS__)                                       \
                                     : f<__nv_bfloat16, 64, 4>(__VA_ARGS__))                                      \
                      : ((NT) == 1   ? f<__nv_bfloat16, 128, 1>(__VA_ARGS__)                                      \
                         : (NT) == 2 ? f<__nv_bfloat16, 128, 2>(__VA_ARGS__)                                      \
                                     : f<__nv_bfloat16, 128, 4>(__VA_ARGS__))))

// kernel<T, D>(args...) for the call's type and head dimension
#define AKV_TD(dtype, D, LAUNCH)                                                     \
    do {                                                                             \
        if ((dtype) == ATLASKV_F32) {                                                \
            if ((D) == 64) LAUNCH(float, 64);                                        \
            else LAUNCH(float, 128);                                                 \
        } else {                                                                     \
            if ((D) == 64) LAUNCH(__nv_bfloat16, 64);                                \
            else LAUNCH(__nv_bfloat16, 128);                                         \
        }                                                                            \
    } while (0)

// What attention over the cache needs of the sequences and of q, without its
// outputs and workspace.  On OK with B > 0, *qs is q's token stride in elements.
atlaskv_status check_attend(const atlaskv_cache *c, const atlaskv_seqs *seqs, int dtype, int H, float scale, const void *q,
                            int64_t q_stride, akv::CacheParams *p, int64_t *qs, size_t *need)
{
    AKV_RET(check_cache(c));
    AKV_RET(cache_params(c, seqs, p));
    AKV_RET(atlaskv_cache_workspace_size(c, dtype, seqs->B, seqs->N, H, need));
    if (!(scale >= 0.f) || std::isinf(scale)) return fail(ATLASKV_EINVAL, "scale must be finite and >= 0");
    if (seqs->B == 0) return ATLASKV_OK;
    AKV_RET(check_rows("q", q, (int64_t)H * c->d.head_dim, dtype, q_stride, qs));
    const long long rows = (long long)p->N * (H / p->H_kv);
    if (rows > (1 << 30)) return fail(ATLASKV_EUNSUPPORTED, "more than 2^30 query rows per KV head");
    if (use_tc(dtype, rows) && tc_blocks(rows) * p->B * p->H_kv > (1 << 30))
        return fail(ATLASKV_EUNSUPPORTED, "too many query rows for one call");
    return ATLASKV_OK;
}

// Attention over the cache into a.out / a.lse or a.oseq / a.lse_seq.
atlaskv_status attend_cache(atlaskv_cache *c, const atlaskv_seqs *seqs, int dtype, int H, float scale,
                            akv::CacheAttendIo a, void *workspace, size_t workspace_bytes, void *stream)
{
    akv::CacheParams p;
    int64_t qs = 0;
    size_t need = 0;
    AKV_RET(check_attend(c, seqs, dtype, H, scale, a.q, a.qs, &p, &qs, &need));
    if (seqs->B == 0) return ATLASKV_OK;
    const int D = c->d.head_dim;
    if (!a.oseq && (!a.out || !aligned16(a.out))) return fail(ATLASKV_EINVAL, "null or unaligned out");
    if (a.lse && !aligned4(a.lse)) return fail(ATLASKV_EINVAL, "unaligned lse");
    if (!workspace || ((uintptr_t)workspace & 255u)) return fail(ATLASKV_EINVAL, "workspace must be 256-byte aligned");
    if (workspace_bytes < need)
        return fail(ATLASKV_ENOMEM, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    a.qs = qs;
    a.H = H;
    a.G = H / p.H_kv;
    a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
    a.ws = static_cast<uint8_t *>(workspace);
    const long long rows = (long long)p.N * a.G;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (use_tc(dtype, rows)) return D == 64 ? launch_tc<64>(c, p, a, s) : launch_tc<128>(c, p, a, s);
    return AKV_CA(dtype, D, row_tiles(dtype, rows), launch_ca, c, p, a, s);
}

}  // namespace

extern "C" {

atlaskv_status atlaskv_rope_init(atlaskv_rope_spec *spec, int32_t layout, int32_t rotary_dim, double base, double factor,
                                 double original_len, double low_turns, double high_turns, double amplitude)
{
    if (!spec) return fail(ATLASKV_EINVAL, "null spec");
    if (layout != ATLASKV_ROPE_HALF && layout != ATLASKV_ROPE_INTERLEAVED)
        return fail(ATLASKV_EINVAL, "rotary layout %d", layout);
    if (rotary_dim < 16 || rotary_dim > 2 * ATLASKV_ROPE_MAX_PAIRS || rotary_dim % 16)
        return fail(ATLASKV_EINVAL, "rotary_dim %d is not a multiple of 16 in [16, %d]", rotary_dim,
                    2 * ATLASKV_ROPE_MAX_PAIRS);
    if (!(base > 0.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor) || !(original_len >= 0.0) ||
        !std::isfinite(original_len) || !(low_turns >= 0.0) || !(high_turns > low_turns) || !std::isfinite(high_turns) ||
        !std::isfinite(amplitude))
        return fail(ATLASKV_EINVAL, "need base > 0, factor > 0, original_len >= 0, 0 <= low_turns < high_turns and a "
                                    "finite amplitude");
    atlaskv_rope_spec r = {};
    r.layout = layout;
    r.rotary_dim = rotary_dim;
    r.amplitude = amplitude;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rotary_dim);
        const double turns = original_len * f / (2.0 * 3.14159265358979323846);
        const double keep =
            original_len == 0.0 ? 0.0 : std::min(1.0, std::max(0.0, (turns - low_turns) / (high_turns - low_turns)));
        r.freq[i] = keep * f + (1.0 - keep) * f / factor;
    }
    *spec = r;
    return ATLASKV_OK;
}

atlaskv_status atlaskv_rope(const atlaskv_rope_spec *spec, const atlaskv_rope_io *io, void *stream)
{
    if (!spec || !io) return fail(ATLASKV_EINVAL, "null spec or io");
    AKV_RET(check_dtype(io->dtype));
    AKV_RET(check_head_dim(io->head_dim));
    if (io->H < 1) return fail(ATLASKV_EINVAL, "H = %d < 1", io->H);
    if (io->H > (1 << 20)) return fail(ATLASKV_EUNSUPPORTED, "more than 2^20 heads");
    if (io->tokens < 0) return fail(ATLASKV_EINVAL, "tokens < 0");
    if (io->backward != 0 && io->backward != 1) return fail(ATLASKV_EINVAL, "backward is 0 or 1");
    akv::RopeParams p;
    AKV_RET(rope_params(spec, io->head_dim, &p));
    if (io->tokens == 0) return ATLASKV_OK;
    akv::RopeIo r = {};
    int64_t xs, ys;
    const int64_t row = (int64_t)io->H * io->head_dim;
    AKV_RET(check_rows("x", io->x, row, io->dtype, io->x_stride, &xs));
    AKV_RET(check_rows("y", io->y, row, io->dtype, io->y_stride, &ys));
    if (io->x == io->y && xs != ys) return fail(ATLASKV_EINVAL, "in place needs equal strides");
    if (!io->positions || !aligned4(io->positions)) return fail(ATLASKV_EINVAL, "null or unaligned positions");
    r.x = io->x;
    r.y = io->y;
    r.pos = io->positions;
    r.tokens = io->tokens;
    r.xs = xs;
    r.ys = ys;
    r.H = io->H;
    r.backward = io->backward;
    r.per_cta = tokens_per_cta(io->tokens, io->H, io->head_dim, num_sms());
    const long long blocks = (io->tokens + r.per_cta - 1) / r.per_cta;
    AKV_RET(check_grid(blocks));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
#define LAUNCH(T, D) AKV_RET(launch_pdl(akv::rope_kernel<T, D>, dim3((unsigned)blocks), akv::kTokThreads, 0, s, p, r))
    AKV_TD(io->dtype, io->head_dim, LAUNCH);
#undef LAUNCH
    return ATLASKV_OK;
}

atlaskv_status atlaskv_cache_page_bytes(int32_t n_kv_heads, int32_t head_dim, int32_t page_size, size_t *bytes)
{
    if (!bytes) return fail(ATLASKV_EINVAL, "null bytes");
    if (n_kv_heads < 1) return fail(ATLASKV_EINVAL, "n_kv_heads = %d < 1", n_kv_heads);
    AKV_RET(check_head_dim(head_dim));
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
        return fail(ATLASKV_EUNSUPPORTED, "page_size %d (16, 32, 64, 128 or 256)", page_size);
    *bytes = (size_t)n_kv_heads * (page_size / 16) * 20 * head_dim;
    return ATLASKV_OK;
}

atlaskv_status atlaskv_create_cache(const atlaskv_cache_desc *d, void *stream, atlaskv_cache **out)
{
    if (!d || !out) return fail(ATLASKV_EINVAL, "null desc or out");
    size_t page = 0;
    AKV_RET(atlaskv_cache_page_bytes(d->n_kv_heads, d->head_dim, d->page_size, &page));
    if (d->n_pages < 1 || d->n_pages > 0x7fffffffLL) return fail(ATLASKV_EINVAL, "n_pages not in [1, 2^31 - 1]");
    if (!d->pages || !aligned16(d->pages)) return fail(ATLASKV_EINVAL, "pages must be a 16-byte aligned device pointer");
    atlaskv_cache *c = new (std::nothrow) atlaskv_cache{};
    if (!c) return fail(ATLASKV_ENOMEM, "out of host memory");
    c->d = *d;
    const auto init = [&]() -> atlaskv_status {
        AKV_CUDA(cudaGetDevice(&c->device));
        c->num_sms = std::min(num_sms(), akv::kMaxCtas / 4);
        AKV_CUDA(cudaMalloc(&c->status, sizeof(int)));
        AKV_CUDA(cudaMemsetAsync(c->status, 0, sizeof(int), static_cast<cudaStream_t>(stream)));
        AKV_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
        return ATLASKV_OK;
    };
    const atlaskv_status st = init();
    if (st != ATLASKV_OK) {
        if (c->status) cudaFree(c->status);
        delete c;
        return st;
    }
    *out = c;
    return ATLASKV_OK;
}

atlaskv_status atlaskv_destroy_cache(atlaskv_cache *c)
{
    if (!c) return ATLASKV_OK;
    const cudaError_t e = cudaFree(c->status);
    delete c;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(ATLASKV_ECUDA, "cudaFree: %s", cudaGetErrorString(e));
    }
    return ATLASKV_OK;
}

atlaskv_status atlaskv_cache_sync_status(atlaskv_cache *c, void *stream)
{
    AKV_RET(check_cache(c));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int v = 0;
    AKV_CUDA(cudaMemcpyAsync(&v, c->status, sizeof(int), cudaMemcpyDeviceToHost, s));
    AKV_CUDA(cudaStreamSynchronize(s));
    if (v == akv::kDevBadPage)
        return fail(ATLASKV_EDEVICE, "a page id, a sequence length or a slot was out of range on the device");
    if (v == akv::kDevNonFinite) return fail(ATLASKV_EDEVICE, "a key or value to store was not finite");
    if (v == akv::kDevTimeout) return fail(ATLASKV_ETIMEOUT, "a bounded device wait gave up");
    if (v != akv::kDevOk) return fail(ATLASKV_EDEVICE, "device status %d", v);
    return ATLASKV_OK;
}

atlaskv_status atlaskv_cache_append(atlaskv_cache *c, const atlaskv_rope_spec *rope, const atlaskv_seqs *seqs,
                                    const atlaskv_append_io *io, void *stream)
{
    AKV_RET(check_cache(c));
    if (!io) return fail(ATLASKV_EINVAL, "null io");
    AKV_RET(check_dtype(io->dtype));
    if (io->H < 0) return fail(ATLASKV_EINVAL, "H = %d < 0", io->H);
    akv::CacheParams p;
    AKV_RET(cache_params(c, seqs, &p));
    akv::RopeParams rp;
    AKV_RET(rope_params(rope, c->d.head_dim, &rp));
    if (seqs->B == 0) return ATLASKV_OK;
    const int D = c->d.head_dim;
    akv::AppendIo a = {};
    int64_t ks, vs, qs = 0;
    AKV_RET(check_rows("k", io->k, (int64_t)p.H_kv * D, io->dtype, io->k_stride, &ks));
    AKV_RET(check_rows("v", io->v, (int64_t)p.H_kv * D, io->dtype, io->v_stride, &vs));
    if (io->H > 0) {
        AKV_RET(check_rows("q", io->q, (int64_t)io->H * D, io->dtype, io->q_stride, &qs));
        if (!io->q_out || !aligned16(io->q_out)) return fail(ATLASKV_EINVAL, "null or unaligned q_out");
        if (io->q_out == io->q && qs != (int64_t)io->H * D) return fail(ATLASKV_EINVAL, "in place needs a dense q");
    }
    if (io->positions && !aligned4(io->positions)) return fail(ATLASKV_EINVAL, "unaligned positions");
    a.k = io->k;
    a.v = io->v;
    a.q = io->q;
    a.q_out = io->q_out;
    a.ks = ks;
    a.vs = vs;
    a.qs = qs;
    a.pos = io->positions;
    a.H = io->H;
    if (2LL * p.H_kv + io->H > (1 << 20)) return fail(ATLASKV_EUNSUPPORTED, "more than 2^20 heads");
    const long long tokens = (long long)p.B * p.N;
    a.kv_per = tokens_per_cta(tokens, 2 * p.H_kv, D, c->num_sms);
    a.q_per = io->H > 0 ? tokens_per_cta(tokens, io->H, D, c->num_sms) : 1;
    const long long kv_ctas = (tokens + a.kv_per - 1) / a.kv_per;
    const long long blocks = kv_ctas + (io->H > 0 ? (tokens + a.q_per - 1) / a.q_per : 0);
    AKV_RET(check_grid(blocks));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.kv_ctas = (int)kv_ctas;
#define LAUNCH(T, D) \
    AKV_RET(launch_pdl(akv::cache_append_kernel<T, D>, dim3((unsigned)blocks), akv::kTokThreads, 0, s, rp, p, a))
    AKV_TD(io->dtype, D, LAUNCH);
#undef LAUNCH
    return ATLASKV_OK;
}

atlaskv_status atlaskv_cache_read(atlaskv_cache *c, const atlaskv_seqs *seqs, int32_t dtype, void *k_out, void *v_out,
                                  void *stream)
{
    AKV_RET(check_cache(c));
    AKV_RET(check_dtype(dtype));
    akv::CacheParams p;
    AKV_RET(cache_params(c, seqs, &p));
    if (!aligned16(k_out) || !aligned16(v_out)) return fail(ATLASKV_EINVAL, "k_out and v_out must be 16-byte aligned");
    if (seqs->B == 0 || (!k_out && !v_out)) return ATLASKV_OK;
    const int D = c->d.head_dim;
    const int wide = (((uintptr_t)k_out | (uintptr_t)v_out) & 31u) == 0;
    // blocks of 16 slots that N consecutive slots can touch
    const int per_seq = (int)std::min<long long>(((long long)p.N + 30) / 16, (long long)p.max_pages * p.page_size / 16);
    const long long warps = (long long)p.B * per_seq * p.H_kv, blocks = (warps + akv::kReadWarps - 1) / akv::kReadWarps;
    AKV_RET(check_grid(blocks));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
#define LAUNCH(T, D)                                                                                                \
    AKV_RET(launch_pdl(akv::cache_read_kernel<T, D>, dim3((unsigned)blocks), 32 * akv::kReadWarps, 0, s, p,         \
                       static_cast<T *>(k_out), static_cast<T *>(v_out), per_seq, wide))
    AKV_TD(dtype, D, LAUNCH);
#undef LAUNCH
    return ATLASKV_OK;
}

atlaskv_status atlaskv_cache_workspace_size(const atlaskv_cache *c, int32_t dtype, int32_t B, int32_t N, int32_t H,
                                            size_t *bytes)
{
    if (!c || !bytes) return fail(ATLASKV_EINVAL, "null cache or bytes");
    AKV_RET(check_dtype(dtype));
    if (B < 0 || N < 1 || H < 1 || H % c->d.n_kv_heads)
        return fail(ATLASKV_EINVAL, "need B >= 0, N >= 1 and H a positive multiple of H_kv = %d", c->d.n_kv_heads);
    *bytes = 0;
    if (B == 0) return ATLASKV_OK;
    const long long rows = (long long)N * (H / c->d.n_kv_heads);
    if (use_tc(dtype, rows)) *bytes = c->d.head_dim == 64 ? tc_workspace<64>(c) : tc_workspace<128>(c);
    else *bytes = AKV_CA(dtype, c->d.head_dim, row_tiles(dtype, rows), ca_workspace, c);
    return ATLASKV_OK;
}

atlaskv_status atlaskv_cache_attend(atlaskv_cache *c, const atlaskv_seqs *seqs, const atlaskv_cache_attend_io *io,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    if (!io) return fail(ATLASKV_EINVAL, "null io");
    akv::CacheAttendIo a = {};
    a.q = io->q;
    a.qs = io->q_stride;
    a.out = io->out;
    a.lse = io->lse;
    return attend_cache(c, seqs, io->dtype, io->H, io->scale, a, workspace, workspace_bytes, stream);
}

}  // extern "C"

atlaskv_status akv_cache_matches(const atlaskv_cache *c, int n_kv_heads, int head_dim)
{
    if (c->d.n_kv_heads != n_kv_heads || c->d.head_dim != head_dim)
        return fail(ATLASKV_EINVAL, "the cache has %d KV heads of %d channels, the tree %d of %d", c->d.n_kv_heads,
                    c->d.head_dim, n_kv_heads, head_dim);
    return check_cache(c);
}

atlaskv_status akv_cache_check(const atlaskv_cache *c, const atlaskv_seqs *seqs, int dtype, int H, const void *q, float scale)
{
    akv::CacheParams p;
    int64_t qs = 0;
    size_t need = 0;
    return check_attend(c, seqs, dtype, H, scale, q, 0, &p, &qs, &need);
}

atlaskv_status akv_cache_part(atlaskv_cache *c, const atlaskv_seqs *seqs, int dtype, int H, const void *q, float scale,
                              float *oseq, float *lse_seq, void *workspace, size_t workspace_bytes, void *stream)
{
    akv::CacheAttendIo a = {};
    a.q = q;
    a.oseq = oseq;
    a.lse_seq = lse_seq;
    return attend_cache(c, seqs, dtype, H, scale, a, workspace, workspace_bytes, stream);
}
