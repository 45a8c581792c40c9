// cache_host.cuh -- host side of the cache operators (include/csa_cache.h):
// validation, launch shapes, the C ABI.  Included once, by csa_indexer.cu.
#pragma once
#include <cmath>

#include "csa_cache.h"
#include "cache_attn_join_kernel.cuh"
#include "cache_attn_unit.cuh"
#include "cache_rows_kernel.cuh"
#include "rotary_kernel.cuh"

namespace {

using csa::cache::CacheView;
using csa::cache::FastDiv;
using csa::cache::PageMap;

constexpr long long kIntLimit = (1ll << 31) - 1024;   // positions and rows, and a tile more, are ints

// Bytes of a row's data and of its scales.
long long cache_row_bytes(const csa_cache_t &c)
{
    return c.dtype == CSA_CACHE_BF16 ? 2ll * c.D : c.dtype == CSA_CACHE_E4M3 ? c.D : c.D / 2;
}

long long cache_scale_bytes(const csa_cache_t &c)
{
    return c.dtype == CSA_CACHE_BF16 ? 0 : c.dtype == CSA_CACHE_E4M3 ? 4 : c.D / 16;
}

csa_status_t validate_cache(const csa_cache_t &c)
{
    if (c.dtype < CSA_CACHE_BF16 || c.dtype > CSA_CACHE_E2M1 || c.H <= 0 || c.D <= 0 ||
        c.num_pages <= 0 || c.page_size <= 0 || c.page_stride < 0 || c.scale_page_stride < 0)
        return CSA_ERR_INVALID_ARG;
    if (c.D % 16 != 0 || c.D > 512 ||
        static_cast<long long>(c.H) * c.page_size >= kIntLimit)
        return CSA_ERR_UNSUPPORTED;
    const bool scaled = c.dtype != CSA_CACHE_BF16;
    if (!c.data || !aligned(c.data, 16) || (scaled && (!c.scale || !aligned(c.scale, 16))))
        return CSA_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(c.H) * c.page_size;
    if (c.page_stride && (c.page_stride % 16 != 0 || c.page_stride < rows * cache_row_bytes(c)))
        return CSA_ERR_INVALID_ARG;
    if (scaled && c.scale_page_stride &&
        (c.scale_page_stride % cache_scale_bytes(c) != 0 ||
         c.scale_page_stride < rows * cache_scale_bytes(c)))
        return CSA_ERR_INVALID_ARG;
    // a row's data must start on 16 bytes: dense pages of E2M1 rows of 8 (mod 16) bytes do not
    if (cache_row_bytes(c) % 16 != 0)
        return CSA_ERR_UNSUPPORTED;
    if (c.dtype == CSA_CACHE_E2M1 && !(c.tensor_scale > 0.0f && std::isfinite(c.tensor_scale)))
        return CSA_ERR_INVALID_ARG;
    return CSA_OK;
}

csa_status_t validate_pages(const int32_t *kv_len, const int32_t *table, int max_pages,
                            long long table_stride, int page_size)
{
    if (max_pages <= 0 || table_stride < max_pages)
        return CSA_ERR_INVALID_ARG;
    if (!kv_len || !table || !aligned(kv_len, 4) || !aligned(table, 4))
        return CSA_ERR_INVALID_ARG;
    if (static_cast<long long>(max_pages) * page_size >= kIntLimit)
        return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

CacheView cache_view(const csa_cache_t &c)
{
    const long long rows = static_cast<long long>(c.H) * c.page_size;
    CacheView v;
    v.data = static_cast<uint8_t *>(c.data);
    v.scale = static_cast<uint8_t *>(c.scale);
    v.row_bytes = static_cast<int>(cache_row_bytes(c));
    v.scale_bytes = static_cast<int>(cache_scale_bytes(c));
    v.page_stride = c.page_stride ? c.page_stride : rows * v.row_bytes;
    v.scale_stride = c.scale_page_stride ? c.scale_page_stride : rows * v.scale_bytes;
    v.tensor_scale = c.dtype == CSA_CACHE_E2M1 ? c.tensor_scale : 1.0f;
    return v;
}

PageMap page_map(const csa_cache_t &c, const int32_t *table, int max_pages, long long table_stride)
{
    PageMap pm;
    pm.table = table;
    pm.table_stride = table_stride;
    pm.max_pages = max_pages;
    pm.num_pages = c.num_pages;
    pm.page_size = c.page_size;
    pm.div = FastDiv::of(static_cast<uint32_t>(c.page_size));
    return pm;
}

bool same_pages(const csa_cache_t &a, const csa_cache_t &b)
{
    return a.dtype == b.dtype && a.H == b.H && a.num_pages == b.num_pages && a.page_size == b.page_size;
}

// Memory in pieces: `count` of them, `bytes` each, `stride` from one to the next.
struct Pieces {
    uintptr_t at;
    long long stride, bytes;
    int count;

    uintptr_t end() const { return at + static_cast<uintptr_t>(count - 1) * stride + bytes; }
};

Pieces data_of(const csa_cache_t &c, const CacheView &v)
{
    return {reinterpret_cast<uintptr_t>(v.data), v.page_stride,
            static_cast<long long>(c.H) * c.page_size * v.row_bytes, c.num_pages};
}

Pieces scale_of(const csa_cache_t &c, const CacheView &v)
{
    return {reinterpret_cast<uintptr_t>(v.scale), v.scale_stride,
            static_cast<long long>(c.H) * c.page_size * v.scale_bytes, c.num_pages};
}

long long floor_div(long long a, long long b) { return a / b - (a % b < 0); }      // b > 0

// Whether two memories share a byte.  Exact, so that caches whose pages interleave in one
// allocation are told from caches that overlap: pages at one distance need one division, others
// (in ranges that overlap) one for each page of the shorter list.
bool share(const Pieces &a, const Pieces &b)
{
    if (a.bytes <= 0 || b.bytes <= 0 || a.end() <= b.at || b.end() <= a.at)
        return false;
    const long long d = static_cast<long long>(b.at - a.at);
    if (a.stride == b.stride && a.count > 1 && b.count > 1) {
        // pieces j of b and i of a meet where -b.bytes < d + (j - i) * stride < a.bytes
        long long k = floor_div(-b.bytes - d, a.stride) + 1;
        k = k > 1 - a.count ? k : 1 - a.count;
        return k < b.count && d + k * a.stride < a.bytes;
    }
    if (a.count > b.count)
        return share(b, a);
    for (int i = 0; i < a.count; ++i) {
        // the first piece of b that ends behind piece i of a begins
        const long long from = i * a.stride - d;
        long long j = b.count > 1 ? floor_div(from - b.bytes, b.stride) + 1 : 0;
        j = j > 0 ? j : 0;
        if (j < b.count && j * b.stride < from + a.bytes && j * b.stride + b.bytes > from)
            return true;
    }
    return false;
}

Pieces one_piece(const void *p, long long bytes)
{
    return {reinterpret_cast<uintptr_t>(p), 0, p ? bytes : 0, 1};
}

// Launches a kernel that may begin while the one before it on the stream ends; it waits
// for that one's results itself (after_kernel_before).
template <typename... P>
void launch_behind(void (*fn)(P...), dim3 grid, int threads, cudaStream_t stream, P... args)
{
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, fn, args...);         // (launched() reports)
}

csa_status_t launched() { return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

} // namespace

// ---------------------------------------------------------------------------
// Rotation frequencies (host).
extern "C" csa_status_t csa_rope_frequencies(int rot_dim, double base, int scaling, double factor,
                                             int original_len, double beta_fast, double beta_slow,
                                             float *inv_freq, float *scale)
{
    const double pi = 3.14159265358979323846;
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base) || !inv_freq ||
        !scale || scaling < CSA_ROPE_PLAIN || scaling > CSA_ROPE_YARN)
        return CSA_ERR_INVALID_ARG;
    if (scaling != CSA_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
        return CSA_ERR_INVALID_ARG;
    if (scaling == CSA_ROPE_NTK && rot_dim == 2)
        return CSA_ERR_INVALID_ARG;
    double lo = 0.0, hi = 0.0;
    if (scaling == CSA_ROPE_YARN) {
        if (original_len <= 0 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast))
            return CSA_ERR_INVALID_ARG;
        // the dimension (in pairs) that turns `turns` times within original_len
        auto pair_of_turns = [&](double turns) {
            return rot_dim * std::log(original_len / (turns * 2.0 * pi)) / (2.0 * std::log(base));
        };
        lo = std::fmax(std::floor(pair_of_turns(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of_turns(beta_slow)), rot_dim - 1.0);
    }
    if (scaling == CSA_ROPE_NTK)
        base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == CSA_ROPE_LINEAR)
            f /= factor;
        if (scaling == CSA_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        inv_freq[i] = static_cast<float>(f);
    }
    *scale = scaling == CSA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return CSA_OK;
}

// ---------------------------------------------------------------------------
// Rotary positions.
namespace {

using csa::rotary::RotaryParams;
using RotaryFn = void (*)(const RotaryParams);

template <typename T, int V>
RotaryFn rotary_fn(bool inter)
{
    return inter ? csa::rotary::rotary_kernel<T, V, true> : csa::rotary::rotary_kernel<T, V, false>;
}

// Position of a head's other elements and the strides allow V elements at a time.
bool rotary_fits(const csa_rotary_args_t *a, int v)
{
    const int unit = a->interleaved ? a->rot_dim : a->rot_dim / 2;
    return unit % v == 0 && a->rot_offset % v == 0 && a->D % v == 0 && a->x_token_stride % v == 0 &&
           a->x_head_stride % v == 0 && a->out_token_stride % v == 0 && a->out_head_stride % v == 0 &&
           aligned(a->x, 16) && aligned(a->out, 16);
}

} // namespace

extern "C" csa_status_t csa_rotary(const csa_rotary_args_t *args, cudaStream_t stream)
{
    EntryRange range("csa_rotary");
    const csa_rotary_args_t *a = args;
    if (!a || a->N < 0 || a->H <= 0 || a->D <= 0 || a->dtype < CSA_ELEM_BF16 || a->dtype > CSA_ELEM_FP32 ||
        a->rot_dim < 2 || a->rot_dim % 2 != 0 || a->rot_offset < 0 || a->rot_offset % 2 != 0 ||
        a->rot_offset > a->D - a->rot_dim || !std::isfinite(a->scale))
        return CSA_ERR_INVALID_ARG;
    if (a->D > 1024 || static_cast<long long>(a->H) * a->D >= kIntLimit / 64)
        return CSA_ERR_UNSUPPORTED;
    if (a->N == 0)
        return CSA_OK;
    const int size = a->dtype == CSA_ELEM_FP32 ? 4 : 2;
    if (!a->x || !a->out || !a->positions || !a->inv_freq || !aligned(a->x, size) ||
        !aligned(a->out, size) || !aligned(a->positions, 4) || !aligned(a->inv_freq, 4))
        return CSA_ERR_INVALID_ARG;
    // rows of out may not overlap: heads within a token or tokens within a head, whichever is outer
    const long long oh = a->out_head_stride, ot = a->out_token_stride;
    if (a->x_head_stride < 0 || a->x_token_stride < 0 || oh < 0 || ot < 0 ||
        (a->H > 1 && oh < a->D) || (a->N > 1 && ot < a->D) ||
        (a->H > 1 && a->N > 1 && ot < (a->H - 1) * oh + a->D && oh < (a->N - 1) * ot + a->D))
        return CSA_ERR_INVALID_ARG;
    if (a->x == a->out && ((a->H > 1 && a->x_head_stride != oh) || (a->N > 1 && a->x_token_stride != ot)))
        return CSA_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0)
        return CSA_ERR_CUDA;
    RotaryParams p;
    std::memset(&p, 0, sizeof p);
    p.x = a->x;
    p.out = a->out;
    p.N = a->N;
    p.H = a->H;
    p.D = a->D;
    p.xt = a->x_token_stride;
    p.xh = a->x_head_stride;
    p.ot = ot;
    p.oh = oh;
    p.positions = a->positions;
    p.inv_freq = a->inv_freq;
    p.half = a->rot_dim / 2;
    p.off = a->rot_offset;
    p.inverse = a->inverse != 0;
    p.scale = a->scale;
    p.copy = a->x != a->out;
    const bool inter = a->interleaved != 0;
    const int wide = 16 / size;
    const int v = rotary_fits(a, wide) ? wide : 1;
    if (inter && v > 1) {
        p.units = (p.copy ? a->D : a->rot_dim) / v;
    } else {
        const int rest = (a->D - a->rot_dim) / v;
        p.pair_units = p.half / v;
        p.units = p.pair_units + (p.copy ? (rest + 1) / 2 : 0);
    }
    p.div_units = FastDiv::of(p.units);
    p.div_half = FastDiv::of(p.half);
    // blocks: about four units a thread; a token's heads are shared out when
    // there are too few tokens to fill the GPU
    const long long per_token = static_cast<long long>(a->H) * p.units;
    const long long want = 4ll * csa::rotary::kThreads;
    long long tokens = per_token >= want ? 1 : want / per_token;
    while (tokens > 1 && (a->N + tokens - 1) / tokens < 4ll * sms)
        tokens = (tokens + 1) / 2;
    const long long most = 32768 / (8ll * p.half);       // cos and sin in 32 KB
    p.tokens = static_cast<int>(tokens < most ? tokens : most);
    const long long blocks = (a->N + p.tokens - 1) / p.tokens;
    long long shares = (2ll * sms + blocks - 1) / blocks;
    const long long most_shares = (per_token * p.tokens + csa::rotary::kThreads - 1) / csa::rotary::kThreads;
    shares = shares < most_shares ? shares : most_shares;
    shares = shares < 1 ? 1 : shares > a->H ? a->H : shares;
    p.heads = static_cast<int>((a->H + shares - 1) / shares);
    p.div_heads = FastDiv::of(p.heads);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((a->H + p.heads - 1) / p.heads));
    if (grid.y > 65535)
        return CSA_ERR_UNSUPPORTED;
    RotaryFn fn;
    if (a->dtype == CSA_ELEM_FP32)
        fn = v > 1 ? rotary_fn<float, 4>(inter) : rotary_fn<float, 1>(inter);
    else if (a->dtype == CSA_ELEM_FP16)
        fn = v > 1 ? rotary_fn<__half, 8>(inter) : rotary_fn<__half, 1>(inter);
    else
        fn = v > 1 ? rotary_fn<__nv_bfloat16, 8>(inter) : rotary_fn<__nv_bfloat16, 1>(inter);
    if (!mark(0, stream))
        return CSA_ERR_CUDA;
    fn<<<grid, csa::rotary::kThreads, p.tokens * p.half * sizeof(float2), stream>>>(p);
    const csa_status_t st = launched();
    return st == CSA_OK && !mark(1, stream) ? CSA_ERR_CUDA : st;
}

// ---------------------------------------------------------------------------
// Appending to and reading from a cache.
namespace {

int row_lanes(int D) { return pow2_ceil(D / 16); }

template <int kType>
void launch_append(const csa::cache::AppendParams &p, bool inter, unsigned grid, size_t smem,
                   cudaStream_t stream)
{
    using namespace csa::cache;
    auto fn = p.half == 0 ? append_kernel<kType, kStill>
              : inter     ? append_kernel<kType, kInterleaved>
              : ((p.off | p.half) & 15) == 0 ? append_kernel<kType, kWhole> : append_kernel<kType, kHalves>;
    fn<<<grid, kRowThreads, smem, stream>>>(p);
}

} // namespace

extern "C" csa_status_t csa_cache_append(const csa_append_args_t *args, cudaStream_t stream)
{
    EntryRange range("csa_cache_append");
    const csa_append_args_t *a = args;
    if (!a || a->N < 0 || a->B < 0 || (!a->cu_tokens && (a->S < 0 || a->N != static_cast<long long>(a->B) * a->S)))
        return CSA_ERR_INVALID_ARG;
    csa_status_t st = validate_cache(a->cache_k);
    if (st == CSA_OK && a->v)
        st = validate_cache(a->cache_v);
    if (st != CSA_OK)
        return st;
    if (a->v && !same_pages(a->cache_k, a->cache_v))
        return CSA_ERR_INVALID_ARG;
    // six tensor scales are what a code of the largest magnitude and a scale of one stand for
    if (a->cache_k.dtype == CSA_CACHE_E2M1 && (!std::isfinite(6.0f * a->cache_k.tensor_scale) ||
                                               (a->v && !std::isfinite(6.0f * a->cache_v.tensor_scale))))
        return CSA_ERR_INVALID_ARG;
    // the lanes that a token's rows take are counted in an int
    if (static_cast<long long>(a->cache_k.H) * row_lanes(a->cache_k.D) >= kIntLimit ||
        (a->v && static_cast<long long>(a->cache_v.H) * row_lanes(a->cache_v.D) >= kIntLimit))
        return CSA_ERR_UNSUPPORTED;
    if (a->inv_freq && (a->rot_dim < 2 || a->rot_dim % 2 != 0 || a->rot_offset < 0 || a->rot_offset % 2 != 0 ||
                        a->rot_offset > a->cache_k.D - a->rot_dim || !std::isfinite(a->rope_scale) ||
                        !aligned(a->inv_freq, 4)))
        return CSA_ERR_INVALID_ARG;
    if (a->N == 0 || a->B == 0)
        return CSA_OK;
    st = validate_pages(a->kv_len, a->page_table, a->max_pages, a->table_stride, a->cache_k.page_size);
    if (st != CSA_OK)
        return st;
    if (!a->k || !aligned(a->k, 16) || (a->v && !aligned(a->v, 16)) || !aligned(a->cu_tokens, 4) ||
        !aligned(a->positions, 4))
        return CSA_ERR_INVALID_ARG;
    if (a->k_token_stride < 0 || a->k_head_stride < 0 || a->k_token_stride % 8 != 0 || a->k_head_stride % 8 != 0 ||
        (a->v && (a->v_token_stride < 0 || a->v_head_stride < 0 || a->v_token_stride % 8 != 0 ||
                  a->v_head_stride % 8 != 0)))
        return CSA_ERR_INVALID_ARG;
    // what is written must be different memory: codes and scales, of keys and of values
    const CacheView ck = cache_view(a->cache_k), cv = a->v ? cache_view(a->cache_v) : ck;
    const csa_cache_t &cache_v = a->v ? a->cache_v : a->cache_k;
    const Pieces written[4] = {data_of(a->cache_k, ck), scale_of(a->cache_k, ck), data_of(cache_v, cv),
                               scale_of(cache_v, cv)};
    for (int i = 0; i < (a->v ? 4 : 2); ++i)
        for (int j = 0; j < i; ++j)
            if (share(written[i], written[j]))
                return CSA_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0)
        return CSA_ERR_CUDA;
    csa::cache::AppendParams p;
    std::memset(&p, 0, sizeof p);
    p.k = static_cast<const __nv_bfloat16 *>(a->k);
    p.v = static_cast<const __nv_bfloat16 *>(a->v);
    p.kt = a->k_token_stride;
    p.kh = a->k_head_stride;
    p.vt = a->v_token_stride;
    p.vh = a->v_head_stride;
    p.N = a->N;
    p.B = a->B;
    p.S = a->S;
    p.H = a->cache_k.H;
    p.Dk = a->cache_k.D;
    p.Dv = a->v ? a->cache_v.D : 0;
    p.cu = a->cu_tokens;
    p.kv_len = a->kv_len;
    p.pm = page_map(a->cache_k, a->page_table, a->max_pages, a->table_stride);
    p.ck = ck;
    if (a->v)
        p.cv = cv;
    p.inv_freq = a->inv_freq;
    p.positions = a->positions;
    p.half = a->inv_freq ? a->rot_dim / 2 : 0;
    p.off = a->rot_offset;
    p.rope_scale = a->rope_scale;
    p.lanes_k = row_lanes(p.Dk);
    p.lanes_v = a->v ? row_lanes(p.Dv) : 1;
    // tokens a block takes: about four rounds of rows, fewer while blocks are few
    int tokens = 4 * csa::cache::kRowThreads / (p.lanes_k * p.H);
    tokens = tokens < 1 ? 1 : tokens > csa::cache::kMaxTile ? csa::cache::kMaxTile : tokens;
    while (tokens > 1 && (static_cast<long long>(a->N) + tokens - 1) / tokens < 4ll * sms)
        tokens = (tokens + 1) / 2;
    const int turns = p.half + (p.half >> 3);            // places of a token's cos and sin (turn_at)
    if (p.half && tokens > 2048 / turns)                 // in 32 KB
        tokens = 2048 / turns;
    p.tokens = tokens;
    p.div_H = FastDiv::of(p.H);
    p.div_half = FastDiv::of(p.half ? p.half : 1);
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(a->N) + tokens - 1) / tokens);
    const size_t smem = static_cast<size_t>(tokens) * turns * sizeof(csa::cache::Turn);
    const bool inter = a->interleaved != 0;
    if (!mark(0, stream))
        return CSA_ERR_CUDA;
    if (a->cache_k.dtype == CSA_CACHE_BF16)
        launch_append<0>(p, inter, grid, smem, stream);
    else if (a->cache_k.dtype == CSA_CACHE_E4M3)
        launch_append<1>(p, inter, grid, smem, stream);
    else
        launch_append<2>(p, inter, grid, smem, stream);
    st = launched();
    return st == CSA_OK && !mark(1, stream) ? CSA_ERR_CUDA : st;
}

extern "C" csa_status_t csa_cache_read(const csa_cache_read_args_t *args, cudaStream_t stream)
{
    EntryRange range("csa_cache_read");
    const csa_cache_read_args_t *a = args;
    if (!a || a->B < 0 || a->T < 0)
        return CSA_ERR_INVALID_ARG;
    csa_status_t st = validate_cache(a->cache);
    if (st != CSA_OK)
        return st;
    if (a->B == 0 || a->T == 0)
        return CSA_OK;
    st = validate_pages(a->kv_len, a->page_table, a->max_pages, a->table_stride, a->cache.page_size);
    if (st != CSA_OK)
        return st;
    if (!a->out || !aligned(a->out, 16))
        return CSA_ERR_INVALID_ARG;
    if (static_cast<long long>(a->T) * a->cache.H >= kIntLimit / 2)
        return CSA_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (sms <= 0)
        return CSA_ERR_CUDA;
    csa::cache::ReadParams p;
    std::memset(&p, 0, sizeof p);
    p.c = cache_view(a->cache);
    p.pm = page_map(a->cache, a->page_table, a->max_pages, a->table_stride);
    p.kv_len = a->kv_len;
    p.B = a->B;
    p.T = a->T;
    p.H = a->cache.H;
    p.D = a->cache.D;
    p.lanes = row_lanes(p.D);
    p.rows = a->T * p.H;
    p.div_H = FastDiv::of(p.H);
    p.out = static_cast<__nv_bfloat16 *>(a->out);
    const int per = csa::cache::kRowThreads / p.lanes * csa::cache::kReadAhead;
    const unsigned rows_y = a->B < 65535 ? a->B : 65535;
    long long need = (static_cast<long long>(p.rows) + per - 1) / per, most = (16ll * sms + rows_y - 1) / rows_y;
    const dim3 grid(static_cast<unsigned>(need < most ? need : most), rows_y);
    if (!mark(0, stream))
        return CSA_ERR_CUDA;
    if (a->cache.dtype == CSA_CACHE_BF16)
        csa::cache::read_kernel<0><<<grid, csa::cache::kRowThreads, 0, stream>>>(p);
    else if (a->cache.dtype == CSA_CACHE_E4M3)
        csa::cache::read_kernel<1><<<grid, csa::cache::kRowThreads, 0, stream>>>(p);
    else
        csa::cache::read_kernel<2><<<grid, csa::cache::kRowThreads, 0, stream>>>(p);
    st = launched();
    return st == CSA_OK && !mark(1, stream) ? CSA_ERR_CUDA : st;
}

// ---------------------------------------------------------------------------
// Attention over a 4-bit cache.
namespace {

using csa::cattn::CattnPlan;

// What turns a product of stored keys and a query (times 2^kQueryBits) into a log2 score.
float log2_scale(const csa_cache_attn_args_t *a)
{
    return a->scale * a->cache_k.tensor_scale * (1.4426950408889634f / (1 << csa::cattn::kQueryBits));
}

// Whether anything that a call writes shares memory with the query, the selection or
// something else that it writes.
bool cattn_overlaps(const csa_cache_attn_args_t *a, const void *workspace, size_t workspace_bytes)
{
    const long long queries = static_cast<long long>(a->B) * a->S, rows = queries * a->HA;
    const Pieces all[5] = {one_piece(a->q, 2 * rows * a->cache_k.D), one_piece(a->idx, 4 * queries * a->topk),
                           one_piece(a->out, 2 * rows * a->cache_v.D), one_piece(a->lse, 4 * rows),
                           one_piece(workspace, static_cast<long long>(workspace_bytes))};
    for (int i = 2; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (share(all[i], all[j]))
                return true;
    return false;
}

csa_status_t validate_cattn(const csa_cache_attn_args_t *a)
{
    if (!a || a->B < 0 || a->S < 0 || a->HA <= 0 || !std::isfinite(a->scale) || (a->idx && a->topk <= 0))
        return CSA_ERR_INVALID_ARG;
    csa_status_t st = validate_cache(a->cache_k);
    if (st == CSA_OK)
        st = validate_cache(a->cache_v);
    if (st != CSA_OK)
        return st;
    if (!same_pages(a->cache_k, a->cache_v) || a->HA % a->cache_k.H != 0)
        return CSA_ERR_INVALID_ARG;
    if (a->cache_k.dtype == CSA_CACHE_E2M1 && !std::isfinite(log2_scale(a)))
        return CSA_ERR_INVALID_ARG;
    const int dk = a->cache_k.D, dv = a->cache_v.D;
    if (a->cache_k.dtype != CSA_CACHE_E2M1 || dk % 64 != 0 || dk > 256 || dv % 64 != 0 || dv > 256 ||
        a->HA / a->cache_k.H > 128)
        return CSA_ERR_UNSUPPORTED;
    if (static_cast<long long>(a->B) * a->S == 0)
        return CSA_OK;
    st = validate_pages(a->kv_len, a->page_table, a->max_pages, a->table_stride, a->cache_k.page_size);
    if (st != CSA_OK)
        return st;
    if (!a->q || !a->out || !aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->idx, 4) ||
        !aligned(a->lse, 4))
        return CSA_ERR_INVALID_ARG;
    if (static_cast<long long>(a->S) * a->HA >= kIntLimit || (a->idx && a->topk >= kIntLimit) ||
        static_cast<long long>(a->B) * a->S * a->HA >= kIntLimit)
        return CSA_ERR_UNSUPPORTED;
    return cattn_overlaps(a, nullptr, 0) ? CSA_ERR_INVALID_ARG : CSA_OK;
}

csa_status_t plan_cattn(const csa_cache_attn_args_t *a, CattnPlan *pl)
{
    const int sms = device_sms();
    if (sms <= 0)
        return CSA_ERR_CUDA;
    const int H = a->cache_k.H, G = a->HA / H;
    pl->rows = a->idx ? G : a->S * G;
    // The tensor-memory kernel takes what does not fit one tile of the register kernel, which reads and
    // converts every key once for 16 rows.  Wide / register (as tiles of 16), us, D = 128, by rows:
    //                                            17-20        32         48         64        128
    //   16 x 16,384 keys, 8 cache heads        228 / 181   230 / 189  232 / 274  225 / 356  280 / 688
    //   the same, ragged                       228 / 118   226 / 127  228 / 181  224 / 235  262 / 451
    //   4 x 4,096 keys, 2 cache heads         18.2 / 14.7 18.9 / 16.1 20.1 / 19.0 20.9 / 22.9 22.7 / 29.1
    //   32 x 2,048 keys, 1 cache head         19.3 / 21.4 20.2 / 22.9 21.5 / 27.4 21.8 / 31.2 23.7 / 46.3
    //   32 x 2,048 selected                   19.0 / 23.0 19.9 / 24.3 20.9 / 30.5 21.8 / 35.0 23.6 / 51.0
    //   512 queries over 2,048 selected        128 / 127   131 / 139  133 / 197  136 / 248  168 / 475
    // For selections the border is where it should be; dense calls over long contexts would gain from a
    // higher one (32 rows, ragged 48), for the wide kernel's shares are even in the table's reach, not
    // in the sequences' keys.
    pl->wide = pl->rows > 16;
    const CacheView ck = cache_view(a->cache_k), cv = cache_view(a->cache_v);
    pl->bulk = !a->idx && a->cache_k.page_size % 16 == 0 && ck.scale_stride % 16 == 0 && cv.scale_stride % 16 == 0;
    pl->tile_rows = pl->rows <= 8 ? 8 : pl->rows <= 16 ? 16 : pl->rows <= 64 ? 64 : csa::cattn::kWideRows;
    pl->tiles = (pl->rows + pl->tile_rows - 1) / pl->tile_rows;
    pl->works = static_cast<long long>(a->B) * (a->idx ? a->S : 1) * H * pl->tiles;
    bool ok = false;
    switch (a->cache_k.D) {
    case 64: ok = csa::cattn::pick_64(a->cache_v.D, pl); break;
    case 128: ok = csa::cattn::pick_128(a->cache_v.D, pl); break;
    case 192: ok = csa::cattn::pick_192(a->cache_v.D, pl); break;
    case 256: ok = csa::cattn::pick_256(a->cache_v.D, pl); break;
    }
    if (!ok)
        return CSA_ERR_UNSUPPORTED;
    const long long most = a->idx ? a->topk : static_cast<long long>(a->max_pages) * a->cache_k.page_size;
    long long splits = 1;
    if (pl->wide) {
        // the share count that ends first: rounds of the persistent grid x tiles
        // of a share, an item costing about three tiles of its own
        const long long tiles = (most + pl->keys - 1) / pl->keys;
        long long best = -1;
        for (long long s = 1; s <= tiles && s <= 256; ++s) {
            const long long cost = (pl->works * s + sms - 1) / sms * ((tiles + s - 1) / s + 3);
            if (best < 0 || cost < best) {
                best = cost;
                splits = s;
            }
        }
    } else {
        // as many CTAs as the GPU holds share the chunks; where no tile has more than kAlone
        // chunks (256 keys each at D = 128), a CTA each, and no second kernel.  Alone / shared and joined,
        // us on the device, 32 heads over 8, by keys:
        //                    256         512         777        1,024
        //   1 sequence    5.5 / 8.4   7.8 / 9.7   10.9 / 9.8  11.1 / 9.8
        //   16 sequences  5.8 / 9.4   7.8 / 10.8  11.0 / 16.9 11.2 / 17.1
        // and 17 / 21 us issued one by one, at each of them: the second launch costs more than the 1.3
        // us that a captured step of one sequence would gain at three or four chunks.
        constexpr long long kAlone = 4;
        const long long chunks = (most + pl->chunk - 1) / pl->chunk;
        const long long held = static_cast<long long>(sms) * pl->ctas;
        pl->most = static_cast<int>(chunks);
        pl->ctas = chunks <= kAlone ? 0 : static_cast<int>(pl->works * chunks < held ? pl->works * chunks : held);
    }
    pl->splits = static_cast<int>(splits < 1 ? 1 : splits > 256 ? 256 : splits);
    if (pl->works * pl->splits >= kIntLimit)
        return CSA_ERR_UNSUPPORTED;
    const long long pieces = pl->wide ? (pl->splits > 1 ? pl->works * pl->splits : 0) : 2ll * pl->ctas;
    pl->piece_rows = pieces * pl->tile_rows;
    pl->workspace = static_cast<size_t>(pl->piece_rows) * (a->cache_v.D + 2) * sizeof(float);
    return CSA_OK;
}

// Whether a kernel's shared memory has been allowed for on the current device; done
// once, by the most the kernel can ask for.
bool is_ready(const CattnPlan &pl)
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev < 64 && pl.ready->load(std::memory_order_acquire) >> dev & 1ull;
}

bool set_ready(const CattnPlan &pl, const void *fn)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, pl.wide ? kSmemLimit : pl.smem) != cudaSuccess)
        return false;
    if (dev < 64)
        pl.ready->fetch_or(1ull << dev, std::memory_order_release);
    return true;
}

// The tiles' launch: the persistent tcgen05 kernel.
csa_status_t launch_wide(const csa_cache_attn_args_t *a, const CattnPlan &pl, const csa::cattn::AttnParams &p,
                         cudaStream_t stream)
{
    using namespace csa::cattn;
    WideParams w;
    std::memset(&w, 0, sizeof w);
    w.a = p;
    w.items = static_cast<int>(pl.works * pl.splits);
    w.k_bytes = pl.keys * a->cache_k.D * 2;
    w.v_bytes = pl.keys * a->cache_v.D * 2;
    const int q_bytes = kWideRows * a->cache_k.D * 2;
    const int x_bytes = pl.tile_rows == kWideRows ? 0 : 4 * kXCols * 32 * 4;
    const int fixed = q_bytes + pl.raw + x_bytes + static_cast<int>(sizeof(WideBarriers)) + 1024;
    // as many stages as fit
    static const int kChoices[4][2] = {{2, 2}, {2, 1}, {1, 2}, {1, 1}};
    for (const auto &c : kChoices)
        if (fixed + c[0] * w.k_bytes + c[1] * w.v_bytes <= kSmemLimit) {
            w.k_stages = c[0];
            w.v_stages = c[1];
            break;
        }
    if (w.k_stages == 0)
        return CSA_ERR_UNSUPPORTED;
    w.off_k = q_bytes;
    w.off_v = w.off_k + w.k_stages * w.k_bytes;
    w.off_raw = w.off_v + w.v_stages * w.v_bytes;
    w.off_x = w.off_raw + pl.raw;
    w.off_bar = w.off_x + x_bytes;
    // more than half of the SM: one CTA a SM, so its TMEM allocation never waits
    int smem = w.off_bar + static_cast<int>(sizeof(WideBarriers)) + 1024;
    smem = smem < kSmemLimit / 2 + 1024 ? kSmemLimit / 2 + 1024 : smem;
    w.wait_limit = static_cast<long long>(g_wait_limit);
    const int sms = device_sms();
    if (sms <= 0)
        return CSA_ERR_CUDA;
    if (!is_ready(pl)) {
        // the warpgroups trade registers (setmaxnreg): only valid for a build with
        // exactly the launch count that the split assumes
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, pl.wide_fn) != cudaSuccess)
            return CSA_ERR_CUDA;
        if (fa.numRegs != kWideLaunchRegs)
            return CSA_ERR_UNSUPPORTED;
        if (!set_ready(pl, reinterpret_cast<const void *>(pl.wide_fn)))
            return CSA_ERR_CUDA;
    }
    pl.wide_fn<<<w.items < sms ? w.items : sms, kWideThreads, smem, stream>>>(w);
    return launched();
}

} // namespace

extern "C" size_t csa_cache_attention_workspace_size(const csa_cache_attn_args_t *args)
{
    CattnPlan pl;
    if (validate_cattn(args) != CSA_OK || static_cast<long long>(args->B) * args->S == 0 ||
        plan_cattn(args, &pl) != CSA_OK)
        return 0;
    return pl.workspace;
}

extern "C" csa_status_t csa_cache_attention(const csa_cache_attn_args_t *args, void *workspace,
                                            size_t workspace_bytes, cudaStream_t stream)
{
    EntryRange range("csa_cache_attention");
    const csa_cache_attn_args_t *a = args;
    csa_status_t st = validate_cattn(a);
    if (st != CSA_OK)
        return st;
    if (static_cast<long long>(a->B) * a->S == 0)
        return CSA_OK;
    CattnPlan pl;
    st = plan_cattn(a, &pl);
    if (st != CSA_OK)
        return st;
    void *ws = workspace;
    if (ws) {
        if (workspace_bytes < pl.workspace)
            return CSA_ERR_WORKSPACE;
        if (!aligned(ws, 256) || cattn_overlaps(a, ws, pl.workspace))
            return CSA_ERR_INVALID_ARG;
    } else if (pl.workspace && cudaMallocAsync(&ws, pl.workspace, stream) != cudaSuccess) {
        return CSA_ERR_CUDA;
    }
    csa::cattn::AttnParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const __nv_bfloat16 *>(a->q);
    p.ck = cache_view(a->cache_k);
    p.cv = cache_view(a->cache_v);
    p.pm = page_map(a->cache_k, a->page_table, a->max_pages, a->table_stride);
    p.kv_len = a->kv_len;
    p.idx = a->idx;
    p.topk = a->topk;
    p.B = a->B;
    p.S = a->S;
    p.HA = a->HA;
    p.H = a->cache_k.H;
    p.G = p.HA / p.H;
    p.causal = a->causal != 0;
    p.sl2 = log2_scale(a);
    p.v_scale = a->cache_v.tensor_scale;
    p.out = static_cast<__nv_bfloat16 *>(a->out);
    p.lse = a->lse;
    p.wait_limit = static_cast<long long>(g_wait_limit);
    p.splits = pl.splits;
    p.ctas = pl.ctas;
    p.most = pl.most;
    p.chunk = pl.chunk;
    p.works = static_cast<int>(pl.works / a->B);
    p.tiles = pl.tiles;
    p.rows = pl.rows;
    p.capacity = a->max_pages * a->cache_k.page_size;
    p.div_splits = FastDiv::of(p.splits);
    p.div_tiles = FastDiv::of(p.tiles);
    p.div_H = FastDiv::of(p.H);
    p.div_S = FastDiv::of(p.S);
    p.div_G = FastDiv::of(p.G);
    p.part = static_cast<float *>(ws);
    p.stat = reinterpret_cast<float2 *>(p.part + pl.piece_rows * a->cache_v.D);
    if (!mark(0, stream)) {
        st = CSA_ERR_CUDA;
    } else if (pl.wide) {
        st = launch_wide(a, pl, p, stream);
    } else if (!is_ready(pl) && !set_ready(pl, reinterpret_cast<const void *>(pl.fn))) {
        st = CSA_ERR_CUDA;
    } else {
        pl.fn<<<static_cast<unsigned>(pl.ctas ? pl.ctas : pl.works), csa::cattn::kThreads, pl.smem, stream>>>(p);
        st = launched();
    }
    if (st == CSA_OK && !mark(1, stream))
        st = CSA_ERR_CUDA;
    const long long rows = static_cast<long long>(a->B) * a->S * a->HA;
    const bool join = pl.wide ? pl.splits > 1 : pl.ctas > 0;
    if (st == CSA_OK && join) {
        if (pl.wide) {
            launch_behind(csa::cattn::cache_attn_join_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, stream, p,
                          a->cache_v.D, pl.tile_rows, rows);
        } else {
            // a block for every row, or several rows a block when there are many
            const int per = a->S * a->HA, most = 32 * device_sms() / a->B;
            const dim3 grid(a->B, per < most ? per : most < 1 ? 1 : most);
            launch_behind(csa::cattn::cache_attn_pieces_kernel, grid, csa::cattn::kThreads, stream, p, a->cache_v.D,
                          pl.tile_rows);
        }
        st = launched();
        if (st == CSA_OK && !mark(2, stream))
            st = CSA_ERR_CUDA;
    }
    if (!workspace && ws && cudaFreeAsync(ws, stream) != cudaSuccess && st == CSA_OK)
        st = CSA_ERR_CUDA;
    return st;
}
