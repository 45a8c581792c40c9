// cache_rows_kernel.cuh -- rows into and out of a paged cache
// (csa_cache_append, csa_cache_read, include/csa_cache.h).
//
// Both are bound by memory.  A row (one position of one head) is worked by
// lanes of 16 elements each -- one E2M1 scale group, 32 bytes of bf16 -- in a
// group of 2^n lanes, which exchange only the row maximum that the E4M3 scale needs.
// A lane moves whole 32-byte sectors (two 16-byte stores at a stride of 32 write half
// sectors: 19.3 us instead of 15.6 for the 4-bit read below, in L2).  Measured, on inputs that do not
// stand in L2: 18 thousand ragged tokens x 8 heads of 128 + 128 bf16, every key element
// rotated, 46 us (3.9 TB/s; the rotation carried in 40 bits is about 300 instructions for 16
// elements, and it is what bounds the append: left out, an earlier version took 48 us instead
// of 64); 8 x 32,768 rows of 128 from 4 bits to bf16 17.0 us (4.8 TB/s).
#pragma once
#include "cache_common.cuh"
#include "ptx.cuh"

namespace csa {
namespace cache {

constexpr int kRowThreads = 128;
constexpr int kMaxTile = 32;             // tokens a block takes at most
constexpr int kReadAhead = 2;           // rows a lane loads before it works on the first (read)

struct AppendParams {
    const __nv_bfloat16 *k, *v;
    long long kt, kh, vt, vh;            // strides in elements
    int N, B, S, H, Dk, Dv;
    const int32_t *cu, *kv_len;
    PageMap pm;
    CacheView ck, cv;
    const float *inv_freq;
    const int32_t *positions;
    int half, off;                       // rot_dim / 2 (0: no rotation)
    float rope_scale;
    int tokens;                          // tokens a block takes
    int lanes_k, lanes_v;                // lanes a row takes (2^n >= D / 16)
    FastDiv div_H, div_half;
};

// cos and sin of one pair, in 40 bits: the high part has 16 bits, so its
// product with a bf16 element is exact in fp32.
struct Turn {
    float ch, cl, sh, sl;
};

// Where pair i's turn lies in shared memory: one place is left out after eight, so that
// lanes 8 or 16 pairs apart do not meet in a bank.
__device__ __forceinline__ int turn_at(int i) { return i + (i >> 3); }

__device__ __forceinline__ Turn make_turn(int pos, float freq, float scale)
{
    double s, c;
    sincospi(half_turns(pos, freq), &s, &c);
    s *= scale;
    c *= scale;
    Turn t;
    t.ch = __uint_as_float(__float_as_uint(static_cast<float>(c)) & 0xFFFFFF00u);
    t.sh = __uint_as_float(__float_as_uint(static_cast<float>(s)) & 0xFFFFFF00u);
    t.cl = static_cast<float>(c - t.ch);
    t.sl = static_cast<float>(s - t.sh);
    return t;
}

// a * c + b * s (s already signed) for bf16 a and b, rounded once: the two high
// products are exact, their sum's rounding error is recovered by the
// two-sum of Knuth and added with the low products.
__device__ __forceinline__ float turned(float a, float ch, float cl, float b, float sh, float sl)
{
    const float x = __fmul_rn(a, ch), y = __fmul_rn(b, sh);
    const float sum = __fadd_rn(x, y);
    const float z = __fsub_rn(sum, x);
    const float err = __fadd_rn(__fsub_rn(x, __fsub_rn(sum, z)), __fsub_rn(y, z));
    const float low = __fmaf_rn(a, cl, __fmul_rn(b, sl));
    return __fadd_rn(sum, __fadd_rn(err, low));
}

// 16 consecutive bf16 elements.
struct Raw16 {
    uint4 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *src) { load32(src, a, b); }
    __device__ __forceinline__ void unpack(float (&x)[16]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = float2_of_bf16x2(w[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
};

// Stores 16 elements of a row in the cache's type.  E4M3: every lane of the
// row's group calls (peak is exchanged), `active` ones store.
template <int kType>
__device__ __forceinline__ void store16(const CacheView &c, uint8_t *data, uint8_t *scale, int lane,
                                        int lanes, bool active, const float (&x)[16])
{
    float peak = 0.0f;
    if constexpr (kType != 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            peak = fmaxf(peak, fabsf(x[j]));
    }
    if constexpr (kType == 0) {
        if (active) {
            uint4 w[2];
            uint32_t *u = reinterpret_cast<uint32_t *>(w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u[j] = bf16x2_of(x[2 * j], x[2 * j + 1]);
            store32(data + 32 * lane, w[0], w[1]);
        }
    } else if constexpr (kType == 1) {
        if (!active)
            peak = 0.0f;
        for (int m = 1; m < lanes; m <<= 1)
            peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, m));
        float s = __fdiv_rn(peak, 448.0f);
        s = s > 0.0f ? s : 1.0f;                        // (0 for a peak below 2^-141, too: codes of zero)
        if (active) {
            uint4 w;
            uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = e4m3x2(__fdiv_rn(x[4 * j], s), __fdiv_rn(x[4 * j + 1], s)) |
                       e4m3x2(__fdiv_rn(x[4 * j + 2], s), __fdiv_rn(x[4 * j + 3], s)) << 16;
            *reinterpret_cast<uint4 *>(data + 16 * lane) = w;
            if (lane == 0)
                *reinterpret_cast<float *>(scale) = s;
        }
    } else if (active) {
        const uint32_t s8 = e4m3x2(__fdiv_rn(peak, __fmul_rn(6.0f, c.tensor_scale)), 0.0f) & 0xFFu;
        const float s = __fmul_rn(float2_of_f16x2(f16x2_of_e4m3x2(s8)).x, c.tensor_scale);
        uint2 w = make_uint2(0u, 0u);
        if (s > 0.0f) {
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                y[j] = __fdiv_rn(x[j], s);
            w = make_uint2(e2m1x8(y), e2m1x8(y + 8));
        }
        *reinterpret_cast<uint2 *>(data + 8 * lane) = w;
        scale[lane] = static_cast<uint8_t>(s8);
    }
}

// How rows are rotated: not at all; interleaved pairs; halves that lanes of 16 elements
// take whole (offset and half multiples of 16: a lane's partners are 16 elements that
// lie together); halves at any even place.
enum Rotation : int { kStill = 0, kInterleaved = 1, kWhole = 2, kHalves = 3 };

// Rotates the 16 elements [e0, e0 + 16) of a head row; src is the row, `partner` the
// elements half a rotation away (kWhole).
template <int kHow>
__device__ __forceinline__ void rotate16(const __nv_bfloat16 *src, int e0, int off, int half,
                                         const Turn *w, const Raw16 &partner, float (&x)[16])
{
    if (kHow == kStill || e0 + 16 <= off || e0 >= off + 2 * half)
        return;
    if constexpr (kHow == kInterleaved) {
        // off is even: a pair lies within the lane's elements
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const int i = (e0 + j - off) >> 1;
            if (i >= 0 && i < half) {
                const Turn t = w[turn_at(i)];
                const float a = x[j], b = x[j + 1];
                x[j] = turned(a, t.ch, t.cl, b, -t.sh, -t.sl);
                x[j + 1] = turned(b, t.ch, t.cl, a, t.sh, t.sl);
            }
        }
    } else if constexpr (kHow == kWhole) {
        const bool first = e0 < off + half;
        float y[16];
        partner.unpack(y);
        const int i0 = first ? e0 - off : e0 - off - half;      // a multiple of 16
        const Turn *u = w + turn_at(i0);
        const float sign = first ? -1.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const Turn t = u[turn_at(j)];
            x[j] = turned(x[j], t.ch, t.cl, sign * y[j], t.sh, t.sl);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int i = e0 + j - off;
            if (i >= 0 && i < 2 * half) {
                const bool first = i < half;
                const Turn t = w[turn_at(first ? i : i - half)];
                const float b = __bfloat162float(src[first ? e0 + j + half : e0 + j - half]);
                x[j] = first ? turned(x[j], t.ch, t.cl, b, -t.sh, -t.sl)
                             : turned(x[j], t.ch, t.cl, b, t.sh, t.sl);
            }
        }
    }
}

// A lane's part of one row on its way from K or V.
struct RowPart {
    Raw16 own, other;                    // 16 elements, and their partners (kWhole)
    int tok, head;                       // head -1: none
};

// How a block goes through the rows of K, or of V: `lanes` lanes a row, round by round.
template <int kHow>
struct RowWalk {
    const __nv_bfloat16 *src;
    long long ts, hs;
    int D, lanes, step, lane, rows, rounds, n0;
    bool partnered;
    int partner;

    __device__ __forceinline__ RowWalk(const AppendParams &p, const __nv_bfloat16 *src_, long long ts_, long long hs_,
                                       int D_, int lanes_, int n0_, int nt)
        : src(src_), ts(ts_), hs(hs_), D(D_), lanes(lanes_), n0(n0_)
    {
        lane = threadIdx.x & (lanes - 1);
        step = kRowThreads / lanes;
        rows = nt * p.H;
        rounds = (rows + step - 1) / step;
        partnered = kHow == kWhole && 16 * lane >= p.off && 16 * lane < p.off + 2 * p.half;
        partner = 16 * lane < p.off + p.half ? 16 * lane + p.half : 16 * lane - p.half;
    }
    __device__ __forceinline__ const __nv_bfloat16 *row(const RowPart &r) const
    {
        return src + (n0 + r.tok) * ts + r.head * hs;
    }
    __device__ __forceinline__ void load(const AppendParams &p, int round, RowPart &r) const
    {
        const int i = round * step + threadIdx.x / lanes;
        r.tok = static_cast<int>(p.div_H.div(i < rows ? i : 0));
        r.head = i < rows && 16 * lane < D ? i - r.tok * p.H : -1;
        if (r.head >= 0 && CSA_CHECK_INDEX(kChkAppendRow, n0 + r.tok, p.cu ? __ldg(p.cu + p.B) : p.N)) {
            r.own.load(row(r) + 16 * lane);
            if (partnered)
                r.other.load(row(r) + partner);
        }
    }
    // (every lane of a warp: store16 exchanges)
    template <int kType>
    __device__ __forceinline__ void work(const AppendParams &p, const CacheView &c, const RowPart &r, const int *page,
                                         const int *off, const Turn *turns) const
    {
        float x[16];
        uint8_t *data = nullptr, *scale = nullptr;
        const int pg = page[r.tok];
        const bool active = r.head >= 0 && pg >= 0;
        if constexpr (kType == 0 && kHow == kStill) {   // bf16 to bf16
            if (active)
                store32(const_cast<uint8_t *>(row_data(c, p.pm, pg, r.head, off[r.tok])) + 32 * lane, r.own.a, r.own.b);
            return;
        }
        if (active) {
            r.own.unpack(x);
            rotate16<kHow>(row(r), 16 * lane, p.off, p.half, turns + r.tok * turn_at(p.half), r.other, x);
            data = const_cast<uint8_t *>(row_data(c, p.pm, pg, r.head, off[r.tok]));
            if (kType != 0)
                scale = const_cast<uint8_t *>(row_scale(c, p.pm, pg, r.head, off[r.tok]));
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[j] = 0.0f;
        }
        store16<kType>(c, data, scale, lane, lanes, active, x);
    }
};

// One block takes p.tokens tokens: their places (one thread a token), their
// cos and sin, then every row of K and of V.  A row's elements are loaded a round
// before they are worked on, the first ones before their places are known.
template <int kType, int kHow>
__global__ void __launch_bounds__(kRowThreads, 8) append_kernel(const AppendParams p)
{
    extern __shared__ Turn turns[];                     // [tokens][half]
    __shared__ int s_page[kMaxTile], s_off[kMaxTile], s_pos[kMaxTile];
    const int n0 = blockIdx.x * p.tokens;
    const int end = p.cu ? min(p.N, __ldg(p.cu + p.B)) : p.N;      // rows behind the last sequence's are not read
    if (n0 >= end)
        return;
    const int nt = min(p.tokens, end - n0);
    const RowWalk<kHow> kw(p, p.k, p.kt, p.kh, p.Dk, p.lanes_k, n0, nt);
    const RowWalk<kStill> vw(p, p.v, p.vt, p.vh, p.Dv, p.lanes_v, n0, nt);
    RowPart cur, next;
    kw.load(p, 0, cur);
    if (threadIdx.x < nt) {
        const int n = n0 + threadIdx.x;
        int b = -1, pos = -1, page = -1, off = 0;
        if (!p.cu) {
            b = n / p.S;
            const int len = __ldg(p.kv_len + b);
            pos = len > 0 ? len - p.S + (n - b * p.S) : -1;
        } else {
            // the last b with cu[b] <= n: the sequence that holds row n
            int lo = 0, hi = p.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.cu + mid) <= n)
                    lo = mid;
                else
                    hi = mid;
            }
            b = lo;
            const int len = __ldg(p.kv_len + b);
            pos = len > 0 ? len - __ldg(p.cu + b + 1) + n : -1;
        }
        if (pos < 0 || !p.pm.locate(p.pm.table + b * p.pm.table_stride, pos, page, off))
            page = -1;
        s_page[threadIdx.x] = page;
        s_off[threadIdx.x] = off;
        s_pos[threadIdx.x] = p.positions ? __ldg(p.positions + n) : pos;
    }
    __syncthreads();
    if constexpr (kHow != kStill) {
        for (int i = threadIdx.x; i < nt * p.half; i += kRowThreads) {
            const int t = static_cast<int>(p.div_half.div(i)), f = i - t * p.half;
            turns[t * turn_at(p.half) + turn_at(f)] = make_turn(s_pos[t], __ldg(p.inv_freq + f), p.rope_scale);
        }
        __syncthreads();
    }
    for (int i = 0; i < kw.rounds; ++i) {
        if (i + 1 < kw.rounds)
            kw.load(p, i + 1, next);
        else if (p.v)
            vw.load(p, 0, next);
        kw.template work<kType>(p, p.ck, cur, s_page, s_off, turns);
        cur = next;
    }
    if (!p.v)
        return;
    for (int i = 0; i < vw.rounds; ++i) {
        if (i + 1 < vw.rounds)
            vw.load(p, i + 1, next);
        vw.template work<kType>(p, p.cv, cur, s_page, s_off, turns);
        cur = next;
    }
}

// ---------------------------------------------------------------- read back

struct ReadParams {
    CacheView c;
    PageMap pm;
    const int32_t *kv_len;
    int B, T, H, D;
    int lanes;
    int rows;                            // T * H, of one sequence
    FastDiv div_H;
    __nv_bfloat16 *out;                  // [B, T, H, D]
};

// 16 stored elements: the codes, and the scale they share.
template <int kType>
struct Held16 {
    uint4 a, b;                          // kType 1: a; 2: a.x, a.y
    float s;
    uint32_t s8;

    __device__ __forceinline__ void load(const uint8_t *data, const uint8_t *scale, int lane)
    {
        if constexpr (kType == 0) {
            load32(data + 32 * lane, a, b);
        } else if constexpr (kType == 1) {
            a = __ldg(reinterpret_cast<const uint4 *>(data) + lane);
            s = __ldg(reinterpret_cast<const float *>(scale));
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(data) + lane);
            a.x = w.x;
            a.y = w.y;
            s8 = __ldg(scale + lane);
        }
    }

    __device__ __forceinline__ void store(uint8_t *dst, float tensor_scale) const
    {
        uint4 w[2];
        uint32_t *u = reinterpret_cast<uint32_t *>(w);
        if constexpr (kType == 0) {
            w[0] = a;
            w[1] = b;
        } else if constexpr (kType == 1) {
            const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 lo = float2_of_f16x2(f16x2_of_e4m3x2(q[j] & 0xFFFFu));
                const float2 hi = float2_of_f16x2(f16x2_of_e4m3x2(q[j] >> 16));
                u[2 * j] = bf16x2_of(lo.x * s, lo.y * s);
                u[2 * j + 1] = bf16x2_of(hi.x * s, hi.y * s);
            }
        } else {
            const float f = float2_of_f16x2(f16x2_of_e4m3x2(s8)).x * tensor_scale;
            const uint32_t q[2] = {a.x, a.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 f0 = float2_of_f16x2(f16x2_of_e2m1x2<0>(q[j]));
                const float2 f1 = float2_of_f16x2(f16x2_of_e2m1x2<1>(q[j]));
                const float2 f2 = float2_of_f16x2(f16x2_of_e2m1x2<2>(q[j]));
                const float2 f3 = float2_of_f16x2(f16x2_of_e2m1x2<3>(q[j]));
                u[4 * j] = bf16x2_of(f0.x * f, f0.y * f);
                u[4 * j + 1] = bf16x2_of(f1.x * f, f1.y * f);
                u[4 * j + 2] = bf16x2_of(f2.x * f, f2.y * f);
                u[4 * j + 3] = bf16x2_of(f3.x * f, f3.y * f);
            }
        }
        store32(dst, w[0], w[1]);
    }
};

// Rows of sequences blockIdx.y, + gridDim.y, ..: a group of lanes takes kReadAhead
// rows at a time (all their loads are on the way before the first is used), a lane
// writes 16 elements of each.
template <int kType>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const ReadParams p)
{
    const int lane = threadIdx.x & (p.lanes - 1);
    const int per = kRowThreads / p.lanes;
    if (16 * lane >= p.D)
        return;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int len = __ldg(p.kv_len + b);
        const int32_t *table = p.pm.table + b * p.pm.table_stride;
        uint8_t *out = reinterpret_cast<uint8_t *>(p.out + static_cast<long long>(b) * p.rows * p.D);
        const unsigned stride = gridDim.x * per * kReadAhead;
        int t[kReadAhead], page[kReadAhead];             // of the rows worked on next
        auto find = [&](unsigned r0) {
#pragma unroll
            for (int k = 0; k < kReadAhead; ++k) {
                const unsigned r = r0 + k * per;
                t[k] = static_cast<int>(p.div_H.div(min(r, static_cast<unsigned>(p.rows - 1))));
                const int n = static_cast<int>(p.pm.div.div(t[k]));
                page[k] = r < p.rows && t[k] < len && n < p.pm.max_pages ? __ldg(table + n) : -1;
            }
        };
        unsigned r0 = blockIdx.x * per * kReadAhead + threadIdx.x / p.lanes;
        find(r0);
        for (; r0 < p.rows; r0 += stride) {
            Held16<kType> x[kReadAhead];
            bool has[kReadAhead];
#pragma unroll
            for (int k = 0; k < kReadAhead; ++k) {
                has[k] = page[k] >= 0 && page[k] < p.pm.num_pages;
                const int h = static_cast<int>(r0 + k * per) - t[k] * p.H;
                const int off = t[k] - static_cast<int>(p.pm.div.div(t[k])) * p.pm.page_size;
                if (has[k])
                    x[k].load(row_data(p.c, p.pm, page[k], h, off), row_scale(p.c, p.pm, page[k], h, off), lane);
            }
            find(r0 + stride);                           // (the next rows' pages come meanwhile)
#pragma unroll
            for (int k = 0; k < kReadAhead; ++k) {
                const unsigned r = r0 + k * per;
                if (r >= p.rows)
                    break;
                uint8_t *dst = out + (static_cast<long long>(r) * p.D + 16 * lane) * 2;
                if (has[k])
                    x[k].store(dst, p.c.tensor_scale);
                else
                    store32(dst, make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u));
            }
        }
    }
}

} // namespace cache
} // namespace csa
