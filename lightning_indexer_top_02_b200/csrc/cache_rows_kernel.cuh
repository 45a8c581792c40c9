// cache_rows_kernel.cuh -- rows into and out of a paged cache
// (csa_cache_append, csa_cache_read, include/csa_cache.h).
//
// Both are bound by memory.  A row (one position of one head) is worked by
// lanes of 16 elements each -- one E2M1 scale group, 32 bytes of bf16 -- in a
// group of 2^n lanes, which exchange only the row maximum that the E4M3 scale needs.
#pragma once
#include "cache_common.cuh"

namespace csa {
namespace cache {

constexpr int kRowThreads = 128;
constexpr int kMaxTile = 32;             // tokens a block takes at most

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
};

// cos and sin of one pair, in 40 bits: the high part has 16 bits, so its
// product with a bf16 element is exact in fp32.
struct Turn {
    float ch, cl, sh, sl;
};

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

// 16 consecutive bf16 elements as floats.
__device__ __forceinline__ void load16(const __nv_bfloat16 *src, float (&x)[16])
{
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src));
    const uint4 b = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 f = float2_of_bf16x2(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}

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
            uint4 *dst = reinterpret_cast<uint4 *>(data + 32 * lane);
            dst[0] = w[0];
            dst[1] = w[1];
        }
    } else if constexpr (kType == 1) {
        if (!active)
            peak = 0.0f;
        for (int m = 1; m < lanes; m <<= 1)
            peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, m));
        const float s = peak > 0.0f ? __fdiv_rn(peak, 448.0f) : 1.0f;
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

// Rotates the 16 elements [e0, e0 + 16) of a head row; src is the row.
template <bool kInter>
__device__ __forceinline__ void rotate16(const __nv_bfloat16 *src, int e0, int off, int half,
                                         const Turn *w, float (&x)[16])
{
    if (e0 + 16 <= off || e0 >= off + 2 * half)
        return;
    if constexpr (kInter) {
        // off is even: a pair lies within the lane's elements
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const int i = (e0 + j - off) >> 1;
            if (i >= 0 && i < half) {
                const Turn t = w[i];
                const float a = x[j], b = x[j + 1];
                x[j] = turned(a, t.ch, t.cl, b, -t.sh, -t.sl);
                x[j + 1] = turned(b, t.ch, t.cl, a, t.sh, t.sl);
            }
        }
    } else if (((off | half) & 15) == 0) {
        // the partners are another lane's 16 elements, read again (they are in L1)
        const bool first = e0 < off + half;
        float y[16];
        load16(src + (first ? e0 + half : e0 - half), y);
        const Turn *u = w + (first ? e0 - off : e0 - off - half);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const Turn t = u[j];
            x[j] = first ? turned(x[j], t.ch, t.cl, y[j], -t.sh, -t.sl)
                         : turned(x[j], t.ch, t.cl, y[j], t.sh, t.sl);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int i = e0 + j - off;
            if (i >= 0 && i < 2 * half) {
                const bool first = i < half;
                const Turn t = w[first ? i : i - half];
                const float b = __bfloat162float(src[first ? e0 + j + half : e0 + j - half]);
                x[j] = first ? turned(x[j], t.ch, t.cl, b, -t.sh, -t.sl)
                             : turned(x[j], t.ch, t.cl, b, t.sh, t.sl);
            }
        }
    }
}

template <int kType, bool kInter, bool kRotate>
__device__ __forceinline__ void append_rows(const __nv_bfloat16 *src, long long ts, long long hs, int D,
                                            int lanes, const CacheView &c, const PageMap &pm, int H,
                                            int n0, int nt, const int *page, const int *off,
                                            const Turn *turns, int rope_off, int half)
{
    const int lane = threadIdx.x & (lanes - 1);
    const int rows = nt * H;
    const int step = kRowThreads / lanes;
    const bool has = 16 * lane < D;
    // every lane of a warp takes the same number of turns (store16 exchanges)
    for (int r0 = 0; r0 < rows; r0 += step) {
        const int r = r0 + threadIdx.x / lanes;
        const int t = r < rows ? r / H : 0, h = r < rows ? r - t * H : 0;
        const bool active = r < rows && has && page[t] >= 0;
        float x[16];
        uint8_t *data = nullptr, *scale = nullptr;
        if (active) {
            const __nv_bfloat16 *row = src + (n0 + t) * ts + h * hs;
            load16(row + 16 * lane, x);
            if (kRotate)
                rotate16<kInter>(row, 16 * lane, rope_off, half, turns + t * half, x);
            data = const_cast<uint8_t *>(row_data(c, pm, page[t], h, off[t]));
            if (kType != 0)
                scale = const_cast<uint8_t *>(row_scale(c, pm, page[t], h, off[t]));
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[j] = 0.0f;
        }
        store16<kType>(c, data, scale, lane, lanes, active, x);
    }
}

// One block takes p.tokens tokens: their places (one thread a token), their
// cos and sin, then every row of K and of V.
template <int kType, bool kInter>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const AppendParams p)
{
    extern __shared__ Turn turns[];                     // [tokens][half]
    __shared__ int s_page[kMaxTile], s_off[kMaxTile], s_pos[kMaxTile];
    const int n0 = blockIdx.x * p.tokens;
    const int nt = min(p.tokens, p.N - n0);
    if (threadIdx.x < nt) {
        const int n = n0 + threadIdx.x;
        int b = -1, pos = -1, page = -1, off = 0;
        if (!p.cu) {
            b = n / p.S;
            const int len = __ldg(p.kv_len + b);
            pos = len > 0 ? len - p.S + (n - b * p.S) : -1;
        } else if (n < __ldg(p.cu + p.B)) {
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
    for (int i = threadIdx.x; i < nt * p.half; i += kRowThreads) {
        const int t = i / p.half;
        turns[i] = make_turn(s_pos[t], __ldg(p.inv_freq + i - t * p.half), p.rope_scale);
    }
    __syncthreads();
    if (p.half)
        append_rows<kType, kInter, true>(p.k, p.kt, p.kh, p.Dk, p.lanes_k, p.ck, p.pm, p.H, n0, nt,
                                         s_page, s_off, turns, p.off, p.half);
    else
        append_rows<kType, kInter, false>(p.k, p.kt, p.kh, p.Dk, p.lanes_k, p.ck, p.pm, p.H, n0, nt,
                                          s_page, s_off, turns, 0, 0);
    if (p.v)
        append_rows<kType, kInter, false>(p.v, p.vt, p.vh, p.Dv, p.lanes_v, p.cv, p.pm, p.H, n0, nt,
                                          s_page, s_off, turns, 0, 0);
}

// ---------------------------------------------------------------- read back

struct ReadParams {
    CacheView c;
    PageMap pm;
    const int32_t *kv_len;
    int B, T, H, D;
    int lanes;
    long long rows;                      // B * T * H
    __nv_bfloat16 *out;                  // [B, T, H, D]
};

// A group of lanes takes a row at a time; a lane writes 16 elements.
template <int kType>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const ReadParams p)
{
    const int lane = threadIdx.x & (p.lanes - 1);
    const int per = kRowThreads / p.lanes;
    if (16 * lane >= p.D)
        return;
    for (long long r = static_cast<long long>(blockIdx.x) * per + threadIdx.x / p.lanes; r < p.rows;
         r += static_cast<long long>(gridDim.x) * per) {
        const long long bt = r / p.H;
        const int h = static_cast<int>(r - bt * p.H);
        const int b = static_cast<int>(bt / p.T), t = static_cast<int>(bt - static_cast<long long>(b) * p.T);
        int page, off;
        uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (t < __ldg(p.kv_len + b) && p.pm.locate(p.pm.table + b * p.pm.table_stride, t, page, off)) {
            const uint8_t *data = row_data(p.c, p.pm, page, h, off);
            uint32_t *u = reinterpret_cast<uint32_t *>(w);
            if constexpr (kType == 0) {
                const uint4 *src = reinterpret_cast<const uint4 *>(data + 32 * lane);
                w[0] = src[0];
                w[1] = src[1];
            } else if constexpr (kType == 1) {
                const uint4 q = *reinterpret_cast<const uint4 *>(data + 16 * lane);
                const float s = *reinterpret_cast<const float *>(row_scale(p.c, p.pm, page, h, off));
                const uint32_t q4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 lo = float2_of_f16x2(f16x2_of_e4m3x2(q4[j] & 0xFFFFu));
                    const float2 hi = float2_of_f16x2(f16x2_of_e4m3x2(q4[j] >> 16));
                    u[2 * j] = bf16x2_of(lo.x * s, lo.y * s);
                    u[2 * j + 1] = bf16x2_of(hi.x * s, hi.y * s);
                }
            } else {
                const uint2 q = *reinterpret_cast<const uint2 *>(data + 8 * lane);
                const float s = float2_of_f16x2(f16x2_of_e4m3x2(
                                    row_scale(p.c, p.pm, page, h, off)[lane])).x * p.c.tensor_scale;
                const uint32_t q2[2] = {q.x, q.y};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 f0 = float2_of_f16x2(f16x2_of_e2m1x2<0>(q2[j]));
                    const float2 f1 = float2_of_f16x2(f16x2_of_e2m1x2<1>(q2[j]));
                    const float2 f2 = float2_of_f16x2(f16x2_of_e2m1x2<2>(q2[j]));
                    const float2 f3 = float2_of_f16x2(f16x2_of_e2m1x2<3>(q2[j]));
                    u[4 * j] = bf16x2_of(f0.x * s, f0.y * s);
                    u[4 * j + 1] = bf16x2_of(f1.x * s, f1.y * s);
                    u[4 * j + 2] = bf16x2_of(f2.x * s, f2.y * s);
                    u[4 * j + 3] = bf16x2_of(f3.x * s, f3.y * s);
                }
            }
        }
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + r * p.D + 16 * lane);
        dst[0] = w[0];
        dst[1] = w[1];
    }
}

} // namespace cache
} // namespace csa
