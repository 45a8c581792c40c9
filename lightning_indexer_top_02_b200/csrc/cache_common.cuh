// cache_common.cuh -- what the cache kernels share: the page lookup and the
// rounding to and from the cache's types (layouts: include/csa_cache.h).
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace csa {
namespace cache {

// n / d for 0 <= n < 2^31 by one multiplication (d >= 1 fixed on the host), after Granlund and
// Montgomery, "Division by invariant integers using multiplication" (1994): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, the quotient is
// (mulhi(m, n) + n) >> l.
struct FastDiv {
    uint32_t d, m, l;
    static FastDiv of(uint32_t d)
    {
        FastDiv f;
        f.d = d;
        f.l = 0;
        while ((1ull << f.l) < d)
            ++f.l;
        f.m = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.l) - d)) / d + 1);
        return f;
    }
    __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const
    {
#if defined(__CUDA_ARCH__)
        return (__umulhi(m, n) + n) >> l;
#else
        return static_cast<uint32_t>(((static_cast<uint64_t>(m) * n >> 32) + n) >> l);
#endif
    }
};

// One cache as the kernels see it.  Row o of head h in page p starts at
// data + p * page_stride + (h * page_size + o) * row_bytes.
struct CacheView {
    uint8_t *data, *scale;
    long long page_stride, scale_stride;
    int row_bytes, scale_bytes;
    float tensor_scale;
};

// Where the positions of the sequences lie.
struct PageMap {
    const int32_t *table;
    long long table_stride;
    int max_pages, num_pages, page_size;
    FastDiv div;

    // Page and row of position pos >= 0 of the sequence with table row `row`;
    // false where there is none.
    __device__ __forceinline__ bool locate(const int32_t *row, int pos, int &page, int &off) const
    {
        const int n = static_cast<int>(div.div(static_cast<uint32_t>(pos)));
        off = pos - n * page_size;
        if (n >= max_pages)
            return false;
        page = __ldg(row + n);
        return page >= 0 && page < num_pages;
    }
};

__device__ __forceinline__ const uint8_t *row_data(const CacheView &c, const PageMap &pm, int page,
                                                   int head, int off)
{
    return c.data + page * c.page_stride +
           (static_cast<long long>(head) * pm.page_size + off) * c.row_bytes;
}

__device__ __forceinline__ const uint8_t *row_scale(const CacheView &c, const PageMap &pm, int page,
                                                    int head, int off)
{
    return c.scale + page * c.scale_stride +
           (static_cast<long long>(head) * pm.page_size + off) * c.scale_bytes;
}

// Four pairs of floats as E2M1 codes, the first of a pair in a byte's low half
// (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e2m1x8(const float *x)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Two floats as E4M3 bytes, lo in the low one (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

// Two E4M3 bytes as f16 (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}

// The two E2M1 codes of byte `which` of w as f16 (exact), the low half's code first.
template <int which>
__device__ __forceinline__ uint32_t f16x2_of_e2m1x2(uint32_t w)
{
    uint32_t r;
    if constexpr (which == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
            : "=r"(r) : "r"(w));
    else if constexpr (which == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
            : "=r"(r) : "r"(w));
    else if constexpr (which == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
            : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}"
            : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float2 float2_of_f16x2(uint32_t h)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ float2 float2_of_bf16x2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// 32 bytes a lane at once where they stand on 32 bytes (a whole sector: two stores of
// 16 at a stride of 32 each write half of every sector they touch).
__device__ __forceinline__ void store32(uint8_t *dst, const uint4 &a, const uint4 &b)
{
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                     "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = a;
        reinterpret_cast<uint4 *>(dst)[1] = b;
    }
}

__device__ __forceinline__ void load32(const void *src, uint4 &a, uint4 &b)
{
    if ((reinterpret_cast<uintptr_t>(src) & 31) == 0) {
        asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
            : "l"(src));
    } else {
        a = __ldg(static_cast<const uint4 *>(src));
        b = __ldg(static_cast<const uint4 *>(src) + 1);
    }
}

// The angle pos * freq as a fraction of half turns, about [-1, 1].  The product has 31 + 24 bits,
// two more than a double: it is kept as a rounded value and its exact remainder (fma), and the
// quotient by 2 pi likewise, with 1 / 2 pi as two doubles.  What is left out is below 2^-104 of
// the turns taken (2^-75 of a turn at the farthest position) beside the result's own rounding.
__device__ __forceinline__ double half_turns(int pos, float freq)
{
    constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;   // 1 / 2 pi
    const double p = pos, f = freq;
    const double hi = p * f, lo = fma(p, f, -hi);
    const double t = hi * kInv;
    const double rest = fma(hi, kInv, -t) + fma(hi, kInvLow, lo * kInv);
    return 2.0 * ((t - rint(t)) + rest);
}

} // namespace cache
} // namespace csa
