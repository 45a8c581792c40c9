// cache_attn_join_kernel.cuh -- the second kernels of attention over a 4-bit
// cache: what several CTAs found for one row tile becomes the rows' outputs.
#pragma once
#include "cache_attn_kernel.cuh"

namespace csa {
namespace cattn {

// Waits until the kernel launched before this one has ended and its results can be
// read.  Every block does, before it returns too: what follows on the stream waits
// for this kernel only.
__device__ __forceinline__ void after_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }


// Joins the pieces of the row tiles that several CTAs of the kernel above share: out =
// sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.  A block takes rows of sequence
// blockIdx.x, its warps every fourth piece of a row.
__global__ void __launch_bounds__(kThreads) cache_attn_pieces_kernel(const AttnParams p, int Dv, int tile_rows)
{
    __shared__ long long scratch[kWarps];
    __shared__ float2 part[kWarps][128 + 1];             // a warp's O, then its maximum and sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x;
    const int all = chunks_of(p, b);
    const long long total = chunks_before(p, p.B, scratch), first = chunks_before(p, b, scratch);
    after_kernel_before();
    if (all == 0)
        return;                                          // written by that kernel
    const int ctas = static_cast<int>(min(static_cast<long long>(p.ctas), total));
    for (int row = blockIdx.y; row < p.S * p.HA; row += gridDim.y) {
        const int i = row / p.HA, head = row - i * p.HA, h = head / p.G;
        const int r = p.idx ? head - h * p.G : i * p.G + head - h * p.G;
        const int w = ((p.idx ? i * p.H : 0) + h) * p.tiles + r / tile_rows;
        const long long start = first + static_cast<long long>(w) * all;
        const int k0 = cta_of(start, total, ctas), k1 = cta_of(start + all - 1, total, ctas);
        if (k0 == k1)
            continue;                                    // one CTA had the whole tile
        if (k0 < 0 || k1 >= p.ctas)
            continue;                                    // (lengths that changed meanwhile: no such pieces)
        // the first CTA's piece begins the tile (its second slot), the others' end or fill it
        auto piece = [&](int k) { return (2ll * k + (k == k0 ? 1 : 0)) * tile_rows + r % tile_rows; };
        float top = -INFINITY;
        for (int k = k0 + threadIdx.x; k <= k1; k += kThreads)
            top = fmaxf(top, p.stat[piece(k)].x);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        __syncthreads();                                 // (the row before has been read)
        if (lane == 0)
            part[warp][128].x = top;
        __syncthreads();
        top = fmaxf(fmaxf(part[0][128].x, part[1][128].x), fmaxf(part[2][128].x, part[3][128].x));
        const float base = top == -INFINITY ? 0.0f : top;
        float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll 4
        for (int k = k0 + warp; k <= k1; k += kWarps) {
            const float *src = p.part + piece(k) * Dv;
            const float2 st = p.stat[piece(k)];
            const float a = ex2_approx(st.x - base);
            sum += a * st.y;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (64 * j < Dv) {
                    const float2 v = *reinterpret_cast<const float2 *>(src + 64 * j + 2 * lane);
                    x[2 * j] += a * v.x;
                    x[2 * j + 1] += a * v.y;
                }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (64 * j < Dv)
                part[warp][32 * j + lane] = make_float2(x[2 * j], x[2 * j + 1]);
        if (lane == 0)
            part[warp][128].y = sum;
        __syncthreads();
        sum = part[0][128].y + part[1][128].y + part[2][128].y + part[3][128].y;
        const float inv = sum > 0.0f ? p.v_scale / sum : 0.0f;
        const long long out_row = static_cast<long long>(b) * p.S * p.HA + row;
        for (int d = threadIdx.x; d < Dv / 2; d += kThreads) {
            const float u = part[0][d].x + part[1][d].x + part[2][d].x + part[3][d].x;
            const float v = part[0][d].y + part[1][d].y + part[2][d].y + part[3][d].y;
            *reinterpret_cast<uint32_t *>(p.out + out_row * Dv + 2 * d) = cache::bf16x2_of(u * inv, v * inv);
        }
        if (p.lse && threadIdx.x == 0)
            p.lse[out_row] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
}

// Joins the wide kernel's shares of one row, one warp a row.
__global__ void __launch_bounds__(128) cache_attn_join_kernel(const AttnParams p, int Dv, int tile_rows,
                                                              long long rows)
{
    after_kernel_before();
    const int lane = threadIdx.x & 31;
    const long long at = blockIdx.x * 4ll + (threadIdx.x >> 5);   // (b, i, head)
    if (at >= rows)
        return;
    const int head = static_cast<int>(at % p.HA);
    const long long bi = at / p.HA;
    const int h = head / p.G;
    const int r = p.idx ? head - h * p.G : static_cast<int>(bi % p.S) * p.G + head - h * p.G;
    const long long group = p.idx ? bi * p.H + h : bi / p.S * p.H + h;
    const long long work = group * p.tiles + r / tile_rows;
    const long long first = work * p.splits * tile_rows + r % tile_rows;
    float top = -INFINITY;
    for (int s = lane; s < p.splits; s += 32)
        top = fmaxf(top, p.stat[first + static_cast<long long>(s) * tile_rows].x);
#pragma unroll
    for (int d = 16; d; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const long long piece = first + static_cast<long long>(s) * tile_rows;
        const float2 st = p.stat[piece];
        const float a = ex2_approx(st.x - base);
        sum += a * st.y;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (64 * j < Dv) {
                const float2 v = *reinterpret_cast<const float2 *>(p.part + piece * Dv + 64 * j + 2 * lane);
                x[2 * j] += a * v.x;
                x[2 * j + 1] += a * v.y;
            }
    }
    const float inv = sum > 0.0f ? p.v_scale / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (64 * j < Dv)
            *reinterpret_cast<uint32_t *>(p.out + at * Dv + 64 * j + 2 * lane) =
                cache::bf16x2_of(x[2 * j] * inv, x[2 * j + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[at] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

} // namespace cattn
} // namespace csa
