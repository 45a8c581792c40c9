// rotary_kernel.cuh -- rotary positions on part of every head
// (csa_rotary, include/csa_cache.h):
//   (a, b) -> (a c - b s, b c + a s),  c + i s = scale * e^(i pos f_i).
//
// Bound by memory: 2 * sizeof(element) bytes an element against about three
// flops.  One block takes a few tokens (and a share of their heads when there
// are few tokens); its threads compute the tokens' cos and sin once, in
// shared memory, and use them for every head, so the angles cost rot_dim / 2
// sincospi a token and no table is read from memory.  What it took to reach memory's
// rate was instructions: packed conversions, one shape for rotated and copied pieces
// (a warp's accesses do not diverge) and kAhead units loaded before the angles are
// waited for.  8,192 tokens x 64 heads of 128 bf16 (64 rotated, interleaved): 45 us,
// 5.9 TB/s; 4,099 x 16 x 192 fp32: 18.4 us, 5.5 TB/s (inputs that do not stand in L2).
#pragma once
#include "cache_common.cuh"

namespace csa {
namespace rotary {

constexpr int kThreads = 128;
constexpr int kAhead = 4;       // units a thread loads before it works on the first

struct RotaryParams {
    const void *x;
    void *out;
    int N, H, D;
    long long xt, xh, ot, oh;   // strides in elements
    const int32_t *positions;
    const float *inv_freq;
    int half;                   // rot_dim / 2
    int off;
    int inverse;
    float scale;
    int tokens;                 // tokens a block takes
    int heads;                  // heads a block takes (a share of H)
    int copy;                   // out != x: the other elements are copied
    int units;                  // work units of a head
    int pair_units;             // of them, those that rotate (all interleaved units of V > 1 stand in order)
    cache::FastDiv div_units, div_heads, div_half;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// V elements, reached two at a time (16-bit types: a packed word).
template <typename T, int V> struct __align__(V * sizeof(T)) Vec {
    T v[V];
    __device__ __forceinline__ float2 pair(int j) const { return make_float2(to_f(v[2 * j]), to_f(v[2 * j + 1])); }
    __device__ __forceinline__ void set(int j, float2 f)
    {
        v[2 * j] = from_f<T>(f.x);
        v[2 * j + 1] = from_f<T>(f.y);
    }
};
template <> struct __align__(16) Vec<__nv_bfloat16, 8> {
    uint32_t w[4];
    __device__ __forceinline__ float2 pair(int j) const { return cache::float2_of_bf16x2(w[j]); }
    __device__ __forceinline__ void set(int j, float2 f) { w[j] = cache::bf16x2_of(f.x, f.y); }
};
template <> struct __align__(16) Vec<__half, 8> {
    uint32_t w[4];
    __device__ __forceinline__ float2 pair(int j) const { return cache::float2_of_f16x2(w[j]); }
    __device__ __forceinline__ void set(int j, float2 f)
    {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
};

// The elements that unit u of a head covers: V from `first` on and (half layout, or
// V = 1) V from `second` on, -1: none.  Every unit has the same shape, rotated or
// copied, so that a warp's loads and stores do not diverge.
struct Unit {
    int first, second, pair;     // pair: the first pair's index, -1: copied
};

template <int V, bool kInter>
__device__ __forceinline__ Unit unit_at(const RotaryParams &p, int u)
{
    Unit r;
    if constexpr (kInter && V >= 2) {
        r.first = u * V + (p.copy ? 0 : p.off);
        r.second = -1;
        const int in = r.first - p.off;
        r.pair = in >= 0 && in < 2 * p.half ? in / 2 : -1;
        return r;
    }
    if (u < p.pair_units) {
        r.first = p.off + u * (kInter ? 2 : V);
        r.second = r.first + (kInter ? 1 : p.half);
        r.pair = u * V;
    } else {                     // two pieces of the rest, around the rotated part
        const int c = u - p.pair_units, n = p.units - p.pair_units;
        r.first = c * V;
        r.second = (c + n) * V;
        r.second = r.second < p.D - 2 * p.half ? r.second : -1;
        r.first += r.first >= p.off ? 2 * p.half : 0;
        r.second += r.second >= p.off ? 2 * p.half : 0;
        r.pair = -1;
    }
    return r;
}

// V elements at a time (V = 1: any alignment).  Half layout: a unit is V elements
// of the first half and their V partners; interleaved: V consecutive elements, V / 2
// pairs (V = 1: one pair, two elements).
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p)
{
    extern __shared__ float2 cs[];                       // [tokens][half]
    using Vt = Vec<T, V>;
    constexpr bool kOne = kInter && V >= 2;              // a unit is one piece
    const int n0 = blockIdx.x * p.tokens;
    const int nt = min(p.tokens, p.N - n0);
    const int h0 = blockIdx.y * p.heads;
    const int nh = min(p.heads, p.H - h0);
    const T *x0 = static_cast<const T *>(p.x);
    T *o0 = static_cast<T *>(p.out);
    const int rows = nt * nh;
    // the thread's place: unit, and row (token and head) of its head; the next one is
    // kThreads units on
    int row = static_cast<int>(p.div_units.div(threadIdx.x)), u = threadIdx.x - row * p.units;
    const int row_step = static_cast<int>(p.div_units.div(kThreads)), u_step = kThreads - row_step * p.units;
    bool ready = false;                                  // cos and sin are there
    while (!ready || row < rows) {
        // kAhead units' loads are on the way before the first is used
        Vt a[kAhead], b[kAhead];
        int tok[kAhead], head[kAhead];
        Unit unit[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            unit[k] = unit_at<V, kInter>(p, u);
            tok[k] = nh == p.heads ? static_cast<int>(p.div_heads.div(row)) : row / nh;
            head[k] = h0 + row - tok[k] * nh;
            const bool in = row < rows;
            row += row_step;
            u += u_step;
            if (u >= p.units) {
                u -= p.units;
                ++row;
            }
            if (!in) {
                head[k] = -1;
                continue;
            }
            const T *x = x0 + (n0 + tok[k]) * p.xt + head[k] * p.xh;
            a[k] = *reinterpret_cast<const Vt *>(x + unit[k].first);
            if (!kOne && unit[k].second >= 0)
                b[k] = *reinterpret_cast<const Vt *>(x + unit[k].second);
        }
        if (!ready) {
            for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
                const int t = static_cast<int>(p.div_half.div(i)), f = i - t * p.half;
                // the angle's fp32 value, and (to first order) what its rounding leaves out, in radians:
                // that is up to 9.4e-8, more than sincospif's own error
                const double h = cache::half_turns(__ldg(p.positions + n0 + t), __ldg(p.inv_freq + f));
                const float near = static_cast<float>(h), rest = static_cast<float>(h - near) * 3.14159265f;
                float s, c;
                sincospif(near, &s, &c);
                const float s1 = fmaf(c, rest, s), c1 = fmaf(-s, rest, c);
                cs[i] = make_float2(c1 * p.scale, (p.inverse ? -s1 : s1) * p.scale);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (head[k] < 0)
                continue;
            T *o = o0 + (n0 + tok[k]) * p.ot + head[k] * p.oh;
            if (unit[k].pair >= 0) {
                const float2 *w = cs + tok[k] * p.half + unit[k].pair;
                if constexpr (kOne) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        const float2 q = w[j], f = a[k].pair(j);
                        a[k].set(j, make_float2(f.x * q.x - f.y * q.y, f.y * q.x + f.x * q.y));
                    }
                } else if constexpr (V >= 2) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        const float2 q = w[2 * j], r = w[2 * j + 1], f = a[k].pair(j), g = b[k].pair(j);
                        a[k].set(j, make_float2(f.x * q.x - g.x * q.y, f.y * r.x - g.y * r.y));
                        b[k].set(j, make_float2(g.x * q.x + f.x * q.y, g.y * r.x + f.y * r.y));
                    }
                } else {
                    const float2 q = w[0];
                    const float fa = to_f(a[k].v[0]), fb = to_f(b[k].v[0]);
                    a[k].v[0] = from_f<T>(fa * q.x - fb * q.y);
                    b[k].v[0] = from_f<T>(fb * q.x + fa * q.y);
                }
            }
            *reinterpret_cast<Vt *>(o + unit[k].first) = a[k];
            if (!kOne && unit[k].second >= 0)
                *reinterpret_cast<Vt *>(o + unit[k].second) = b[k];
        }
    }
}

} // namespace rotary
} // namespace csa
