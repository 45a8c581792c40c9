// rotary_kernel.cuh -- rotary positions on part of every head
// (csa_rotary, include/csa_cache.h):
//   (a, b) -> (a c - b s, b c + a s),  c + i s = scale * e^(i pos f_i).
//
// Bound by memory: 2 * sizeof(element) bytes an element against about three
// flops.  One block takes kTokens tokens (and a share of their heads when there
// are few tokens); its threads compute the tokens' cos and sin once, in
// shared memory, and use them for every head, so the angles cost rot_dim / 2
// sincospi a token and no table is read from memory.
#pragma once
#include "cache_common.cuh"

namespace csa {
namespace rotary {

constexpr int kThreads = 256;

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
    int units;                  // work units a head: pair units, then copy units
    int pair_units;
    cache::FastDiv div_units, div_heads;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V> struct __align__(V * sizeof(T)) Vec { T v[V]; };

// V elements at a time (V = 1: any alignment).  Half layout: a pair unit is
// V elements of the first half and their V partners; interleaved: V
// consecutive elements, V / 2 pairs (V = 1: one pair, two elements).
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p)
{
    extern __shared__ float2 cs[];                       // [tokens][half]
    using Vt = Vec<T, V>;
    constexpr int kPair = V / 2 > 0 ? V / 2 : 1;          // interleaved: pairs of a unit
    const int n0 = blockIdx.x * p.tokens;
    const int nt = min(p.tokens, p.N - n0);
    const int h0 = blockIdx.y * p.heads;
    const int nh = min(p.heads, p.H - h0);
    for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
        const int t = i / p.half, f = i - t * p.half;
        float s, c;
        sincospif(static_cast<float>(cache::half_turns(__ldg(p.positions + n0 + t), __ldg(p.inv_freq + f))),
                  &s, &c);
        cs[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
    }
    __syncthreads();
    const T *x0 = static_cast<const T *>(p.x);
    T *o0 = static_cast<T *>(p.out);
    const int total = nt * nh * p.units;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int row = static_cast<int>(p.div_units.div(i));
        const int u = i - row * p.units;
        const int t = nh == p.heads ? static_cast<int>(p.div_heads.div(row)) : row / nh;
        const int h = h0 + row - t * nh;
        const T *x = x0 + (n0 + t) * p.xt + h * p.xh;
        T *o = o0 + (n0 + t) * p.ot + h * p.oh;
        const float2 *w = cs + t * p.half;
        if (u < p.pair_units) {
            if constexpr (!kInter) {
                const int e = p.off + u * V;
                const Vt a = *reinterpret_cast<const Vt *>(x + e);
                const Vt b = *reinterpret_cast<const Vt *>(x + e + p.half);
                Vt ra, rb;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 k = w[u * V + j];
                    const float fa = to_f(a.v[j]), fb = to_f(b.v[j]);
                    ra.v[j] = from_f<T>(fa * k.x - fb * k.y);
                    rb.v[j] = from_f<T>(fb * k.x + fa * k.y);
                }
                *reinterpret_cast<Vt *>(o + e) = ra;
                *reinterpret_cast<Vt *>(o + e + p.half) = rb;
            } else if constexpr (V >= 2) {
                const int e = p.off + u * V;
                const Vt a = *reinterpret_cast<const Vt *>(x + e);
                Vt r;
#pragma unroll
                for (int j = 0; j < kPair; ++j) {
                    const float2 k = w[u * kPair + j];
                    const float fa = to_f(a.v[2 * j]), fb = to_f(a.v[2 * j + 1]);
                    r.v[2 * j] = from_f<T>(fa * k.x - fb * k.y);
                    r.v[2 * j + 1] = from_f<T>(fb * k.x + fa * k.y);
                }
                *reinterpret_cast<Vt *>(o + e) = r;
            } else {
                const int e = p.off + 2 * u;
                const float2 k = w[u];
                const float fa = to_f(x[e]), fb = to_f(x[e + 1]);
                o[e] = from_f<T>(fa * k.x - fb * k.y);
                o[e + 1] = from_f<T>(fb * k.x + fa * k.y);
            }
        } else {
            int e = (u - p.pair_units) * V;               // past the rotated part
            if (e >= p.off)
                e += 2 * p.half;
            *reinterpret_cast<Vt *>(o + e) = *reinterpret_cast<const Vt *>(x + e);
        }
    }
}

} // namespace rotary
} // namespace csa
