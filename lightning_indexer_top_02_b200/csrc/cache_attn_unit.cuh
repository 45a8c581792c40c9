// cache_attn_unit.cuh -- what the translation units that hold the attention
// kernels (one for each key width: cache_attn_unit.cu) give the host code.  One
// unit for all of them takes minutes to compile.
#pragma once
#include <atomic>

#include "cache_attn_kernel.cuh"
#include "cache_attn_wide_kernel.cuh"

namespace csa {
namespace cattn {

using CattnFn = void (*)(const AttnParams);
using CattnWideFn = void (*)(const WideParams);

// How a call runs: the shape of its tiles (set before pick_*), the kernel that
// takes them and what that needs (pick_*), the shares (after it).
struct CattnPlan {
    bool wide;
    bool bulk;              // tiles of 16 keys lie together in a page (the register kernel)
    int keys, raw;          // of the wide kernel: keys of a tile, staging bytes
    int tile_rows, tiles, rows, splits;
    long long works, piece_rows;
    size_t workspace;
    int chunk;              // keys that are shared out together
    int most;               // of the register kernel: chunks of a row tile, at most
    int ctas;               // of the register kernel: those that share the chunks, 0: one a row tile
    CattnFn fn;
    CattnWideFn wide_fn;
    int smem;
    std::atomic<unsigned long long> *ready;  // devices that the kernel has been set up on, one bit each
};

// Fill in the kernel for keys of 64 .. 256 elements and values of dv; false: there is none.
bool pick_64(int dv, CattnPlan *pl);
bool pick_128(int dv, CattnPlan *pl);
bool pick_192(int dv, CattnPlan *pl);
bool pick_256(int dv, CattnPlan *pl);
// The unit's device error word (ptx.cuh; h is left as it was while no call has used the unit), cleared
// when it holds an error; false: a CUDA call failed.
bool error_64(int (&h)[4]);
bool error_128(int (&h)[4]);
bool error_192(int (&h)[4]);
bool error_256(int (&h)[4]);

} // namespace cattn
} // namespace csa
