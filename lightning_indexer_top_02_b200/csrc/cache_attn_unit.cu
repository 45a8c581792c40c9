// cache_attn_unit.cu -- the attention kernels for keys of CSA_UNIT_DK elements;
// compiled once for each width.
#include <cuda_runtime.h>

#include "cache_attn_unit.cuh"

#define CSA_CAT_(a, b) a##b
#define CSA_CAT(a, b) CSA_CAT_(a, b)

namespace csa {
namespace cattn {

namespace {

std::atomic<bool> g_asked;                  // a call has asked for a kernel of this unit

template <int kDk, int kDv>
void cattn_pick(CattnPlan *pl)
{
    static std::atomic<unsigned long long> ready[6];
    pl->ready = &ready[pl->wide ? 4 + (pl->tile_rows == kWideRows) : 2 * (pl->tile_rows > 8) + pl->bulk];
    if (pl->wide) {
        pl->keys = WideShape<kDk, kDv>::kKeys;
        pl->raw = 2 * kGatherWarps * WideShape<kDk, kDv>::kRaw;
        pl->wide_fn = pl->tile_rows == kWideRows ? cache_attn_wide_kernel<kDk, kDv, false>
                                                 : cache_attn_wide_kernel<kDk, kDv, true>;
    } else if (pl->tile_rows == 8) {
        pl->fn = pl->bulk ? cache_attn_kernel<kDk, kDv, 1, true> : cache_attn_kernel<kDk, kDv, 1, false>;
        pl->smem = Shape<kDk, kDv, 1>::kSmem;
        pl->ctas = Shape<kDk, kDv, 1>::kCtas;
        pl->chunk = Shape<kDk, kDv, 1>::kChunk;
    } else {
        pl->fn = pl->bulk ? cache_attn_kernel<kDk, kDv, 2, true> : cache_attn_kernel<kDk, kDv, 2, false>;
        pl->smem = Shape<kDk, kDv, 2>::kSmem;
        pl->ctas = Shape<kDk, kDv, 2>::kCtas;
        pl->chunk = Shape<kDk, kDv, 2>::kChunk;
    }
}

template <int kDk>
bool cattn_pick_dv(int dv, CattnPlan *pl)
{
    switch (dv) {
    case 64: cattn_pick<kDk, 64>(pl); return true;
    case 128: cattn_pick<kDk, 128>(pl); return true;
    case 192: cattn_pick<kDk, 192>(pl); return true;
    case 256: cattn_pick<kDk, 256>(pl); return true;
    }
    return false;
}

} // namespace

bool CSA_CAT(pick_, CSA_UNIT_DK)(int dv, CattnPlan *pl)
{
    if (!g_asked.load(std::memory_order_relaxed))
        g_asked.store(true, std::memory_order_relaxed);
    return cattn_pick_dv<CSA_UNIT_DK>(dv, pl);
}

bool CSA_CAT(error_, CSA_UNIT_DK)(int (&h)[4])
{
    if (!g_asked.load(std::memory_order_relaxed))
        return true;                        // (a copy costs a synchronisation: none for the indexer's callers)
    const int zero[4] = {0, 0, 0, 0};
    return cudaMemcpyFromSymbol(h, g_csa_error, sizeof h) == cudaSuccess &&
           (h[0] == 0 || cudaMemcpyToSymbol(g_csa_error, zero, sizeof zero) == cudaSuccess);
}

} // namespace cattn
} // namespace csa
