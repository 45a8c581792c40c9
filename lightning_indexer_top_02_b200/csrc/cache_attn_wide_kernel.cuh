// cache_attn_wide_kernel.cuh -- attention over a cache held in 4 bits, more
// than 16 query rows per cached row (csa_cache_attention, include/csa_cache.h):
// up to 128 heads that share a row, or several queries of grouped heads.
//
// 2 rows (Dk + Dv) flops for each 9/16 (Dk + Dv) bytes: from about 64 rows on
// the work is bound by the tensor cores, and by what feeds them.  Tiles of 128
// query rows (TMEM lanes) x 128 keys on tcgen05:
//   S = Q . K^T    A = Q from TMEM (written there once an item), B = K from shared memory
//   O += P . V     A = P from TMEM (over its S slot), B = V from shared memory (MN-major)
// so that shared memory's bandwidth is left to the keys and values: written
// once as f16, read once by an MMA.
//
// One persistent CTA a SM walks work items (a group's row tile x a share of
// the keys).  Warps:
//   0-3   softmax: thread = TMEM lane = query row.  Q row to f16 (scaled by a power of
//         two, see cache_attn_kernel.cuh) into TMEM; per tile the row's maximum, then
//         P over the slot's first columns; O / l at the item's end.  S is read twice
//         (maximum, then exponentials), 64 columns at a time, so that 128 registers do.
//   4-11  gather: 16 tile rows each; codes and scales to registers one tile
//         ahead (their pages two, their list entries three tiles ahead), converted and
//         stored as the 128-byte-swizzled operands; rows without a key are zeros.
//   12    MMA issue and TMEM.
// Up to 64 rows (kSplit) the rows stand in lanes 0-63 and again in lanes
// 64-127: the copy takes the tile's other 64 keys with its own maximum, sum and
// O, so that all four softmax warps work; the halves are joined at the end.
// Waits are bounded (ptx.cuh).
#pragma once
#include "cache_attn_kernel.cuh"

namespace csa {
namespace cattn {

constexpr int kWideThreads = 512;
constexpr int kWideKeys = 128;              // keys of a tile
constexpr int kWideRows = 128;              // query rows of a tile (TMEM lanes)
constexpr int kGatherWarps = 8;
constexpr int kGatherRows = kWideKeys / kGatherWarps;
constexpr int kWideMmaWarp = 4 + kGatherWarps;
constexpr int kWideStages = 3;              // at most, per ring (keys, values)
constexpr int kMaskRing = 8;                // validity words kept: stages + S slots + what is in use

enum WideRole : int { kWideGather = 31, kWideMma = 32, kWideSoftmax = 33 };

struct WideParams {
    AttnParams a;
    int items;                              // works * splits
    int k_stages, v_stages, k_bytes, v_bytes;
    int off_v, off_x, off_bar;              // shared memory: K ring, V ring, exchange, barriers
    int slots;                              // S slots in TMEM
    int col_o, col_q;                       // TMEM columns
    long long wait_limit;
};

struct WideBarriers {
    uint64_t k_full[kWideStages], k_empty[kWideStages];
    uint64_t v_full[kWideStages], v_empty[kWideStages];
    uint64_t s_full[2], s_empty[2], p_full[2];
    uint64_t q_full, pv_done, o_empty, drain;
    uint64_t xbar[2][2];                    // kSplit: per row quarter, two phases in turn
    float xchg[4][32][2];                   // kSplit: a row copy's maximum and sum
    uint16_t valid[kMaskRing][kGatherWarps];
    uint32_t tmem_addr;
    int abort;
};

// What every role needs to know of an item.
struct Item {
    Group g;
    int len;
    int t0, t1;                             // its tiles
    int slots;                              // key slots of the group
    int limit;                              // positions the tile's last row sees
};

__device__ __forceinline__ Item item_of(const AttnParams &p, int item, int tile_rows)
{
    Item it;
    const int work = item / p.splits, split = item - work * p.splits;
    it.g = group_of(p, work, tile_rows);
    it.len = __ldg(p.kv_len + it.g.b);
    const int r_last = min(it.g.r0 + tile_rows, p.rows) - 1;
    it.limit = it.len > 0 ? seen(p, it.len, it.g.i0 + r_last / p.G) : 0;
    it.slots = p.idx ? (it.limit > 0 ? p.topk : 0) : min(max(it.limit, 0), p.capacity);
    const long long tiles = (static_cast<long long>(it.slots) + kWideKeys - 1) / kWideKeys;
    it.t0 = static_cast<int>(tiles * split / p.splits);
    it.t1 = static_cast<int>(tiles * (split + 1) / p.splits);
    return it;
}

// ---------------------------------------------------------------- gather

// A row's place in one of the caches: byte offsets of its data and scales.
template <int kD>
__device__ __forceinline__ void wide_load(const CacheView &c, const PageMap &pm, int h, int page, int off,
                                          int lane, uint4 (&w)[kD / 64], uint32_t (&s)[kD / 64])
{
    constexpr int kQ = kD / 32;             // 32-element pieces of a row
#pragma unroll
    for (int k = 0; k < kD / 64; ++k) {
        const int combo = 4 * k + (lane >> 3);
        const int q = combo % kQ, r = (lane & 7) + 8 * (combo / kQ);
        const int pg = __shfl_sync(0xffffffffu, page, r), of = __shfl_sync(0xffffffffu, off, r);
        w[k] = make_uint4(0u, 0u, 0u, 0u);
        s[k] = 0u;
        if (pg >= 0) {
            w[k] = __ldg(reinterpret_cast<const uint4 *>(cache::row_data(c, pm, pg, h, of)) + q);
            s[k] = __ldg(reinterpret_cast<const uint16_t *>(cache::row_scale(c, pm, pg, h, of)) + q);
        }
    }
}

// Converts and stores what wide_load fetched: element e of tile row r at
// stage + (e / 64) * 128 * 128 + r * 128 + ((e / 8 % 8) ^ (r & 7)) * 16.
// Eight lanes in a row store the same unit of eight different tile rows, whose
// swizzled places differ: no bank conflicts.
template <int kD>
__device__ __forceinline__ void wide_store(uint32_t stage, int row0, int lane, const uint4 (&w)[kD / 64],
                                           const uint32_t (&s)[kD / 64])
{
    constexpr int kQ = kD / 32;
#pragma unroll
    for (int k = 0; k < kD / 64; ++k) {
        const int combo = 4 * k + (lane >> 3);
        const int q = combo % kQ, r = row0 + (lane & 7) + 8 * (combo / kQ);
        const uint32_t dst = stage + (q >> 1) * kWideKeys * 128 + r * 128;
        const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t sc = cache::f16x2_of_e4m3x2((s[k] >> (8 * (j >> 1)) & 0xFFu) * 0x0101u);
            const uint32_t a = hmul2(pair_of(x[j], 0), sc), b = hmul2(pair_of(x[j], 1), sc);
            const uint32_t c = hmul2(pair_of(x[j], 2), sc), d = hmul2(pair_of(x[j], 3), sc);
            const uint32_t u = 4 * (q & 1) + j;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((u ^ (r & 7)) << 4)),
                         "r"(a), "r"(b), "r"(c), "r"(d)
                         : "memory");
        }
    }
}

// Walks the CTA's tiles in order.
struct TileCursor {
    int item, t;
    Item it;
    const int32_t *list, *table;

    __device__ __forceinline__ void enter(const AttnParams &p, int tile_rows)
    {
        it = item_of(p, item, tile_rows);
        t = it.t0;
        table = p.pm.table + it.g.b * p.pm.table_stride;
        list = p.idx ? p.idx + (static_cast<long long>(it.g.b) * p.S + it.g.i0) * p.topk : nullptr;
    }
    // the first tile at or behind the cursor; false: none left
    __device__ __forceinline__ bool settle(const AttnParams &p, int items, int tile_rows)
    {
        while (t >= it.t1) {
            item += gridDim.x;
            if (item >= items)
                return false;
            enter(p, tile_rows);
        }
        return true;
    }
};

template <int kDk, int kDv>
__device__ void wide_gather(const WideParams &wp, uint8_t *smem, WideBarriers *bars, const WaitCtl &ctl,
                            int tile_rows)
{
    const AttnParams &p = wp.a;
    const int lane = threadIdx.x & 31;
    const int gw = (threadIdx.x >> 5) - 4;
    const int row0 = gw * kGatherRows;
    const uint32_t k_base = smem_u32(smem), v_base = k_base + wp.off_v;

    TileCursor cur;                         // the tile whose list entry is fetched next
    cur.item = blockIdx.x;
    bool more = cur.item < wp.items;
    if (more) {
        cur.enter(p, tile_rows);
        more = cur.settle(p, wp.items, tile_rows);
    }
    // three tiles ahead: this lane's position; two ahead: its page; one ahead: codes
    int pos3 = -1, lim3 = 0, h3 = 0, page2 = -1, off2 = 0, h2 = 0;
    const int32_t *table3 = nullptr;
    bool have3 = false, have2 = false, have1 = false;
    uint4 kw[kDk / 64], vw[kDv / 64];
    uint32_t ks[kDk / 64], vs[kDv / 64];
    uint32_t bits = 0;
    auto fetch_pos = [&]() {
        have3 = more;
        if (!more)
            return;
        const int slot = cur.t * kWideKeys + row0 + lane;
        pos3 = lane < kGatherRows && slot < cur.it.slots ? (cur.list ? __ldg(cur.list + slot) : slot) : -1;
        lim3 = cur.it.limit;
        h3 = cur.it.g.h;
        table3 = cur.table;
        ++cur.t;
        more = cur.settle(p, wp.items, tile_rows);
    };
    auto fetch_page = [&]() {
        have2 = have3;
        h2 = h3;
        page2 = -1;
        off2 = 0;
        if (have3 && pos3 >= 0 && pos3 < lim3 && !p.pm.locate(table3, pos3, page2, off2))
            page2 = -1;
    };
    auto fetch_codes = [&]() {
        have1 = have2;
        if (!have2)
            return;
        bits = __ballot_sync(0xffffffffu, page2 >= 0);
        wide_load<kDk>(p.ck, p.pm, h2, page2, off2, lane, kw, ks);
        wide_load<kDv>(p.cv, p.pm, h2, page2, off2, lane, vw, vs);
    };
    fetch_pos();
    fetch_page();
    fetch_pos();
    fetch_codes();
    fetch_page();
    fetch_pos();
    bool ok = true;
    for (int gt = 0; have1; ++gt) {
        uint4 kc[kDk / 64], vc[kDv / 64];
        uint32_t ksc[kDk / 64], vsc[kDv / 64];
        const uint32_t cbits = bits;
#pragma unroll
        for (int k = 0; k < kDk / 64; ++k) {
            kc[k] = kw[k];
            ksc[k] = ks[k];
        }
#pragma unroll
        for (int k = 0; k < kDv / 64; ++k) {
            vc[k] = vw[k];
            vsc[k] = vs[k];
        }
        fetch_codes();
        fetch_page();
        fetch_pos();
        const int kst = gt % wp.k_stages, vst = gt % wp.v_stages;
        if (lane == 0)
            ok = wait_bounded(&bars->k_empty[kst], ((gt / wp.k_stages) & 1) ^ 1, ctl, kWideGather, gt);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok)
            break;
        wide_store<kDk>(k_base + kst * wp.k_bytes, row0, lane, kc, ksc);
        if (lane == 0)
            bars->valid[gt % kMaskRing][gw] = static_cast<uint16_t>(cbits);
        fence_proxy_async_smem();           // these writes before the tensor core's reads
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bars->k_full[kst]);
            ok = wait_bounded(&bars->v_empty[vst], ((gt / wp.v_stages) & 1) ^ 1, ctl, kWideGather, gt);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok)
            break;
        wide_store<kDv>(v_base + vst * wp.v_bytes, row0, lane, vc, vsc);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bars->v_full[vst]);
    }
    if (!ok)
        *ctl.abort = 1;
}

// ---------------------------------------------------------------- MMA issue

template <int kDk, int kDv>
__device__ void wide_mma(const WideParams &wp, uint8_t *smem, WideBarriers *bars, uint32_t tmem,
                         const WaitCtl &ctl, int tile_rows)
{
    const AttnParams &p = wp.a;
    const uint32_t idesc_s = instr_desc_f16(kWideKeys, 0);
    const uint32_t idesc_pv = instr_desc_f16(kDv, 0) | (1u << 16);   // B (V) MN-major
    const uint32_t k_base = smem_u32(smem), v_base = k_base + wp.off_v;
    const int slots = wp.slots;
    int gt = 0, used = 0;                   // tiles, items with tiles
    auto issue_pv = [&](int g, bool first) -> bool {
        const int vst = g % wp.v_stages, slot = g % slots;
        if (!wait_bounded(&bars->p_full[slot], (g / slots) & 1, ctl, kWideMma, g) ||
            !wait_bounded(&bars->v_full[vst], (g / wp.v_stages) & 1, ctl, kWideMma, g))
            return false;
        // the item's first P.V overwrites O: the item before must have read its own
        if (first && used > 0 && !wait_bounded(&bars->o_empty, (used - 1) & 1, ctl, kWideMma, g))
            return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kWideKeys / 16; ++k)
            mma_f16_ts(tmem + wp.col_o, tmem + slot * kWideKeys + 8 * k,
                       smem_desc_mn_sw128(v_base + vst * wp.v_bytes + k * 16 * 128, kWideKeys * 128, 1024),
                       idesc_pv, !first || k > 0 ? 1u : 0u);
        mma_commit(&bars->v_empty[vst]);
        mma_commit(&bars->s_empty[slot]);   // the slot (S, then P) is free
        mma_commit(&bars->pv_done);
        return true;
    };
    bool ok = true;
    for (int item = blockIdx.x; item < wp.items && ok; item += gridDim.x) {
        const Item it = item_of(p, item, tile_rows);
        if (it.t0 >= it.t1)
            continue;
        ok = wait_bounded(&bars->q_full, used & 1, ctl, kWideMma, item);
        const int g0 = gt;
        for (int t = it.t0; t < it.t1 && ok; ++t, ++gt) {
            const int kst = gt % wp.k_stages, slot = gt % slots;
            // one S slot: the P.V that frees it goes first
            if (slots == 1 && gt > g0 && !(ok = issue_pv(gt - 1, gt - 1 == g0)))
                break;
            ok = wait_bounded(&bars->k_full[kst], (gt / wp.k_stages) & 1, ctl, kWideMma, gt) &&
                 wait_bounded(&bars->s_empty[slot], ((gt / slots) & 1) ^ 1, ctl, kWideMma, gt);
            if (!ok)
                break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kDk / 16; ++k)
                mma_f16_ts(tmem + slot * kWideKeys, tmem + wp.col_q + 8 * k,
                           smem_desc_kmajor(k_base + kst * wp.k_bytes + (k >> 2) * kWideKeys * 128 + (k & 3) * 32, 128),
                           idesc_s, k > 0 ? 1u : 0u);
            mma_commit(&bars->s_full[slot]);
            mma_commit(&bars->k_empty[kst]);
            // S(t) is queued: P(t-1) . V(t-1) runs beside the softmax of tile t
            if (slots > 1 && gt > g0)
                ok = issue_pv(gt - 1, gt - 1 == g0);
        }
        if (!ok)
            break;
        ok = issue_pv(gt - 1, gt - 1 == g0);
        ++used;
    }
    if (!ok)
        *ctl.abort = 1;
    mma_commit(&bars->drain);
    wait_drain(&bars->drain, 0);
}

// ---------------------------------------------------------------- softmax

// Largest of 32 scores whose bits are set.
template <bool kMasked>
__device__ __forceinline__ float max32(const uint32_t (&v)[32], uint32_t bits)
{
    float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 32; ++j)
        a[j & 3] = fmaxf(a[j & 3], !kMasked || (bits >> j & 1u) ? __uint_as_float(v[j]) : -INFINITY);
    return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
}

// 32 scores to packed f16 probabilities 2^(f v - m); returns their sum.
template <bool kMasked>
__device__ __forceinline__ float probs32(const uint32_t (&v)[32], uint32_t bits, float f, float m,
                                         uint32_t *pk)
{
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        float a = ex2_approx(fmaf(__uint_as_float(v[j]), f, -m));
        float b = ex2_approx(fmaf(__uint_as_float(v[j + 1]), f, -m));
        if (kMasked) {
            a = bits >> j & 1u ? a : 0.0f;
            b = bits >> (j + 1) & 1u ? b : 0.0f;
        }
        s[(j >> 1) & 1] += a + b;
        pk[j / 2] = f16x2_of(a, b);
    }
    return s[0] + s[1];
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// The row's query in f16 over its power of two, into TMEM (two elements a
// column); returns the factor that turns a score into the log2 domain (>= 0:
// the scale's sign goes with the query).
template <int kDk>
__device__ __forceinline__ float wide_query(const AttnParams &p, const __nv_bfloat16 *src, uint32_t taddr)
{
    float peak = 0.0f;
    if (src) {
#pragma unroll 8
        for (int j = 0; j < kDk / 8; ++j) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src) + j);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = cache::float2_of_bf16x2(u[e]);
                peak = fmaxf(peak, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
        }
    }
    const int e = min(max(static_cast<int>(__float_as_uint(peak) >> 23), 1), 253);
    float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
    if (p.sl2 < 0.0f)
        down = -down;
#pragma unroll 1
    for (int c = 0; c < kDk / 32; ++c) {
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 x = src ? __ldg(reinterpret_cast<const uint4 *>(src) + 4 * c + j)
                                : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 y = cache::float2_of_bf16x2(u[q]);
                v[4 * j + q] = f16x2_of(y.x * down, y.y * down);
            }
        }
        tmem_st_32x32b_x16(taddr + 16 * c, v);
    }
    return up * fabsf(p.sl2);
}

template <int kDk, int kDv, bool kSplit>
__device__ void wide_softmax(const WideParams &wp, uint8_t *smem, WideBarriers *bars, uint32_t tmem,
                             const WaitCtl &ctl)
{
    constexpr int kTileRows = kSplit ? kWideRows / 2 : kWideRows;
    constexpr int NC = kSplit ? kWideKeys / 2 : kWideKeys;    // keys a thread takes of a tile
    const AttnParams &p = wp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = kSplit ? warp & 1 : warp;
    const int half = kSplit ? warp >> 1 : 0;
    const int row = 32 * quarter + lane;                      // of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int slots = wp.slots;
    float *xo = reinterpret_cast<float *>(smem + wp.off_x);   // kSplit: [warp][32 columns][32 lanes]
    int gt = 0, xc = 0;
    bool ok = true;
    // both warps of a pair have arrived (kSplit)
    auto pair_sync = [&]() -> bool {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bars->xbar[quarter][xc & 1]);
        const bool good = wait_bounded(&bars->xbar[quarter][xc & 1], (xc >> 1) & 1, ctl, kWideSoftmax, xc);
        ++xc;
        return __all_sync(0xffffffffu, good);
    };
    auto wait_pv = [&](int g) -> bool {
        const bool good = wait_bounded(&bars->pv_done, g & 1, ctl, kWideSoftmax, g);
        return __all_sync(0xffffffffu, good);
    };
    for (int item = blockIdx.x; item < wp.items && ok; item += gridDim.x) {
        const Item it = item_of(p, item, kTileRows);
        const int r = it.g.r0 + row;
        const bool real = r < p.rows;
        int i = 0, head = 0;
        if (real)
            row_of(p, it.g, r, i, head);
        const long long at = (static_cast<long long>(it.g.b) * p.S + i) * p.HA + head;
        float m = -INFINITY, l = 0.0f;
        if (it.t0 < it.t1) {
            // every S of the item before has been waited for: its query may go
            const float f = wide_query<kDk>(p, real ? p.q + at * kDk : nullptr, lanes + wp.col_q);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars->q_full);
            // a dense row sees the slots below its own limit; a list's entries are checked when gathered
            const int see = p.idx ? it.slots : (real ? seen(p, it.len, i) : 0);
            for (int t = it.t0; t < it.t1; ++t, ++gt) {
                const int slot = gt % slots;
                ok = wait_bounded(&bars->s_full[slot], (gt / slots) & 1, ctl, kWideSoftmax, gt);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t scol = lanes + slot * kWideKeys + half * NC;
                // the thread's keys: gathered, and visible to its row
                uint32_t bits[NC / 32];
                bool whole = true;
#pragma unroll
                for (int w = 0; w < NC / 32; ++w) {
                    const int c = half * NC + 32 * w;
                    const uint32_t *vw = reinterpret_cast<const uint32_t *>(bars->valid[gt % kMaskRing]);
                    const int n = see - t * kWideKeys - c;
                    const uint32_t below = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
                    bits[w] = *reinterpret_cast<const volatile uint32_t *>(vw + (c >> 5)) & below;
                    whole = whole && bits[w] == 0xFFFFFFFFu;
                }
                whole = __all_sync(0xffffffffu, whole);
                float best = -INFINITY;
#pragma unroll
                for (int w = 0; w < NC / 32; w += 2) {
                    uint32_t v[2][32];
                    tmem_ld_32x32b_x32(scol + 32 * w, v[0]);
                    tmem_ld_32x32b_x32(scol + 32 * w + 32, v[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            reg_fence(v[e][j]);
                        best = fmaxf(best, whole ? max32<false>(v[e], 0u) : max32<true>(v[e], bits[w + e]));
                    }
                }
                const float top = best == -INFINITY ? -INFINITY : best * f;
                float alpha = 1.0f;
                if (top > m + kLag) {                          // (first keys: m is -inf)
                    alpha = ex2_approx(m - top);
                    m = top;
                }
                // a raised maximum rescales O once the tile before is in it
                if (t > it.t0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                    if (!(ok = wait_pv(gt - 1)))
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kDv; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(lanes + wp.col_o + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            reg_fence(o[j]);
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        }
                        tmem_st_32x32b_x32(lanes + wp.col_o + c, o);
                    }
                    tmem_st_wait();
                }
                const float m0 = m == -INFINITY ? 0.0f : m;
                float sum = 0.0f;
                const uint32_t pcol = lanes + slot * kWideKeys;
                // P over columns whose S has been read: 32 keys take 16 columns
#pragma unroll
                for (int w = 0; w < NC / 32; ++w) {
                    uint32_t v[32], pk[16];
                    tmem_ld_32x32b_x32(scol + 32 * w, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        reg_fence(v[j]);
                    sum += whole ? probs32<false>(v, 0u, f, m0, pk) : probs32<true>(v, bits[w], f, m0, pk);
                    if constexpr (kSplit) {
                        // the second half's P lies on columns that the same warp reads first
                        tmem_st_32x32b_x16(pcol + 32 * half + 16 * w, pk);
                    } else {
                        tmem_st_32x32b_x16(pcol + 16 * w, pk);
                    }
                }
                if constexpr (kSplit) {
                    uint32_t z[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        z[j] = 0u;
                    tmem_st_32x32b_x32(pcol + 32 * (1 - half), z);
                }
                l = l * alpha + sum;
                tmem_st_wait();
                // every tile waits for the P.V before it, so that the parity waits on
                // pv_done stay within one phase of the barrier
                if (gt > 0 && !(ok = wait_pv(gt - 1)))
                    break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars->p_full[slot]);
            }
            if (!ok || !(ok = wait_pv(gt - 1)))
                break;
            tc_fence_after();
        }
        const bool any = it.t0 < it.t1;
        float scale = 1.0f;                                    // of this copy's O
        if (kSplit) {
            bars->xchg[warp][lane][0] = m;
            bars->xchg[warp][lane][1] = l;
            if (!(ok = pair_sync()))
                break;
            const float m2 = bars->xchg[warp ^ 2][lane][0], l2 = bars->xchg[warp ^ 2][lane][1];
            const float top = fmaxf(m, m2);
            scale = m == -INFINITY ? 0.0f : ex2_approx(m - top);
            l = l * scale + (m2 == -INFINITY ? 0.0f : l2 * ex2_approx(m2 - top));
            m = top;
        }
        const bool part = p.splits > 1;
        const float norm = part ? 1.0f : (l > 0.0f ? p.v_scale / l : 0.0f);
        float *dst = part ? p.part + (static_cast<long long>(item) * kTileRows + row) * (kDv + 2) : nullptr;
        __nv_bfloat16 *out = p.out + at * kDv;
        auto put = [&](int c, const float (&x)[32]) {
            if (!real)
                return;
            if (part) {
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    *reinterpret_cast<float2 *>(dst + c + j) = make_float2(x[j], x[j + 1]);
            } else {
#pragma unroll
                for (int j = 0; j < 32; j += 8)
                    *reinterpret_cast<uint4 *>(out + c + j) =
                        make_uint4(cache::bf16x2_of(x[j] * norm, x[j + 1] * norm),
                                   cache::bf16x2_of(x[j + 2] * norm, x[j + 3] * norm),
                                   cache::bf16x2_of(x[j + 4] * norm, x[j + 5] * norm),
                                   cache::bf16x2_of(x[j + 6] * norm, x[j + 7] * norm));
            }
        };
        auto take = [&](int c, float (&x)[32]) {               // O's columns c.., scaled
            uint32_t o[32];
            if (any) {
                tmem_ld_32x32b_x32(lanes + wp.col_o + c, o);
                tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (any)
                    reg_fence(o[j]);
                x[j] = any ? __uint_as_float(o[j]) * scale : 0.0f;
            }
        };
        if constexpr (kSplit) {
            // each copy writes half of the columns: its own plus the other's, sent 32 at a time
            float *mine = xo + warp * 32 * 32;
            const float *theirs = xo + (warp ^ 2) * 32 * 32;
            for (int c = 0; c < kDv / 2; c += 32) {
                float x[32];
                take((1 - half) * (kDv / 2) + c, x);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    mine[j * 32 + lane] = x[j];
                if (!(ok = pair_sync()))
                    break;
                take(half * (kDv / 2) + c, x);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j] += theirs[j * 32 + lane];
                put(half * (kDv / 2) + c, x);
                if (!(ok = pair_sync()))                       // the buffer may be rewritten
                    break;
            }
            if (!ok)
                break;
        } else {
#pragma unroll 1
            for (int c = 0; c < kDv; c += 32) {
                float x[32];
                take(c, x);
                put(c, x);
            }
        }
        if (real && half == 0) {
            if (part) {
                dst[kDv] = m;
                dst[kDv + 1] = l;
            } else if (p.lse) {
                p.lse[at] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
        }
        if (any) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars->o_empty);
        }
    }
    if (!ok)
        *ctl.abort = 1;
}

// ---------------------------------------------------------------- kernel

template <int kDk, int kDv, bool kSplit>
__global__ void __launch_bounds__(kWideThreads, 1) cache_attn_wide_kernel(const WideParams wp)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    WideBarriers *bars = reinterpret_cast<WideBarriers *>(smem + wp.off_bar);
    constexpr int kTileRows = kSplit ? kWideRows / 2 : kWideRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWideStages; ++s) {
            mbar_init(&bars->k_full[s], kGatherWarps);
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->v_full[s], kGatherWarps);
            mbar_init(&bars->v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->s_full[s], 1);
            mbar_init(&bars->s_empty[s], 1);
            mbar_init(&bars->p_full[s], 4);
            mbar_init(&bars->xbar[s][0], 2);
            mbar_init(&bars->xbar[s][1], 2);
        }
        mbar_init(&bars->q_full, 4);
        mbar_init(&bars->pv_done, 1);
        mbar_init(&bars->o_empty, 4);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == kWideMmaWarp) {
        tmem_alloc(&bars->tmem_addr, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_addr;
    const WaitCtl ctl{&bars->abort, wp.wait_limit};
    if (warp < 4)
        wide_softmax<kDk, kDv, kSplit>(wp, smem, bars, tmem, ctl);
    else if (warp < kWideMmaWarp)
        wide_gather<kDk, kDv>(wp, smem, bars, ctl, kTileRows);
    else if (warp == kWideMmaWarp && lane == 0)
        wide_mma<kDk, kDv>(wp, smem, bars, tmem, ctl, kTileRows);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWideMmaWarp) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

} // namespace cattn
} // namespace csa
