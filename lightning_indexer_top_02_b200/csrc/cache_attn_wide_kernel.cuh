// cache_attn_wide_kernel.cuh -- attention over a cache held in 4 bits, more
// than 16 query rows per cached row (csa_cache_attention, include/csa_cache.h):
// up to 128 heads that share a row, or several queries of grouped heads.
//
// 2 rows (Dk + Dv) flops for each 9/16 (Dk + Dv) bytes: from about 64 rows on
// the work is bound by the tensor cores, and by what feeds them.  Tiles of 128
// query rows (TMEM lanes) x 128 keys on tcgen05:
//   S = Q . K^T    A = Q, B = K from shared memory
//   O += P . V     A = P from TMEM (over its S slot), B = V from shared memory (MN-major)
//
// One persistent CTA a SM walks work items (a group's row tile x a share of
// the keys).  Warps:
//   0-3   softmax: thread = TMEM lane = query row.  Q row to f16 (scaled by a power of
//         two, see cache_attn_kernel.cuh) into shared memory; per tile the row's maximum,
//         then P over the slot's first columns; O / l at the item's end.
//   4-11  gather: a share of the tile's rows each.  A tile's codes and scales come
//         by cp.async one tile ahead (their pages two, their list entries three tiles
//         ahead) into the warp's own staging rows, and are converted from there to
//         the 128-byte-swizzled operands; rows without a key are zeros.  (Held in
//         registers, the loads shared the six scoreboards with everything else and
//         each wait became a wait for memory.)
//   12    MMA issue and TMEM (13-15 complete its warpgroup).
// Nothing may spill: beside 200 KB of shared memory little L1 is left, and a spilled
// value comes back from L2.  Registers move from the gather warpgroups and the MMA's to
// the softmax's (setmaxnreg).
// Tiles have 128 keys, 64 where a head is wider than 128 elements (shared memory).
// Up to 64 rows (kSplit) the rows stand in lanes 0-63 and again in lanes
// 64-127: the copy takes the tile's other keys with its own maximum, sum and
// O, so that all four softmax warps work; the halves are joined at the end.
// Waits are bounded (ptx.cuh).
//
// Measured at D = 128: a tile of 128 keys takes 2.2 us with 64 rows (a prompt chunk of
// 1,024 queries x 64 heads over 2,048 selected keys: 231 us, 298 TFLOP/s), 2.4 us with 128 rows
// (32 sequences x 128 heads over 2,048 keys: 26 us, of which about 11 are the start and
// end of an item and 4 the join).  The tensor cores are busy 26 % of the time and the
// issue slots 44 %: the tile's chain of waits bounds it.  Leaving out the loads and
// conversions, the softmax or the MMAs takes only 10 to 20 % off.  Tried and slower: two CTAs an
// SM at 80 registers (spills: 447 us), warps that only copy (386 us) or only look up
// pages with one barrier for keys and values (315 us).
#pragma once
#include "cache_attn_kernel.cuh"

namespace csa {
namespace cattn {

constexpr int kWideThreads = 512;
constexpr int kWideRows = 128;              // query rows of a tile (TMEM lanes)
constexpr int kGatherWarps = 8;
constexpr int kWideMmaWarp = 4 + kGatherWarps;
// register split: launched with kWideLaunchRegs a thread; the increase takes what the
// decreases release
constexpr int kWideLaunchRegs = 128, kWideSoftmaxRegs = 200, kWideGatherRegs = 104, kWideMmaRegs = 104;
static_assert(kWideSoftmaxRegs >= kWideLaunchRegs && kWideGatherRegs <= kWideLaunchRegs &&
                  kWideMmaRegs <= kWideLaunchRegs && kWideSoftmaxRegs % 8 == 0 && kWideGatherRegs % 8 == 0 &&
                  kWideMmaRegs % 8 == 0 && kWideSoftmaxRegs <= 256 && kWideMmaRegs >= 24,
              "setmaxnreg counts: increases from, decreases to at most, the launch count");
static_assert(kWideSoftmaxRegs + 2 * kWideGatherRegs + kWideMmaRegs <= 4 * kWideLaunchRegs,
              "the register split must fit in the launch's registers");
constexpr int kWideStages = 2;              // at most, per ring (keys, values)
constexpr int kMaskRing = 8;                // validity words kept: stages + S slots + what is in use
constexpr int kXCols = 32;                  // O columns that two row copies exchange at a time

enum WideRole : int { kWideGather = 31, kWideMma = 32, kWideSoftmax = 33 };

struct WideParams {
    AttnParams a;
    int items;                              // works * splits
    int k_stages, v_stages, k_bytes, v_bytes;
    int off_k, off_v, off_raw, off_x, off_bar; // shared memory: Q, K ring, V ring, staging, exchange, barriers
    long long wait_limit;
};

template <int kDk, int kDv>
struct WideShape {
    static constexpr int kKeys = kDk <= 128 && kDv <= 128 ? 128 : 64;    // keys of a tile
    static constexpr int kRows = kKeys / kGatherWarps;                   // of it, a gather warp's
    // TMEM columns: two S slots, then O
    static constexpr int kO = 2 * kKeys;
    static_assert(kO + kDv <= 512, "TMEM columns");
    // staging of one gather warp and tile: K codes, V codes, K scales, V scales
    static constexpr int kRawV = kRows * kDk / 2, kRawKs = kRawV + kRows * kDv / 2;
    static constexpr int kRawVs = kRawKs + kRows * kDk / 16, kRaw = kRawVs + kRows * kDv / 16;
    static_assert(kRaw % 16 == 0, "staging rows start on 16 bytes");
};

// Position in a ring of n entries and the parity of its present round.
struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n)
    {
        if (++at == n) {
            at = 0;
            phase ^= 1;
        }
    }
};

struct WideBarriers {
    uint64_t k_full[kWideStages], k_empty[kWideStages];
    uint64_t v_full[kWideStages], v_empty[kWideStages];
    uint64_t s_full[2], s_empty[2], p_full[2];   // s_empty: the slot's P.V is done
    uint64_t q_full, o_empty, drain;
    uint64_t xbar[2][2];                    // kSplit: per row quarter, two phases in turn
    float xchg[4][32][2];                   // kSplit: a row copy's maximum and sum
    uint32_t valid[kMaskRing][4];           // a tile's keys, one bit each
    uint32_t tmem_addr;
    int abort;
};

// Every thread calls this once, when it has started what needs neither barriers nor
// TMEM (the first loads): the barriers are there from here on.  Returns TMEM's address.
__device__ __forceinline__ uint32_t wide_ready(const WideBarriers *bars)
{
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return bars->tmem_addr;
}

// What every role needs to know of an item.
struct Item {
    Group g;
    int len;
    int t0, t1;                             // its tiles
    int slots;                              // key slots of the group
    int limit;                              // positions the tile's last row sees
};

__device__ __forceinline__ Item item_of(const AttnParams &p, int item, int tile_rows, int keys)
{
    Item it;
    const int work = static_cast<int>(p.div_splits.div(item)), split = item - work * p.splits;
    it.g = group_of(p, work, tile_rows);
    it.len = __ldg(p.kv_len + it.g.b);
    const int r_last = min(it.g.r0 + tile_rows, p.rows) - 1;
    it.limit = it.len > 0 ? seen(p, it.len, it.g.i0 + static_cast<int>(p.div_G.div(r_last))) : 0;
    it.slots = p.idx ? (it.limit > 0 ? p.topk : 0) : min(max(it.limit, 0), p.capacity);
    const unsigned tiles = (static_cast<unsigned>(it.slots) + keys - 1) / keys;   // (keys: a power of two)
    // even shares, the first ones a tile larger
    const int each = static_cast<int>(p.div_splits.div(tiles)), more = static_cast<int>(tiles) - each * p.splits;
    it.t0 = each * split + min(split, more);
    it.t1 = it.t0 + each + (split < more ? 1 : 0);
    return it;
}

// ---------------------------------------------------------------- gather

// Converts staged rows to an operand stage: element e of tile row r goes to
// stage + (e / 64) * kKeys * 128 + r * 128 + ((e / 8 % 8) ^ (r & 7)) * 16.  Eight
// lanes in a row store the same unit of eight different tile rows, whose swizzled
// places differ: no bank conflicts.
template <int kD, int kKeys, int kRows>
__device__ __forceinline__ void convert_rows(uint32_t stage, const uint8_t *codes, const uint8_t *scales, int row0,
                                             int lane)
{
    constexpr int kQ = kD / 32, kN = kQ * kRows;
#pragma unroll
    for (int k = 0; k < (kN + 31) / 32; ++k) {
        const int combo = 4 * k + (lane >> 3);
        const int q = combo % kQ, r = (lane & 7) + 8 * (combo / kQ);
        if (kN % 32 != 0 && combo >= kN / 8)
            break;
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + staged_at<kQ>(r, q));
        const uint32_t two = cache::f16x2_of_e4m3x2(*reinterpret_cast<const uint16_t *>(scales + r * (kD / 16) + 2 * q));
        const uint32_t dst = stage + (q >> 1) * kKeys * 128 + (row0 + r) * 128;
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        // both scales of the piece, each in both halves
        const uint32_t sc[2] = {__byte_perm(two, 0u, 0x1010), __byte_perm(two, 0u, 0x3232)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = hmul2(pair_of(x[j], 0), sc[j >> 1]), b = hmul2(pair_of(x[j], 1), sc[j >> 1]);
            const uint32_t c = hmul2(pair_of(x[j], 2), sc[j >> 1]), d = hmul2(pair_of(x[j], 3), sc[j >> 1]);
            const uint32_t u = 4 * (q & 1) + j;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((u ^ (r & 7)) << 4)), "r"(a), "r"(b),
                         "r"(c), "r"(d)
                         : "memory");
        }
    }
}

// Walks the CTA's tiles in order.
struct TileCursor {
    int item, t;
    Item it;
    const int32_t *list, *table;

    __device__ __forceinline__ void enter(const AttnParams &p, int tile_rows, int keys)
    {
        it = item_of(p, item, tile_rows, keys);
        t = it.t0;
        table = p.pm.table + it.g.b * p.pm.table_stride;
        list = p.idx ? p.idx + (static_cast<long long>(it.g.b) * p.S + it.g.i0) * p.topk : nullptr;
    }
    // the first tile at or behind the cursor; false: none left
    __device__ __forceinline__ bool settle(const AttnParams &p, int items, int tile_rows, int keys)
    {
        while (t >= it.t1) {
            item += gridDim.x;
            if (item >= items)
                return false;
            enter(p, tile_rows, keys);
        }
        return true;
    }
};

template <int kDk, int kDv>
__device__ void wide_gather(const WideParams &wp, uint8_t *smem, WideBarriers *bars, const WaitCtl &ctl,
                            int tile_rows)
{
    using Sh = WideShape<kDk, kDv>;
    constexpr int kKeys = Sh::kKeys, kRows = Sh::kRows;
    const AttnParams &p = wp.a;
    const int lane = threadIdx.x & 31;
    const int gw = (threadIdx.x >> 5) - 4;
    const int row0 = gw * kRows;
    const uint32_t k_base = smem_u32(smem) + wp.off_k, v_base = smem_u32(smem) + wp.off_v;
    uint8_t *raw = smem + wp.off_raw + gw * 2 * Sh::kRaw;     // two tiles in turn

    TileCursor cur;                         // the tile whose list entry is fetched next
    cur.item = blockIdx.x;
    bool more = cur.item < wp.items;
    if (more) {
        cur.enter(p, tile_rows, kKeys);
        more = cur.settle(p, wp.items, tile_rows, kKeys);
    }
    // Three tiles ahead: this lane's position; two ahead: its page.  Nothing that
    // a load brought is looked at before the step that needs it.
    int pos3 = -1, page2 = -1, row2 = 0, lim3 = 0, h3 = 0;
    const int32_t *table3 = nullptr;
    bool have3 = false, have2 = false;
    auto fetch_pos = [&]() {
        have3 = more;
        if (!more)
            return;
        const int slot = cur.t * kKeys + row0 + lane;
        pos3 = lane < kRows && slot < cur.it.slots ? (cur.list ? __ldg(cur.list + slot) : slot) : -1;
        lim3 = cur.it.limit;
        h3 = cur.it.g.h;
        table3 = cur.table;
        ++cur.t;
        more = cur.settle(p, wp.items, tile_rows, kKeys);
    };
    auto fetch_page = [&]() {
        have2 = have3;
        if (!have3)
            return;
        const bool in = pos3 >= 0 && pos3 < lim3;
        const int n = in ? static_cast<int>(p.pm.div.div(pos3)) : 0;
        const bool has = in && n < p.pm.max_pages;
        page2 = has ? __ldg(table3 + n) : -1;
        row2 = h3 * p.pm.page_size + (has ? pos3 - n * p.pm.page_size : 0);
    };
    // starts the copies of tile g (if there is one); one cp.async group in any case
    auto start = [&](int g) -> bool {
        if (have2) {
            const int page = page2 >= 0 && page2 < p.pm.num_pages ? page2 : -1;
            const uint32_t bits = __ballot_sync(0xffffffffu, page >= 0);
            uint8_t *mask = reinterpret_cast<uint8_t *>(bars->valid[g % kMaskRing]);
            if (lane == 0) {
                if constexpr (kRows == 16)
                    reinterpret_cast<uint16_t *>(mask)[gw] = static_cast<uint16_t>(bits);
                else
                    mask[gw] = static_cast<uint8_t>(bits);
            }
            const uint32_t to = smem_u32(raw + (g & 1) * Sh::kRaw);
            stage_codes<kDk, kRows>(to, data_at(p.ck, page, row2), bits, lane);
            stage_codes<kDv, kRows>(to + Sh::kRawV, data_at(p.cv, page, row2), bits, lane);
            // scales: the keys' by lanes 0.., the values' by lanes 16..
            const int pg = __shfl_sync(0xffffffffu, page, lane & 15), ro = __shfl_sync(0xffffffffu, row2, lane & 15);
            if ((lane & 15) < kRows) {
                if (lane < 16)
                    stage_scales<kDk>(to + Sh::kRawKs, lane, scale_at(p.ck, pg, ro), pg >= 0);
                else
                    stage_scales<kDv>(to + Sh::kRawVs, lane - 16, scale_at(p.cv, pg, ro), pg >= 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return have2;
    };
    fetch_pos();
    fetch_page();
    fetch_pos();
    bool have = start(0), ok = true;
    fetch_page();
    fetch_pos();
    wide_ready(bars);
    Ring kr, vr;
    for (int gt = 0; have; ++gt) {
        const bool next = start(gt + 1);
        fetch_page();
        fetch_pos();
        asm volatile("cp.async.wait_group 1;" ::: "memory");   // this tile's have landed
        __syncwarp();                                          // every lane's
        if (lane == 0)
            ok = wait_bounded(&bars->k_empty[kr.at], kr.phase ^ 1, ctl, kWideGather, gt);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok)
            break;
        const uint8_t *from = raw + (gt & 1) * Sh::kRaw;
        convert_rows<kDk, kKeys, kRows>(k_base + kr.at * wp.k_bytes, from, from + Sh::kRawKs, row0, lane);
        fence_proxy_async_smem();           // these writes before the tensor core's reads
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bars->k_full[kr.at]);
            ok = wait_bounded(&bars->v_empty[vr.at], vr.phase ^ 1, ctl, kWideGather, gt);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok)
            break;
        convert_rows<kDv, kKeys, kRows>(v_base + vr.at * wp.v_bytes, from + Sh::kRawV, from + Sh::kRawVs, row0, lane);
        fence_proxy_async_smem();
        __syncwarp();                       // (the staging may be written again)
        if (lane == 0)
            mbar_arrive(&bars->v_full[vr.at]);
        kr.step(wp.k_stages);
        vr.step(wp.v_stages);
        have = next;
    }
    if (!ok)
        *ctl.abort = 1;
    cp_async_wait_all();                    // every copy lands before the CTA can exit
}

// ---------------------------------------------------------------- MMA issue

template <int kDk, int kDv>
__device__ void wide_mma(const WideParams &wp, uint8_t *smem, WideBarriers *bars, uint32_t tmem,
                         const WaitCtl &ctl, int tile_rows)
{
    using Sh = WideShape<kDk, kDv>;
    constexpr int kKeys = Sh::kKeys;
    const AttnParams &p = wp.a;
    constexpr uint32_t idesc_s = instr_desc_f16(kKeys, 0);
    constexpr uint32_t idesc_pv = instr_desc_f16(kDv, 0) | (1u << 16);   // B (V) MN-major
    const uint64_t q_desc = smem_desc_kmajor(smem_u32(smem), 128);
    const uint64_t k_desc = smem_desc_kmajor(smem_u32(smem) + wp.off_k, 128);
    const uint64_t v_desc = smem_desc_mn_sw128(smem_u32(smem) + wp.off_v, kKeys * 128, 1024);
    // ring positions are kept, not divided for: one thread issues everything, and
    // its latency between MMAs is the tensor cores' idle time
    Ring kr, vr, sr, pr;                    // K, V, S slots, P slots
    int used = 0;                           // items with tiles
    auto issue_pv = [&](bool first) -> bool {
        if (!wait_bounded(&bars->p_full[pr.at], pr.phase, ctl, kWideMma, used) ||
            !wait_bounded(&bars->v_full[vr.at], vr.phase, ctl, kWideMma, used))
            return false;
        // the item's first P.V overwrites O: the item before must have read its own
        if (first && used > 0 && !wait_bounded(&bars->o_empty, (used - 1) & 1, ctl, kWideMma, used))
            return false;
        tc_fence_after();
        const uint64_t b = v_desc + static_cast<uint64_t>((vr.at * wp.v_bytes) >> 4);
        const uint32_t a = tmem + pr.at * kKeys;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
            mma_f16_ts(tmem + Sh::kO, a + 8 * k, b + (k * 16 * 128 >> 4), idesc_pv, !first || k > 0 ? 1u : 0u);
        mma_commit(&bars->v_empty[vr.at]);
        mma_commit(&bars->s_empty[pr.at]);  // the slot (S, then P) is free
        vr.step(wp.v_stages);
        pr.step(2);
        return true;
    };
    bool ok = true;
    for (int item = blockIdx.x; item < wp.items && ok; item += gridDim.x) {
        const Item it = item_of(p, item, tile_rows, kKeys);
        if (it.t0 >= it.t1)
            continue;
        ok = wait_bounded(&bars->q_full, used & 1, ctl, kWideMma, item);
        for (int t = it.t0; t < it.t1 && ok; ++t) {
            ok = wait_bounded(&bars->k_full[kr.at], kr.phase, ctl, kWideMma, t) &&
                 wait_bounded(&bars->s_empty[sr.at], sr.phase ^ 1, ctl, kWideMma, t);
            if (!ok)
                break;
            tc_fence_after();
            const uint64_t b = k_desc + static_cast<uint64_t>((kr.at * wp.k_bytes) >> 4);
            const uint32_t d = tmem + sr.at * kKeys;
#pragma unroll
            for (int k = 0; k < kDk / 16; ++k)
            {
                const uint32_t in = (k & 3) * 32;
                mma_f16_ss(d, q_desc + (((k >> 2) * kWideRows * 128 + in) >> 4), b + (((k >> 2) * kKeys * 128 + in) >> 4), idesc_s, k > 0 ? 1u : 0u);
            }
            mma_commit(&bars->s_full[sr.at]);
            mma_commit(&bars->k_empty[kr.at]);
            kr.step(wp.k_stages);
            sr.step(2);
            // S(t) is queued: P(t-1) . V(t-1) runs beside the softmax of tile t
            if (t > it.t0)
                ok = issue_pv(t - 1 == it.t0);
        }
        if (!ok)
            break;
        ok = issue_pv(it.t1 - 1 == it.t0);
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

// The row's query in f16 over its power of two, into the swizzled A operand
// (row `row` of the tile at smem address dst); returns the factor that turns a score
// into the log2 domain (>= 0: the scale's sign goes with the query).  Rows
// of more than 64 elements are read twice (the second time from L1).
template <int kDk>
__device__ __forceinline__ float wide_query(const AttnParams &p, const __nv_bfloat16 *src, uint32_t dst, int row)
{
    constexpr bool kKeep = kDk <= 64;
    constexpr int kPart = 64;                            // elements in registers at a time
    uint4 w[kPart / 8];
    float peak = 0.0f;
    auto fetch = [&](int c) {
#pragma unroll
        for (int j = 0; j < kPart / 8; ++j)
            w[j] = src ? __ldg(reinterpret_cast<const uint4 *>(src + c) + j) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int c = 0; c < kDk; c += kPart) {
        fetch(c);
#pragma unroll
        for (int j = 0; j < kPart / 8; ++j) {
            const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = cache::float2_of_bf16x2(u[e]);
                peak = fmaxf(peak, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
        }
    }
    float down, up;
    query_scale(peak, down, up);
    if (p.sl2 < 0.0f)
        down = -down;
#pragma unroll
    for (int c = 0; c < kDk; c += kPart) {
        if (!kKeep)
            fetch(c);
#pragma unroll
        for (int j = 0; j < kPart / 8; ++j) {
            const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 y = cache::float2_of_bf16x2(u[q]);
                v[q] = f16x2_of(y.x * down, y.y * down);
            }
            const int unit = c / 8 + j;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             dst + (unit >> 3) * kWideRows * 128 + row * 128 + (((unit & 7) ^ (row & 7)) << 4)),
                         "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                         : "memory");
        }
    }
    return up * fabsf(p.sl2);
}

// What a softmax thread keeps of its row of an item.
struct WideRow {
    int item, t0, t1;
    int see;                                // slots below this are visible to the row
    float f;
    bool real;
    long long at;                           // (b, i, head)
};

template <int kDk, int kDv, bool kSplit>
__device__ void wide_softmax(const WideParams &wp, uint8_t *smem, WideBarriers *bars, const WaitCtl &ctl)
{
    constexpr int kTileRows = kSplit ? kWideRows / 2 : kWideRows;
    using Sh = WideShape<kDk, kDv>;
    constexpr int kKeys = Sh::kKeys;
    constexpr int NC = kSplit ? kKeys / 2 : kKeys;            // keys a thread takes of a tile
    const AttnParams &p = wp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = kSplit ? warp & 1 : warp;
    const int half = kSplit ? warp >> 1 : 0;
    const int row = 32 * quarter + lane;                      // of the tile
    uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;  // the warp's TMEM lanes
    Ring sr;
    float *xo = reinterpret_cast<float *>(smem + wp.off_x);   // kSplit: [warp][kXCols columns][32 lanes]
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
    // P.V of the CTA's tile g is done.  Its slot's barrier has completed the phase
    // before (S of that tile waited for it) and cannot complete the next without a P of
    // this warp, so the parity is exact.
    auto wait_pv = [&](int g) -> bool {
        const bool good = wait_bounded(&bars->s_empty[g & 1], (g >> 1) & 1, ctl, kWideSoftmax, g);
        return __all_sync(0xffffffffu, good);
    };
    // An item's row.  Its query is on its way to L2 from here on.
    auto look = [&](int item) -> WideRow {
        WideRow w;
        w.item = item;
        w.t0 = w.t1 = 0;
        if (item >= wp.items)
            return w;
        const Item it = item_of(p, item, kTileRows, kKeys);
        const int r = it.g.r0 + row;
        int i = 0, head = 0;
        w.real = r < p.rows;
        if (w.real)
            row_of(p, it.g, r, i, head);
        w.at = (static_cast<long long>(it.g.b) * p.S + i) * p.HA + head;
        w.t0 = it.t0;
        w.t1 = it.t1;
        // a dense row sees the slots below its own limit; a list's entries are checked when gathered
        w.see = p.idx ? it.slots : (w.real ? seen(p, it.len, i) : 0);
        if (w.real && w.t0 < w.t1)
            for (int c = 0; c < kDk; c += 64)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + w.at * kDk + c));
        return w;
    };
    // Writes its query as an operand.  Called when every S of the item before has
    // been waited for, and before that item's O is written out, so that the next
    // item's S runs meanwhile.
    auto begin = [&](WideRow &w) {
        if (w.t0 < w.t1) {
            w.f = wide_query<kDk>(p, w.real ? p.q + w.at * kDk : nullptr, smem_u32(smem), 32 * warp + lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars->q_full);
        }
    };
    WideRow cur = look(blockIdx.x);
    lanes += wide_ready(bars);
    begin(cur);
    while (cur.item < wp.items && ok) {
        float m = -INFINITY, l = 0.0f;
        const bool any = cur.t0 < cur.t1;
        WideRow next = look(cur.item + gridDim.x);
        if (any) {
            const float f = cur.f;
            const int see = cur.see;
            for (int t = cur.t0; t < cur.t1; ++t, ++gt) {
                const int slot = sr.at;
                ok = wait_bounded(&bars->s_full[slot], sr.phase, ctl, kWideSoftmax, gt);
                sr.step(2);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t scol = lanes + slot * kKeys + half * NC;
                // the thread's keys: gathered, and visible to its row
                uint32_t bits[NC / 32];
                bool whole = true;
#pragma unroll
                for (int w = 0; w < NC / 32; ++w) {
                    const int c = half * NC + 32 * w;
                    const int n = see - t * kKeys - c;
                    const uint32_t below = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
                    bits[w] = *reinterpret_cast<const volatile uint32_t *>(&bars->valid[gt % kMaskRing][c >> 5]) & below;
                    whole = whole && bits[w] == 0xFFFFFFFFu;
                }
                whole = __all_sync(0xffffffffu, whole);
                // up to 64 scores stay in registers, 128 are read twice, for the maximum and for the
                // probabilities: kept, they would not fit beside the rest
                constexpr int kAt = NC < 64 ? NC : 64;
                uint32_t v[kAt / 32][32];
                auto scores = [&](int c) {
#pragma unroll
                    for (int e = 0; e < kAt / 32; ++e)
                        tmem_ld_32x32b_x32(scol + c + 32 * e, v[e]);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < kAt / 32; ++e)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            reg_fence(v[e][j]);
                };
                float best = -INFINITY;
#pragma unroll
                for (int w = 0; w < NC / 32; w += kAt / 32) {
                    scores(32 * w);
#pragma unroll
                    for (int e = 0; e < kAt / 32; ++e)
                        best = fmaxf(best, whole ? max32<false>(v[e], 0u) : max32<true>(v[e], bits[w + e]));
                }
                const float top = best == -INFINITY ? -INFINITY : best * f;
                float alpha = 1.0f;
                if (top > m + kLag) {                          // (first keys: m is -inf)
                    alpha = ex2_approx(m - (top - kHead));
                    m = top - kHead;
                }
                // a raised maximum rescales O once the tile before is in it
                if (t > cur.t0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                    if (!(ok = wait_pv(gt - 1)))
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kDv; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(lanes + Sh::kO + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            reg_fence(o[j]);
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        }
                        tmem_st_32x32b_x32(lanes + Sh::kO + c, o);
                    }
                    tmem_st_wait();
                }
                const float m0 = m == -INFINITY ? 0.0f : m;
                float sum = 0.0f;
                const uint32_t pcol = lanes + slot * kKeys;
                // P over columns whose S has been read: 32 keys take 16 columns (kSplit: the
                // second copy's keys go to columns 32.., its S stands in columns 64..)
#pragma unroll
                for (int w = 0; w < NC / 32; w += kAt / 32) {
                    if (NC > kAt)
                        scores(32 * w);
#pragma unroll
                    for (int e = 0; e < kAt / 32; ++e) {
                        uint32_t pk[16];
                        sum += whole ? probs32<false>(v[e], 0u, f, m0, pk)
                                     : probs32<true>(v[e], bits[w + e], f, m0, pk);
                        tmem_st_32x32b_x16(pcol + NC / 2 * half + 16 * (w + e), pk);
                    }
                }
                if constexpr (kSplit) {
                    uint32_t z[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        z[j] = 0u;
#pragma unroll
                    for (int w = 0; w < NC / 32; ++w)
                        tmem_st_32x32b_x16(pcol + NC / 2 * (1 - half) + 16 * w, z);
                }
                l = l * alpha + sum;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars->p_full[slot]);
            }
            if (!ok)
                break;
        }
        begin(next);
        const bool real = cur.real;
        const long long at = cur.at;
        if (any) {
            if (!(ok = wait_pv(gt - 1)))
                break;
            tc_fence_after();
        }
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
        const long long piece = static_cast<long long>(cur.item) * kTileRows + row;
        float *dst = p.part + piece * kDv;
        __nv_bfloat16 *out = p.out + at * kDv;
        auto put = [&](int c, const float (&x)[kXCols]) {
            if (!real)
                return;
            if (part) {
#pragma unroll
                for (int j = 0; j < kXCols; j += 8) {
                    const uint32_t *u = reinterpret_cast<const uint32_t *>(x + j);
                    cache::store32(reinterpret_cast<uint8_t *>(dst + c + j), make_uint4(u[0], u[1], u[2], u[3]),
                                   make_uint4(u[4], u[5], u[6], u[7]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < kXCols; j += 16) {
                    uint32_t u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        u[e] = cache::bf16x2_of(x[j + 2 * e] * norm, x[j + 2 * e + 1] * norm);
                    cache::store32(reinterpret_cast<uint8_t *>(out + c + j), make_uint4(u[0], u[1], u[2], u[3]),
                                   make_uint4(u[4], u[5], u[6], u[7]));
                }
            }
        };
        auto take = [&](int c, float (&x)[kXCols]) {           // O's columns c.., scaled
            uint32_t o[kXCols];
            if (any) {
                tmem_ld_32x32b_x32(lanes + Sh::kO + c, o);
                tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < kXCols; ++j) {
                if (any)
                    reg_fence(o[j]);
                x[j] = any ? __uint_as_float(o[j]) * scale : 0.0f;
            }
        };
        if constexpr (kSplit) {
            // each copy writes half of the columns: its own plus the other's, sent kXCols at a time
            float *mine = xo + warp * kXCols * 32;
            const float *theirs = xo + (warp ^ 2) * kXCols * 32;
            for (int c = 0; c < kDv / 2; c += kXCols) {
                float x[kXCols];
                take((1 - half) * (kDv / 2) + c, x);
#pragma unroll
                for (int j = 0; j < kXCols; ++j)
                    mine[j * 32 + lane] = x[j];
                if (!(ok = pair_sync()))
                    break;
                take(half * (kDv / 2) + c, x);
#pragma unroll
                for (int j = 0; j < kXCols; ++j)
                    x[j] += theirs[j * 32 + lane];
                put(half * (kDv / 2) + c, x);
                if (!(ok = pair_sync()))                       // the buffer may be rewritten
                    break;
            }
            if (!ok)
                break;
        } else {
#pragma unroll 1
            for (int c = 0; c < kDv; c += kXCols) {
                float x[kXCols];
                take(c, x);
                put(c, x);
            }
        }
        if (real && half == 0) {
            if (part) {
                p.stat[piece] = make_float2(m, l);
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
        cur = next;
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
        mbar_init(&bars->o_empty, 4);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == kWideMmaWarp) {
        tmem_alloc(&bars->tmem_addr, 512);
        tmem_relinquish();
    }
    const WaitCtl ctl{&bars->abort, wp.wait_limit};
    next_kernel_may_begin();
    uint32_t tmem = 0;
    if (warp < 4) {
        regs_inc<kWideSoftmaxRegs>();
        wide_softmax<kDk, kDv, kSplit>(wp, smem, bars, ctl);
    } else if (warp < kWideMmaWarp) {
        regs_dec<kWideGatherRegs>();
        wide_gather<kDk, kDv>(wp, smem, bars, ctl, kTileRows);
    } else {
        regs_dec<kWideMmaRegs>();
        tmem = wide_ready(bars);
        if (warp == kWideMmaWarp && lane == 0)
            wide_mma<kDk, kDv>(wp, smem, bars, tmem, ctl, kTileRows);
    }
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
