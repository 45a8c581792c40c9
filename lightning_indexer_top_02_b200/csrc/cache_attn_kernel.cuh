// cache_attn_kernel.cuh -- attention over a cache held in 4 bits, few query
// rows per cached row (csa_cache_attention, include/csa_cache.h).
//
// The query rows that share cached rows (all the queries and heads of one
// cache head; with a selection, the heads of one query) go in tiles of 8 * kNT
// rows, the N of mma.m16n8k16; the cached rows are its M:
//   S^T [16 keys x 8 rows]  = K  [16 x Dk] . Q^T [Dk x 8]
//   O^T [16 dims x 8 rows] += V^T [16 x 16 keys] . P^T [16 keys x 8]
// With at most 16 rows the work is bound by reading the cache (9/16 byte an
// element against 4 rows' flops an element), so what matters is how few
// instructions stand between a code and its use.  A warp takes blocks of 64 keys (32 where
// a key and a value have more than 256 elements together); their codes and scales come one block
// ahead (two ahead) into the warp's own staging rows and go from there into registers in the layout of the MMA's A
// operand: no transposition, and no barrier between warps.
//   K: the contraction's order is free, so thread (g, t) of a warp takes the
//     16 * NG consecutive elements 16 * NG * t.. of the rows of its two keys --
//     whole scale groups, one wide load -- and the query fragments are laid
//     out to match.
//   V: a key's place in the tile is free too: thread (g, t) reads rows
//     4t .. 4t+3 of 16 keys (two of them swapped for t > 1, which keeps the reads
//     free of bank conflicts), elements VU * g.. of each; two keys' codes of one
//     dimension are merged into a byte (one and-or for eight codes) that
//     converts to the f16 pair that the A operand wants.
//   P^T: the S^T accumulator holds (key g, rows 2t, 2t+1); movmatrix
//     transposes the packed pairs into the B operand.
// Values are exact in f16: an E2M1 code times an E4M3 scale has six
// significant bits and lies within 2^-10 .. 2688 or is zero.  A query row is scaled by a
// power of two to a largest magnitude in [2^14, 2^15): what bf16 holds down to
// 2^-28 of it stays exact, smaller elements are off by at most 2^-39 of the largest.
// P is f16 (11 bits), relative to a reference 2^7 below the running maximum: the row's
// largest is 2^7 at first and 2^13 at most where the maximum lags, so that half of f16's
// smallest step is at most 2^-32 of the largest weight (relative to the maximum itself it would
// be 2^-25, and what 2^17 keys that far below one leave would be lost).  P's 11 bits move one
// bf16 output in ten by its last bit (relative difference 8.5e-4 to fp32 probabilities, distance
// from 64-bit values 1.670e-3 instead of 1.658e-3); more would take a second P . V.  Sums,
// maxima and O are fp32.
//
// Tensor-core work here is mma.sync on purpose: tcgen05 reads operands from
// shared memory, where writing the converted tile and reading it back would
// move 4 bytes an element for each 9/16 byte that memory delivers, more than
// shared memory's 128 bytes a clock allow at the memory's rate.
//
// Where every key is read and pages hold whole tiles of 16 keys (kBulk), a tile is
// 16 rows of one page, and a lane for each of a tile's four arrays (16 lanes a block of 64
// keys, 8 one of 32) fetches it with one bulk copy; else every row is found by itself and
// copied 16 bytes at a time.  Instructions are the same within 1 % (21.7 and 21.9 million at
// 8 sequences x 16,384 keys x 8 cache heads of 128).  Time there, bulk / row by row: 128+128
// 46.6 / 45.1 us, 192+128 55.3 / 57.7, 192+192 66.6 / 76.9, 128+256 66.0 / 65.3; 32 ragged
// sequences (below) 155 / 151; one of 777 keys 10.7 / 10.1.  So the bulk copies pay where
// rows have 192 elements (six pieces, staged without a conflict-free place) and cost up to
// 5 % elsewhere.
//
// Measured at 32 sequences of 512 .. 32,768 keys, 64 heads over 8, D = 128 (615 MB of
// cache): 155 us, 4.0 TB/s.  Memory alone (the arithmetic left out) takes 111 us, the
// arithmetic alone 115: some 1,330 instructions a block of 64 keys with everything around it,
// of which 512 are the conversions (128 + 128 of codes, 128 + 128 multiplications by scales, both
// on half-rate pipes).  12 warps an SM; 8 or 16 warps, deeper staging or shorter blocks were
// slower (150 -> 158 .. 188 us).
//
// The CTAs that the GPU holds share out all the chunks (256 or 128 keys) of all row tiles,
// evenly and in order, whatever the sequences' lengths: a CTA's share is a run of
// chunks, which ends one tile, takes whole ones and begins another.  In a tile the
// warps take blocks of keys in turn and keep their own running maxima, sums and O,
// which are joined in shared memory; the pieces of a tile that several CTAs share
// are joined by a second kernel.
#pragma once
#include "cache_common.cuh"
#include "ptx.cuh"

namespace csa {
namespace cattn {

using cache::CacheView;
using cache::FastDiv;
using cache::PageMap;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kHead = 7.0f;               // a row's reference: its maximum / 2^kHead when it was last raised
constexpr float kLag = 13.0f;               // and it is raised when a weight would pass 2^kLag (f16: below 2^16)
constexpr int kNoKey = 0x7FFFFFFF;          // a position no query sees
constexpr int kStatic = 128;                // static shared memory of a block, at most

struct AttnParams {
    const __nv_bfloat16 *q;                 // [B, S, HA, Dk]
    CacheView ck, cv;
    PageMap pm;
    const int32_t *kv_len;
    const int32_t *idx;                     // [B, S, topk] or null
    int topk;
    int B, S, HA, H, G;                     // G = HA / H
    int causal;
    float sl2;                              // scale * k tensor scale * log2(e) / 2^kQueryBits
    float v_scale;
    __nv_bfloat16 *out;
    float *lse;
    long long wait_limit;
    int splits;                             // wide kernel: shares of the keys
    int ctas;                               // CTAs that share the chunks; 0: one a row tile
    int most;                               // chunks of a row tile, at most
    int works;                              // row tiles of a sequence
    int chunk;                              // keys that are shared out together
    int tiles;                              // row tiles of a group
    int rows;                               // query rows of a group: S * G, or G with idx
    int capacity;                           // positions the page table reaches
    float *part;                            // [piece][rows of a tile][Dv]: O before it is divided
    float2 *stat;                           // [piece][rows of a tile]: its maximum (log2) and sum
    FastDiv div_splits, div_tiles, div_H, div_S, div_G;
};

// The group of query rows that a work item belongs to.
struct Group {
    int b, h, i0;                           // sequence, cache head, first query
    int r0;                                 // first row of the tile
};

__device__ __forceinline__ Group group_of(const AttnParams &p, int w, int tile_rows)
{
    Group g;
    int q = static_cast<int>(p.div_tiles.div(w));
    g.r0 = (w - q * p.tiles) * tile_rows;
    w = q;
    q = static_cast<int>(p.div_H.div(w));
    g.h = w - q * p.H;
    g.b = q;
    g.i0 = 0;
    if (p.idx) {
        g.b = static_cast<int>(p.div_S.div(q));
        g.i0 = q - g.b * p.S;
    }
    return g;
}

// Query and head of row r of a group.
__device__ __forceinline__ void row_of(const AttnParams &p, const Group &g, int r, int &i, int &head)
{
    const int k = static_cast<int>(p.div_G.div(r));
    i = g.i0 + k;
    head = g.h * p.G + r - k * p.G;
}

// Positions below this are seen by query i (len > 0).
__device__ __forceinline__ int seen(const AttnParams &p, int len, int i)
{
    return p.causal ? len - p.S + i + 1 : len;
}

// 16-byte piece q of a row among rows of kQ pieces: where it is staged, so that
// eight rows' pieces q lie in eight different 16-byte places of a bank row.
template <int kQ>
__device__ __forceinline__ uint32_t staged_at(int r, int q)
{
    const int x = kQ == 2 ? (r >> 2) & 1 : kQ == 4 ? (r >> 1) & 3 : kQ == 8 ? r & 7 : 0;
    return static_cast<uint32_t>((r * kQ + (q ^ x)) * 16);
}

__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

template <int kBytes>
__device__ __forceinline__ void cp_async_small_zfill(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes),
                 "r"(ok ? kBytes : 0)
                 : "memory");
}

// Copies kRows rows of one operand to the warp's staging: a lane's piece is 16
// bytes (32 elements) of a row.  Lane r < kRows holds row r's address; rows whose bit in
// `has` is clear are staged as zeros.
template <int kD, int kRows>
__device__ __forceinline__ void stage_codes(uint32_t codes, const uint8_t *row, uint32_t has, int lane)
{
    constexpr int kQ = kD / 32, kN = kQ * kRows;          // pieces of a row, and in all
    static_assert(kRows % 8 == 0, "eight lanes in a row take eight rows");
#pragma unroll
    for (int k = 0; k < (kN + 31) / 32; ++k) {
        const int combo = 4 * k + (lane >> 3);
        const int q = combo % kQ, r = (lane & 7) + 8 * (combo / kQ);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r & (kRows - 1)));
        if (kN % 32 == 0 || combo < kN / 8)
            cp_async_zfill(codes + staged_at<kQ>(r, q), src + 16 * q, has >> r & 1u);
    }
}

template <int kD>
__device__ __forceinline__ void stage_scales(uint32_t scales, int r, const uint8_t *src, bool ok)
{
    constexpr int kS = kD / 16;                           // scale bytes of a row
    if constexpr (kS == 16) {
        cp_async_zfill(scales + r * kS, src, ok);
    } else if constexpr (kS == 8) {
        cp_async_small_zfill<8>(scales + r * kS, src, ok);
    } else {
#pragma unroll
        for (int j = 0; j < kS; j += 4)
            cp_async_small_zfill<4>(scales + r * kS + j, src + j, ok);
    }
}

// Addresses of row `row` (head * page_size + offset) of a page; page < 0: of page 0.
__device__ __forceinline__ const uint8_t *data_at(const CacheView &c, int page, int row)
{
    return c.data + max(page, 0) * c.page_stride + static_cast<long long>(row) * c.row_bytes;
}

__device__ __forceinline__ const uint8_t *scale_at(const CacheView &c, int page, int row)
{
    return c.scale + max(page, 0) * c.scale_stride + static_cast<long long>(row) * c.scale_bytes;
}

// 16 * n bytes global -> shared by the copy engine, counted on `bar`.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// N bytes of staged row r from byte `at` on (whole pieces, or within one; rows of
// kQ = 6 pieces, and bulk copies, are staged as they are).
template <int kQ, bool kBulk>
__device__ __forceinline__ uint32_t staged(int r, int q)
{
    return kBulk ? static_cast<uint32_t>((r * kQ + q) * 16) : staged_at<kQ>(r, q);
}

template <int kQ, int N, bool kBulk>
__device__ __forceinline__ void read_staged(const uint8_t *rows, int r, int at, uint32_t (&w)[(N + 3) / 4])
{
    if constexpr (N % 16 == 0) {
#pragma unroll
        for (int j = 0; j < N / 16; ++j) {
            const uint4 v = *reinterpret_cast<const uint4 *>(rows + staged<kQ, kBulk>(r, (at >> 4) + j));
            w[4 * j] = v.x;
            w[4 * j + 1] = v.y;
            w[4 * j + 2] = v.z;
            w[4 * j + 3] = v.w;
        }
    } else if constexpr (N % 8 == 0) {
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
            const int b = at + 8 * j;
            const uint2 v = *reinterpret_cast<const uint2 *>(rows + staged<kQ, kBulk>(r, b >> 4) + (b & 15));
            w[2 * j] = v.x;
            w[2 * j + 1] = v.y;
        }
    } else {
        static_assert(N == 4, "4, 8 or 16 bytes at a time");
        w[0] = *reinterpret_cast<const uint32_t *>(rows + staged<kQ, kBulk>(r, at >> 4) + (at & 15));
    }
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A query row of largest magnitude `peak` is held in f16 times `down`, a power of two: its largest
// is then in [2^14, 2^15), or smaller for a peak below 2^-112.  2^14 / down is `up`, both are normal
// numbers, and 2^-14 is part of AttnParams::sl2 (as a step of its own here it cost the wide kernel
// 1.1 us of 27 at 32 sequences x 128 heads x 2,048 keys).
constexpr int kQueryBits = 14;
__device__ __forceinline__ void query_scale(float peak, float &down, float &up)
{
    const int e = min(max(static_cast<int>(__float_as_uint(peak) >> 23), kQueryBits), 254);
    down = __uint_as_float(static_cast<uint32_t>(254 + kQueryBits - e) << 23);
    up = __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Byte j (constant after unrolling) of a packed word as an f16 pair.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int j)
{
    switch (j) {
    case 0: return cache::f16x2_of_e2m1x2<0>(w);
    case 1: return cache::f16x2_of_e2m1x2<1>(w);
    case 2: return cache::f16x2_of_e2m1x2<2>(w);
    default: return cache::f16x2_of_e2m1x2<3>(w);
    }
}

template <int kDk, int kDv, int kNT>
struct Shape {
    static constexpr int NG = kDk / 64;                  // K: scale groups a thread takes of a row
    static constexpr int VU = kDv % 128 == 0 ? 16 : 8;   // V: consecutive elements a thread takes
    static constexpr int NU = kDv / (8 * VU);            // and how many times
    static constexpr int MT = kDv / 16;                  // output m-tiles
    static constexpr int kRows = 8 * kNT;
    // keys a warp takes at a time: what a block costs beside its keys (finding, copying
    // and waiting, about 170 instructions) is spread over 64 where shared memory allows
    static constexpr int kBlock = kDk + kDv <= 256 ? 64 : 32;
    static constexpr int kTiles = kBlock / 16, kSets = kBlock / 32;      // MMA tiles; keys a lane looks up
    static constexpr int kStages = kBlock == 64 ? 2 : 3;                 // blocks in use and on their way
    static constexpr int kChunk = kBlock * kWarps;                       // keys that are shared out together
    // staging of a block: K codes, V codes, K scales, V scales
    static constexpr int kV = kBlock * kDk / 2, kKs = kV + kBlock * kDv / 2;
    static constexpr int kVs = kKs + kBlock * kDk / 16, kStage = kVs + kBlock * kDv / 16;
    // the warps' joined results take the staging's place
    static constexpr int kJoin = kWarps * kRows * (kDv + 2) * 4, kStaging = kWarps * kStages * kStage;
    static constexpr int kBars = kJoin > kStaging ? kJoin : kStaging;    // barriers, abort flag
    static constexpr int kSmem = kBars + kWarps * kStages * 8 + 16;
    // blocks an SM holds: as many as its 228 KB take beside a block's own kilobyte and static words
    // (three up to widths of 320 together, two beyond), at most those whose O and query find registers.
    // (Shares for one CTA more than the SMs hold run in a second round: 8 sequences of 16,384 keys, 8 cache
    // heads of 192 + 192, take 92 us with three planned and 66 with two.)
    static constexpr int kHeld = 233472 / (kSmem + 1024 + kStatic);
    static constexpr int kCtas = kHeld < (kNT == 1 ? 3 : 2) ? kHeld : (kNT == 1 ? 3 : 2);
    static_assert(kCtas >= 1, "a block fits an SM");
};

// The kernel that joins the pieces may take the SMs' free places from here on.
__device__ __forceinline__ void next_kernel_may_begin()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Chunks of one row tile of sequence b.  (A tile of early queries sees less of the
// sequence; the chunks past that find nothing to do.)
__device__ __forceinline__ int chunks_of(const AttnParams &p, int b)
{
    const int len = __ldg(p.kv_len + b);
    const int n = len > 0 ? (p.idx ? p.topk : min(len, p.capacity)) : 0;
    return static_cast<int>((static_cast<unsigned>(n) + p.chunk - 1) / p.chunk);   // (a power of two)
}

// Sum over the block's kThreads threads (scratch: kWarps words).
__device__ __forceinline__ long long block_sum(long long v, long long *scratch)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return scratch[0] + scratch[1] + scratch[2] + scratch[3];
}
static_assert(kWarps == 4, "block_sum");

// Chunks of the sequences before `upto`.
__device__ __forceinline__ long long chunks_before(const AttnParams &p, int upto, long long *scratch)
{
    long long v = 0;
    for (int b = threadIdx.x; b < upto; b += kThreads)
        v += chunks_of(p, b);
    return block_sum(v, scratch) * p.works;
}

// The sequence that holds chunk x of all, and x's place in it (found: shared memory).
struct Found {
    int b;
    long long y;
};

__device__ __forceinline__ void find_chunk(const AttnParams &p, long long x, Found *found, long long *scratch)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long carry = 0;
    if (threadIdx.x == 0)
        *found = Found{0, 0};                            // (lengths that changed meanwhile: x may be nowhere)
    for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + threadIdx.x;
        const long long v = b < p.B ? static_cast<long long>(chunks_of(p, b)) * p.works : 0;
        long long upto = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, upto, d);
            upto += lane >= d ? u : 0;
        }
        __syncthreads();
        if (lane == 31)
            scratch[warp] = upto;
        __syncthreads();
        long long start = carry + upto - v;
        for (int w = 0; w < kWarps; ++w) {
            start += w < warp ? scratch[w] : 0;
            carry += scratch[w];
        }
        if (x >= start && x < start + v) {
            found->b = b;
            found->y = x - start;
        }
    }
    __syncthreads();
}

// The CTA whose share holds chunk x of `total`: shares start at total * k / ctas.
__device__ __forceinline__ int cta_of(long long x, long long total, int ctas)
{
    return static_cast<int>(((x + 1) * ctas - 1) / total);
}

template <int kDk, int kDv, int kNT, bool kBulk>
__global__ void __launch_bounds__(kThreads, Shape<kDk, kDv, kNT>::kCtas)
    cache_attn_kernel(const AttnParams p)
{
    using Sh = Shape<kDk, kDv, kNT>;
    constexpr int NG = Sh::NG, VU = Sh::VU, NU = Sh::NU, MT = Sh::MT, RT = Sh::kRows;
    constexpr int kBlock = Sh::kBlock, kTiles = Sh::kTiles, kSets = Sh::kSets, kStages = Sh::kStages;
    extern __shared__ __align__(16) uint8_t smem_raw[];  // staging, then [warp][row][Dv + 2]
    __shared__ long long scratch[kWarps];
    __shared__ Found found;
    static_assert(sizeof(scratch) + sizeof(found) <= kStatic, "kStatic");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + Sh::kBars) + warp * kStages;
    int *abort = reinterpret_cast<int *>(smem_raw + Sh::kBars + kWarps * kStages * 8);
    const WaitCtl ctl{abort, p.wait_limit};
    if constexpr (kBulk) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s)
                mbar_init(&bars[s], 1);
            fence_mbar_init();
        }
        if (threadIdx.x == 0)
            *abort = 0;
    }
    __syncthreads();
    next_kernel_may_begin();
    // the CTA's share: `left` chunks from chunk y of sequence `seq` on
    long long left = p.most, y = 0;
    int seq = 0;
    if (p.ctas) {
        const long long total = chunks_before(p, p.B, scratch);
        const int ctas = static_cast<int>(min(static_cast<long long>(p.ctas), total));   // no share is empty
        left = 0;
        if (blockIdx.x < ctas) {
            const long long x = total * blockIdx.x / ctas;
            left = total * (blockIdx.x + 1) / ctas - x;
            find_chunk(p, x, &found, scratch);
            seq = found.b;
            y = found.y;
        }
        // sequences without a key: zeros
        for (int b = blockIdx.x; b < p.B; b += p.ctas) {
            if (chunks_of(p, b) > 0)
                continue;
            const long long at = static_cast<long long>(b) * p.S * p.HA, n = static_cast<long long>(p.S) * p.HA;
            for (long long e = threadIdx.x; e < n * (kDv / 8); e += kThreads)
                reinterpret_cast<uint4 *>(p.out + at * kDv)[e] = make_uint4(0u, 0u, 0u, 0u);
            for (long long e = threadIdx.x; p.lse && e < n; e += kThreads)
                p.lse[at + e] = -INFINITY;
        }
    }
    uint32_t phase = 0;                                  // of the staging barriers
    int at = 0;                                          // stage of the next block
    while (left > 0) {
        int work = blockIdx.x, lo = 0, hi = p.most, all = p.most;   // the segment: chunks lo .. hi - 1 of `all`
        if (p.ctas) {
            // (lengths that change meanwhile are not allowed, but lead neither out of the
            // batch nor into an endless loop)
            all = seq < p.B ? chunks_of(p, seq) : 0;
            if (all <= 0 || y >= static_cast<long long>(all) * p.works)
                break;
            const int w = static_cast<int>(y / all);
            lo = static_cast<int>(y - static_cast<long long>(w) * all);
            hi = static_cast<int>(min(static_cast<long long>(all), lo + left));
            work = seq * p.works + w;
            y += hi - lo;
            if (y == static_cast<long long>(all) * p.works) {
                y = 0;
                do
                    ++seq;
                while (seq < p.B && chunks_of(p, seq) == 0);
            }
        }
        left -= hi - lo;
        const Group gr = group_of(p, work, RT);
        const int len = __ldg(p.kv_len + gr.b);
        const int32_t *table = p.pm.table + gr.b * p.pm.table_stride;
        const int32_t *list = p.idx ? p.idx + (static_cast<long long>(gr.b) * p.S + gr.i0) * p.topk : nullptr;

        // the tile's rows: what the last and the first of them see
        const int r_last = min(gr.r0 + RT, p.rows) - 1;
        const int see_hi = len > 0 ? seen(p, len, gr.i0 + static_cast<int>(p.div_G.div(r_last))) : 0;
        const int see_lo = len > 0 ? seen(p, len, gr.i0 + static_cast<int>(p.div_G.div(gr.r0))) : 0;
        const int slots = p.idx ? (see_hi > 0 ? p.topk : 0) : min(max(see_hi, 0), p.capacity);
        const int blocks = (slots + kBlock - 1) / kBlock;
        const int b_lo = lo * kWarps, b_hi = min(hi * kWarps, blocks);

        // query fragments: row g of each n-tile, elements 16 NG t.., scaled by a power of two
        uint32_t qf[kNT][4 * NG][2];
        float f[kNT][2];                                     // factor of rows 2t, 2t+1 (log2 domain)
        int lim[kNT][2];                                     // and the positions they see
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
            const int r = gr.r0 + 8 * n + g;
            float x[16 * NG];
            float peak = 0.0f;
            int i = 0, head = 0;
            if (r < p.rows) {
                row_of(p, gr, r, i, head);
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    p.q + ((static_cast<long long>(gr.b) * p.S + i) * p.HA + head) * kDk + 16 * NG * t);
#pragma unroll
                for (int j = 0; j < 2 * NG; ++j) {
                    const uint4 w = __ldg(src + j);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = cache::float2_of_bf16x2(u[e]);
                        x[8 * j + 2 * e] = v.x;
                        x[8 * j + 2 * e + 1] = v.y;
                        peak = fmaxf(peak, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16 * NG; ++j)
                    x[j] = 0.0f;
            }
            peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
            peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 2));
            float down, up;
            query_scale(peak, down, up);
            if (p.sl2 < 0.0f)
                down = -down;
#pragma unroll
            for (int s = 0; s < 4 * NG; ++s) {
                qf[n][s][0] = f16x2_of(x[4 * s] * down, x[4 * s + 1] * down);
                qf[n][s][1] = f16x2_of(x[4 * s + 2] * down, x[4 * s + 3] * down);
            }
            // the scale's sign goes with the query, and the factor is not zero, so that a masked
            // score times it is -inf
            const float fr = fmaxf(up * fabsf(p.sl2), 1.17549435e-38f);
            const int see = r < p.rows && len > 0 ? seen(p, len, i) : 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f[n][c] = __shfl_sync(0xffffffffu, fr, 4 * (2 * t + c));
                lim[n][c] = __shfl_sync(0xffffffffu, see, 4 * (2 * t + c));
            }
        }

        float o[MT][kNT][4];
        float m[kNT][2], l[kNT][2];
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[j][n][c] = 0.0f;
        }

        // rows of a tile of 16 keys: K rows k0, k0 + 2 (MMA rows g, g + 8), V rows 4t + (0, 1, 2, 3)
        // with the pairs swapped for t > 1
        const int k0 = 4 * (g >> 1) + ((g & 1) ^ (g >> 2));
        const int v0 = 4 * t + (t >> 1), v1 = 4 * t + 1 - (t >> 1);
        uint8_t *stage = smem_raw + warp * kStages * Sh::kStage;

        // Bulk: lane kTiles * a + i copies array a (K codes, V codes, K scales, V scales) of tile i.
        const int tile = lane % kTiles, array = lane / kTiles;
        const CacheView &view = array & 1 ? p.cv : p.ck;
        const int b_row = array < 2 ? view.row_bytes : view.scale_bytes;
        const long long b_page = array < 2 ? view.page_stride : view.scale_stride;
        const uint8_t *b_base = (array < 2 ? view.data : view.scale) + static_cast<long long>(gr.h) * p.pm.page_size * b_row;
        const int b_to = (array == 0 ? 0 : array == 1 ? Sh::kV : array == 2 ? Sh::kKs : Sh::kVs) + tile * 16 * b_row;

        // A lane's keys of a block (bulk: its tile), found ahead of the copies: first the
        // position, then its page.  Nothing that a load brought is looked at before the
        // step that needs it.
        constexpr int kLook = kBulk ? 1 : kSets;
        int pos_f[kLook], pos_p[kLook], page_p[kLook], off_p[kLook];
        auto fetch_pos = [&](int blk) {
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                pos_f[i] = -1;
                if (blk < b_hi) {
                    const int slot = blk * kBlock + (kBulk ? 16 * tile : 32 * i + lane);
                    if (slot < slots)
                        pos_f[i] = !kBulk && list ? __ldg(list + slot) : slot;
                }
            }
        };
        auto fetch_page = [&]() {
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const bool in = pos_f[i] >= 0 && pos_f[i] < see_hi;
                const int n = in ? static_cast<int>(p.pm.div.div(pos_f[i])) : 0;
                const bool has = in && n < p.pm.max_pages;
                page_p[i] = has ? __ldg(table + n) : -1;
                off_p[i] = has ? pos_f[i] - n * p.pm.page_size : 0;
                pos_p[i] = pos_f[i];
            }
        };
        // starts a block's copies; pos: the lane's positions in it (kNoKey: none)
        auto start = [&](int blk, int at, int (&pos)[kSets]) {
#pragma unroll
            for (int i = 0; i < kSets; ++i)
                pos[i] = kNoKey;
            if (blk < b_hi) {
                const uint32_t to = smem_u32(stage + at * Sh::kStage);
                if constexpr (kBulk) {
                    const bool ok = page_p[0] >= 0 && page_p[0] < p.pm.num_pages;
                    const uint32_t has = __ballot_sync(0xffffffffu, ok) & ((1u << kTiles) - 1u);
#pragma unroll
                    for (int i = 0; i < kSets; ++i) {
                        const int slot = blk * kBlock + 32 * i + lane;
                        if (has >> (2 * i + (lane >> 4)) & 1u && slot < slots)
                            pos[i] = slot;
                    }
                    if (lane == 0)
                        mbar_arrive_expect_tx(&bars[at], Sh::kStage / kTiles * __popc(has));
                    __syncwarp();
                    if (lane < 4 * kTiles && ok)
                        bulk_copy(to + b_to, b_base + page_p[0] * b_page + static_cast<long long>(off_p[0]) * b_row,
                                  16 * b_row, &bars[at]);
                } else {
#pragma unroll
                    for (int i = 0; i < kSets; ++i) {
                        const int page = page_p[i] >= 0 && page_p[i] < p.pm.num_pages ? page_p[i] : -1;
                        const int row = gr.h * p.pm.page_size + off_p[i];
                        const uint32_t has = __ballot_sync(0xffffffffu, page >= 0);
                        pos[i] = page >= 0 ? pos_p[i] : kNoKey;
                        stage_codes<kDk, 32>(to + 16 * i * kDk, data_at(p.ck, page, row), has, lane);
                        stage_codes<kDv, 32>(to + Sh::kV + 16 * i * kDv, data_at(p.cv, page, row), has, lane);
                        stage_scales<kDk>(to + Sh::kKs + 2 * i * kDk, lane, scale_at(p.ck, page, row), page >= 0);
                        stage_scales<kDv>(to + Sh::kVs + 2 * i * kDv, lane, scale_at(p.cv, page, row), page >= 0);
                    }
                }
            }
            if constexpr (!kBulk)
                asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto after = [](int s) { return s == kStages - 1 ? 0 : s + 1; };
        // all but one stage are filled before the first block, one block behind another
        int blk = b_lo + warp, pos[kStages][kSets], to = at;
        fetch_pos(blk);
        fetch_page();
        fetch_pos(blk + kWarps);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            start(blk + i * kWarps, to, pos[i]);
            fetch_page();
            fetch_pos(blk + (i + 2) * kWarps);
            to = after(to);
        }
        for (; blk < b_hi; blk += kWarps) {
            // the stage that the block before has left takes the next copies
            start(blk + (kStages - 1) * kWarps, to, pos[kStages - 1]);
            fetch_page();
            fetch_pos(blk + (kStages + 1) * kWarps);
            if constexpr (kBulk) {
                const bool landed = wait_bounded(&bars[at], phase, ctl, 30, blk);
                if (!__all_sync(0xffffffffu, landed))
                    break;
                // what lies behind the sequence in its page may be anything, a NaN scale too:
                // those keys' P is zero, so their V is made zero
                bool all_there = true;
#pragma unroll
                for (int i = 0; i < kSets; ++i)
                    all_there = all_there && pos[0][i] != kNoKey;
                if (!__all_sync(0xffffffffu, all_there)) {
#pragma unroll
                    for (int i = 0; i < kSets; ++i)
                        if (pos[0][i] == kNoKey)
                            for (int j = 0; j < kDv / 16; j += 4)
                                *reinterpret_cast<uint32_t *>(stage + at * Sh::kStage + Sh::kVs +
                                                              (32 * i + lane) * (kDv / 16) + j) = 0u;
                    fence_proxy_async_smem();                      // before the stage's next copies
                    __syncwarp();
                }
            } else {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");   // this block's have landed
                __syncwarp();                                      // every lane's
            }
            const uint8_t *cur = stage + at * Sh::kStage;
            phase ^= at == kStages - 1;
            at = after(at);
            to = after(to);
            // S^T of the tiles of 16 keys, two at a time: their MMAs' chains of sums alternate
            float s[kTiles][kNT][4];
#pragma unroll
            for (int a0 = 0; a0 < kTiles; a0 += 2) {
                uint32_t kw[2][2][2 * NG], sc[2][2][NG];      // [tile][row]: the thread's parts of its rows
#pragma unroll
                for (int a = 0; a < 2; ++a) {
#pragma unroll
                    for (int n = 0; n < kNT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            s[a0 + a][n][c] = 0.0f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 16 * (a0 + a) + k0 + 2 * e;
                        read_staged<kDk / 32, 8 * NG, kBulk>(cur, r, 8 * NG * t, kw[a][e]);
                        const uint8_t *s8 = cur + Sh::kKs + r * (kDk / 16) + NG * t;
#pragma unroll
                        for (int c = 0; c < NG; c += 2) {     // scales, each in both halves
                            const uint32_t two = cache::f16x2_of_e4m3x2(
                                NG % 2 == 0 ? *reinterpret_cast<const uint16_t *>(s8 + c)
                                            : s8[c] | (c + 1 < NG ? s8[c + 1] << 8 : 0));
                            sc[a][e][c] = __byte_perm(two, 0u, 0x1010);
                            if (c + 1 < NG)
                                sc[a][e][c + 1] = __byte_perm(two, 0u, 0x3232);
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < NG; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            const uint32_t w0 = kw[a][0][2 * c + (q >> 1)], w1 = kw[a][1][2 * c + (q >> 1)];
                            const int j = 2 * (q & 1);
                            const uint32_t x0 = hmul2(pair_of(w0, j), sc[a][0][c]);
                            const uint32_t x1 = hmul2(pair_of(w1, j), sc[a][1][c]);
                            const uint32_t x2 = hmul2(pair_of(w0, j + 1), sc[a][0][c]);
                            const uint32_t x3 = hmul2(pair_of(w1, j + 1), sc[a][1][c]);
#pragma unroll
                            for (int n = 0; n < kNT; ++n)
                                mma16816(s[a0 + a][n], x0, x1, x2, x3, qf[n][4 * c + q][0], qf[n][4 * c + q][1]);
                        }
            }
            // masks: the positions of the thread's keys
            bool seen_all = true;
#pragma unroll
            for (int i = 0; i < kSets; ++i)
                seen_all = seen_all && pos[0][i] < see_lo;
            if (!__all_sync(0xffffffffu, seen_all)) {
#pragma unroll
                for (int a = 0; a < kTiles; ++a)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at_key = __shfl_sync(0xffffffffu, pos[0][a >> 1], 16 * (a & 1) + k0 + 2 * e);
#pragma unroll
                        for (int n = 0; n < kNT; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (at_key >= lim[n][c])
                                    s[a][n][2 * e + c] = -INFINITY;
                    }
            }
            bool raise = false;
            float top[kNT][2];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float best = -INFINITY;
#pragma unroll
                    for (int a = 0; a < kTiles; ++a)
                        best = fmaxf(best, fmaxf(s[a][n][c], s[a][n][2 + c]));
                    top[n][c] = best * f[n][c];
                    raise = raise || top[n][c] > m[n][c] + kLag;   // (-inf > -inf is false)
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float best = top[n][c];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
                        best -= kHead;
                        if (best > m[n][c]) {
                            const float a = ex2_approx(m[n][c] - best);   // first keys: 2^-inf = 0
                            m[n][c] = best;
                            l[n][c] *= a;
#pragma unroll
                            for (int j = 0; j < MT; ++j) {
                                o[j][n][c] *= a;
                                o[j][n][2 + c] *= a;
                            }
                        }
                    }
            }
            // P, its sums, and P^T as the B operand
            uint32_t pb[kTiles][kNT][2];
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                // a row without a key yet: 2^-inf is 0
                const float m0 = m[n][0] == -INFINITY ? 0.0f : m[n][0];
                const float m1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
#pragma unroll
                for (int a = 0; a < kTiles; ++a)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = ex2_approx(fmaf(s[a][n][2 * e], f[n][0], -m0));
                        const float p1 = ex2_approx(fmaf(s[a][n][2 * e + 1], f[n][1], -m1));
                        l[n][0] += p0;
                        l[n][1] += p1;
                        pb[a][n][e] = transpose8x8(f16x2_of(p0, p1));
                    }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int a = 0; a < kTiles; ++a)
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    uint32_t vw[4][VU / 8], sc[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        read_staged<kDv / 32, VU / 2, kBulk>(cur + Sh::kV, 16 * a + ((e & 1) ? v1 : v0) + (e & 2), 4 * VU * u + (VU / 2) * g,
                                                      vw[e]);
                    const uint8_t *s8 = cur + Sh::kVs + (VU / 2) * u + (VU * g) / 16;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        sc[e] = cache::f16x2_of_e4m3x2(s8[(16 * a + v0 + 2 * e) * (kDv / 16)] |
                                                       s8[(16 * a + v1 + 2 * e) * (kDv / 16)] << 8);
#pragma unroll
                    for (int w = 0; w < VU / 8; ++w) {
                        uint32_t lo[2], hi[2];              // even and odd dimensions, a byte = two keys
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = vw[2 * e][w], y = vw[2 * e + 1][w];
                            lo[e] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
                            hi[e] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a0 = hmul2(pair_of(lo[0], j), sc[0]), a1 = hmul2(pair_of(hi[0], j), sc[0]);
                            const uint32_t a2 = hmul2(pair_of(lo[1], j), sc[1]), a3 = hmul2(pair_of(hi[1], j), sc[1]);
#pragma unroll
                            for (int n = 0; n < kNT; ++n)
                                mma16816(o[(VU / 2) * u + 4 * w + j][n], a0, a1, a2, a3, pb[a][n][0], pb[a][n][1]);
                        }
                    }
                }
#pragma unroll
            for (int i = 0; i + 1 < kStages; ++i)
#pragma unroll
                for (int j = 0; j < kSets; ++j)
                    pos[i][j] = pos[i + 1][j];
            __syncwarp();                                          // the block's stage is free
        }
        // after a wait that ran out: the copies still on their way land before the CTA goes on
        for (int s = at, ph = phase; kBulk && blk < b_hi; blk += kWarps) {
            wait_drain(&bars[s], ph);
            ph ^= s == kStages - 1;
            s = after(s);
            if (s == at)
                break;
        }
        cp_async_wait_all();
        __syncthreads();                                     // the staging becomes the join's buffer
        const bool failed = kBulk && *ctl.abort;             // (the same for every warp)

        // join the warps: every warp's O, maxima and sums go to shared memory
        float *smem = reinterpret_cast<float *>(smem_raw);
        float *mine = smem + warp * RT * (kDv + 2);
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float sum = l[n][c];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, d);
                float *row = mine + (8 * n + 2 * t + c) * (kDv + 2);
                if (g == 0) {
                    row[kDv] = m[n][c];
                    row[kDv + 1] = sum;
                }
                // m-tile j of unit u: rows g, g + 8 are dimensions 8 VU u + VU g + 2j, + 1
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const int d = 8 * VU * (j / (VU / 2)) + VU * g + 2 * (j % (VU / 2));
                    *reinterpret_cast<float2 *>(row + d) = make_float2(o[j][n][c], o[j][n][2 + c]);
                }
            }
        __syncthreads();
        for (int r = warp; r < RT && gr.r0 + r < p.rows; r += kWarps) {
            const float *row = smem + r * (kDv + 2);
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top = fmaxf(top, row[w * RT * (kDv + 2) + kDv]);
            float a[kWarps], sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *wr = row + w * RT * (kDv + 2);
                a[w] = top == -INFINITY ? 0.0f : ex2_approx(wr[kDv] - top);
                sum += a[w] * wr[kDv + 1];
            }
            if (hi - lo < all) {
                // a piece: the CTA's first one ends a tile that another began, or it begins one
                const long long piece = static_cast<long long>(2 * blockIdx.x + (lo > 0 ? 0 : 1)) * RT + r;
                float *dst = p.part + piece * kDv;
                for (int d = lane; d < kDv; d += 32) {
                    float x = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        x += a[w] * row[w * RT * (kDv + 2) + d];
                    dst[d] = x;
                }
                if (lane == 0)
                    p.stat[piece] = make_float2(top, sum);
                continue;
            }
            int i, head;
            row_of(p, gr, gr.r0 + r, i, head);
            const long long out_row = (static_cast<long long>(gr.b) * p.S + i) * p.HA + head;
            const float inv = sum > 0.0f ? p.v_scale / sum : 0.0f;
            for (int d = lane; d < kDv; d += 32) {
                float x = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    x += a[w] * row[w * RT * (kDv + 2) + d];
                p.out[out_row * kDv + d] = __float2bfloat16_rn(x * inv);
            }
            if (p.lse && lane == 0)
                p.lse[out_row] = sum > 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        }
        fence_proxy_async_smem();                            // before the next segment's bulk copies
        __syncthreads();
        if (failed)
            break;
    }
}

} // namespace cattn
} // namespace csa
