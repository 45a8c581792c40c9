/*
 * csa_cache.h -- C ABI of the cache operators beside the indexer: rotary
 * positions, appending keys and values to a paged cache (the rotation applied
 * on the way), reading cached rows back as bf16, and attention over a cache
 * held in 4 bits.  Status codes, streams and error behaviour are those of
 * csa_indexer.h: every call validates its arguments before any launch, is
 * stream-ordered on `stream`, allocates nothing unless stated, never throws
 * and never synchronises.  Kernels run on the current device, which the
 * pointers must belong to.  Floating-point inputs must be finite (other
 * values give unspecified but memory-safe results), except where a row is
 * masked: what lies in a cache outside a sequence's rows is never used.  Lengths, page
 * tables and lists must not change while a call's work runs (results are then
 * unspecified, the access stays within the caches and outputs).
 *
 * The cache.  A page holds page_size rows for each of H heads, head by head:
 * row o of head h in page p starts at
 *   data  + p * page_stride       + (h * page_size + o) * (bytes of a row)
 *   scale + p * scale_page_stride + (h * page_size + o) * (scale bytes of a row)
 * and holds the D elements x of one position:
 *   CSA_CACHE_BF16  D bf16 values; no scale
 *   CSA_CACHE_E4M3  D bytes and one fp32 scale: x ~ scale * E4M3, scale =
 *                   max|x| / 448 (1 where that is 0 in fp32) -- the indexer's keys:
 *                   with H = 1 and one page of T rows a sequence, data is
 *                   csa_indexer's k [B,T,d] and scale its k_scale [B,T]
 *   CSA_CACHE_E2M1  D/2 bytes (the even element in a byte's low half) and
 *                   D/16 E4M3 scale bytes, one for 16 elements:
 *                   x ~ tensor_scale * E4M3 scale * E2M1, scale =
 *                   max|x| / (6 * tensor_scale) rounded to E4M3 (at most 448)
 * Rounding is to nearest, ties to even, and saturates.
 *
 * Position s of sequence b is row s % page_size of page
 * page_table[b * table_stride + s / page_size].  A position past max_pages
 * pages, or whose entry is outside [0, num_pages), has no row: an append
 * drops it, a read gives zeros, attention does not see it.  kv_len[b] is the
 * number of the sequence's tokens, those of the present step among them (they
 * are the last ones); 0 (or less) marks an unused place of a padded batch.
 * Pages of different sequences may be shared for reading; the positions that one
 * append writes must not be (which value stays is then unspecified).
 */
#ifndef CSA_CACHE_H
#define CSA_CACHE_H

#include "csa_indexer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CSA_CACHE_BF16 = 0, CSA_CACHE_E4M3 = 1, CSA_CACHE_E2M1 = 2 } csa_cache_dtype_t;
typedef enum { CSA_ELEM_BF16 = 0, CSA_ELEM_FP16 = 1, CSA_ELEM_FP32 = 2 } csa_elem_dtype_t;
typedef enum {
    CSA_ROPE_PLAIN = 0,  /* base^(-2i/rot_dim)                                      */
    CSA_ROPE_LINEAR = 1, /* positions divided by factor                             */
    CSA_ROPE_NTK = 2,    /* base raised to base * factor^(rot_dim / (rot_dim - 2))  */
    CSA_ROPE_YARN = 3    /* by parts: a ramp between plain and linear frequencies   */
} csa_rope_scaling_t;

/* One cache (of keys, or of values). */
typedef struct {
    void *data;                  /* device, 16-byte aligned                              */
    void *scale;                 /* device, 16-byte aligned; NULL for CSA_CACHE_BF16     */
    int dtype;                   /* csa_cache_dtype_t                                    */
    int H, D;                    /* D a multiple of 16 (E2M1: of 32), at most 512        */
    int num_pages, page_size;
    long long page_stride;       /* bytes from page to page, a multiple of 16; 0: dense  */
    long long scale_page_stride; /* bytes, a multiple of a row's scale bytes; 0: dense   */
    float tensor_scale;          /* CSA_CACHE_E2M1: > 0 and finite (an append: 6 times   */
                                 /* it, too); others ignore it                           */
} csa_cache_t;

/*
 * Rotation frequencies (HOST memory, computed in double, rounded to fp32):
 * inv_freq[i], i < rot_dim / 2, and *scale, the factor on cos and sin that
 * csa_rotary and csa_cache_append take (1 except for CSA_ROPE_YARN, where it is
 * 0.1 ln(factor) + 1).  CSA_ROPE_YARN keeps dimensions that turn more than
 * beta_fast times within original_len, divides by factor those that turn less
 * than beta_slow times, and ramps linearly between them.  original_len,
 * beta_fast and beta_slow are read by CSA_ROPE_YARN only.
 */
csa_status_t csa_rope_frequencies(int rot_dim, double base, int scaling, double factor,
                                  int original_len, double beta_fast, double beta_slow,
                                  float *inv_freq, float *scale);

/*
 * Rotary positions.  For every token n, head h and pair i < rot_dim / 2, with
 * c = scale * cos(positions[n] * inv_freq[i]) and s the same of sin:
 *   (a, b) -> (a c - b s, b c + a s)       (inverse: s negated)
 * a and b are elements rot_offset + i and rot_offset + i + rot_dim/2 of the
 * head, or rot_offset + 2i and + 2i + 1 (interleaved); the head's other
 * elements are copied.  The inverse applied to the gradient of the output is
 * the gradient of x.  Angles are reduced in two doubles, so the farthest positions
 * lose nothing; cos, sin and the products are fp32, rounded once to the element
 * type.  out == x (with equal strides) rotates in place; otherwise they must
 * not overlap.  rot_dim and rot_offset are even, rot_dim >= 2,
 * rot_offset + rot_dim <= D <= 1024; strides are in elements, heads and tokens must not
 * overlap in out.
 */
typedef struct {
    const void *x;               /* [N, H, D] at the strides below                       */
    void *out;
    int dtype;                   /* csa_elem_dtype_t of x and out                        */
    int N, H, D;
    long long x_token_stride, x_head_stride, out_token_stride, out_head_stride;
    const int32_t *positions;    /* [N], may be negative                                 */
    const float *inv_freq;       /* [rot_dim / 2], device                                */
    int rot_dim, rot_offset;
    int interleaved, inverse;
    float scale;
} csa_rotary_args_t;

csa_status_t csa_rotary(const csa_rotary_args_t *args, cudaStream_t stream);

/*
 * Appends new keys (and values) to paged caches.  The tokens are [B, S]
 * (cu_tokens NULL; N = B * S), or packed: sequence b's are rows
 * cu_tokens[b] .. cu_tokens[b+1]-1 of N, ascending from cu_tokens[0] = 0, rows
 * (and positions) from cu_tokens[B] on are not read.  A sequence's n new tokens go to
 * positions kv_len[b] - n .. kv_len[b] - 1 (those below 0 are dropped).
 * With inv_freq, keys are rotated as csa_rotary says by positions[n], or
 * by the token's position in the cache when positions is NULL; values are
 * not.  A rotated element is rounded once to fp32 (the products are carried
 * in more than 32 bits, so that a stored code does not depend on the order of
 * operations) and then to the cache's type.  The two caches have the same num_pages,
 * page_size, H and dtype.  Their codes and scales are four different memories (pages may
 * interleave in one allocation; a shared byte is refused), and no row that is
 * written overlaps k or v.  Rows that no token goes to are left as they were.
 */
typedef struct {
    const void *k;               /* bf16 [N, H, Dk] at the strides below, 16-byte aligned */
    const void *v;               /* bf16 [N, H, Dv], or NULL (keys only)                 */
    long long k_token_stride, k_head_stride, v_token_stride, v_head_stride; /* elements, multiples of 8 */
    int N, B, S;                 /* S is read when cu_tokens is NULL                     */
    const int32_t *cu_tokens;    /* [B + 1] device, or NULL                              */
    const int32_t *kv_len;       /* [B] device                                           */
    const int32_t *page_table;   /* [B, max_pages] device                                */
    int max_pages;
    long long table_stride;      /* entries from row to row                              */
    csa_cache_t cache_k, cache_v; /* cache_v is read when v is given                     */
    const float *inv_freq;       /* device, or NULL: no rotation                         */
    const int32_t *positions;    /* [N] device, or NULL                                  */
    int rot_dim, rot_offset, interleaved;
    float rope_scale;
} csa_append_args_t;

csa_status_t csa_cache_append(const csa_append_args_t *args, cudaStream_t stream);

/*
 * Reads positions 0 .. T-1 of every sequence back as bf16: out [B, T, H, D]
 * (dense, 16-byte aligned, over no row that is read; with H = 1 csa_sparse_attention's
 * k or v), zeros at positions from kv_len[b] on and where there is no row.
 */
typedef struct {
    csa_cache_t cache;
    const int32_t *kv_len, *page_table;
    int max_pages;
    long long table_stride;
    int B, T;
    void *out;
} csa_cache_read_args_t;

csa_status_t csa_cache_read(const csa_cache_read_args_t *args, cudaStream_t stream);

/*
 * Attention over a cache held in 4 bits (both caches CSA_CACHE_E2M1).  Query row
 * i of sequence b stands at position kv_len[b] - S + i and sees the positions
 * up to its own (causal) or below kv_len[b]; with idx, of these only the ones
 * that idx[b,i,0..topk) lists (the indexer's out_idx: entries outside the
 * sequence are padding wherever they stand; a key listed twice counts twice).
 * Heads h * HA/H .. of HA query heads share head h of the cache.
 *   out[b,i,g,:] = sum_j softmax_j(scale * q[b,i,g,:] . k_j) * v_j
 *   lse[b,i,g]   = ln sum_j exp(scale * q[b,i,g,:] . k_j)
 * (zeros and -inf where a row sees no key).  Arithmetic: the stored values
 * are exact in the tensor cores' 16-bit types; q.k and P.V accumulate in fp32, softmax
 * is fp32, the probabilities are rounded to 16 bits for P.V, out to bf16.
 * scale times the keys' tensor_scale is finite in fp32.
 * D of each cache is 64, 128, 192 or 256; HA a multiple of H, HA / H <= 128;
 * the caches have the same H, num_pages and page_size, and may be the same one
 * (values that are the keys).  out, lse and the workspace overlap neither one another
 * nor q, idx (refused) or a cache.
 * `workspace` is device memory of csa_cache_attention_workspace_size(args)
 * bytes (shapes and the device's SM count decide it, not the data; 0 for arguments
 * that the call rejects, or when it needs none), 256-byte
 * aligned, used by the enqueued work only and with no state to keep; NULL
 * allocates and frees it stream-ordered.  Calls that may overlap, replays of captured
 * graphs among them, need workspaces of their own.
 */
typedef struct {
    const void *q;               /* [B, S, HA, Dk] bf16, dense, 16-byte aligned          */
    csa_cache_t cache_k, cache_v;
    const int32_t *kv_len, *page_table;
    int max_pages;
    long long table_stride;
    const int32_t *idx;          /* [B, S, topk], or NULL: every visible key             */
    int topk;
    int B, S, HA;
    int causal;
    float scale;
    void *out;                   /* [B, S, HA, Dv] bf16, 16-byte aligned                 */
    float *lse;                  /* [B, S, HA], or NULL                                  */
} csa_cache_attn_args_t;

csa_status_t csa_cache_attention(const csa_cache_attn_args_t *args, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream);
size_t csa_cache_attention_workspace_size(const csa_cache_attn_args_t *args);

#ifdef __cplusplus
}
#endif

#endif /* CSA_CACHE_H */
