/*
 * rr_cache.h -- C ABI of the paged, quantised key/value cache and the
 * attention that reads it (librr.so).
 *
 * The cache keeps keys and values of past tokens in pages of `chunk` tokens --
 * the chunk that the router selects (rr.h) -- so a route names pages of a
 * sequence directly.  A sequence's page table maps its chunk j (positions
 * j*chunk ..) to a page of the pool.
 *
 * Formats, both with power-of-two scales, so that storing rounds exactly once:
 *   RR_E4M3  8-bit floats (4 exponent, 3 mantissa bits), one scale per row of
 *            dh elements; largest value M = 448
 *   RR_E2M1  4-bit floats (2 exponent, 1 mantissa bit), one scale per 32
 *            elements; M = 6; element 2i in the low half of byte i
 * A group with largest magnitude a gets the least exponent e >= -127 with
 * a <= M 2^e; its elements x are stored as x 2^-e rounded to nearest, ties to
 * even, its scale as the byte e + 127.  A group that holds an infinity or a
 * NaN gets the byte 255 and reads back as NaN.  (The format's own NaN codes,
 * 0x7F and 0xFF, are never stored; in a pool that holds them in places that a
 * sequence has reached, they can reach query tokens that do not see them.)
 *
 * Conventions of rr.h: device memory is the caller's, a call enqueues on
 * `stream` and returns without synchronising, argument errors come back before
 * any CUDA call.  Page ids outside the pool (-1 among them) name no page:
 * tokens there are neither written nor attended, and read as zeros.
 */
#ifndef RR_CACHE_H
#define RR_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "rr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RR_E4M3 = 0, RR_E2M1 = 1 } rr_cache_format;

/* One pool of pages.  Limits: pages >= 0; 1 <= heads <= 65535; dh in {64, 128}; chunk in
 * {16, 32, 64, 128}. */
typedef struct {
    int32_t pages;
    int32_t heads;   /* key / value heads */
    int32_t dh;      /* head dimension */
    int32_t chunk;   /* tokens per page */
    int32_t format;  /* rr_cache_format */
} rr_cache_config;

/* The pool's two arrays, owned by the caller.  R = dh (e4m3) or dh/2 (e2m1)
 * bytes and G = 1 or dh/32 scales per row:
 *   codes  [pages, heads, 2, chunk, R] bytes, 16-byte aligned   (0: keys, 1: values)
 *   scales [pages, heads, 2, chunk, G] bytes, 16-byte aligned */
typedef struct {
    void *codes;
    void *scales;
} rr_cache_pool;

/* Bytes of the two arrays (0 if the config is invalid).  Host arithmetic. */
size_t rr_cache_codes_bytes(const rr_cache_config *cfg);
size_t rr_cache_scales_bytes(const rr_cache_config *cfg);

/* A ragged batch of tokens: rows cu[b] .. cu[b+1]-1 of the row arrays belong to
 * sequence b, at positions start[b], start[b]+1, ...  Rows outside
 * [cu[0], cu[batch]) belong to none.  Two rows of one write must not fall on
 * the same place of the pool: what that place then holds is undefined. */
typedef struct {
    int32_t batch;              /* sequences, >= 0 */
    int32_t rows;               /* rows of the row arrays, >= 0 */
    const int32_t *cu;          /* [batch + 1], not decreasing */
    const int32_t *start;       /* [batch] */
    const int32_t *page_table;  /* [batch, table_stride] page ids */
    int32_t table_width;        /* entries read per sequence; later positions have no page */
    int32_t table_stride;       /* >= max(table_width, 1) */
} rr_cache_rows;

/* Quantises and stores the rows of k and v (each [rows, heads, dh] of `dtype`:
 * RR_F32, RR_BF16 or RR_F16; strides of row and head in elements (of a size of one:
 * any), rows 16-byte aligned, dh contiguous).  Only places that a row falls on are written.
 * Errors: RR_EINVAL, RR_ECUDA. */
rr_status rr_cache_write(const rr_cache_config *cfg, const rr_cache_pool *pool, const rr_cache_rows *rows,
                         const void *d_k, const int64_t k_stride[2], const void *d_v,
                         const int64_t v_stride[2], int32_t dtype, void *stream);

/* Reads the rows back as `dtype` (rounded to nearest where its range or
 * precision is short of the stored value).  Either output may be NULL.  Rows
 * that belong to no sequence are left as they were.  The rows of an output lie
 * apart: the smaller stride is at least dh, the other at least what the smaller
 * one's dimension spans.  Errors as above. */
rr_status rr_cache_read(const rr_cache_config *cfg, const rr_cache_pool *pool, const rr_cache_rows *rows,
                        void *d_k, const int64_t k_stride[2], void *d_v, const int64_t v_stride[2],
                        int32_t dtype, void *stream);

/* Attention of the newest q_tokens tokens of each sequence over its cached
 * tokens.  Query token i of a sequence of seq_len cached tokens (its own among
 * them) has position p = seq_len - q_tokens + i and sees the positions s <= p;
 * with a route, of those only the ones in the chunks that it lists for the
 * sequence and key head (ids outside the sequence are skipped, repeated ones
 * count once per occurrence).
 *   x = cap * tanh(scale * q.k / cap) - slope_h * (p - s),  o, lse as in rr_attention.h
 * A token with no visible key gets zeros and lse -inf.
 * Weights are rounded to f16 for the product with the values (below 2^-21 of a
 * row's largest weight * scale to 2^-32 of it), the result once to dtype; scores,
 * softmax and sums are fp32.  The same call gives the same bits.
 * Limits: batch, q_tokens >= 0; q_heads a multiple of cache heads, q_heads /
 * heads * q_tokens <= 256; batch * heads <= 65535; table_width * chunk <=
 * 2^24; 0 <= width <= 2^20, route_stride >= max(width, 1); scale >= 0 and at
 * most 1e30; soft_cap 0 or in [1e-3, 1e30]; dtype RR_BF16 or RR_F16; q strides >= 0,
 * multiples of 8 (of a size of one: any).  A query row's largest magnitude times scale (with a cap, times
 * scale / cap) is 0 or in [2^-112, 2^108], the keys' scales 2^e at most 2^100:
 * outside of this, scores can lose bits or become infinite, which makes a row NaN. */
typedef struct {
    int32_t batch;
    int32_t q_tokens;
    int32_t q_heads;
    int32_t dtype;         /* rr_dtype of q and out */
    int32_t table_width;   /* page table entries per sequence */
    int32_t table_stride;
    int32_t width;         /* route entries read per sequence and key head */
    int32_t route_stride;
    float scale;           /* 0 selects 1/sqrt(dh) */
    float soft_cap;        /* 0: no cap */
    int64_t q_stride[3];   /* elements from one sequence, token, head to the next */
} rr_cached_attn_config;

typedef struct {
    const void *q;              /* [batch, q_tokens, q_heads, dh] by q_stride; 16-byte aligned */
    const int32_t *seq_lens;    /* [batch] */
    const int32_t *page_table;  /* [batch, table_stride] */
    const int32_t *route;       /* optional [batch, heads, route_stride]; NULL: every chunk (width 0: none) */
    const float *slopes;        /* optional [q_heads], in [0, 1e30] */
    void *out;                  /* [batch, q_tokens, q_heads, dh], contiguous; 16-byte aligned */
    float *lse;                 /* optional [batch, q_tokens, q_heads] */
} rr_cached_attn_args;

/* Bytes of device workspace a call needs (may be 0): the partial results of
 * sequences whose tokens are split over blocks; `routed`: whether the call has
 * a route (it splits the route instead of the table).  It is written and read within
 * the call only; calls that can overlap on the GPU need one each. */
size_t rr_cached_attention_workspace_bytes(const rr_cache_config *cfg, const rr_cached_attn_config *attn,
                                           int32_t routed);

/* Enqueues the attention; `workspace` is 256-byte aligned.  Errors: RR_EINVAL,
 * RR_ENOMEM (workspace too small), RR_ECUDA. */
rr_status rr_cached_attention(const rr_cache_config *cfg, const rr_cache_pool *pool,
                              const rr_cached_attn_config *attn, const rr_cached_attn_args *args,
                              void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RR_CACHE_H */
