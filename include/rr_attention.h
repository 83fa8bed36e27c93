/*
 * rr_attention.h -- C ABI of the sparse attention that consumes a route
 * (librr.so).
 *
 * Method: "RouteRelay: Event-Triggered Cross-Layer Route Reuse for Efficient
 * Dynamic Sparse Attention" (arXiv 2609.07306), cited as RouteRelay §x.
 * The router's output is a route per query chunk: the ids of the key chunks
 * it attends (§2.1 Eq. 2; the first k ids of a ledger row, rr.h).  The
 * selected chunks are expanded into token indices and attended with an
 * online softmax (§2.1); every layer attends with its own q, K, V over the
 * (possibly reused) route (§2.2 Eq. 3):
 *
 *     o_t = softmax(q_t K_T^T * scale) V_T,   T = tokens of the route's chunks
 *
 * Conventions (the page leaves them to the attention backend, §4.3):
 *  - Chunk j covers tokens j*chunk .. j*chunk + chunk - 1, for queries and
 *    keys alike; query token t belongs to query chunk t / chunk.
 *  - causal != 0: key token s is visible to query token t iff s <= t.
 *  - Route ids that are negative (-1 padding) or >= the number of key
 *    chunks are skipped; with causal, so are ids greater than the query
 *    chunk's own (they hold no visible token).  Every other entry
 *    contributes its chunk once per occurrence.
 *  - A query token with no visible key gets a zero output row.
 *  - Same stream, ownership and error conventions as rr.h: device memory is
 *    the caller's, the call enqueues on `stream` and returns without
 *    synchronising, argument errors return before any CUDA call.
 */
#ifndef RR_ATTENTION_H
#define RR_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "rr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of one sparse-attention call.  Limits: bh, nq_tokens, nk_tokens >= 0
 * (bh == 0 or nq_tokens == 0: nothing to do); dh in {64, 128}; chunk in
 * {16, 32, 64, 128}; nq_tokens and nk_tokens multiples of chunk;
 * 0 <= width <= 1024; route_stride >= max(width, 1);
 * bh * (nq_tokens / chunk) <= 2^31 - 1; scale finite and >= 0. */
typedef struct {
    int32_t bh;           /* heads (batch x heads) */
    int32_t nq_tokens;    /* query tokens per head */
    int32_t nk_tokens;    /* key / value tokens per head */
    int32_t dh;           /* head dimension of q, k, v */
    int32_t chunk;        /* tokens per chunk */
    int32_t width;        /* route entries read per query chunk */
    int32_t route_stride; /* int32 elements from one query chunk's route to the next */
    int32_t causal;       /* nonzero: token-level causal mask (s <= t) */
    float scale;          /* softmax scale; 0 selects 1/sqrt(dh) (Eq. 3) */
} rr_attn_config;

/* Sparse attention over a route (RouteRelay §2.1, §2.2 Eq. 3).
 *   d_q     bf16 [bh, nq_tokens, dh], row-major, 16-byte aligned
 *   d_k     bf16 [bh, nk_tokens, dh], the same layout (may be NULL when nk_tokens == 0)
 *   d_v     bf16 [bh, nk_tokens, dh], the same layout
 *   d_route int32 [bh, nq_tokens / chunk, route_stride]; entries 0..width-1 of
 *           each query chunk's row are read.  A ledger's ids (rr_ledger_device_view)
 *           serve directly: route_stride = c, width = k.
 *   d_out   fp32 [bh, nq_tokens, dh], 16-byte aligned; written in full.
 * The scores and the softmax are fp32; P is rounded to bf16 before the
 * P.V product (both products run on the tensor cores with fp32
 * accumulation), so each output element is within about 2^-8 of the
 * softmax-weighted mean of |v| of the exact result.  Errors: RR_EINVAL
 * (bad shape, null or misaligned pointer), RR_ECUDA (launch). */
rr_status rr_sparse_attention(const rr_attn_config *cfg, const void *d_q, const void *d_k,
                              const void *d_v, const int32_t *d_route, float *d_out,
                              void *stream);

/* ---- masked attention over a route ---------------------------------------
 * The attention above with the score terms and masks of a prompt:
 *
 *   x(t, s) = cap * tanh(scale * q_t . k_s / cap)        (cap > 0; else the product)
 *             - slope_h * |p_t - s|,                      p_t = t + q_offset
 *   s is visible to t iff s belongs to a chunk of the route of t's query chunk,
 *     causal == 0, or s <= p_t, or s < prefix_b, and
 *     doc_q(t) == doc_k(s) >= 0 where documents are given;
 *   o_t = sum_s e^x(t,s) v_s / sum_s e^x(t,s),   lse_t = log sum_s e^x(t,s)
 *
 * over the visible s, an entry that the route repeats counting once per
 * occurrence.  A token with no visible key gets a zero row and lse -inf.
 * Query chunk i holds query tokens i*chunk .. i*chunk + chunk - 1 (positions
 * q_offset later), key chunk j key tokens j*chunk ..; the last chunk of either
 * may be short.  Key/value heads and routes may be shared: query head h uses
 * route head h / (q_heads / route_heads) and key head h / (q_heads / kv_heads).
 * What a masked key or value row holds is never read into a result, infinities
 * and NaN included. */

/* Limits: batch, nq_tokens, nk_tokens >= 0; kv_heads divides route_heads
 * divides q_heads; dh in {64, 128}; chunk in {16, 32, 64, 128}; 0 <= width <=
 * 1024; route_stride >= max(width, 1); dtype RR_BF16 or RR_F16; q_offset >= 0
 * and q_offset + nq_tokens, nk_tokens <= 2^24 (positions are exact in fp32);
 * scale >= 0 and at most 1e30; soft_cap 0 or in [1e-3, 1e30]; rows of a unit,
 * q_heads / route_heads * chunk, <= 2^24, and 16ths of them times batch * route_heads *
 * query chunks <= 2^31 - 1; strides in elements, >= 0 and multiples of 8; those of a size of one count nothing.  The
 * rows of `out` lie apart: by dimensions from the smallest stride up, each stride
 * is at least what the ones before it span. */
typedef struct {
    int32_t batch;
    int32_t q_heads;      /* query (and output) heads */
    int32_t kv_heads;     /* key / value heads */
    int32_t route_heads;  /* routes per batch entry */
    int32_t nq_tokens;    /* query tokens */
    int32_t nk_tokens;    /* key / value tokens */
    int32_t dh;           /* head dimension */
    int32_t chunk;        /* tokens per chunk */
    int32_t width;        /* route entries read per query chunk */
    int32_t route_stride; /* int32 elements from one query chunk's route to the next */
    int32_t causal;       /* nonzero: causal mask, with the prefix's exception */
    int32_t dtype;        /* rr_dtype of q, k, v and out */
    int32_t q_offset;     /* position of query token 0 */
    float scale;          /* 0 selects 1/sqrt(dh) */
    float soft_cap;       /* 0: no cap */
    int64_t q_stride[3];  /* elements from one batch entry, head, token to the next */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t out_stride[3];
} rr_masked_attn_config;

/* Device pointers of one call; those marked optional may be NULL. */
typedef struct {
    const void *q;           /* [batch, q_heads, nq_tokens, dh] by q_stride; 16-byte aligned */
    const void *k;           /* [batch, kv_heads, nk_tokens, dh] by k_stride; 16-byte aligned */
    const void *v;           /* the same by v_stride */
    const int32_t *route;    /* [batch, route_heads, ceil(nq_tokens / chunk), route_stride] */
    const float *slopes;     /* optional [q_heads]: bias by distance, in [0, 1e30] */
    const int32_t *doc_q;    /* optional [batch, nq_tokens]: document of each query token */
    const int32_t *doc_k;    /* [batch, nk_tokens], given iff doc_q is */
    const int32_t *prefix;   /* optional [batch]: keys below it are visible under causal */
    void *out;               /* [batch, q_heads, nq_tokens, dh] by out_stride; 16-byte aligned */
    float *lse;              /* optional [batch, q_heads, nq_tokens] */
} rr_masked_attn_args;

/* Enqueues the attention. Scores, softmax and sums are fp32; the weights are
 * rounded to the inputs' type for the product with v, and the result to that
 * type once. Units of more than 64 rows (q_heads / route_heads * chunk; at dh
 * 128 without a cap of 64 too) run on tcgen05, smaller ones on mma.sync; both
 * give the same bits from call to call. Rows whose result is not finite, and
 * rows whose route's chunks hold an infinity or a NaN in a value row that they
 * do not see, take a slow path: 610 cycles a key and row at dh 128, hundreds of
 * times the usual. `out` must not overlap the inputs. Every wait inside the
 * kernels is bounded (by one second to nine); should one run out, the rows not
 * yet written become NaN. Errors: RR_EINVAL (shape, stride, null or misaligned
 * pointer), RR_ECUDA (launch). */
rr_status rr_masked_attention(const rr_masked_attn_config *cfg, const rr_masked_attn_args *args,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RR_ATTENTION_H */
