/*
 * gsample_tokens.h -- C ABI of libgsample's operators on sequences of tokens:
 * layer normalisation, dropout, and attention with a learned relative
 * position bias by buckets, forward and backward.
 *
 * They are what a model computes on the feature maps that gsample.h's
 * operators sample, once their positions are read as a sequence of tokens.
 * Status codes and element types are gsample.h's.  The conventions of that
 * header hold here too (device pointers owned by the caller, host
 * descriptors, every argument validated before anything is enqueued, no
 * allocation, no state, no synchronisation, no overlap of outputs with
 * inputs), with one difference: tensors named with strides may be strided.
 * A stride counts elements; the last axis is always contiguous.  A stride
 * may be any value >= 0, 0 only in tensors that are read (a broadcast).
 *
 * Sums, means, softmax statistics and gradients are accumulated in fp32 or
 * wider.  No entry point adds in an order that varies: the same call on the
 * same device gives the same bits.
 */
#ifndef GSAMPLE_TOKENS_H
#define GSAMPLE_TOKENS_H

#include "gsample.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Layer normalisation
 * --------------------------------------------------------------------- */

/*
 * For each row x of `cols` elements:
 *   mean = sum(x) / cols,  var = sum((x - mean)^2) / cols,
 *   inv_std = 1 / sqrt(var + epsilon),
 *   y = (x - mean) * inv_std * scale + bias.
 *
 *   X, dtype     device, rows x cols, element type dtype (GS_F32, GS_F16,
 *                GS_BF16), row r at r * x_stride.
 *   scale, bias  device (cols), element type param_dtype: dtype or GS_F32.
 *                bias may be NULL (zeros).
 *   Y            device, rows x cols, element type dtype, row r at
 *                r * y_stride.
 *   mean, inv_std  device fp32 (rows), or NULL where they are not wanted.
 *
 * Errors: GS_ERR_NULL, GS_ERR_SHAPE (negative extent; a row stride smaller
 * than cols in Y, negative in X; cols 0 with rows), GS_ERR_DTYPE,
 * GS_ERR_ATTR (epsilon negative or not finite), GS_ERR_TOO_LARGE (cols above
 * 2^24, rows above 2^31 - 1), GS_ERR_HIP.
 */
int gs_layer_norm(const void *X, int dtype, int64_t rows, int64_t cols, int64_t x_stride,
                  const void *scale, const void *bias, int param_dtype, float epsilon, void *Y,
                  int64_t y_stride, float *mean, float *inv_std, void *stream);

/*
 * Gradients of gs_layer_norm.  With xh = (x - mean) * inv_std and g = dy * scale:
 *   dx = inv_std * (g - mean_row(g) - xh * mean_row(g * xh)),
 *   dscale = sum over rows of dy * xh,  dbias = sum over rows of dy.
 *
 *   dY, X        device, rows x cols, dtype, rows dy_stride and x_stride apart.
 *   mean, inv_std  device fp32 (rows), as gs_layer_norm wrote them.
 *   dX           device, rows x cols, dtype, rows dx_stride apart.
 *   dscale, dbias  device (cols), param_dtype; both, or both NULL.  They are
 *                overwritten (rows = 0 writes zeros).
 *   workspace    device, 256-byte aligned, at least
 *                gs_layer_norm_backward_workspace_size() bytes; needed where
 *                dscale is wanted.  Overwritten.
 *
 * Errors: as gs_layer_norm; GS_ERR_NULL for a missing workspace,
 * GS_ERR_ATTR for one that is too small or misaligned.
 */
int gs_layer_norm_backward(const void *dY, const void *X, int dtype, int64_t rows, int64_t cols,
                           int64_t dy_stride, int64_t x_stride, const void *scale, int param_dtype,
                           const float *mean, const float *inv_std, void *dX, int64_t dx_stride,
                           void *dscale, void *dbias, void *workspace, int64_t workspace_bytes,
                           void *stream);

/* Bytes of workspace gs_layer_norm_backward needs for these extents, written
 * to *bytes (host). */
int gs_layer_norm_backward_workspace_size(int64_t rows, int64_t cols, int64_t *bytes);

/* ------------------------------------------------------------------------
 * Dropout
 * --------------------------------------------------------------------- */

/*
 * The numbers behind both dropouts: Philox4x32-10 (Salmon, Moraes, Dror and
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) under the key
 * (seed mod 2^32, seed / 2^32).  Its 128 bits are eight 16-bit numbers, low
 * half of the first word first.  An element whose number is below
 * t = floor(ratio * 65536 + 0.5) is dropped (0); a kept one is multiplied by
 * 65536 / (65536 - t), so that the mean is kept for the ratio as rounded.
 * No mask is stored: the same seed and call give the same mask again.  A
 * program gives each use of a step its own `call`, each step its own seed.
 */

/*
 * Y = residual + dropout(X): element n of the tensor uses number n % 8 of the
 * counter (n / 8 mod 2^32, n / 8 / 2^32, 0, call).  The gradient with respect
 * to X is the same call on dY without a residual; with respect to the
 * residual it is dY.
 *
 *   X, residual, Y  device, `count` contiguous elements, element type dtype
 *                (GS_F32, GS_F16, GS_BF16).  residual may be NULL (zeros).
 *                Y may be X or residual itself (in place).
 *   ratio        0 <= ratio, floor(ratio * 65536 + 0.5) <= 65535.
 *
 * A dropped element contributes 0 whatever it holds (NaN and infinities
 * included).  The sum is made in fp32 and rounded once.
 * Errors: GS_ERR_NULL, GS_ERR_SHAPE (count negative), GS_ERR_DTYPE,
 * GS_ERR_ATTR (ratio), GS_ERR_TOO_LARGE (count above 2^40), GS_ERR_HIP.
 */
int gs_dropout(const void *X, int dtype, int64_t count, const void *residual, float ratio,
               uint64_t seed, uint32_t call, void *Y, void *stream);

/* ------------------------------------------------------------------------
 * Attention with a relative position bias
 * --------------------------------------------------------------------- */

/*
 * Bucket of a relative position r = key position - query position.  With
 * `bidirectional`, half of the buckets (n = num_buckets / 2) serve r <= 0 and
 * the other half r > 0, by d = |r|; otherwise n = num_buckets and
 * d = max(-r, 0).  The first e = n / 2 buckets of a side hold one distance
 * each; bucket e + j begins at the smallest d >= e with
 * (d / e)^(n - e) >= (max_distance / e)^j, and the last one has no end.
 *
 * Host only: the bucket is written to *bucket.  Errors: GS_ERR_NULL,
 * GS_ERR_ATTR (num_buckets below 2, above 512, or with bidirectional odd or
 * below 4; max_distance <= e), GS_ERR_TOO_LARGE (the last border lies beyond
 * 1024).
 */
int gs_relative_bucket(int64_t r, int num_buckets, int max_distance, int bidirectional,
                       int *bucket);

/*
 * One attention call.  Element (b, h, i, d) of a tensor with strides s lies
 * at b * s[0] + h * s[1] + i * s[2] + d.  Query head h reads key / value head
 * h / (q_heads / kv_heads).
 */
typedef struct {
    int dtype;             /* of Q, K, V, O and their gradients: GS_F32, GS_F16, GS_BF16 */
    int table_dtype;       /* of table and dtable: dtype or GS_F32 */
    int64_t batch, q_heads, kv_heads, q_len, kv_len, head_dim;
    int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3];
    int64_t do_stride[3], dq_stride[3], dk_stride[3], dv_stride[3]; /* backward only */
    float scale;           /* of the scores */
    int causal;            /* 1: a key after the query's position is masked */
    int q_from_end;        /* 0: query i is at position q_position + i of the keys;
                              1: at position length_b - q_len + i */
    int64_t q_position;
    int num_buckets;       /* 0: no bias */
    int max_distance;
    int bidirectional;
    float ratio;           /* dropout of the probabilities */
    uint32_t call;
    uint64_t seed;
} gs_attention_desc;

/*
 * For each query i of head h and sequence b, over the keys j that it sees
 * (j < length_b, and j <= position of i when causal):
 *   s_j = scale * (q_i . k_j) + table[bucket(j - position of i)][h],
 *   p_j = exp(s_j) / sum of exp(s),  o_i = sum of dropout(p_j) * v_j.
 * Key j of query i uses number j % 8 of the counter
 * (j / 8, i, b * q_heads + h, call).  A query that sees no key gives 0.
 * A bias of any finite size may serve as a mask: a query whose every key has
 * one keeps the softmax of its products, which a constant does not change.
 * (Values beyond 2.35e38 count as that; -inf hides a key as a mask does.)
 *
 *   Q            device (batch, q_heads, q_len, head_dim)
 *   K, V         device (batch, kv_heads, kv_len, head_dim)
 *   lengths      device int32 (batch): keys of each sequence, held to
 *                0 .. kv_len; NULL: kv_len.  Keys at and beyond a sequence's
 *                length are not read: they may hold anything.
 *   table        device (num_buckets, q_heads); NULL with num_buckets 0.
 *   O            device (batch, q_heads, q_len, head_dim)
 *   lse          device fp32 (batch, q_heads, q_len), contiguous: log of the
 *                sum of exp(s), -inf for a query that sees no key; or NULL.
 *   workspace    device, 256-byte aligned, of gs_attention_workspace_size()
 *                bytes; without it (NULL, 0), or with less, a long key axis of
 *                few queries is not split over thread blocks: slower, and the
 *                sums in another order.
 *
 * The probabilities are rounded to dtype before they multiply V (with
 * GS_F32 not at all).  A NaN or infinity in V reaches every query of the
 * call whose mask leaves its key, and may reach the other queries of its head.
 * (In gs_attention_backward so may one in Q, K, V or dO.  Keys past a length and,
 * with causal, queries before position 0 reach nothing, whatever they hold.)
 * Errors: GS_ERR_NULL, GS_ERR_SHAPE (an extent negative, q_heads no multiple
 * of kv_heads, head_dim 0, a negative stride, one below head_dim along an axis
 * of more than one element of an output: rows must not overlap), GS_ERR_DTYPE, GS_ERR_ATTR
 * (scale not finite, a flag not 0 or 1, ratio, buckets as in
 * gs_relative_bucket, a workspace that is misaligned), GS_ERR_TOO_LARGE
 * (head_dim above 128, q_len, kv_len or |q_position| above 2^29, heads above
 * 2^20, the last border as in gs_relative_bucket, 2^24 thread blocks or
 * more: a block has at least 32 queries or keys of a head), GS_ERR_HIP.
 */
int gs_attention(const gs_attention_desc *desc, const void *Q, const void *K, const void *V,
                 const int32_t *lengths, const void *table, void *O, float *lse, void *workspace,
                 int64_t workspace_bytes, void *stream);

/* Bytes of workspace that gs_attention uses for this descriptor (0: none),
 * written to *bytes (host). */
int gs_attention_workspace_size(const gs_attention_desc *desc, int64_t *bytes);

/*
 * Gradients of gs_attention from dO, its inputs, and the O and lse that it
 * wrote, under the same descriptor.  dQ, dK, dV and dtable (num_buckets,
 * q_heads; contiguous, table_dtype) are overwritten whole; keys that no query
 * sees get 0, as do the scores of a query that sees one key (its probability
 * is 1 whatever they are).  Probabilities are made again from lse: its fp32
 * rounding is a relative error of up to |lse| 2^-23 of theirs.  dtable may be NULL where it is not wanted.  dS is
 * rounded to dtype before it multiplies Q and K (with GS_F32 not at all).  The
 * workspace (256-byte aligned) is required.  Errors as gs_attention; GS_ERR_ATTR for a
 * workspace that is too small, GS_ERR_TOO_LARGE for a dtable of 2^24 - 8200
 * elements or more.
 */
int gs_attention_backward(const gs_attention_desc *desc, const void *dO, const void *Q,
                          const void *K, const void *V, const void *O, const float *lse,
                          const int32_t *lengths, const void *table, void *dQ, void *dK, void *dV,
                          void *dtable, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace that gs_attention_backward needs for this descriptor,
 * written to *bytes (host). */
int gs_attention_backward_workspace_size(const gs_attention_desc *desc, int64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* GSAMPLE_TOKENS_H */
