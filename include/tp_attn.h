/*
 * tp_attn.h -- C ABI of equivariant neighbour attention on the receiver-sorted graph of tp.h,
 * with a learned bias by distance buckets and dropout of the probabilities, and of the
 * distance buckets themselves.
 *
 * Attention.  Rows q, k follow irreps_qk, rows v and y follow irreps_v (layouts as in tp.h).
 * Every block's channels are divided evenly among H heads, head h owning the h-th part with
 * all its components m; <a, b>_h is the sum over a head's floats.  It is invariant under
 * rotations (the Wigner-D matrices are orthogonal), so the probabilities are scalars and y
 * transforms as v does.  For receiver i and its edges e = (j -> i), rowptr[i] <= e < rowptr[i+1]:
 *
 *   s[e,h] = scale <q[i], k[j]>_h + table[bucket[e], h]       p[e,h] = softmax of s over e
 *   y[i]_h = sum_e r[e,h] p[e,h] v[j]_h                       lse[i,h] = log sum_e exp s[e,h]
 *
 * r = 1 without dropout.  With it r[e,h] is 0 or 1/(1-p_drop): value number e H + h of the
 * generator below.  tp_attn_bwd takes y and lse of the forward call, forms the probabilities
 * again as exp(s - lse), and returns, against gy and with ds = p (r <gy[i], v[j]>_h - <gy[i], y[i]>_h),
 *
 *   gq[i] = scale sum_e ds k[j]      gk[j] = scale sum_{e from j} ds q[i]
 *   gv[j] = sum_{e from j} r p gy[i] gtable[b,h] = sum_{e: bucket[e] = b} ds[e,h]
 *
 * Where |lse| >= 2^10 (a large constant in the table, a mask of the lowest float on every edge of a
 * row), lse in 32 bits no longer holds the row's sum; the backward pass then forms it again from q, k
 * and table, in one more sweep over those rows' edges.
 *
 * First order only.  The bias is constant within a bucket: no gradient reaches the edge vectors.
 *
 * What takes no part.  An edge whose bucket lies outside [0, n_buckets) (tp_distance_buckets
 * gives -1 from the cutoff on: the skin of a neighbour list), an edge whose sender lies outside
 * [0, N), and, for its head, an edge whose table entry is -inf: neither k[j] nor v[j] reaches
 * any result there, not even as a NaN.  Edges outside [rowptr[0], rowptr[N]) (the spare tail of
 * a list of fixed capacity E) belong to no row.  A row without any other edge gives y = 0,
 * lse = -inf and no gradient.  rowptr, perm and colptr entries are clamped to [0, E]: bad ones
 * give unspecified results, never an access outside the arrays.
 *
 * Generator.  Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
 * 1, 2, 3", SC 2011): value number n is word n mod 4 of the block with counter
 * (n div 4, rng[1] + site) as two 64-bit halves, low words first, and key rng[0]; it is kept
 * when it is >= round(p_drop 2^32).  rng is {seed, offset} in device memory, so a captured
 * call draws anew when the program advances the offset; `site` tells the calls of one step
 * apart.  No mask is stored: the backward pass draws the same values again.
 *
 * Layouts: fp32, q/k/v and gq/gk/gv rows ld* floats apart (ld >= the row's width: the three
 * may be slices of one [N, 2 qk_dim + v_dim] array); y, gy [N, v_dim], lse [N, H], table
 * [n_buckets, H], bucket [E] int32.  Outputs are fully overwritten, rows without edges with
 * zeros.  No output (the workspace is one) may share memory with an input or another output: rows
 * of q, k, v and gy are read until the call ends, by other rows' sums too.  Results do not depend on
 * the schedule: no floating-point atomics, fixed orders.
 *
 * Ownership, streams and errors as in tp.h; the library owns only the handle (host memory).
 * Calls on one handle from several threads or streams are independent as long as their
 * workspaces are.  Pointers need 4-byte alignment; when every pointer is 16-byte (8-byte)
 * aligned and every width (a head's floats in each block) and ld is a multiple of 4 (2), rows
 * move 16 (8) bytes at a time, else 4.  The workspace needs 256-byte alignment.  Row strides
 * stay below 2^30 floats, E and N * heads below 2^31 - 2^22.
 */
#ifndef TP_ATTN_H_
#define TP_ATTN_H_

#include "tp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tp_attn_s* tp_attn_t;

/* Builds an attention.  heads in [1, 32] divides every multiplicity of both strings; at most 16
 * blocks each; a head has at most 4,096 floats in a row of q or v; n_buckets in [0, 4096], 0 for
 * an attention without buckets; n_buckets * heads <= 32768.  Errors: TP_ERR_INVALID_ARG (syntax,
 * heads that do not divide), TP_ERR_UNSUPPORTED (l > 3, beyond the limits). */
tp_status_t tp_attn_create(tp_attn_t* attn, const char* irreps_qk, const char* irreps_v, int32_t heads,
                           int32_t n_buckets);
tp_status_t tp_attn_destroy(tp_attn_t attn);
tp_status_t tp_attn_query(tp_attn_t attn, int64_t* qk_dim, int64_t* v_dim);

/* Device workspace bytes of a call of kind op (TP_OP_FWD or TP_OP_BWD) for N nodes and E edges.
 * Forward: partial rows of receivers with very many edges (0 for E <= 320), node-sized in all.
 * Backward: those, two floats per edge and head, the receiver of each edge, partials of gtable,
 * and room for the transpose. */
tp_status_t tp_attn_workspace_size(tp_attn_t attn, int64_t N, int64_t E, int32_t op, size_t* bytes);

/* Forward.  bucket may be NULL (every edge takes part; then table must be NULL), table may be
 * NULL (no bias; bucket is then only a mask).  rng may be NULL when p_drop = 0; p_drop in
 * [0, 1).  lse may be NULL when no backward call follows. */
tp_status_t tp_attn_fwd(tp_attn_t attn, int64_t N, int64_t E, const int32_t* rowptr, const int32_t* src,
                        const int32_t* bucket, const float* q, int64_t ldq, const float* k, int64_t ldk,
                        const float* v, int64_t ldv, const float* table, float scale, double p_drop,
                        const int64_t* rng, int64_t site, float* y, float* lse, void* ws, size_t ws_bytes,
                        tp_stream_t stream);

/* Backward against gy.  colptr/perm: a transpose from tp_csr_transpose, or both NULL to have it
 * built in the workspace (only needed for gk and gv).  Each NULL output is skipped. */
tp_status_t tp_attn_bwd(tp_attn_t attn, int64_t N, int64_t E, const int32_t* rowptr, const int32_t* src,
                        const int32_t* colptr, const int32_t* perm, const int32_t* bucket, const float* q,
                        int64_t ldq, const float* k, int64_t ldk, const float* v, int64_t ldv, const float* table,
                        float scale, double p_drop, const int64_t* rng, int64_t site, const float* y,
                        const float* lse, const float* gy, float* gq, int64_t ldgq, float* gk, int64_t ldgk,
                        float* gv, int64_t ldgv, float* gtable, void* ws, size_t ws_bytes, tp_stream_t stream);

/* bucket[e] = number of bounds[k] <= |vec[e]| (so n_bounds + 1 buckets; bounds ascending, device
 * memory, n_bounds in [0, 1023]), or -1 when |vec[e]| >= cutoff or is NaN; cutoff = +inf for none
 * (an infinite distance is then -1 too).  Lengths are compared as squares in 64 bits, where the
 * products of 32-bit floats are exact: the choice does not depend on the hardware's rounding of
 * a square root, and a bound belongs to the bucket above it. */
tp_status_t tp_distance_buckets(int64_t E, const float* vec, int32_t n_bounds, const float* bounds, float cutoff,
                                int32_t* bucket, tp_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* TP_ATTN_H_ */
