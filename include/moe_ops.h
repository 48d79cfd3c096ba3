/*
 * moe_ops.h -- C ABI of the operators around the quantised MoE decode step
 * (GB300, sm_103a): products whose weights stay in 16 bits, and the slot
 * bookkeeping of a router other than the step's own.
 *
 *   moe_linear          out = act(x W^T + bias) [* (x Wup^T + bias_up)] [+ residual]
 *   moe_grouped_linear  the same product with one weight matrix per expert,
 *                       over rows grouped by expert
 *   moe_group_slots     top-k expert ids -> rows grouped by expert
 *   moe_combine_slots   out[t] = sum_j w[t,j] y[slot_of[t,j]] [+ residual[t]]
 *   moe_route           router logits -> top-k expert ids and weights, for routers
 *                       other than the step's: sigmoid scores, a bias for balance,
 *                       groups of experts
 *   moe_quantize_rows   rows of 16-bit values -> 8-bit codes with a scale per row
 *   moe_linear_q8       moe_linear on 8-bit codes, scales per row of x and of W
 *   moe_grouped_linear_q8   moe_grouped_linear likewise
 *
 * Together they run a layer that moe_decode_forward does not: a shared expert
 * beside the routed ones, the projections around the step, experts that a
 * checkpoint leaves unquantised or keeps in 8 bits, and any router (the grouping
 * and the combine take ids and weights, from moe_route or anywhere else). The
 * sources of the step (mlxcel issues #1616 and #1859) have the routed block only;
 * grouping and combine follow the same readings:
 * #1616 Leading hypothesis (slots sorted by expert id), Current Behavior
 * (moe_weighted_sum), Implementation Notes (f32 partials with a single final
 * rounding; decline unsupported shapes, validate before dispatch).
 *
 * Conventions
 *   - Every pointer inside the argument lists is a DEVICE pointer on the
 *     current device unless a comment says host; the stream belongs to that
 *     device too. The calls keep nothing of their arguments, own no workspace,
 *     allocate nothing, and may be captured into a CUDA graph (make a first
 *     call on the device before a capture: it loads the kernels). Calls on
 *     different streams or from several host threads are independent.
 *   - Calls are asynchronous on the stream. Argument errors are returned by the
 *     host checks and nothing is launched. moe_ops_check reports a device-side
 *     wait that gave up.
 *   - Results do not depend on timing: the order of every sum is fixed by the
 *     sizes, types and alignment alone.
 *   - Sums run in f32; each result is rounded once, to the output's type. A
 *     product of two 16-bit values is exact in f32. Infinities and NaN of an
 *     input reach only the outputs that read it. An activation adds a relative
 *     error of about 2^-18, also where it is tiny.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of the operators besides MOE_DTYPE_BF16 (MOE_DTYPE_F32 is
 * declined by the products and the combine) */
enum { MOE_DTYPE_F16 = 2 };

/* activation of a product's epilogue */
enum {
    MOE_EPI_NONE = 0,
    MOE_EPI_SILU = 1,      /* z / (1 + exp(-z)) */
    MOE_EPI_GELU = 2,      /* z/2 (1 + erf(z / sqrt 2)) */
    MOE_EPI_GELU_TANH = 3  /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
};

/* The weights and the epilogue of a product (host struct). With w_up the
 * product is gated: out = act(x w^T + bias) * (x w_up^T + bias_up). All 16-bit
 * arrays have the type `dtype`. */
typedef struct {
    int dtype;              /* MOE_DTYPE_BF16 or MOE_DTYPE_F16: x, weights, biases,
                               residual and out */
    int E;                  /* experts, 1..1024 (moe_linear: 1) */
    int N;                  /* output columns, >= 1 */
    int K;                  /* input columns, >= 8, a multiple of 8 */
    const void *w;          /* [E, N, K], 16-byte aligned */
    const void *w_up;       /* [E, N, K], or NULL (not gated); strides as w's */
    int64_t ldw;            /* elements from row to row, >= K, a multiple of 8 */
    int64_t stride_e;       /* elements from expert to expert, a multiple of 8, >= 0
                               (E = 1: ignored) */
    const void *bias;       /* [E, N] dense, or NULL */
    const void *bias_up;    /* [E, N] dense, or NULL; needs w_up */
    int activation;         /* MOE_EPI_* */
    float act_limit;        /* 0: no clamp. > 0 (gated products only): the clamp
                               bound L, act(min(g, L)) * min(max(u, -L), L) */
} moe_product;

/* out[r] = epilogue(x[r]) (+ residual[r]) for r in 0..n-1.
 *   x         [n, K], rows ldx elements apart (>= K, a multiple of 8), 16-byte aligned
 *   residual  [n, N], rows ldr elements apart (>= N), or NULL
 *   out       [n, N], rows ldo elements apart (>= N); columns N.. of a row are not
 *             written. It may be `residual` itself (same pointer and row distance);
 *             it overlaps no other input.
 * Alignment of residual and out beyond their type's is not needed; rows at
 * multiples of 16 bytes are faster. n = 0 launches nothing.
 * INVALID_ARG: a null pointer (p, w, x, out), negative n, a bad field of *p, a
 * bad row distance, a misaligned pointer, E != 1. UNSUPPORTED: dtype f32, K not
 * a multiple of 8, K > 65536, N > 1048576, n > 16777216, E > 1024. */
moe_status moe_linear(const moe_product *p, const void *x, int64_t ldx, int n,
                      const void *residual, int64_t ldr, void *out, int64_t ldo, void *stream);

/* out[r] = epilogue of expert e for the rows r in offsets[e]..offsets[e+1]-1,
 * for every e. The row's input is x[r], or x[row_token[r]] with row_token.
 *   offsets    [E + 1] int32, ascending, 0 <= offsets[e] <= rows, as
 *              moe_group_slots writes them
 *   row_token  [rows] int32 in 0..x_rows-1 for the rows in use, or NULL
 *   x          [x_rows, K] (without row_token x_rows >= rows), as for moe_linear
 *   out        [rows, N] as for moe_linear. Rows outside every group
 *              (offsets[E].. ) are left as they were.
 * The offsets are read on the device only. Values outside their bounds are
 * clamped to them and a token outside 0..x_rows-1 is replaced by one inside:
 * nothing out of range is read or written, and the rows concerned hold values
 * that mean nothing. rows = 0 launches nothing. Errors as for moe_linear;
 * x_rows = 0 with rows > 0 is INVALID_ARG. */
moe_status moe_grouped_linear(const moe_product *p, const int32_t *offsets, const int32_t *row_token,
                              const void *x, int64_t ldx, int x_rows, int rows,
                              void *out, int64_t ldo, void *stream);

/* Group the n * top_k slots (token t, rank j) by the expert topk_idx[t, j]:
 * slots in the order of their expert, then token, then rank.
 *   topk_idx    [n, top_k] int32; ids outside expert_begin..expert_end-1 (other
 *               shards' experts, -1 for a dropped slot) belong to no group
 *   offsets     [E + 1]: the groups' first rows; offsets[E] is the number of rows
 *   slot_token  [n * top_k]: the row's token; -1 from offsets[E] on
 *   slot_k      [n * top_k]: the row's rank; -1 from offsets[E] on; or NULL
 *   slot_of     [n, top_k]: the slot's row; -1 where it belongs to no group
 * An id that a token lists twice makes two rows. n = 0 writes offsets only. The
 * outputs overlap neither topk_idx nor one another.
 * INVALID_ARG: a null pointer, negative n, top_k < 1, E < 1, an expert range
 * other than 0 <= expert_begin <= expert_end <= E, a pointer that is not 4-byte
 * aligned. UNSUPPORTED: E > 1024, top_k > 64, n * top_k > 16777216. */
moe_status moe_group_slots(const int32_t *topk_idx, int n, int top_k, int E, int expert_begin,
                           int expert_end, int32_t *offsets, int32_t *slot_token, int32_t *slot_k,
                           int32_t *slot_of, void *stream);

/* out[t] = sum over the ranks j in order of topk_w[t,j] * y[slot_of[t,j]]
 * (+ residual[t]). A slot_of outside 0..rows-1 adds nothing, whatever its weight.
 *   y         [rows, N] of dtype, rows ldy elements apart (>= N)
 *   slot_of   [n, top_k] int32; topk_w [n, top_k] f32
 *   residual  [n, N] or NULL; out [n, N]; ldr, ldo, aliasing and alignment as
 *             for moe_linear
 * n = 0 launches nothing; rows may be 0 (every slot then adds nothing).
 * INVALID_ARG: a null pointer (y with rows = 0 excepted), a negative size, top_k
 * < 1, N < 1, a bad row distance, a misaligned pointer. UNSUPPORTED: dtype not
 * bf16 or f16, top_k > 64, N > 1048576, n > 16777216. */
moe_status moe_combine_slots(int dtype, const void *y, int64_t ldy, int rows, const int32_t *slot_of,
                             const float *topk_w, int n, int top_k, int N, const void *residual,
                             int64_t ldr, void *out, int64_t ldo, void *stream);

/* ---- routing ---------------------------------------------------------------------- */

enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };

/* How a router's logits become ids and weights (host struct). For one row l:
 *   s_e = exp(l_e) / sum exp(l), or 1 / (1 + exp(-l_e))          the scores
 *   c_e = s_e + bias_e                                           what decides
 * With groups > 1 the experts form that many groups of neighbours, a group's score
 * is its best c (group_best 1) or the sum of its best two (2; of one where it has
 * one), and only the top_groups best groups stay. The ids are those of the top_k
 * largest c that stay, in falling order; ties, of groups too, go to the lower number.
 * The weights are the s of those ids (without the bias), divided by their sum with
 * renormalize, times scale.
 * An expert whose logit is -inf or NaN, or whose bias is, takes no part; where
 * fewer than top_k are left, the last ids are -1 and their weights 0 (moe_group_slots
 * and moe_combine_slots leave such slots out). Logits of +inf are the limit: they
 * share a softmax's whole mass. The choice is that of exact scores: without a bias the
 * order of the logits, with one that of c in f64. */
typedef struct {
    int E;              /* experts, 1..1024 */
    int top_k;          /* 1..64, at most the experts of top_groups groups */
    int score;          /* MOE_SCORE_* */
    int groups;         /* 1..32, a divisor of E */
    int top_groups;     /* 1..groups */
    int group_best;     /* 1 or 2 */
    int renormalize;    /* 0 or 1 */
    float scale;        /* finite */
    const float *bias;  /* [E] on the device, or NULL */
} moe_router;

/* Route n rows of logits.
 *   logits    [n, E] of dtype (bf16, f16 or f32), rows ldl elements apart (>= E)
 *   topk_idx  [n, top_k] int32; topk_w [n, top_k] f32; they overlap no input
 * Alignment beyond the type's is not needed; rows at multiples of 16 bytes are faster.
 * n = 0 launches nothing. INVALID_ARG: a null pointer, negative n, a bad field of *r,
 * a bad row distance, a misaligned pointer, another dtype. UNSUPPORTED: E > 1024, top_k > 64,
 * groups > 32, n * top_k > 16777216. */
moe_status moe_route(const moe_router *r, int dtype, const void *logits, int64_t ldl, int n, int32_t *topk_idx,
                     float *topk_w, void *stream);

/* ---- products of 8-bit codes ------------------------------------------------------ */

/* codes[r,k] = round(127 x[r,k] / m), scale[r] = m / 127 with m = max_k |x[r,k]|: the
 * codes of the exact quotient, halves to even, so that x is about codes * scale and
 * no code is -128. Rows of weights are quantised the same way.
 *   x      [n, K] of dtype (bf16 or f16), rows ldx elements apart (>= K)
 *   codes  [n, K] int8, rows ldc apart (>= K; moe_linear_q8 wants a multiple of 16)
 *   scale  [n] f32
 * A row of zeros has codes and scale 0. A row with an infinity or a NaN has codes 0 and
 * an infinite or NaN scale: a product makes NaN of it, in that row alone. The outputs
 * overlap nothing. Alignment beyond the types' is not needed; rows of x at multiples of
 * 16 bytes and of codes at 8, with K a multiple of 8, are faster. n = 0 launches nothing.
 * INVALID_ARG: a null pointer, negative n, K < 1, a bad row distance, a misaligned
 * pointer. UNSUPPORTED: another dtype, K > 1048576, n > 16777216. */
moe_status moe_quantize_rows(int dtype, const void *x, int64_t ldx, int n, int K, int8_t *codes, int64_t ldc,
                             float *scale, void *stream);

/* The weights and the epilogue of a product of codes (host struct), as moe_product:
 *   z[r,c] = x_scale[r] scale[c] sum_k x[r,k] w[c,k] + bias[c]
 * (and z_up likewise from w_up, scale_up and bias_up), out = act(z) [* z_up]. Any int8
 * value may occur, -128 too. */
typedef struct {
    int dtype;              /* MOE_DTYPE_BF16 or MOE_DTYPE_F16: biases, residual and out */
    int E;                  /* experts, 1..1024 (moe_linear_q8: 1) */
    int N;                  /* output columns, >= 1 */
    int K;                  /* input columns, >= 16, a multiple of 16 */
    const int8_t *w;        /* [E, N, K], 16-byte aligned */
    const int8_t *w_up;     /* [E, N, K], or NULL (not gated); strides as w's */
    int64_t ldw;            /* bytes from row to row, >= K, a multiple of 16 */
    int64_t stride_e;       /* bytes from expert to expert, a multiple of 16, >= 0
                               (E = 1: ignored) */
    const float *scale;     /* [E, N] dense */
    const float *scale_up;  /* [E, N] dense, with w_up */
    const void *bias;       /* [E, N] dense, or NULL */
    const void *bias_up;    /* [E, N] dense, or NULL; needs w_up */
    int activation;         /* MOE_EPI_* */
    float act_limit;        /* as moe_product's */
} moe_product_q8;

/* moe_linear and moe_grouped_linear on codes: x is int8 with rows ldx bytes apart (>= K, a
 * multiple of 16), 16-byte aligned, and x_scale holds a scale for each row of x. All
 * else, limits and errors included, is as there. The sum of products is exact up to
 * 2^24 in magnitude (whatever the codes for K <= 1024) and otherwise an f32 sum, and is
 * scaled (by a weight's scale first: with scales of W up to 2^97 nothing overflows that the row's
 * scale brings back into range), activated and rounded once. An infinite or NaN scale reaches its
 * own row or column only. UNSUPPORTED: K not a multiple of 16. */
moe_status moe_linear_q8(const moe_product_q8 *p, const int8_t *x, int64_t ldx, const float *x_scale, int n,
                         const void *residual, int64_t ldr, void *out, int64_t ldo, void *stream);
moe_status moe_grouped_linear_q8(const moe_product_q8 *p, const int32_t *offsets, const int32_t *row_token,
                                 const int8_t *x, int64_t ldx, const float *x_scale, int x_rows, int rows, void *out,
                                 int64_t ldo, void *stream);

/* Synchronise `stream` and report a device-side wait of these operators on the
 * current device that gave up (MOE_ERR_TIMEOUT: every wait inside a kernel is
 * bounded, about 1 s; outputs since the last check are then invalid), then
 * clear it. The word is the device's: one check reports, once, for the calls of
 * every stream and thread, so a program has one place that checks. Not for a
 * stream that is being captured. */
moe_status moe_ops_check(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
