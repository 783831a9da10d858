/*
 * sparse_ffn_experts.h -- expert layers with 8-bit weights, beside the neuron-sparse FFN of
 * sparse_ffn.h (same library, same conventions).
 *
 * sparse_ffn.h computes the part of one FFN that a predictor selects, neuron by neuron. A
 * mixture-of-experts layer selects whole FFNs: a router scores E experts for every token
 * (sparse_ffn_route), and each token goes through its k experts only (sparse_ffn_experts).
 * The experts' weights, and any other weight matrix (sparse_ffn_i8_matmul), are held in 8
 * bits with one scale per output channel, and the activations that meet them in 8 bits with
 * one scale per token; the products are sums of whole numbers on the matrix cores.
 *
 * Conventions of sparse_ffn.h hold: device pointers owned by the caller, `stream` a
 * hipStream_t of the current device, nothing synchronizes or allocates, every argument is
 * checked on the host before anything is enqueued, and every result is bitwise reproducible.
 * Outputs and work must not overlap each other or the inputs (sparse_ffn_experts may write its y
 * over its x). Calls can be captured in a HIP graph. Calls that share a `work` buffer must be ordered, and
 * so must the replays of graphs that hold such calls.
 *
 * 8-bit rows. A row r of numbers is held as q and s: s is max|r| times the 32-bit float
 * nearest to 1 / 127, rounded to 32 bits, and q_j the whole number nearest to r_j / s, ties to
 * even, decided exactly (|q| <= 127). A row whose largest magnitude is below 2^-100 is held as zeros with
 * s = 0; a row with an infinity or a NaN as zeros with s = NaN, so that everything computed
 * from it is NaN.
 *
 * Layout: int8 matrices are row-major with one row per output channel; a row starts at a
 * multiple of 16 bytes and `ld` bytes after the one before it (ld a multiple of 16, at least
 * the row length rounded up to 16; above 2^24 SFFN_ERR_UNSUPPORTED). Bytes between a row's end and the next multiple of 16 are
 * read and have no effect.
 */
#ifndef SPARSE_FFN_EXPERTS_H
#define SPARSE_FFN_EXPERTS_H

#include "sparse_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further values of dtype arguments, for the calls of this header only. */
enum { SFFN_BF16 = 2, SFFN_I8 = 3 };

enum { SFFN_SCORE_SOFTMAX = 0, SFFN_SCORE_SIGMOID = 1 };

#define SFFN_MAX_EXPERTS 1024 /* experts of one layer */
#define SFFN_MAX_TOPK 64      /* experts of one token */
/* longest row of an 8-bit product: its sums fit 32 bits for any 8-bit values */
#define SFFN_I8_MAX_K 131071

/* Router: for each of T tokens the k experts it goes to, best first, and their weights.
 *   s_e = softmax or sigmoid (score) of the token's logits
 *   c_e = s_e + bias_e; without a bias the logit itself (the order of the scores)
 *   groups > 1: experts form `groups` groups of E / groups neighbours; a group is worth its
 *     best c_e (group_top 1) or the sum of its two best scores c_e (group_top 2; without a
 *     bias the two best s_e); only the top_groups most valuable groups stay
 *   idx: the k largest c_e of what stays, in descending order; weights: their s_e (without
 *     the bias), divided by their sum when renormalize is 1 (all 0 where that sum is 0, as it
 *     is for sigmoids of logits below -709.78, which are 0 in 64 bits), times scale.
 * Scores are compared in 64 bits; ties go to the lower index. Weights are computed in 32 bits
 * (in 64 where the choice needed them): off by a few 2^-24 of their value where the logits lie
 * close together, and by less than 2^-15 of it, or 2^-126 scale, wherever they lie. An expert
 * whose logit is minus infinity or NaN takes no part in the softmax. Neither it nor one whose
 * c_e is minus infinity or NaN (by its bias) is ever chosen or counts in its group's worth;
 * slots for which no expert is left hold idx -1 and weight 0.
 * logits: device [T] rows of E values (dtype SFFN_F32, SFFN_F16 or SFFN_BF16), ld elements
 * apart (ld >= E); bias: device [E] fp32 or NULL; idx: device int32 [T][k]; weights: device
 * fp32 [T][k]. T >= 0 (0: nothing happens), 1 <= k <= min(E, SFFN_MAX_TOPK), E <=
 * SFFN_MAX_EXPERTS, groups divides E and is at most 64. */
int sparse_ffn_route(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                     int32_t k, int32_t score, const float* bias, int32_t groups,
                     int32_t top_groups, int32_t group_top, int32_t renormalize, float scale,
                     int32_t* idx, float* weights, void* stream);

/* Rows of numbers into 8 bits (see above): q row r at q + r * ldq, scale[r]. For weights
 * offline (a row per output channel) and for activations that several products share (a row
 * per token). x: device, `rows` rows of `cols` values (SFFN_F32, SFFN_F16 or SFFN_BF16), ldx
 * elements apart; q: device, 16-byte aligned, ldq a multiple of 16 and at least cols rounded
 * up to 16 (the bytes from cols to that multiple are written as zeros); scale: device fp32
 * [rows]. rows >= 0; cols above 2^31 - 1024: SFFN_ERR_UNSUPPORTED. */
int sparse_ffn_quantize_rows(const void* x, int32_t dtype, int64_t ldx, int32_t rows,
                             int32_t cols, int8_t* q, int64_t ldq, float* scale, void* stream);

/* y = x W^T (+ bias) with 8-bit weights:
 *   y[t][n] = (sum_j qx[t][j] w[n][j]) * (sx[t] * w_scale[n]) + bias[n]
 * the sum exact in 32-bit whole numbers, the rest in fp32, rounded once to y_dtype.
 * x: device, M rows of K values, ldx elements apart. SFFN_F32, SFFN_F16, SFFN_BF16: each row
 * is held in 8 bits as above first (x_scale NULL). SFFN_I8: the rows are qx already and
 * x_scale is sx, device fp32 [M]. w: device int8, N rows of K, 16-byte aligned, ldw bytes
 * apart; w_scale: device fp32 [N]; bias: device fp32 [N] or NULL; y: device, M rows of N
 * values of y_dtype (SFFN_F32, SFFN_F16, SFFN_BF16), ldy elements apart; what lies between
 * the rows is left as it was. work: device scratch, 256-byte aligned, of at least
 * sparse_ffn_i8_matmul_work_bytes() (0 bytes: may be NULL). M >= 0, 1 <= K <= SFFN_I8_MAX_K.
 * SFFN_ERR_UNSUPPORTED: K above that, M or N above 2^31 - 1024, or more tiles of output than one
 * launch holds (possible from 2^36 outputs on). The size query returns (size_t)-1 for an argument
 * it cannot size. */
size_t sparse_ffn_i8_matmul_work_bytes(int32_t x_dtype, int32_t M, int32_t N, int32_t K);
int sparse_ffn_i8_matmul(const void* x, int32_t x_dtype, const float* x_scale, int64_t ldx,
                         int32_t M, int32_t K, const int8_t* w, int64_t ldw,
                         const float* w_scale, const float* bias, int32_t N, void* y,
                         int32_t y_dtype, int64_t ldy, void* work, size_t work_bytes,
                         void* stream);

/* E ReLU FFNs with 8-bit weights. The call reads the descriptor and keeps nothing of it. */
typedef struct {
  int32_t experts;  /* E, 1 .. SFFN_MAX_EXPERTS */
  int32_t d;        /* model dimension */
  int32_t d_ffn;    /* neurons of one expert */
  int32_t gated;    /* 0: h = relu(W_up x + b);  1: h = relu(W_gate x + b) * (W_up x) */
  const int8_t* w_act;      /* device [E][d_ffn][d], gated [E][d_ffn][2][d] (a neuron's gate
                               row, then its up row), rows ld_act bytes apart throughout */
  int64_t ld_act;
  const float* act_scale;   /* device [E][d_ffn], gated [E][d_ffn][2] */
  const float* b_act;       /* device [E][d_ffn]: bias inside the ReLU; NULL = 0 */
  const int8_t* w_down;     /* device [E][d][d_ffn], rows ld_down bytes apart throughout */
  int64_t ld_down;
  const float* down_scale;  /* device [E][d] */
} sffn_experts_desc;

/* The routed experts' FFNs: y_t = sum over the slots s of token t, in slot order, of
 *   weights[t][s] * W_down[e] h,  e = idx[t][s],  h = relu(...) as above for expert e,
 * x_t and h held in 8 bits as described above; h is the 32-bit float nearest to its value
 * before that (computed in 64 bits from the exact sums), the down product is scaled and summed
 * in fp32. A slot whose idx is negative or at least E has no expert: it adds nothing, and its
 * weight is not read. A token with no expert gets y = 0. An expert named twice counts twice.
 * With E = 1, idx 0 and weight 1 this is one dense FFN with 8-bit weights.
 * x: device, T rows of d values (SFFN_F32, SFFN_F16, SFFN_BF16), ldx elements apart; idx:
 * device int32 [T][k]; weights: device fp32 [T][k]; y: device, T rows of d values of y_dtype,
 * ldy elements apart, fully overwritten (what lies between the rows is left as it was). work:
 * device scratch, 256-byte aligned, of work_bytes >= sparse_ffn_experts_work_bytes(desc, 1,
 * k): the tokens go through in chunks of the most that fit, so pass the size for T tokens
 * where memory allows. y may lie over x, in rows of any distance; where the tokens go through in
 * chunks and no order of them would keep the inputs of later ones, SFFN_ERR_INVALID (an order is
 * found whenever y begins where x does). T >= 0, 1 <= k <= SFFN_MAX_TOPK, d and d_ffn at most SFFN_I8_MAX_K.
 * The size query returns 0 for an argument it cannot size. */
size_t sparse_ffn_experts_work_bytes(const sffn_experts_desc* desc, int32_t tokens, int32_t k);
int sparse_ffn_experts(const sffn_experts_desc* desc, const void* x, int32_t x_dtype,
                       int64_t ldx, int32_t T, const int32_t* idx, const float* weights,
                       int32_t k, void* y, int32_t y_dtype, int64_t ldy, void* work,
                       size_t work_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_FFN_EXPERTS_H */
