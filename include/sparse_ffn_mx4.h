/*
 * sparse_ffn_mx4.h -- rows in 4-bit blocks, products of such rows, and the norm in front of 8- and
 * 4-bit products, beside the FFNs of sparse_ffn.h and the 8-bit rows of sparse_ffn_experts.h (same
 * library, same conventions).
 *
 * A norm stands before every layer, and the products after it read its output in 8 bits
 * (sparse_ffn_i8_matmul) or in 4 (sparse_ffn_mx4_matmul): sparse_ffn_rms_norm adds the residual,
 * normalises and writes the row in the form that they read. Weights in 4-bit blocks are half as
 * many bytes as weights in 8 bits.
 *
 * Conventions of sparse_ffn.h hold: device pointers owned by the caller, `stream` a hipStream_t of
 * the current device, nothing synchronizes or allocates, every argument is checked on the host
 * before anything is enqueued, and every result is bitwise reproducible. Outputs and work must not
 * overlap each other or the inputs, but where it is said. Calls can be captured in a HIP graph.
 * Calls that share a `work` buffer must be ordered, and so must the replays of graphs that hold
 * such calls.
 *
 * 4-bit blocks. A row of K numbers is held in ceil(K / 32) blocks of 32, the last one filled up
 * with zeros. A block is 16 bytes of codes and a byte E, its scale 2^(E - 127). With m the block's
 * largest magnitude, E - 127 is the e with 3.5 * 2^e <= m < 7 * 2^e, and at least -127 (E 0, for
 * zeros too). A code stands for 0, 0.5, 1, 1.5, 2, 3, 4 or 6 (codes 0 to 7; plus 8: negative) times
 * the scale: the one nearest to the number, ties to the even code. Two codes are a byte, the first
 * one in its low half. A block with an infinity or a NaN has E = 255 and codes 0: everything
 * computed from it is NaN. These are the elements (E2M1) and scales (E8M0) of the microscaling
 * format MXFP4; rows from elsewhere may hold any codes and scales.
 *
 * Layout: codes are row-major bytes; a row starts at a multiple of 16 bytes, ldq bytes after the
 * one before it (a multiple of 16, at least 16 bytes for every block; above 2^24
 * SFFN_ERR_UNSUPPORTED). Scales are row-major bytes too; a row starts at a multiple of 16 bytes,
 * lds after the one before it (a multiple of 16, at least a byte for every block; above 2^24
 * SFFN_ERR_UNSUPPORTED). Bytes between the scales' end and the next multiple of 16 are read and
 * have no effect.
 */
#ifndef SPARSE_FFN_MX4_H
#define SPARSE_FFN_MX4_H

#include "sparse_ffn_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further value of dtype arguments, for the calls of this header only. */
enum { SFFN_MX4 = 4 };

/* longest row of a 4-bit product */
#define SFFN_MX4_MAX_K (1 << 20)

/* Root-mean-square norm, with the residual's addition in front of it:
 *   v = x, or x + residual rounded to x's type, written to sum: the residual as it goes on
 *   y_j = v_j w_j / sqrt((v_0^2 + ... + v_{cols-1}^2) / cols + eps)
 * in 64 bits up to one rounding: to y_dtype (SFFN_F32, SFFN_F16, SFFN_BF16), or to 32 bits before
 * the row is held in 8 bits (SFFN_I8) or in 4-bit blocks (SFFN_MX4), which gives bitwise what
 * sparse_ffn_quantize_rows or sparse_ffn_quantize_mx4 gives for the SFFN_F32 output.
 * x: device, `rows` rows of `cols` values of dtype (SFFN_F32, SFFN_F16, SFFN_BF16), ldx elements
 * apart; residual and sum: device, rows of the same type, ldr and ldsum elements apart, both or
 * neither (NULL). w: device, cols values of w_dtype (SFFN_F32, SFFN_F16, SFFN_BF16), or NULL (1).
 * eps: 0, or a positive normal number. y: device, rows ldy elements (SFFN_I8, SFFN_MX4: bytes) apart; what
 * lies between the rows is left as it was, but that 8-bit rows are filled with zeros to a multiple
 * of 16. scale: SFFN_I8: device fp32 [rows] (lds is not read); SFFN_MX4: device, rows of scales lds
 * bytes apart; otherwise NULL. sum may lie over residual or over x, row on row; a float y of x's
 * type over x or residual likewise (not where sum does). rows >= 0 (0: nothing happens); cols
 * above 2^31 - 1024: SFFN_ERR_UNSUPPORTED. */
int sparse_ffn_rms_norm(const void* x, int32_t dtype, int64_t ldx, const void* residual,
                        int64_t ldr, int32_t rows, int32_t cols, const void* w, int32_t w_dtype,
                        double eps, void* sum, int64_t ldsum, void* y, int32_t y_dtype,
                        int64_t ldy, void* scale, int64_t lds, void* stream);

/* Rows of numbers into 4-bit blocks. For weights offline (a row per output channel) and for
 * activations that several products share (a row per token). x: device, `rows` rows of `cols`
 * values (SFFN_F32, SFFN_F16 or SFFN_BF16), ldx elements apart; q, scale: device, as above; what
 * lies between the rows is left as it was. rows >= 0; cols above 2^31 - 1024:
 * SFFN_ERR_UNSUPPORTED. */
int sparse_ffn_quantize_mx4(const void* x, int32_t dtype, int64_t ldx, int32_t rows, int32_t cols,
                            uint8_t* q, int64_t ldq, uint8_t* scale, int64_t lds, void* stream);

/* The values that rows in 4-bit blocks stand for, the first `cols` of each: y: device, rows ldy
 * elements apart (SFFN_F32: exact, but infinite from 2^128 on, which E 253 and 254 reach; SFFN_F16,
 * SFFN_BF16: those rounded once). */
int sparse_ffn_dequantize_mx4(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds,
                              int32_t rows, int32_t cols, void* y, int32_t dtype, int64_t ldy,
                              void* stream);

/* y = x W^T (+ bias) with x and W in 4-bit blocks:
 *   y[t][n] = sum over blocks b of 2^(Ex[t][b] + Ew[n][b] - 254) sum_j x_j w_j  (+ bias[n])
 * The products are exact; the sums are held in 32 bits, in an order that M, N and K decide; rounded
 * once to y_dtype. Rows that the call holds in 4-bit blocks and the same rows held before give the
 * same bits.
 * x: device, M rows of K values, ldx elements apart. SFFN_F32, SFFN_F16, SFFN_BF16: each row is
 * held in 4-bit blocks as above first (x_scale NULL, ldxs is not read). SFFN_MX4: codes, ldx bytes
 * apart, with their scales x_scale, ldxs bytes apart; K is then 32 for each block. w: device, codes
 * of N rows of ceil(K / 32) blocks, ldw bytes apart, w_scale: their scales, ldws bytes apart; bias:
 * device fp32 [N] or NULL; y: device, M rows of N values of y_dtype (SFFN_F32, SFFN_F16,
 * SFFN_BF16), ldy elements apart; what lies between the rows is left as it was. work: device
 * scratch, 256-byte aligned, of at least sparse_ffn_mx4_matmul_work_bytes() (0 bytes: may be
 * NULL). M >= 0, 1 <= K <= SFFN_MX4_MAX_K. SFFN_ERR_UNSUPPORTED: K above that, M or N above
 * 2^31 - 1024, or 2^23 - 8 tiles of 256 x 256 outputs or more, which no launch holds. The size
 * query returns (size_t)-1 for an argument it cannot size. */
size_t sparse_ffn_mx4_matmul_work_bytes(int32_t x_dtype, int32_t M, int32_t N, int32_t K);
int sparse_ffn_mx4_matmul(const void* x, int32_t x_dtype, const uint8_t* x_scale, int64_t ldx,
                          int64_t ldxs, int32_t M, int32_t K, const uint8_t* w, int64_t ldw,
                          const uint8_t* w_scale, int64_t ldws, const float* bias, int32_t N,
                          void* y, int32_t y_dtype, int64_t ldy, void* work, size_t work_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPARSE_FFN_MX4_H */
