/*
 * f8.h — the E4M3 part of the library's C ABI (libq4.so): 8-bit floating-point
 * matrices with one f32 scale for each block of 128.
 *
 * Format. E4M3: 1 sign, 4 exponent (bias 7) and 3 fraction bits; subnormals
 * down to 2^-9, largest value 448 (0x7E), no infinities, 0x7F and 0xFF are NaN.
 *   - Activations: codes [M, K], one byte each, and scales [M, ceil(K / 128)]
 *     f32: element (m, k) = code * scale[m, k / 128].
 *   - Weights: codes [N, K] and scales [ceil(N / 128), ceil(K / 128)] f32:
 *     element (n, k) = code * scale[n / 128, k / 128].
 *   All arrays are dense and row-major. K is a positive multiple of 32; the
 *   last block of a row, and the last row of tiles, may be short.
 *
 * The conventions of q4.h hold here too: device pointers owned by the caller
 * and 16-byte aligned, arguments checked before anything is launched, outputs
 * that overlap no input, asynchronous work on `stream`, nothing allocated, no
 * state kept, the same Q4_* status codes, empty problems Q4_OK. Every entry
 * point may be captured in a HIP graph, needs no workspace, and is
 * deterministic. Inputs are finite, where an entry point states nothing else.
 */
#ifndef Q4MI_F8_H
#define Q4MI_F8_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns of a block, and the largest K of the products. */
#define F8_BLOCK 128
#define F8_MAX_K 4194304

/*
 * f8_quantize — f32 [M, K] to E4M3 codes and scales.
 *   x           [M, K] f32.
 *   block_rows  1: one scale per 128 columns of a row (activations);
 *               128: one per 128 x 128 tile (weights). Else Q4_ERR_SHAPE.
 *   q, q_bytes  codes; q_bytes == M * K (else Q4_ERR_SIZE).
 *   s, s_elems  scales; s_elems == ceil(M / block_rows) * ceil(K / 128) (else
 *               Q4_ERR_SIZE; also when that is 2^31 or more). q and s must
 *               not overlap (Q4_ERR_ALIAS).
 * Per block: scale = max|x| / 448, rounded to f32; code = the E4M3 value
 * nearest to x / scale, ties to even, where the quotient is first rounded to
 * f32 and clamped to [-448, 448] (the scale is rounded, so the largest quotient
 * can be a step of f32 past 448; farther only for a subnormal scale). -0 and
 * negative quotients that round to zero are 0x80. A block whose scale is 0
 * stores codes 0. Bit-exact. NaN elements get a NaN code (0x7F or 0xFF), the scale
 * comes from the others; a block with an infinity has the scale inf.
 */
int f8_quantize(const float *x, int M, int K, int block_rows, void *q, size_t q_bytes, float *s,
                size_t s_elems, void *stream);

/* f8_quantize_bf16 — f8_quantize of bfloat16 values (raw 16-bit patterns). */
int f8_quantize_bf16(const uint16_t *x, int M, int K, int block_rows, void *q, size_t q_bytes,
                     float *s, size_t s_elems, void *stream);

/*
 * f8_dequant — codes and scales to f32: out[m, k] = code * scale, rounded
 * once. Arguments and errors as f8_quantize, with out [M, K] f32 and
 * out_elems == M * K (else Q4_ERR_SIZE). Bit-exact.
 */
int f8_dequant(const void *q, size_t q_bytes, const float *s, size_t s_elems, int M, int K,
               int block_rows, float *out, size_t out_elems, void *stream);

/*
 * f8_gemm — y = a @ w^T for any M >= 1:
 *   y[m, n] = sum_b a_s[m, b] w_s[n / 128, b] sum_{k in block b} a[m, k] w[n, k].
 *   a, a_s      activations: codes [M, K], scales [M, ceil(K / 128)].
 *   w, w_bytes  weight codes, w_bytes == N * K (else Q4_ERR_SIZE).
 *   w_s         weight scales [ceil(N / 128), ceil(K / 128)].
 *   y           [M, N] bfloat16, as raw 16-bit patterns.
 *   M, N >= 0; K >= 32, K % 32 == 0, K <= F8_MAX_K (else Q4_ERR_SHAPE).
 * Accuracy, per element, with P the sum over k of |a w| (scales included):
 *   |y - exact| <= 2^-8 |exact| + 1.01 (7 * 2^-13 + (24 + K / 128) 2^-23) P.
 * The first term is y's rounding to bfloat16 (at most half a step). The second
 * is the matrix core's: it adds eight products at a time and drops what is
 * below 2^-13 of the largest one's power of two. On normal data that is about
 * 2^-16 of the result, far below the first term. The blocks are added in f32,
 * each times a_s w_s, which is formed in f32: below 2^-126 it is a multiple of
 * 2^-149, and the bound is 2^-150 (sum over k of the codes' |a w| + K / 64) +
 * 2^-134 wider; from 2^128 on its block counts as infinite, or NaN where the
 * codes' sum is 0. f8_quantize makes such scales of values near f32's ends only.
 */
int f8_gemm(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes, const float *w_s,
            uint16_t *y, int M, int N, int K, void *stream);

/* f8_gemv — f8_gemm for 1 <= M <= Q4_GEMV_MAX_ROWS rows (else Q4_ERR_SHAPE;
 * M == 0 is an empty problem): the decode-shaped call. */
int f8_gemv(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes, const float *w_s,
            uint16_t *y, int M, int N, int K, void *stream);

/*
 * f8_gemm_grouped — q4.h's q4_gemm_grouped over E4M3 weights and activations:
 *   y[r, n] = sum_b a_s[r / share, b] w_s[e, n / 128, b] sum_{k in b} a w
 * for the rows r of each group e.
 *   a, a_s      codes [ceil(M / share), K], scales [.., ceil(K / 128)]; the
 *               codes span less than 2^31 bytes (else Q4_ERR_SHAPE).
 *   w, w_bytes  G weight matrices [N, K], w_bytes == G * N * K.
 *   w_s         their scales, [G, ceil(N / 128), ceil(K / 128)].
 *   y           [M, N] bfloat16. Rows that no group names are left as they were.
 *   offsets, order, share, G, M, and what wrong list contents do: as
 *   q4_gemm_grouped. K as f8_gemm. No workspace.
 * Accuracy: as f8_gemm. Deterministic for rows named once.
 */
int f8_gemm_grouped(const uint8_t *a, const float *a_s, const uint8_t *w, size_t w_bytes,
                    const float *w_s, const int32_t *offsets, const int32_t *order, int share,
                    uint16_t *y, int G, int M, int N, int K, void *stream);

/*
 * f8_norm, f8_norm_bf16 — q4.h's q4_norm (q4_norm_bf16) with y as E4M3 codes and a
 * scale for each 128 columns: what f8_quantize with block_rows 1 makes of its f32
 * y, bit for bit.
 *   q, q_bytes, s, s_elems  as f8_quantize (block_rows 1).
 *   y         [M, K] f32 (f8_norm_bf16: bfloat16) as well, or NULL (for a router,
 *             say).
 */
int f8_norm(const float *x, const float *weights, int share, const float *residual, float *sum,
            const float *gamma, float eps, float *y, void *q, size_t q_bytes, float *s,
            size_t s_elems, int M, int K, void *stream);
int f8_norm_bf16(const uint16_t *x, const float *weights, int share, const uint16_t *residual,
                 uint16_t *sum, const float *gamma, float eps, uint16_t *y, void *q, size_t q_bytes,
                 float *s, size_t s_elems, int M, int K, void *stream);

/*
 * f8_act, f8_act_bf16 — q4.h's q4_act (q4_act_bf16) with y as E4M3 codes and a
 * scale for each 128 columns: what f8_quantize with block_rows 1 makes of its f32
 * y, bit for bit. q, q_bytes, s, s_elems as there.
 */
int f8_act(const float *gate, const float *up, int ld, int act, void *q, size_t q_bytes, float *s,
           size_t s_elems, int M, int K, void *stream);
int f8_act_bf16(const uint16_t *gate, const uint16_t *up, int ld, int act, void *q, size_t q_bytes,
                float *s, size_t s_elems, int M, int K, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4MI_F8_H */
