/*
 * retro_mx.h - C ABI of the microscaled 4-bit operators and the
 * mixture-of-experts layer of the MI355X (gfx950) OUT_PROD library.
 *
 * The library's other calls contract F32 operands with a packed weight. These
 * make the 4-bit forms from float tensors, contract two 4-bit operands on the
 * scaled matrix cores, and run a whole expert layer over 4-bit experts.
 *
 * Microscaled 4-bit elements (OCP Microscaling, the MXFP4 element and scale of
 * retro_out_prod.h): 32 consecutive elements along the contraction share a
 * power-of-two scale byte e (value 2^(e - 127), e = 255 NaN); an element is an
 * E2M1 code q (sign, magnitude in {0, 0.5, 1, 1.5, 2, 3, 4, 6}); the value is
 * e2m1(q) * 2^(e - 127). Quantising a block with largest magnitude amax:
 *     e    = clamp(floor(log2(amax)) - 2 + 127, 0, 254), 0 when amax = 0
 *     q[i] = x[i] * 2^(127 - e) rounded to the nearest E2M1 value, a tie to
 *            the even code, magnitudes above 6 to 6; the sign bit is x[i]'s, also
 *            of what rounds to zero
 * A block that holds an infinity or a NaN gets e = 255: all of it is NaN, and its
 * codes are unspecified. These are exact statements: every call below returns
 * those bytes.
 *
 * A microscaled matrix of `rows` x K is two arrays, with C = ceil(K / 256):
 *   codes   rows x C x 128 bytes: element 2i of a row in the low nibble of its
 *           byte i, element 2i + 1 in the high nibble; zeros past K
 *   scales  C x rows x 8 bytes: the scale byte of block 8c + j of row r at
 *           (c * rows + r) * 8 + j; past K any byte but 255
 * Both must be 16-byte aligned. Rows of 128-byte steps keep every 16-byte load
 * of a block aligned, which the 17-byte packed blocks do not, and the scales of
 * a 256-element step of neighbouring rows lie side by side.
 *
 * Float tensors are RETRO_F32, RETRO_F16 or RETRO_BF16 with contiguous rows a
 * given number of elements apart (ld >= the row's length, any alignment of
 * whole elements).
 *
 * Execution and errors are those of retro_out_prod.h: asynchronous on the
 * stream, no allocation, no CPU fallback, negative codes, all checks made on
 * the host before any launch. An empty output returns RETRO_OK and touches
 * nothing. Sizes: every dimension below 2^31 and every array below 2^62 bytes;
 * the products also need ceil(T / 32) * ceil(N / 32) below 2^30 (RETRO_E_SHAPE).
 */
#ifndef RETRO_MX_H
#define RETRO_MX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the two arrays of a microscaled matrix; -1 for a size out of
 * range. Touch no device. */
int64_t retro_mx_code_bytes(int64_t rows, int64_t K);
int64_t retro_mx_scale_bytes(int64_t rows, int64_t K);

/*
 * Packed blocks from floats: row n of W (retro_row_bytes(type, K) bytes) holds
 * the blocks of X[n][0..K). type RETRO_MXFP4 (the rule above, K % 32 == 0) or
 * RETRO_NVFP4 (K % 64 == 0): per 16 elements the E4M3 scale S nearest to
 * amax / 6 (ties to even, at most 448) and each x[i] / S rounded to the nearest
 * E2M1 value (ties to the even code, at most 6, the sign bit x[i]'s); S = 0 gives
 * zeros with x's signs; an infinity or a NaN gives S = NaN (byte 0x7f) and
 * unspecified codes. The inverse of retro_dequantize up to the rounding. xtype is
 * X's type, ldx its row stride in elements.
 */
int retro_quantize(int type, int xtype, const void *X, int64_t ldx, void *W, int64_t K, int64_t N, void *stream);

/*
 * Microscaled matrices from X (rows x cols floats): along its rows (row_codes,
 * row_scales: a rows x cols matrix, blocks along a row), along its columns
 * (col_codes, col_scales: the cols x rows matrix of X's transpose, blocks along
 * a column), or both from one reading of X. Either pair may be NULL (one array
 * of a pair alone, or both pairs, is RETRO_E_NULL).
 */
int retro_mx_quantize(int xtype, const void *X, int64_t ldx, int64_t rows, int64_t cols, void *row_codes,
                      void *row_scales, void *col_codes, void *col_scales, void *stream);

/* Y[r][k] = the value of element k of row r (ytype, rounded to nearest even
 * where ytype cannot hold it). */
int retro_mx_dequantize(int ytype, const void *codes, const void *scales, void *Y, int64_t ldy, int64_t K,
                        int64_t rows, void *stream);

/* The microscaled matrix of the same values as N rows of packed RETRO_MXFP4
 * blocks (K % 32 == 0): a resident weight laid out for the calls below. */
int retro_mx_from_blocks(const void *W, void *codes, void *scales, int64_t K, int64_t N, void *stream);

/*
 * Y[t][n] = sum_k A[t][k] B[n][k] for t < T, n < N: A a T x K and B an N x K
 * microscaled matrix, Y of ytype with rows ldy elements apart. The sum of a block
 * pair's products is exact; the sum over blocks is taken in F32 and rounded to
 * ytype (to nearest) once. The matrix cores add two or four blocks' sums to an F32
 * accumulator at a time, not always to the nearest F32 (1 + 1.5 * 2^-24 gives 1
 * or 1 + 2^-23, by which of the two came first): before the rounding to ytype
 * the error is at most ceil(K / 64) * 2^-22 * sum_k |A[t][k] B[n][k]| (or 2^-149).
 * K == 0 writes zeros.
 */
int retro_mx_mul_mat(int ytype, const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales,
                     void *Y, int64_t ldy, int64_t K, int64_t N, int64_t T, void *stream);

/*
 * Kernels of the product, for tests and benchmarks (retro_mx_mul_mat chooses
 * one by shape):
 *   RETRO_MX_VARIANT_SIMPLE   a wave a 32 x 32 tile, operands from memory; any
 *                             shape, and the only one for T > 32 where offsets
 *                             pass 32 bits within a tile or the tiles' threads
 *                             2^32
 *   RETRO_MX_VARIANT_TILE_*   rows of A x rows of B a workgroup, staged in LDS;
 *                             _K4: four groups of waves take K's steps in turn
 *                             and add their sums
 *   RETRO_MX_VARIANT_SKINNY   T <= 32: 16 rows of B a workgroup, K dealt to its
 *                             waves, B read once from memory
 */
enum {
    RETRO_MX_VARIANT_AUTO = 0,
    RETRO_MX_VARIANT_SIMPLE = 1,
    RETRO_MX_VARIANT_TILE_256x256 = 2,
    RETRO_MX_VARIANT_TILE_128x128 = 3,
    RETRO_MX_VARIANT_TILE_64x128 = 4,
    RETRO_MX_VARIANT_TILE_64x64 = 5,
    RETRO_MX_VARIANT_SKINNY = 6,
    RETRO_MX_VARIANT_TILE_64x64_K4 = 7,
    RETRO_MX_VARIANT_TILE_32x64_K4 = 8,
    RETRO_MX_VARIANT_TILE_256x192 = 9
};

/* retro_mx_mul_mat with a forced kernel; RETRO_E_VARIANT when it does not take
 * the shape. */
int retro_mx_mul_mat_variant(int variant, int ytype, const void *a_codes, const void *a_scales, const void *b_codes,
                             const void *b_scales, void *Y, int64_t ldy, int64_t K, int64_t N, int64_t T,
                             void *stream);

/* The kernel retro_mx_mul_mat runs for a shape, or a negative error code.
 * Touches no device. */
int retro_mx_mul_mat_choice(int ytype, int64_t ldy, int64_t K, int64_t N, int64_t T);

/*
 * retro_mx_mul_mat with A quantised from X (T x K floats of xtype) in the call,
 * Y of X's type. workspace holds the quantised X where the kernel chosen for
 * the shape needs it: retro_mx_linear_workspace_size bytes (0 when it needs
 * none), 16-byte aligned, overlapping no operand (RETRO_E_WORKSPACE otherwise).
 */
int retro_mx_linear(int xtype, const void *X, int64_t ldx, const void *b_codes, const void *b_scales, void *Y,
                    int64_t ldy, int64_t K, int64_t N, int64_t T, void *workspace, int64_t workspace_bytes,
                    void *stream);
int64_t retro_mx_linear_workspace_size(int xtype, int64_t K, int64_t N, int64_t T);

/*
 * A whole mixture-of-experts layer for T <= RETRO_MOE_MAX_T tokens:
 *     l[t][e]  = sum_d x[t][d] R[e][d]                          (F32)
 *     the top_k largest l[t][.] choose the experts; a tie goes to the lower index
 *     p[t][j]  = exp(l[t][e_j] - m) / sum exp(l - m), the sum over the chosen
 *                experts (renormalize != 0) or over all E
 *     h[t][j]  = silu(gate[e_j] x[t]) * (up[e_j] x[t])          silu(v) = v / (1 + exp(-v))
 *     y[t]     = sum_j p[t][j] down[e_j] h[t][j]
 * x and y are T x D of xtype with rows ldx and ldy elements apart; R is E x D of
 * rtype (RETRO_F32 or xtype) with contiguous rows ldr elements apart; gate_up is
 * a microscaled matrix of E * 2F rows x D (an expert's F gate rows, then its F
 * up rows), down one of E * D rows x F. x enters the products as it is, in bf16
 * parts that add up to it. h, computed in F32 and times its p, is rounded to two
 * bf16 parts (16 bits) for BF16 and F16, whose own rounding to 8 and 11 bits y
 * takes at the end, and to three (24 bits) for F32. The sums are F32.
 * Not-a-number logits sort below every number.
 * 1 <= top_k <= min(E, RETRO_MOE_MAX_TOP_K), E <= RETRO_MOE_MAX_E, 1 <= D, F < 2^22
 * (RETRO_E_SHAPE otherwise). workspace: retro_moe_workspace_size bytes, 16-byte
 * aligned, overlapping no operand (RETRO_E_WORKSPACE otherwise); it needs no
 * initial value and holds nothing between calls.
 */
enum { RETRO_MOE_MAX_T = 64, RETRO_MOE_MAX_E = 256, RETRO_MOE_MAX_TOP_K = 16 };
int retro_moe(int xtype, const void *X, int64_t ldx, int rtype, const void *R, int64_t ldr, const void *gate_up_codes,
              const void *gate_up_scales, const void *down_codes, const void *down_scales, void *Y, int64_t ldy,
              int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k, int renormalize, void *workspace,
              int64_t workspace_bytes, void *stream);
int64_t retro_moe_workspace_size(int xtype, int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k);

#ifdef __cplusplus
}
#endif
#endif
