/*
 * fp4.h -- C ABI of the dense part of a decoder layer in block-scaled FP4, for
 * GB300 (sm_103a).  Same library, same conventions as moe.h: device pointers
 * owned by the caller, no state and no allocation, `stream` a cudaStream_t as
 * void*, a moe_status as the return value.  Calls launch on the current device,
 * which has to be the one that the pointers and the stream belong to.
 *
 * Products whose two operands are FP4 (projections, a shared expert, logits),
 * and what stands between them:
 *   fp4_quantize      rows of 16 or 32 bits -> an FP4 matrix
 *   fp4_dequantize    ... and back to the values that the codes stand for
 *   fp4_swiglu        SiLU(gate) * up, into 16 bits and / or an FP4 matrix
 *   fp4_linear        FP4 matrix x FP4 matrix
 *   fp4_linear_rows   rows of 16 or 32 bits, quantised, x FP4 matrix
 *   fp4_block_norm    norm behind a block, gate, residual sum, norm before the
 *                     next block, into 16 bits and / or an FP4 matrix
 *   fp4_tile_scales   row-major block scales -> the layout that products read
 *
 * No output may share bytes with an input, another output or a workspace
 * (MOE_ERR_INVALID_ARG); views of one buffer whose rows lie between one another's do not.  Only
 * the 16- and 32-bit outputs of fp4_swiglu and fp4_block_norm may lie where an input with
 * elements of the same size does, from the same address on and with the same stride.
 */
#ifndef FP4_GB300_H
#define FP4_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows.  Element c of row r of an argument x is x[r * x_stride
 * + c]; rows are 16-B aligned, and a stride (which plays no part for a single row) is a
 * multiple of 16 bytes and at least a row's length, unless it is said otherwise. */
enum { FP4_BF16 = 0, FP4_FP16 = 1, FP4_FP32 = 2 };

/* A matrix in FP4.
 * codes [rows x cols / 2]: e2m1, two to a byte, the even column in the low
 *   nibble (the packing of an expert record), 16-B aligned.
 * scales, fp4_scale_bytes() of them, 16-B aligned: one byte for each block of
 *   16 columns (E4M3, not negative, MOE_FMT_NVFP4) or 32 (UE8M0, MOE_FMT_MXFP4), in tiles of
 *   128 rows x 4 blocks.  With kt = ceil(blocks of a row / 4), block b of row r
 *   is byte ((r / 128) * kt + b / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4.
 *   Blocks of a last tile past cols hold 0; rows past `rows` hold anything.
 * row_scale [rows] FP32, or NULL (1).
 * The value of an element is code * block scale * row scale.
 * Supported: cols a multiple of 32 from 32 to 32768, rows up to 2^24. */
typedef struct {
  void* codes;
  void* scales;
  float* row_scale;
  int32_t rows, cols;
  int32_t format; /* MOE_FMT_NVFP4 or MOE_FMT_MXFP4 */
} fp4_matrix;

/* Bytes of the scales of a matrix; 0 where it is not supported or has no rows. */
size_t fp4_scale_bytes(int rows, int cols, int format);

/* scales [rows x cols / 16 (MXFP4: 32)], row-major (as checkpoints and expert
 * records hold them) -> tiled, fp4_scale_bytes() bytes, 16-B aligned. */
int fp4_tile_scales(const uint8_t* scales, int rows, int cols, int format, uint8_t* tiled, void* stream);

/* Quantises rows of x into every row of `out`.
 * NVFP4 (row_scale is required): with a the largest magnitude of a row, its row
 *   scale is 2^E for the smallest E >= -126 with 2688 * 2^E >= a (2688 = 448 * 6);
 *   with a block's largest magnitude b: s = E4M3_rn(b * 2^-E / 6), codes =
 *   e2m1_rn(x * 2^-E / s), +0 where s is 0 (FP32 quotients).  A row with an
 *   infinity or a NaN gets a NaN as row scale, and codes and scales of 0.
 * MXFP4 (row_scale, where given, becomes 1): s = 2^e for the smallest e >= -127
 *   with 6 * 2^e >= b; codes = e2m1_rn(x / s).  A block with an infinity or a NaN
 *   gets s = NaN (byte 255) and codes of 0.
 * Round to nearest, ties to even; nothing saturates.  The rules of
 * fp4_pack_expert, but for the row's power of two. */
int fp4_quantize(const void* x, long long x_stride, int x_type, const fp4_matrix* out, void* stream);

/* The values of m's elements: code * block scale, exactly, times the row scale in FP32, rounded
 * to out's type (in BF16 that changes nothing in what fp4_quantize made, but for magnitudes
 * below 2^-126). */
int fp4_dequantize(const fp4_matrix* m, void* out, long long out_stride, int out_type, void* stream);

/* a = gate / (1 + exp(-gate)) * up, in FP32, for rows x cols elements; the quotient is
 * -0 where exp(-gate) is 2^128 or more (gates below -88.72).
 * out (BF16 or FP16) gets a rounded, m gets a quantised as by fp4_quantize;
 * either may be NULL, not both.  gate and up are of one type. */
int fp4_swiglu(const void* gate, long long gate_stride, const void* up, long long up_stride, int type, int rows,
               int cols, void* out, long long out_stride, int out_type, const fp4_matrix* m, void* stream);

/* r' = r + scale * gate * N(y; post_weight),  h = N(r'; weight), with
 * N(x; w) = x / sqrt(mean(x^2) + eps) * w over a row, in FP32.
 * y NULL: r' = r.  post_weight NULL: y without a norm.  gate NULL: 1; gate_cols
 * = cols: an element for each element (gate_stride 0: one row for all rows); gate_cols =
 * 1: an element for each row, at any stride.  gate is of y's type.  weight NULL: 1.  Weights
 * are FP32 [cols], 16-B aligned.
 * r_out, of r's type, gets r' rounded (NULL: it is not kept; it may be r itself,
 * with r's stride, or y or a gate for each element, as said above).  h (BF16 or
 * FP16) and m (FP4) get h, either may be NULL, not both; they are made from r'
 * before it is rounded. */
int fp4_block_norm(const void* r, long long r_stride, int r_type, const void* y, long long y_stride, int y_type,
                   const float* post_weight, const void* gate, long long gate_stride, int gate_cols, double scale,
                   const float* weight, double eps, int rows, int cols, void* r_out, long long r_out_stride, void* h,
                   long long h_stride, int h_type, const fp4_matrix* m, void* stream);

/* y[t, n] = x.row_scale[t] * w.row_scale[n] * sum_k x[t, k] w[n, k] + bias[n],
 * for the x.rows rows of y and w.rows columns, rounded once to y's type (BF16,
 * FP16 or FP32).  Codes and block scales meet on the tensor cores (tcgen05,
 * block-scaled MMA), the products exactly and the sums in FP32; the row scales are
 * multiplied in that order in FP32.  x and w have the same cols and format.
 * bias [w.rows] FP32 or NULL.  y's stride: any that is at least w.rows; its
 * data only has to be aligned to its elements.
 * Results are bit-identical between repeated calls.
 * A wait that runs out sets MOE_DEV_TIMEOUT in dev_status (device int32 or NULL)
 * and makes the outputs that it was for NaN. */
int fp4_linear(const fp4_matrix* x, const fp4_matrix* w, const float* bias, void* y, long long y_stride, int y_type,
               int32_t* dev_status, void* stream);

/* Workspace bytes of fp4_linear_rows for up to `rows` rows of x; 0 where it is
 * not supported.  It needs no initial value and may be shared by calls of one
 * stream. */
size_t fp4_linear_rows_workspace(const fp4_matrix* w, int rows);

/* fp4_linear of fp4_quantize(x) in w's format. */
int fp4_linear_rows(const void* x, long long x_stride, int x_type, int rows, const fp4_matrix* w, const float* bias,
                    void* y, long long y_stride, int y_type, void* workspace, size_t ws_bytes, int32_t* dev_status,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4_GB300_H */
