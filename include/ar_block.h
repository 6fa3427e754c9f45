/*
 * ar_block.h -- the operators around the all-reduce of a tensor-parallel
 * layer, over R rank buffers on one MI355X.
 *
 * Tensor-parallel inference runs an all-reduce after the attention and after
 * the MLP of every layer ("SGLang 中的 MSCCL++ All-Reduce 基准测试与推理集成指南",
 * blog.gitcode.com, section 1).  What surrounds it in the layer is here, with
 * the rank buffers of ar_allreduce.h as the common form:
 *
 *   arAllReduceNorm   the sum over the ranks, the residual's addition and the
 *                     root-mean-square norm in one pass over the data, with
 *                     an output in the element type or in 8 bits with scales;
 *   arGateQuant       SiLU gate (or nothing) with an 8-bit output, per rank;
 *   arMatmulScaled    the product of 8-bit activations and 8-bit weights with
 *                     a scale per block of 128, per rank (its outputs are the
 *                     next all-reduce's send buffers, or the gate's inputs),
 *                     or summed over the ranks into every rank's output (a
 *                     row-parallel layer with its all-reduce in one kernel).
 *
 * 8-bit values are e4m3 as the OCP 8-bit floating point specification defines
 * it (largest finite value 448, no infinities).  A value stands for
 * q * scale.  Two layouts of scales, both binary32:
 *
 *   activations [rows, cols]: one scale per row and 128 columns, laid out
 *       [ceil(cols / 128)][rows] -- a block's scales of consecutive rows are
 *       next to each other, which is how a tile of the product reads them;
 *   weights [n, k]: one scale per 128 x 128 block, laid out
 *       [ceil(n / 128)][ceil(k / 128)].
 *
 * Quantisation of a block of values y:
 *     s = max(max|y| / 448, 2^-126);  q = y / s rounded to nearest even
 * (both quotients are rounded to binary32 first; the second may be a unit off in
 * blocks whose scale is above 2^100).
 * A block that holds a NaN has the scale NaN; one that holds an infinity and
 * no NaN the scale infinity, with which its finite values become 0 and its
 * infinities NaN.  A block of zeros has the scale 2^-126.
 *
 * The rules of ar_allreduce.h apply to every entry point here: errors are
 * return codes; nothing allocates, synchronises or records a memset, so calls
 * can be captured into a HIP graph; arguments are checked without touching
 * the device; the communicator has to be on the current device (arInvalidUsage)
 * and is used from one host thread at a time.  These calls use none of the
 * communicator's packet memory, so they may overlap with one another and with
 * all-reduces.  rows == 0 (or n == 0) returns arSuccess and enqueues nothing.
 * arCommGetLastLaunch keeps describing the last all-reduce.
 */
#ifndef AR_BLOCK_H
#define AR_BLOCK_H

#include "ar_allreduce.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns (and, for weights, rows) that share a scale. */
#define AR_SCALE_BLOCK 128
/* The widest row arAllReduceNorm serves: a row is kept in registers. */
#define AR_NORM_MAX_COLS 32768

/* All-reduce, residual, root-mean-square norm.  For every row t and column i,
 * in binary32 with one rounding per output:
 *
 *     a = x_0 + x_1 + .. + x_{R-1}           (in this order, as arAllReduce)
 *     h = a + residual[t][i]                 (h = a without a residual)
 *     residualOut_r[t][i] = h                (for every rank r)
 *     y = h / sqrt(mean_i(h^2) + eps) * weight[i]
 *     out_r[t][i] = y, or 8-bit values and scales of y
 *
 * The norm is taken of h before its rounding to the element type.  The sum of
 * squares is binary32, or binary64 for rows whose mean that does not hold, so
 * that rows of any finite values have a norm.  A row that holds an infinity
 * gives zeros but NaN at the infinity; a row with a NaN is NaN, and so is a row
 * of zeros with eps 0.
 *
 *  sendbufs     host array of nranks device pointers, each [rows, cols] dense.
 *  residual     device pointer, [rows, cols] dense: the residual stream, which
 *               is the same on every rank and read once; NULL: none.
 *  weight       device pointer, [cols].
 *  eps          finite, >= 0.
 *  residualOut  host array of nranks device pointers, or NULL: h is not kept.
 *  outbufs      host array of nranks device pointers: [rows, cols] of dtype, or
 *               of 8-bit values when scalebufs is given.
 *  scalebufs    host array of nranks device pointers, each
 *               [ceil(cols / 128)][rows] floats, or NULL.
 *  dtype        of sendbufs, residual, weight, residualOut (and outbufs
 *               without scalebufs): arBfloat16, arFloat16 or arFloat32.
 *  cols         1 .. AR_NORM_MAX_COLS (else arUnsupported).
 *  nranks       1 .. 32 (else arUnsupported); 1 is a plain norm.
 *
 * Rules (arInvalidArgument when broken): no NULL pointer but those named;
 * every pointer 16-byte aligned; no written range overlaps another written or
 * read one, except that a residualOut_r, or an out_r of dtype, may be exactly
 * the residual or exactly the same rank's send buffer. */
arResult_t arAllReduceNorm(const void *const *sendbufs, const void *residual, const void *weight,
                           float eps, void *const *residualOut, void *const *outbufs,
                           float *const *scalebufs, size_t rows, size_t cols, arDataType_t dtype,
                           int nranks, arComm_t comm, arStream_t stream);

typedef enum { arActNone = 0, arActSiLU = 1 } arActivation_t;

/* Activation and quantisation, for every rank r:
 *
 *     arActSiLU:  y = g / (1 + exp(-g)) * u, in binary32, with an input row
 *                 holding g in its first `cols` columns and u in the next
 *                 (g = -infinity gives NaN, as the formula does);
 *     arActNone:  y = x, an input row holds `cols` columns;
 *     out_r, scales_r = 8-bit values and scales of y.
 *
 *  inbufs     host array of nranks device pointers, each [rows, cols] or
 *             [rows, 2 * cols] of dtype, dense.
 *  outbufs    host array of nranks device pointers, [rows, cols] 8-bit values.
 *  scalebufs  host array of nranks device pointers, [ceil(cols / 128)][rows].
 * Rules (arInvalidArgument when broken): no NULL pointer; every pointer
 * 16-byte aligned; no written range overlaps another written or read one.
 * arUnsupported for another dtype, activation or rank count. */
arResult_t arGateQuant(const void *const *inbufs, void *const *outbufs, float *const *scalebufs,
                       size_t rows, size_t cols, arDataType_t dtype, arActivation_t act,
                       int nranks, arComm_t comm, arStream_t stream);

/* The product of 8-bit matrices with scales per block of 128:
 *
 *     c_r[t][j] = sum_b as_r[b][t] * bs_r[j / 128][b] *
 *                     sum_{i in block b} a_r[t][i] * b_r[j][i]
 *     reduce 0:  out_r = c_r
 *     reduce 1:  out_r = c_0 + .. + c_{R-1}, the same for every rank r
 *
 * with binary32 sums and one rounding to outDtype.  The order of a sum follows
 * from rows, n, k, outDtype, reduce, nranks and the card's number of compute
 * units, never from values or from other calls.  as * bs is rounded to binary32
 * before the block's sum is multiplied by it.
 * Where outDtype is arFloat32 every product is exact; for the 16-bit types the
 * matrix instruction adds eight products at a time after cutting each, toward
 * zero, at 2^-13 of the leading bit of the largest of them, which on normally
 * distributed values leaves the sums 1.4e-5 off (the rounding to bfloat16 or
 * float16 leaves 1.7e-3 or 2.1e-4).
 *
 *  abufs, ascales  host arrays of nranks device pointers: activations
 *                  [rows, k] of 8-bit values, dense, and [ceil(k / 128)][rows].
 *  bbufs, bscales  host arrays of nranks device pointers: weights [n, k] of
 *                  8-bit values, dense, and [ceil(n / 128)][ceil(k / 128)].
 *  outbufs         host array of nranks device pointers, [rows, n] of outDtype
 *                  (with reduce 1 they may hold partial sums while the call
 *                  runs).
 *  k               a multiple of 16 in 16 .. 2^23 (else arUnsupported).
 *  outDtype        arBfloat16, arFloat16 or arFloat32 (else arUnsupported).
 *  rows, n         where ceil(rows / 128) * ceil(n / 128) is above 15000000 a
 *                  launch may not hold the tiles (arUnsupported).
 * Rules (arInvalidArgument when broken): no NULL pointer; every pointer
 * 16-byte aligned; rows and n at most 2^30 and rows * n at most 2^38; no
 * written range overlaps another written or read one (inputs may be shared
 * between ranks). */
arResult_t arMatmulScaled(const void *const *abufs, const float *const *ascales,
                          const void *const *bbufs, const float *const *bscales,
                          void *const *outbufs, size_t rows, size_t n, size_t k,
                          arDataType_t outDtype, int reduce, int nranks, arComm_t comm,
                          arStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AR_BLOCK_H */
