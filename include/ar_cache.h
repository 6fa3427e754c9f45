/*
 * ar_cache.h -- the paged key-value cache of a tensor-parallel layer, over R
 * rank buffers on one MI355X: writing it, reading it back, and the attention
 * of one new token a sequence over it.
 *
 * Between the first product of a tensor-parallel layer and the product whose
 * partial sums the all-reduce adds ("SGLang 中的 MSCCL++ All-Reduce 基准测试与推理集成指南",
 * blog.gitcode.com, section 1) a decode step runs
 *
 *   arCacheWrite      the new tokens' keys and values into the pages, in the
 *                     element type or in 8 bits with scales;
 *   arCacheAttention  softmax attention of one new token a sequence over the
 *                     pages, each rank for its share of the heads, with an
 *                     output in the element type or in the 8-bit form that
 *                     arMatmulScaled takes;
 *   arCacheRead       (a prefill that continues a cached prefix) the cached
 *                     rows back as dense ones.
 *
 * Every rank holds its own heads in its own pages; slots, page table and
 * lengths are the same on every rank and given once.  Place o of page p is
 * slot p * pageTokens + o.
 *
 * 8-bit values are those of ar_block.h (e4m3, a value stands for q * scale),
 * with one binary32 scale per token and head, for keys and for values, laid
 * out [pages][heads][pageTokens], and quantised by its rule:
 *     s = max(max|y| / 448, 2^-126);  q = y / s rounded to nearest even
 * over the `dim` values of a token and head.
 *
 * The rules of ar_block.h apply: errors are return codes; nothing allocates,
 * synchronises or records a memset; arguments are checked without touching
 * the device; the communicator has to be on the current device
 * (arInvalidUsage).  These calls use none of the communicator's packet memory.
 */
#ifndef AR_CACHE_H
#define AR_CACHE_H

#include "ar_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The widest head. */
#define AR_CACHE_MAX_DIM 256
/* What has to be zero of a workspace before its first use: its first bytes. */
#define AR_CACHE_WORKSPACE_ZEROS 65536

/* How keys and values lie in their pages: element (p, h, o, d) of page p, head
 * h, place o is at p * pageStride + h * headStride + o * tokenStride + d.  The
 * same for keys and values and for every rank.  Keys and values may be in one
 * allocation, next to each other inside each page, head or token. */
typedef struct {
    size_t pages;
    size_t pageTokens;  /* places of a page; pages * pageTokens < 2^31 */
    size_t heads;       /* key-value heads of a rank, at most 4096 */
    size_t dim;         /* a multiple of 16 in 16 .. AR_CACHE_MAX_DIM */
    size_t pageStride;  /* in elements, as the other strides; multiples of 16 bytes */
    size_t headStride;
    size_t tokenStride;
} arCacheLayout_t;

/* Keys and values of `tokens` tokens into the cache.  A token whose slot is
 * negative, or not a slot of the cache, is skipped (padding of a batch).  Slots
 * that are given twice hold one of the tokens' values in each element, and one
 * of their scales.
 *
 *  keys, values            host arrays of nranks device pointers: [tokens][heads][dim]
 *                          of dtype, rows rowStride elements apart.
 *  rowStride               at least heads * dim, a multiple of 16 bytes: the rows
 *                          may be parts of the wider ones of a product.
 *  slots                   device pointer, [tokens].
 *  cache                   the layout; read during the call only.
 *  keyPages, valuePages    host arrays of nranks device pointers: elements of
 *                          dtype, or 8-bit values when the scales are given.
 *  keyScales, valueScales  host arrays of nranks device pointers, or both NULL.
 *  dtype                   arBfloat16, arFloat16 or arFloat32 (else arUnsupported).
 * Rules (arInvalidArgument when broken): no NULL pointer but those named; every
 * pointer 16-byte aligned, slots 8-byte aligned; rows of a layout apart; no
 * written range overlaps another written or read one. */
arResult_t arCacheWrite(const void *const *keys, const void *const *values, size_t rowStride,
                        const int64_t *slots, size_t tokens, const arCacheLayout_t *cache,
                        void *const *keyPages, void *const *valuePages, float *const *keyScales,
                        float *const *valueScales, arDataType_t dtype, int nranks, arComm_t comm,
                        arStream_t stream);

/* The inverse: rows of `tokens` slots as [tokens][heads][dim] of dtype, 8-bit
 * values as q * scale rounded to dtype.  Rows whose slot is none of the cache's
 * are left as they were.  Arguments and rules as for arCacheWrite, with keys and
 * values written (they may be parts of the same rows) and the cache read; a slot
 * may be given twice. */
arResult_t arCacheRead(const int64_t *slots, size_t tokens, const arCacheLayout_t *cache,
                       const void *const *keyPages, const void *const *valuePages,
                       const float *const *keyScales, const float *const *valueScales,
                       void *const *keys, void *const *values, size_t rowStride,
                       arDataType_t dtype, int nranks, arComm_t comm, arStream_t stream);

/* Attention of one new token a sequence.  Sequence i has lengths[i] = n tokens in
 * the cache, its new one among them; token t lies in page pageTable[i][t /
 * pageTokens], place t % pageTokens.  With first = max(0, n - window) (window 0:
 * 0), for every rank, sequence i, query head j and its key-value head
 * j / (heads / cache->heads):
 *
 *     x_t = scale * sum_d q[i][j][d] * k_t[d]                first <= t < n
 *     out[i][j] = sum_t exp(x_t) v_t / sum_t exp(x_t)
 *     lse[i][j] = log(sum_t exp(x_t))
 *
 * Scores, exponentials, sums and accumulators are binary32; the scores are taken times
 * log2 e, those of 8-bit keys first without their scales.  (The products of the
 * exponentials with values of 16 and 8 bits take the exponentials in three parts of bfloat16,
 * which hold all of their 24 bits, or, for values of float16, in two parts of that, which are
 * within 2^-23 of an exponential or 2^-33 of the largest.)
 * An infinite value makes its column an infinity, or NaN beside a NaN or an infinity of the
 * other sign; of a token whose weight is less than binary32 holds, either.  A score of
 * infinity makes lse one, NaN beside a NaN, and out NaN.
 * The order of a sum follows from the sizes, the lengths and the card's number of
 * compute units, never from values or from other calls.  Only tokens first .. n - 1
 * and the table's entries for them are read, whatever the other places hold (and place 0
 * of page 0, for a page number that is none).
 *
 * n = 0 gives zeros and lse -infinity.  A length that is negative or above
 * tablePages * pageTokens, and a page number of a token that is none of the
 * cache's, gives NaN in every value of the sequence (8 bits: in every scale).
 *
 *  queries      host array of nranks device pointers: [seqs][heads][dim] of dtype,
 *               rows queryStride elements apart (at least heads * dim, a multiple of
 *               16 bytes).
 *  pageTable    device pointer, [seqs][tablePages].
 *  lengths      device pointer, [seqs].
 *  heads        query heads of a rank, a multiple of cache->heads, at most 4096.
 *  scale        at most 2^126 in magnitude.
 *  window       tokens that are attended to, the last ones; 0: all.
 *  outbufs      host array of nranks device pointers: [seqs][heads][dim] dense, of
 *               dtype, or 8-bit values when outScales is given.
 *  outScales    host array of nranks device pointers, or NULL:
 *               [heads * dim / 128][seqs], the activation scales of arMatmulScaled
 *               for rows of heads * dim columns.  Needs dim 128 or 256 (else
 *               arUnsupported; arGateQuant quantises other outputs).
 *  lse          host array of nranks device pointers [seqs][heads], or NULL.
 *  workspace    device memory of at least the bytes that arCacheAttentionWorkspace
 *               names for this dim and heads / cache->heads, its first
 *               AR_CACHE_WORKSPACE_ZEROS zero before its first use; every call leaves it
 *               fit for the next.  One call at a time may use it: calls that may run at
 *               once, in graphs as well, need one each.
 *  seqs         at most 65536, and seqs * heads * nranks at most 2^24 (else
 *               arUnsupported).
 * Rules (arInvalidArgument when broken): no NULL pointer but those named; every
 * pointer 16-byte aligned, pageTable and lengths 4-byte aligned; tablePages >= 1;
 * no written range (the workspace's is one) overlaps another. */
arResult_t arCacheAttention(const void *const *queries, size_t queryStride,
                            const arCacheLayout_t *cache, const void *const *keyPages,
                            const void *const *valuePages, const float *const *keyScales,
                            const float *const *valueScales, const int32_t *pageTable,
                            size_t tablePages, const int32_t *lengths, size_t seqs, size_t heads,
                            float scale, size_t window, void *const *outbufs,
                            float *const *outScales, float *const *lse, void *workspace,
                            size_t workspaceBytes, arDataType_t dtype, int nranks, arComm_t comm,
                            arStream_t stream);

/* Bytes of workspace that arCacheAttention needs on the communicator's device for
 * heads of `dim` and `group` query heads to a key-value head (1 .. 4096), whatever its
 * other arguments.  One that is large enough for several calls may serve them in turn. */
arResult_t arCacheAttentionWorkspace(size_t dim, size_t group, arComm_t comm, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* AR_CACHE_H */
