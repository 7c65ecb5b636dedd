/*
 * ropekv_serving.h -- C ABI of the serving operators around the paged KV cache
 * (libropekv_serving.so, beside the writes of ropekv.h): rotary positions with
 * several axes, an 8-bit cache with one scale per token and head, reading a
 * cache back, and the attention of a batch whose sequences share a long prefix.
 *
 * The common rules of ropekv.h hold: device pointers owned by the caller and
 * 16-byte aligned, dense row-major layouts, asynchronous launches on the
 * caller's stream that may be captured in a CUDA graph, ropekv_status results
 * (0 or negative, nothing launched when the host rejects the arguments), no
 * allocation, no synchronisation. Invalid indices found on the device are
 * skipped. headDim is 64, 128 or 256.
 *
 * Caches. [numBlocks, blockSize, Hkv, D] of the slot-mapping calls is one plane
 * of the paged pool [2, numPages, tokensPerPage, Hkv, D] (plane 0 = K, plane
 * 1 = V): a pool's planes can be passed to the slot-mapping calls as key and
 * value cache, and what they write is found through a page table.
 *
 * Cache formats. FP16 needs no scales. The 8-bit formats hold one code per
 * element and one FP32 scale per token and KV head; an element's value is
 * code * scale. Scales are laid out [numBlocks, Hkv, blockSize] per plane: an
 * attention call walks the tokens of one head, whose scales are then
 * consecutive.
 */
#ifndef ROPEKV_SERVING_H
#define ROPEKV_SERVING_H

#include "ropekv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a cache. */
typedef enum {
    ROPEKV_CACHE_F16 = 0,  /* IEEE binary16, no scales                             */
    ROPEKV_CACHE_E4M3 = 1, /* OCP E4M3 ("e4m3fn") codes with scales, max 448        */
    ROPEKV_CACHE_INT8 = 2  /* signed 8-bit codes in [-127, 127] with scales         */
} ropekv_cache_format;

/*
 * rope_write_kv_slot_mapping with several position axes, as images and video
 * use them (time, height, width): frequency i of a token is taken from the
 * cos/sin row of the token's position on axis freqAxis[i].
 *   cosSin       [cosSinRows, rotaryDim] FP32, row = position on any axis.
 *   positions    [numAxes, numTokens] INT64.
 *   freqAxis     [rotaryDim / 2] INT32 in HOST memory: the axis of each
 *                frequency, in [0, numAxes). Read during the call (a captured
 *                graph keeps the values).
 *   numAxes      1 to 4.
 * The other arguments are those of rope_write_kv_slot_mapping. A token with a
 * position outside [0, cosSinRows) on any axis is skipped whole.
 * Host errors, besides that call's: numAxes outside 1..4 or an axis outside
 * [0, numAxes) -> ROPEKV_ERR_SHAPE.
 */
ROPEKV_API int rope_write_kv_mrope(const float* cosSin, const int64_t* positions,
                                   const int32_t* freqAxis, int32_t numAxes, const uint16_t* q,
                                   int64_t qTokenStride, const uint16_t* k, int64_t kTokenStride,
                                   const uint16_t* v, int64_t vTokenStride,
                                   const int64_t* slotMapping, uint16_t* keyCache,
                                   uint16_t* valueCache, uint16_t* qOut, uint16_t* kOut,
                                   int32_t numTokens, int32_t numQHeads, int32_t numKVHeads,
                                   int32_t headDim, int32_t rotaryDim, int32_t cosSinRows,
                                   int64_t numBlocks, int32_t blockSize, int32_t style,
                                   void* stream);

/*
 * rope_write_kv_slot_mapping into an 8-bit cache whose scales are found as it
 * is written. For every token and KV head, with x the rotated K head (FP32, not
 * rounded to FP16) or the V head and M = 448 (E4M3) or 127 (INT8):
 *   scale = max|x| / M,   code = x * (M / max|x|), rounded to the nearest code (ties to
 *                                                  the even one);
 * both quotients and the product are rounded to FP32 first, so that an element next to the
 * border between two codes may get another one than x / scale has.
 * A head of zeros (or whose largest magnitude is below 2^-100) gets scale 0 and
 * codes 0; a head that holds an infinity or a NaN gets scale NaN and codes 0,
 * so that every element reads back as NaN.
 *   keyCache8, valueCache8  [numBlocks, blockSize, Hkv, D] 8-bit codes, written.
 *   keyScales, valueScales  [numBlocks, Hkv, blockSize] FP32, written.
 *   cacheFormat             ROPEKV_CACHE_E4M3 or ROPEKV_CACHE_INT8, else
 *                           ROPEKV_ERR_STYLE.
 * Slots of one call that are in range are distinct: of two tokens with the same slot
 * either may stay, and codes and scale need not come from the same one.
 * The other arguments, skip rules and errors are those of
 * rope_write_kv_slot_mapping.
 */
ROPEKV_API int rope_write_kv_slot_mapping_quant(
    const float* cosSin, const int64_t* positions, const uint16_t* q, int64_t qTokenStride,
    const uint16_t* k, int64_t kTokenStride, const uint16_t* v, int64_t vTokenStride,
    const int64_t* slotMapping, uint8_t* keyCache8, uint8_t* valueCache8, float* keyScales,
    float* valueScales, uint16_t* qOut, int32_t numTokens, int32_t numQHeads, int32_t numKVHeads,
    int32_t headDim, int32_t rotaryDim, int32_t cosSinRows, int64_t numBlocks, int32_t blockSize,
    int32_t cacheFormat, int32_t style, void* stream);

/*
 * Rows of a paged cache read back as FP16 (the inverse of
 * paged_kv_delta_update's placement): row t takes the K and V of position
 * rowPositions[t] of sequence rowSequences[t].
 *   kvCache       [2, numPages, tokensPerPage, Hkv, D] in cacheFormat.
 *   kvScales      [2, numPages, Hkv, tokensPerPage] FP32 (8-bit formats; NULL
 *                 for FP16).
 *   pageTable     [batchSize, 2, maxPagesPerSeq] INT32, as paged_kv_delta_update.
 *   kOut, vOut    [numRows, Hkv, D] FP16: the bits of an FP16 cache, or
 *                 code * scale rounded to FP32 and then to FP16.
 * A row is skipped, and its kOut and vOut rows left as they were, when its
 * position or sequence is negative or out of range; each plane is skipped on
 * its own when its page is unmapped.
 * Host errors: as paged_kv_delta_update, and 2 * numPages * tokensPerPage >=
 * 2^31 -> ROPEKV_ERR_SHAPE; an unknown cacheFormat -> ROPEKV_ERR_STYLE.
 */
ROPEKV_API int paged_kv_read(const void* kvCache, const float* kvScales, const int32_t* pageTable,
                             const int32_t* rowPositions, const int32_t* rowSequences,
                             uint16_t* kOut, uint16_t* vOut, int32_t numRows, int32_t batchSize,
                             int32_t numKVHeads, int32_t headDim, int32_t numPages,
                             int32_t maxPagesPerSeq, int32_t tokensPerPage, int32_t cacheFormat,
                             void* stream);

/* Sizes of paged_attention_shared_prefix. */
typedef struct {
    int32_t batch;          /* B: sequences                                         */
    int32_t seqLen;         /* S: query tokens per sequence (1 = decode)            */
    int32_t numQHeads;      /* Hq, a multiple of Hkv                                */
    int32_t numKVHeads;     /* Hkv                                                  */
    int32_t headDim;        /* D                                                    */
    int32_t numPages;       /* pages per plane of the pool                          */
    int32_t tokensPerPage;  /* tokens per page                                      */
    int32_t maxPagesPerSeq; /* columns of pageTable                                 */
    int32_t prefixLen;      /* P: tokens that all sequences share (0 = none)        */
    int32_t maxPrefixPages; /* columns of prefixTable                               */
    int32_t cacheFormat;    /* a ropekv_cache_format                                */
} ropekv_attention_dims;

/* Bytes of workspace that paged_attention_shared_prefix needs for these sizes,
 * or a negative ropekv_status. Host only. */
ROPEKV_API int64_t paged_attention_workspace_size(const ropekv_attention_dims* dims);

/*
 * Attention of S new tokens per sequence over a paged cache in which all
 * sequences begin with the same P tokens. The prefix is stored once, read once
 * per KV head and multiplied with the queries of the whole batch together;
 * each sequence's own tokens follow, and both parts share one softmax:
 *   out = sum_t softmax_t(smScale * q . k_t) v_t.
 * Query s of sequence b sits at position p = kvLens[b] - S + s (kvLens counts
 * the new tokens, whose K and V are already in the cache) and sees positions
 * 0..p: positions below P through prefixTable, the others through its row of
 * pageTable, whose column is position / tokensPerPage (columns that hold only
 * prefix positions are not read).
 *   q            [B, S, Hq, D] FP16.
 *   kvCache      [2, numPages, tokensPerPage, Hkv, D] in dims->cacheFormat.
 *   kvScales     [2, numPages, Hkv, tokensPerPage] FP32 (8-bit formats; NULL for FP16).
 *   prefixTable  [2, maxPrefixPages] INT32 page ids of the prefix, as one row of
 *                pageTable (NULL when P = 0).
 *   pageTable    [B, 2, maxPagesPerSeq] INT32.
 *   kvLens       [B] INT32, read on the device.
 *   out          [B, S, Hq, D] FP16, every row written.
 *   lse          [B, S, Hq] FP32 natural logarithm of the softmax sum, or NULL.
 *   workspace    paged_attention_workspace_size bytes; its content needs no
 *                preparation and means nothing afterwards. Calls that may run
 *                at the same time, from graphs too, need workspaces of their own.
 * A position whose K or V page is unmapped, or past maxPagesPerSeq, is not
 * seen. A query whose position lies before P (an inactive sequence, kvLens[b] =
 * 0, for one) or that sees nothing gets a zero row and lse = -infinity. What
 * lies in cache slots that no query sees does not matter, whatever its bits.
 * Scales may have either sign. A V scale below 2^-40 in magnitude may count as 0 (such a
 * token adds less than 2^-31 to an element of out). A token whose V scale is infinite or NaN
 * leaves no finite element in the rows that see it; their lse does not depend on it. V
 * scales between 2^60 and infinity are not supported (elements may be NaN).
 * Sums, softmax and partial results are FP32; the weights of V are rounded to
 * FP16 once. out may be q itself. The call is two or three launches; the split of the
 * work follows from the sizes alone (pageTable's columns stand for the lengths: a table
 * much wider than kvLens costs time, not correctness; 16384 to 131072 columns x tokens for
 * sequences of 3000 to 9000 took up to 2.7 times as long as exact tables), so equal calls
 * give equal bits.
 * The status is that of the launches. Waits inside the kernels are bounded; should one run
 * out, which no argument makes it do, the rows concerned are NaN in out and lse.
 * Host errors: sizes negative, tokensPerPage <= 0, seqLen > 2^15, prefixLen >
 * maxPrefixPages * tokensPerPage, 2 * numPages * tokensPerPage >= 2^31,
 * prefixLen or maxPagesPerSeq * tokensPerPage > 2^30, or more than 2^30 query
 * rows -> ROPEKV_ERR_SHAPE; workspaceBytes too small -> ROPEKV_ERR_CAPACITY; an unknown
 * cacheFormat -> ROPEKV_ERR_STYLE; smScale not finite -> ROPEKV_ERR_SHAPE.
 */
ROPEKV_API int paged_attention_shared_prefix(
    const uint16_t* q, const void* kvCache, const float* kvScales, const int32_t* prefixTable,
    const int32_t* pageTable, const int32_t* kvLens, uint16_t* out, float* lse, void* workspace,
    int64_t workspaceBytes, const ropekv_attention_dims* dims, float smScale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ROPEKV_SERVING_H */
