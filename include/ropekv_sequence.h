/*
 * ropekv_sequence.h -- C ABI of the operators on whole sequences
 * (libropekv_serving.so, beside ropekv_serving.h): causal attention of packed
 * prompts, attention of one or more new tokens per sequence (a chain or a tree of
 * drafts) over the contiguous cache, moving the rows of accepted drafts to the
 * front, and copying, forking and freeing pages of the paged cache.
 *
 * The common rules of ropekv.h hold: device pointers owned by the caller and
 * 16-byte aligned, asynchronous launches on the caller's stream that may be
 * captured in a CUDA graph, ropekv_status results (0 or negative, nothing launched
 * when the host rejects the arguments), no allocation, no synchronisation. Invalid
 * indices found on the device are skipped. headDim is 64, 128 or 256.
 *
 * Both attention calls take a workspace, whose content needs no preparation and
 * means nothing afterwards; calls that may run at the same time, from graphs too,
 * need workspaces of their own. They are one or two launches whose split follows
 * from the sizes and lengths alone, so equal calls give equal bits. Scores, sums and
 * partial results are FP32; the weights of V are rounded to FP16 once, which is 2^-11 of a
 * weight, or 2^-32 of the row's largest where that is more. A value that is not finite
 * reaches only the rows that see its token; an infinity in V is one in out whatever its
 * weight, and one or a NaN costs such rows, and those of the same tile that do not see it, a
 * much slower path. Waits inside the kernels are bounded; should one run out, which takes a
 * fault and no argument, all rows that a CTA had taken on, and all rows of units that it
 * shares with others, are NaN in out and lse, but for such as it had finished.
 */
#ifndef ROPEKV_SEQUENCE_H
#define ROPEKV_SEQUENCE_H

#include "ropekv_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes of prompt_attention. */
typedef struct {
    int32_t numTokens;    /* rows of q, out and lse                               */
    int32_t numKVTokens;  /* rows of k and v                                      */
    int32_t batch;        /* B: sequences                                         */
    int32_t numQHeads;    /* Hq, a multiple of Hkv                                */
    int32_t numKVHeads;   /* Hkv                                                  */
    int32_t headDim;      /* D                                                    */
} ropekv_prompt_dims;

/* Bytes of workspace that prompt_attention needs for these sizes, or a negative
 * ropekv_status. Host only. */
ROPEKV_API int64_t prompt_attention_workspace_size(const ropekv_prompt_dims* dims);

/*
 * Causal attention of B sequences packed one behind another. Sequence b has the
 * queries qStarts[b] .. qStarts[b+1]-1 (nq of them) and the keys kvStarts[b] ..
 * kvStarts[b+1]-1 (nk); its queries are its last tokens, so that query i sees its
 * keys 0 .. nk-nq+i (a whole prompt: nq = nk; a chunk behind a context: nq < nk):
 *   out = sum_t softmax_t(smScale * q . k_t) v_t.
 *   q            [numTokens, Hq, D] FP16, token stride qTokenStride elements
 *                (>= Hq*D, a multiple of 8); k, v [numKVTokens, Hkv, D] likewise
 *                with strides of their own. They may be views of one packed
 *                projection, and k and v what paged_kv_read returns.
 *   qStarts      [B + 1] INT32, ascending, read on the device.
 *   kvStarts     [B + 1] INT32, or NULL: qStarts.
 *   out          [numTokens, Hq, D] FP16, may not overlap q, k or v.
 *   lse          [numTokens, Hq] FP32 natural logarithm of the softmax sum, or NULL.
 * Starts are taken within [0, numTokens] and [0, numKVTokens]. Rows of no sequence
 * (before the first start, behind the last) are left as they were. A query that sees
 * nothing (nk < nq), or whose scores are all -infinity, gets a zero row and lse =
 * -infinity; a score of +infinity makes its row NaN.
 * Host errors: negative sizes, numTokens or numKVTokens > 2^28, batch > 2^20,
 * strides too small, not multiples of 8 or > 2^36, numTokens * Hq > 2^31 - 1, smScale
 * or smScale * log2 e not finite, out overlapping q, k or v -> ROPEKV_ERR_SHAPE;
 * workspaceBytes too small -> ROPEKV_ERR_CAPACITY.
 */
ROPEKV_API int prompt_attention(const uint16_t* q, int64_t qTokenStride, const uint16_t* k,
                                int64_t kTokenStride, const uint16_t* v, int64_t vTokenStride,
                                const int32_t* qStarts, const int32_t* kvStarts, uint16_t* out,
                                float* lse, void* workspace, int64_t workspaceBytes,
                                const ropekv_prompt_dims* dims, float smScale, void* stream);

/* Sizes of tree_attention. */
typedef struct {
    int32_t batch;        /* B: sequences                                         */
    int32_t seqLen;       /* S: new tokens per sequence (1 = decode)              */
    int32_t numQHeads;    /* Hq, a multiple of Hkv                                */
    int32_t numKVHeads;   /* Hkv                                                  */
    int32_t headDim;      /* D                                                    */
    int32_t kvCapacity;   /* slots per sequence in the cache                      */
} ropekv_tree_dims;

/* Bytes of workspace that tree_attention needs for these sizes, or a negative
 * ropekv_status. Host only. */
ROPEKV_API int64_t tree_attention_workspace_size(const ropekv_tree_dims* dims);

/*
 * Attention of S new tokens per sequence over the contiguous cache, after
 * rope_write_kv_tree or rope_write_kv_continuous has written them: token j of
 * sequence b is at slot kvCacheEndLens[b] - S + j. A token sees every slot before
 * the new ones, and of the new ones those that treeMask names (its ancestors and
 * itself, for a tree), or without a mask itself and those before it.
 *   q               [B, S, Hq, D] FP16.
 *   kvCache         [B, 2, Hkv, kvCapacity, D] FP16.
 *   kvCacheEndLens  [B] INT32, read on the device.
 *   treeMask        [B, S, ceil(S / 32)] INT32, or NULL: bit j % 32 of word j / 32 of
 *                   row i says that token i sees token j. Bits past S mean nothing.
 *   out             [B, S, Hq, D] FP16, every row written; may not overlap q or kvCache.
 *   lse             [B, S, Hq] FP32 natural logarithm of the softmax sum, or NULL.
 * Slots outside [0, kvCapacity) are not seen. A token that sees nothing (an inactive
 * sequence, kvCacheEndLens[b] = 0, for one), or whose scores are all -infinity, gets a zero
 * row and lse = -infinity; a score of +infinity makes its row NaN. What lies in slots that no token sees does not matter, whatever its bits.
 * Host errors: negative sizes, seqLen > 2^15, kvCapacity > 2^28, batch * seqLen * Hq >
 * 2^31 - 1, kvCapacity * Hkv * D > 2^37 or, times batch, 2^40, smScale or smScale *
 * log2 e not finite, out overlapping q or kvCache -> ROPEKV_ERR_SHAPE; workspaceBytes too
 * small -> ROPEKV_ERR_CAPACITY.
 */
ROPEKV_API int tree_attention(const uint16_t* q, const uint16_t* kvCache,
                              const int32_t* kvCacheEndLens, const int32_t* treeMask, uint16_t* out,
                              float* lse, void* workspace, int64_t workspaceBytes,
                              const ropekv_tree_dims* dims, float smScale, void* stream);

/*
 * After drafts were verified: the rows of the accepted ones move to the front of the
 * new tokens, in the contiguous cache. With base = kvCacheEndLens[b] - S, entry j <
 * acceptedLens[b] of sequence b moves K and V (bits, already rotated) from slot base +
 * accepted[b, j] to slot base + j, in the order of j.
 *   kvCache         [B, 2, Hkv, kvCapacity, D] FP16, in and out.
 *   kvCacheEndLens  [B] INT32, read.
 *   accepted        [B, maxAccepted] INT32 numbers of the accepted tokens in [0, S).
 *   acceptedLens    [B] INT32, taken within [0, min(maxAccepted, S)].
 *   endLensOut      [B] INT32 or NULL: kvCacheEndLens[b] - S + acceptedLens[b], the end
 *                   behind the accepted rows; may be kvCacheEndLens itself. Left as it
 *                   was where kvCacheEndLens[b] < S.
 * An entry outside [j, S) (a path down a tree whose parents come before their children
 * has none, and no row is then overwritten before it has moved), or whose source or
 * destination slot is outside [0, kvCapacity), is skipped.
 * Host errors: negative sizes, seqLen or maxAccepted > 2^15 -> ROPEKV_ERR_SHAPE.
 */
ROPEKV_API int kv_accept_drafts(uint16_t* kvCache, const int32_t* kvCacheEndLens,
                                const int32_t* accepted, const int32_t* acceptedLens,
                                int32_t* endLensOut, int32_t batch, int32_t seqLen,
                                int32_t maxAccepted, int32_t numKVHeads, int32_t headDim,
                                int32_t kvCapacity, void* stream);

/*
 * The same in a paged cache of any format, codes and scales as bits: positions in place
 * of slots, found through the page table; each plane is skipped on its own where
 * the source's or the destination's page is unmapped.
 *   kvCache    [2, numPages, tokensPerPage, Hkv, D] in cacheFormat, in and out.
 *   kvScales   [2, numPages, Hkv, tokensPerPage] FP32 (8-bit formats; NULL for FP16).
 *   pageTable  [B, 2, maxPagesPerSeq] INT32, as paged_kv_delta_update. No two
 *              positions moved by one call share a slot.
 *   kvLens     [B] INT32 lengths with the S new tokens, read; kvLensOut as endLensOut.
 * Host errors: as kv_accept_drafts and paged_kv_read.
 */
ROPEKV_API int paged_kv_accept_drafts(void* kvCache, float* kvScales, const int32_t* pageTable,
                                      const int32_t* kvLens, const int32_t* accepted,
                                      const int32_t* acceptedLens, int32_t* kvLensOut,
                                      int32_t batch, int32_t seqLen, int32_t maxAccepted,
                                      int32_t numKVHeads, int32_t headDim, int32_t numPages,
                                      int32_t maxPagesPerSeq, int32_t tokensPerPage,
                                      int32_t cacheFormat, void* stream);

/*
 * Pages in pairs. The three calls below take page p to be the K page p together with
 * the V page numPages + p, as a slot mapping does (one block for K and V). Of a page
 * table they read the K plane and write both. refCounts [numPages] INT32 says how many
 * table entries name a page; a page with 0 is free.
 */

/*
 * Copies pages: pair dstPages[i] becomes a copy of pair srcPages[i], scales too.
 *   srcPages, dstPages  [numCopies] INT32 in [0, numPages); an entry with either
 *                       outside is skipped. No page is destination twice, or both
 *                       source and destination (except of itself: nothing to do).
 * Host errors: as paged_kv_read.
 */
ROPEKV_API int paged_kv_copy_pages(void* kvCache, float* kvScales, const int32_t* srcPages,
                                   const int32_t* dstPages, int32_t numCopies, int32_t numKVHeads,
                                   int32_t headDim, int32_t numPages, int32_t tokensPerPage,
                                   int32_t cacheFormat, void* stream);

/* Bytes of workspace that paged_kv_fork needs, or a negative ropekv_status. Host only. */
ROPEKV_API int64_t paged_kv_fork_workspace_size(int32_t numForks, int32_t batch);

/*
 * Sequence children[i] becomes a copy of sequence parents[i], for beam search and for
 * several samples of one prompt. With n = kvLens[parent] (at most maxPagesPerSeq *
 * tokensPerPage), whole pages are shared: the child's entries are the parent's and
 * their refCounts grow by one. A partly filled last page is copied: its first n %
 * tokensPerPage tokens go to a free page, which gets refCounts 1; forks take the
 * lowest free pages in the order of i. Where none is left, or the parent's partly
 * filled page is unmapped, the child ends with its last whole page. The child's
 * other entries become -1, kvLens[child] its length. Pages that an empty child's row
 * still names (as paged_kv_accept_drafts leaves them where nothing is accepted) are
 * given up, their refCounts shrink by one; they are free for later calls, not for
 * forks of this one.
 *   pageTable  [batch, 2, maxPagesPerSeq] INT32, in and out.
 *   kvLens     [batch] INT32, in and out.
 *   parents, children  [numForks] INT32.
 * Skipped, without a sign but that table and lengths stay as they were: a fork whose parent
 * or child is out of range, whose child is not empty (kvLens[child] > 0; see paged_kv_free),
 * is named by two forks, or is a parent too. So beams that go on take empty sequences, and
 * the old ones are given up afterwards: a beam search keeps twice its sequences in the table.
 * Host errors: as paged_kv_read; batch > 2^18 or numForks > 2^20 -> ROPEKV_ERR_SHAPE;
 * workspaceBytes too small -> ROPEKV_ERR_CAPACITY.
 */
ROPEKV_API int paged_kv_fork(void* kvCache, float* kvScales, int32_t* pageTable, int32_t* kvLens,
                             int32_t* refCounts, const int32_t* parents, const int32_t* children,
                             void* workspace, int64_t workspaceBytes, int32_t numForks,
                             int32_t batch, int32_t numKVHeads, int32_t headDim, int32_t numPages,
                             int32_t maxPagesPerSeq, int32_t tokensPerPage, int32_t cacheFormat,
                             void* stream);

/*
 * Gives up the pages of sequences, whole or behind a length to keep: every entry of
 * sequence s = sequences[i] from column ceil(keepLens[i] / tokensPerPage) on becomes
 * -1, its page's refCounts shrinks by one, and kvLens[s] becomes min(kvLens[s],
 * keepLens[i]). A sequence may be named more than once: the smallest length counts.
 *   keepLens  [numSequences] INT32, or NULL: 0 for all. Negative ones count as 0.
 * A page that keepLens ends in stays, shared as it was: before tokens are written behind a
 * shorter length into a page of refCounts above 1, the sequence needs a copy of its own.
 * Sequences out of range are skipped.
 * Host errors: as paged_kv_read.
 */
ROPEKV_API int paged_kv_free(int32_t* pageTable, int32_t* kvLens, int32_t* refCounts,
                             const int32_t* sequences, const int32_t* keepLens,
                             int32_t numSequences, int32_t batch, int32_t numPages,
                             int32_t maxPagesPerSeq, int32_t tokensPerPage, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ROPEKV_SEQUENCE_H */
