// ropekv_sequence.cu -- host side of prompt_attention and tree_attention: argument
// checks, tensor maps, the choice of launch shape and the launches
// (include/ropekv_sequence.h). Nothing allocates or synchronises.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "ropekv_rows_kernel.cuh"
#include "ropekv_sequence.h"

namespace {

using ropekv_attn::make_divisor;
using ropekv_rows::RowsArgs;
using ropekv_rows::RowsConfig;

constexpr int kSMs = 152;

std::atomic<int> failing{0};      // ropekv_sequence_fail

bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// A kernel's dynamic shared memory limit is raised once per device.
template <auto Kern>
bool raise_smem(int bytes)
{
    static std::atomic<unsigned long long> raised{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return false;
    const unsigned long long bit = (dev >= 0 && dev < 64) ? 1ULL << dev : 0;
    if (bit && (raised.load(std::memory_order_relaxed) & bit))
        return true;
    if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return false;
    raised.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

template <typename Kern, typename... A>
int launch(Kern kern, long long grid, int threads, int smem, bool dependent, cudaStream_t st, const A&... args)
{
    if (grid > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = dependent ? attr : nullptr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? ROPEKV_OK : ROPEKV_ERR_LAUNCH;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library does not link with the driver).
EncodeTiled encoder()
{
    static std::atomic<void*> found{nullptr};
    void* f = found.load(std::memory_order_relaxed);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(f, std::memory_order_relaxed);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// [d3][d2][d1][D] FP16 with strides in elements, read in boxes of 64 dims x b1 x b2 in rows of
// 128 swizzled bytes; what lies outside reads as zeros.
bool make_map(CUtensorMap* map, const uint16_t* p, int D, int64_t d1, int64_t s1, int64_t d2, int64_t s2, int64_t d3,
              int64_t s3, int b1, int b2)
{
    const EncodeTiled encode = encoder();
    if (encode == nullptr)
        return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)d1, (cuuint64_t)d2, (cuuint64_t)d3};
    const cuuint64_t strides[3] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2, (cuuint64_t)s3 * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<uint16_t*>(p), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is cut, from its sizes alone (the shares follow from the lengths, on the device).
struct Plan {
    int mt;                   // row tiles of a CTA
    int perSm;                // CTAs of an SM
    int G, heads, tokens;     // heads of a tile, head groups, tokens of a CTA's tiles
    int tilesSeq;             // tree: CTA tiles of a sequence
    int ctas;
    bool whole;               // no unit is split: there is nothing to join
    int leastShare;
};

// Rows of a tile: the heads that share a KV head, or a divisor of them that fits.
int group_of(int Hq, int Hkv)
{
    const int all = Hq / Hkv;
    for (int m = 1;; ++m)
        if (all % m == 0 && all / m <= 128)
            return all / m;
}

Plan make_plan(bool tree, int64_t T, int B, int S, int Hq, int Hkv, int D, int64_t keys)
{
    Plan p = {};
    p.G = group_of(Hq, Hkv);
    p.heads = Hq / p.G;
    const int64_t rows = (tree ? S : (T + B - 1) / std::max(1, B)) * (int64_t)p.G;     // of a sequence, in mean
    // Two row tiles share K and V and alternate. One tile in their place, D = 128: 32 prompts of
    // 300 tokens 77 us instead of 62, one of 8000 460 instead of 345; 64 of 100 tokens 50 instead of 39.
    p.mt = D != 256 && rows > 128 ? 2 : 1;
    p.tokens = 128 * p.mt / p.G;
    p.tilesSeq = (S + p.tokens - 1) / p.tokens;
    // at most so many units, of so many K/V tiles
    const int64_t units = (tree ? (int64_t)B * p.tilesSeq : T / p.tokens + std::min<int64_t>(B, T)) * p.heads;
    const int64_t tiles = std::max<int64_t>(1, (keys + (D == 256 ? 63 : 127)) / (D == 256 ? 64 : 128));
    p.whole = tiles + ropekv_rows::kSwitch <= 2 + (p.mt == 2 ? ropekv_rows::kSplit<2> : ropekv_rows::kSplit<1>);
    p.leastShare = 4;
    // One row tile: two CTAs of an SM overlap what a step and a change of units wait for, at the
    // cost of scores looked ahead and of stages in flight, which few units, and long ones of
    // 128 dims, need more. One against two, 32 query and 8 KV heads: 200 prompts of 30 tokens 50
    // against 38 us (D = 128), 44 against 27 (D = 64); 64 decoding sequences of 100 to 200 tokens 27
    // against 18; 128 of 2000 to 4000, D = 64, 152 against 130; 16 trees of 26 drafts behind 2000
    // to 4000, D = 128, 48 against 53; one decoding sequence of 16000, D = 64, 17 against 19.
    const int64_t mean = tree ? tiles : (tiles + B - 1) / std::max(1, B);
    p.perSm = p.mt == 1 && D != 256 && units >= kSMs / 2 && (D == 64 || mean <= 8) ? 2 : 1;
    p.ctas = (int)std::min<int64_t>(kSMs * p.perSm, p.whole ? units : units * ((tiles + ropekv_rows::kSwitch + p.leastShare - 1) / p.leastShare));
    return p;
}

// Workspace: joints, partL, partO, each on a 256-byte boundary.
struct Layout {
    int64_t partL, partO, size;
};

Layout make_layout(const Plan& p, int D)
{
    if (p.whole)
        return {0, 0, 16};
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    const int64_t rows = 2LL * p.ctas * p.mt * 128;
    Layout w;
    w.partL = up(p.ctas * (int64_t)sizeof(ropekv_rows::Joint));
    w.partO = w.partL + up(rows * 4);
    w.size = w.partO + up(rows * D * 4);
    return w;
}

template <int D, int MT, int PER, bool TREE>
int launch_rows(const RowsArgs& a, const Plan& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                cudaStream_t st)
{
    constexpr auto kern = ropekv_rows::rows_kernel<D, MT, PER, TREE>;
    using C = RowsConfig<D, MT, PER>;
    if (!raise_smem<kern>(C::kSmem))
        return ROPEKV_ERR_LAUNCH;
    const int rc = launch(kern, p.ctas, C::kThreads, C::kSmem, true, st, a, q, k, v);
    if (rc != ROPEKV_OK || p.whole)
        return rc;
    return launch(ropekv_rows::rows_join_kernel<D, MT>, p.ctas * (long long)(MT * 16 * (D / 32) / 8), 256, 0, true, st, a);
}

template <bool TREE>
int run(RowsArgs& a, const Plan& p, int D, int Hkv, int64_t kvTokens, int64_t kvBatches, void* workspace, cudaStream_t st)
{
    a.G = p.G;
    a.heads = p.heads;
    a.headsPerKv = p.heads / Hkv;
    a.tokens = p.tokens;
    a.tilesSeq = p.tilesSeq;
    a.ctas = p.ctas;
    a.whole = p.whole;
    a.leastShare = p.leastShare;
    a.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    a.fail = failing.load(std::memory_order_relaxed);
    a.divG = make_divisor(p.G);
    const Layout at = make_layout(p, D);
    a.joints = (ropekv_rows::Joint*)workspace;
    a.partL = (float*)((uint8_t*)workspace + at.partL);
    a.partO = (float*)((uint8_t*)workspace + at.partO);
    const int tile = D == 256 ? 64 : 128;
    CUtensorMap q, k, v;
    const int64_t batchStride = TREE ? a.kvBatch : 8;     // of a single batch any will do
    if (!make_map(&q, a.q, D, p.G, D, a.T, a.qStride, p.heads, (int64_t)p.G * D, p.G, p.tokens) ||
        !make_map(&k, a.k, D, kvTokens, a.kTok, Hkv, a.kvHead, kvBatches, batchStride, tile, 1) ||
        !make_map(&v, a.v, D, kvTokens, a.vTok, Hkv, a.kvHead, kvBatches, batchStride, tile, 1))
        return ROPEKV_ERR_LAUNCH;
    switch (D) {
    case 64:
        return p.mt == 2 ? launch_rows<64, 2, 1, TREE>(a, p, q, k, v, st)
             : p.perSm == 2 ? launch_rows<64, 1, 2, TREE>(a, p, q, k, v, st) : launch_rows<64, 1, 1, TREE>(a, p, q, k, v, st);
    case 128:
        return p.mt == 2 ? launch_rows<128, 2, 1, TREE>(a, p, q, k, v, st)
             : p.perSm == 2 ? launch_rows<128, 1, 2, TREE>(a, p, q, k, v, st) : launch_rows<128, 1, 1, TREE>(a, p, q, k, v, st);
    default: return launch_rows<256, 1, 1, TREE>(a, p, q, k, v, st);
    }
}

int check_heads(int32_t Hq, int32_t Hkv, int32_t D)
{
    if (D != 64 && D != 128 && D != 256)
        return ROPEKV_ERR_HEAD_DIM;
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0)
        return ROPEKV_ERR_HEADS;
    return (long long)Hq * D > (1LL << 24) ? ROPEKV_ERR_SHAPE : ROPEKV_OK;
}

int check_prompt(const ropekv_prompt_dims* d)
{
    if (d == nullptr)
        return ROPEKV_ERR_NULL_POINTER;
    const int rc = check_heads(d->numQHeads, d->numKVHeads, d->headDim);
    if (rc != ROPEKV_OK)
        return rc;
    if (d->numTokens < 0 || d->numKVTokens < 0 || d->batch < 0 || d->numTokens > (1 << 28) ||
        d->numKVTokens > (1 << 28) || d->batch > (1 << 20) || (long long)d->numTokens * d->numQHeads > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    return ROPEKV_OK;
}

Plan plan_of(const ropekv_prompt_dims* d)
{
    return make_plan(false, d->numTokens, d->batch, 0, d->numQHeads, d->numKVHeads, d->headDim, d->numKVTokens);
}

int check_tree(const ropekv_tree_dims* d)
{
    if (d == nullptr)
        return ROPEKV_ERR_NULL_POINTER;
    const int rc = check_heads(d->numQHeads, d->numKVHeads, d->headDim);
    if (rc != ROPEKV_OK)
        return rc;
    if (d->batch < 0 || d->seqLen < 0 || d->seqLen > (1 << 15) || d->kvCapacity < 0 || d->kvCapacity > (1 << 28) ||
        (long long)d->batch * d->seqLen > 0x7FFFFFFFLL / d->numQHeads ||
        (long long)d->kvCapacity * d->numKVHeads > (1LL << 37) / d->headDim ||
        (long long)d->kvCapacity * d->numKVHeads * d->headDim > (1LL << 40) / std::max(1, d->batch))
        return ROPEKV_ERR_SHAPE;
    return ROPEKV_OK;
}

Plan plan_of(const ropekv_tree_dims* d)
{
    return make_plan(true, (int64_t)d->batch * d->seqLen, d->batch, d->seqLen, d->numQHeads, d->numKVHeads, d->headDim,
                     d->kvCapacity);
}

// Scores are held in binary digits.
float scale_log2(float smScale)
{
    return smScale * 1.4426950408889634f;
}

bool overlap(const uint16_t* p, int64_t n, const uint16_t* q, int64_t m)
{
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + 2 * m && b < a + 2 * n;
}

}  // namespace

extern "C" {

// Not part of the interface, for tests of what a wait that runs out leaves: with `on`, the attention
// calls from now on end as if one had done so before anything is in flight. Returns what was set.
ROPEKV_API int ropekv_sequence_fail(int on)
{
    return failing.exchange(on != 0, std::memory_order_relaxed);
}

int64_t prompt_attention_workspace_size(const ropekv_prompt_dims* dims)
{
    const int rc = check_prompt(dims);
    if (rc != ROPEKV_OK)
        return rc;
    if (dims->numTokens == 0 || dims->batch == 0)
        return 0;
    return make_layout(plan_of(dims), dims->headDim).size;
}

int prompt_attention(const uint16_t* q, int64_t qTokenStride, const uint16_t* k, int64_t kTokenStride,
                     const uint16_t* v, int64_t vTokenStride, const int32_t* qStarts,
                     const int32_t* kvStarts, uint16_t* out, float* lse, void* workspace,
                     int64_t workspaceBytes, const ropekv_prompt_dims* dims, float smScale, void* stream)
{
    const int rc = check_prompt(dims);
    if (rc != ROPEKV_OK)
        return rc;
    const int64_t most = 1LL << 36, Hq = dims->numQHeads, Hkv = dims->numKVHeads, D = dims->headDim;
    if (qTokenStride < Hq * D || kTokenStride < Hkv * D || vTokenStride < Hkv * D || qTokenStride % 8 != 0 ||
        kTokenStride % 8 != 0 || vTokenStride % 8 != 0 || qTokenStride > most || kTokenStride > most ||
        vTokenStride > most || !isfinite(scale_log2(smScale)))
        return ROPEKV_ERR_SHAPE;
    if (dims->numTokens == 0 || dims->batch == 0)
        return ROPEKV_OK;
    if (!q || !qStarts || !out || !workspace || (dims->numKVTokens > 0 && (!k || !v)))
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(qStarts) || !aligned16(kvStarts) ||
        !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
        return ROPEKV_ERR_MISALIGNED;
    const int64_t size = dims->numTokens * Hq * D, last = std::max(0, dims->numKVTokens - 1);
    if (overlap(q, (dims->numTokens - 1) * qTokenStride + Hq * D, out, size) ||
        (dims->numKVTokens > 0 && (overlap(k, last * kTokenStride + Hkv * D, out, size) ||
                                   overlap(v, last * vTokenStride + Hkv * D, out, size))))
        return ROPEKV_ERR_SHAPE;
    const Plan p = plan_of(dims);
    if (workspaceBytes < make_layout(p, dims->headDim).size)
        return ROPEKV_ERR_CAPACITY;
    RowsArgs a = {};
    a.q = q;
    // without keys nothing is read; the maps still need an address
    a.k = dims->numKVTokens > 0 ? k : q;
    a.v = dims->numKVTokens > 0 ? v : q;
    a.out = out;
    a.lse = lse;
    a.qStarts = qStarts;
    a.kvStarts = kvStarts != nullptr ? kvStarts : qStarts;
    a.qStride = qTokenStride;
    a.kTok = kTokenStride;
    a.vTok = vTokenStride;
    a.kvHead = D;
    a.kvBatch = 0;            // one run of keys for all sequences
    a.scaleLog2 = scale_log2(smScale);
    a.T = dims->numTokens;
    a.Tk = dims->numKVTokens;
    a.B = dims->batch;
    a.Hq = dims->numQHeads;
    return run<false>(a, p, dims->headDim, dims->numKVHeads, std::max(1, dims->numKVTokens), 1, workspace,
                      (cudaStream_t)stream);
}

int64_t tree_attention_workspace_size(const ropekv_tree_dims* dims)
{
    const int rc = check_tree(dims);
    if (rc != ROPEKV_OK)
        return rc;
    if (dims->batch == 0 || dims->seqLen == 0)
        return 0;
    return make_layout(plan_of(dims), dims->headDim).size;
}

int tree_attention(const uint16_t* q, const uint16_t* kvCache, const int32_t* kvCacheEndLens,
                   const int32_t* treeMask, uint16_t* out, float* lse, void* workspace,
                   int64_t workspaceBytes, const ropekv_tree_dims* dims, float smScale, void* stream)
{
    const int rc = check_tree(dims);
    if (rc != ROPEKV_OK)
        return rc;
    if (!isfinite(scale_log2(smScale)))
        return ROPEKV_ERR_SHAPE;
    if (dims->batch == 0 || dims->seqLen == 0)
        return ROPEKV_OK;
    if (!q || !kvCacheEndLens || !out || !workspace || (!kvCache && dims->kvCapacity > 0))
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(kvCache) || !aligned16(kvCacheEndLens) || !aligned16(treeMask) ||
        !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
        return ROPEKV_ERR_MISALIGNED;
    const int64_t T = (int64_t)dims->batch * dims->seqLen, row = (int64_t)dims->numQHeads * dims->headDim;
    const int64_t cap = std::max(1, dims->kvCapacity), plane = cap * dims->numKVHeads * dims->headDim;
    if (overlap(q, T * row, out, T * row) ||
        (dims->kvCapacity > 0 && overlap(kvCache, 2LL * dims->batch * plane, out, T * row)))
        return ROPEKV_ERR_SHAPE;
    const Plan p = plan_of(dims);
    if (workspaceBytes < make_layout(p, dims->headDim).size)
        return ROPEKV_ERR_CAPACITY;
    RowsArgs a = {};
    a.q = q;
    a.k = dims->kvCapacity > 0 ? kvCache : q;
    a.v = dims->kvCapacity > 0 ? kvCache + plane : q;
    a.out = out;
    a.lse = lse;
    a.endLens = kvCacheEndLens;
    a.treeMask = treeMask;
    a.qStride = row;
    a.kTok = a.vTok = dims->headDim;
    a.kvHead = cap * dims->headDim;
    a.kvBatch = 2 * plane;
    a.scaleLog2 = scale_log2(smScale);
    a.T = (int32_t)T;
    a.B = dims->batch;
    a.S = dims->seqLen;
    a.W = (dims->seqLen + 31) / 32;
    a.cap = dims->kvCapacity;
    a.Hq = dims->numQHeads;
    return run<true>(a, p, dims->headDim, dims->numKVHeads, cap, dims->batch, workspace, (cudaStream_t)stream);
}

}  // extern "C"
