// ropekv_attention.cu -- host side of paged_attention_shared_prefix: argument
// checks, the choice of launch shape and the launches
// (include/ropekv_serving.h). Nothing allocates or synchronises.
#include <cuda_runtime.h>

#include <atomic>
#include <math.h>
#include <stdint.h>

#include "ropekv_attention_kernels.cuh"
#include "ropekv_prefix_kernel.cuh"
#include "ropekv_serving.h"

namespace {

using ropekv_attn::Args;
using ropekv_attn::PrefixConfig;
using ropekv_attn::RowsConfig;

constexpr int kSMs = 152;

bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

int check_dims(const ropekv_attention_dims* d)
{
    if (d == nullptr)
        return ROPEKV_ERR_NULL_POINTER;
    if (d->cacheFormat < ROPEKV_CACHE_F16 || d->cacheFormat > ROPEKV_CACHE_INT8)
        return ROPEKV_ERR_STYLE;
    if (d->headDim != 64 && d->headDim != 128 && d->headDim != 256)
        return ROPEKV_ERR_HEAD_DIM;
    if (d->numQHeads <= 0 || d->numKVHeads <= 0 || d->numQHeads % d->numKVHeads != 0)
        return ROPEKV_ERR_HEADS;
    if (d->batch < 0 || d->seqLen < 0 || d->seqLen > (1 << 15) || d->numPages < 0 ||
        d->tokensPerPage <= 0 || d->maxPagesPerSeq < 0 || d->prefixLen < 0 || d->maxPrefixPages < 0)
        return ROPEKV_ERR_SHAPE;
    if (2LL * d->numPages * d->tokensPerPage > 0x7FFFFFFFLL ||
        (long long)d->maxPagesPerSeq * d->tokensPerPage > (1LL << 30) ||
        d->prefixLen > (1 << 30) ||
        d->prefixLen > (long long)d->maxPrefixPages * d->tokensPerPage ||
        (long long)d->batch * d->seqLen > (1LL << 30) / d->numQHeads)
        return ROPEKV_ERR_SHAPE;
    return ROPEKV_OK;
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

// CTAs of a cluster that share one tile's tokens: enough of them for two CTAs
// per SM, but at least one step of 16 tokens for each of their warps.
int cluster_size(long long tiles, long long tokens, int warps)
{
    int c = 1;
    while (c < ropekv_attn::kMaxCluster && tiles * c < 2 * kSMs && tokens > 16LL * warps * c)
        c *= 2;
    return c;
}

template <int D, int FMT, int NT, bool PREFIX>
int launch_rows(const Args& a, long long tiles, long long tokens, bool dependent, cudaStream_t st)
{
    constexpr auto kern = ropekv_attn::rows_kernel<D, FMT, NT, PREFIX>;
    constexpr int smem = RowsConfig<D, FMT, NT>::kSmem;
    if (!raise_smem<kern>(smem))
        return ROPEKV_ERR_LAUNCH;
    constexpr int warps = RowsConfig<D, FMT, NT>::kWarps;
    const int c = cluster_size(tiles, tokens, warps);
    if (tiles * c > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * c));
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (c > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = c;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? ROPEKV_OK : ROPEKV_ERR_LAUNCH;
}

// How the prefix is cut: `tensor` rows take tcgen05 tiles of 128 (or 2 x 128)
// rows, fewer take the rows kernel, whose cluster leaves one partial.
struct PrefixPlan {
    bool tensor;
    int tiles;   // row tiles per KV head
    int parts;   // ranges of the prefix = partials in the workspace
};

// Ranges of the prefix: their number p minimises the K/V tiles that the busiest
// SM walks, waves(units * p) * ceil(tiles / p), where each CTA costs about three
// tiles more to start and to write its partial.
PrefixPlan plan_prefix(const ropekv_attention_dims* d)
{
    PrefixPlan plan = {false, 0, 0};
    if (d->prefixLen <= 0 || d->batch == 0 || d->seqLen == 0)
        return plan;
    const long long rows = (long long)d->batch * d->seqLen * (d->numQHeads / d->numKVHeads);
    plan.tensor = rows > 8;
    plan.parts = 1;
    if (!plan.tensor) {
        plan.tiles = (int)((rows + 7) / 8);
        return plan;
    }
    const int tileRows = d->headDim != 256 && rows > 128 ? 256 : 128;
    const int tokens = d->headDim == 256 ? 64 : 128;
    plan.tiles = (int)((rows + tileRows - 1) / tileRows);
    const long long units = (long long)plan.tiles * d->numKVHeads;
    const long long kv = ((long long)d->prefixLen + tokens - 1) / tokens;
    double best = 1e30;
    for (int p = 1; p <= ropekv_attn::kMaxParts && p <= kv; ++p) {
        const double waves = (double)((units * p + kSMs - 1) / kSMs);
        const double cost = waves * ((double)((kv + p - 1) / p) + 3.0) + 0.25 * p;
        if (cost < best) {
            best = cost;
            plan.parts = p;
        }
    }
    return plan;
}

template <int D, int FMT, int MT>
int launch_prefix(const Args& a, long long ctas, cudaStream_t st)
{
    constexpr auto kern = ropekv_attn::prefix_kernel<D, FMT, MT>;
    using C = PrefixConfig<D, FMT, MT>;
    if (!raise_smem<kern>(C::kSmem))
        return ROPEKV_ERR_LAUNCH;
    if (ctas > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? ROPEKV_OK : ROPEKV_ERR_LAUNCH;
}

// The sequences' own tokens: tiles of 8 rows, or of 16 or 32 (D = 256: 16) where
// a sequence has more, so that its tokens are fetched once.
template <int D, int FMT, int NT>
int launch_own(Args& a, bool dependent, cudaStream_t st)
{
    a.tilesPerUnit = (a.S * a.G + 8 * NT - 1) / (8 * NT);
    const long long own = (long long)a.mpps * a.tpp - a.P;
    return launch_rows<D, FMT, NT, false>(a, (long long)a.B * a.tilesPerUnit * a.Hkv, own, dependent, st);
}

template <int D, int FMT>
int launch_all(Args a, const PrefixPlan& plan, cudaStream_t st)
{
    int rc = ROPEKV_OK;
    a.numParts = plan.parts;
    if (plan.tensor) {
        const long long ctas = (long long)plan.tiles * a.Hkv * plan.parts;
        if constexpr (D != 256) {
            rc = a.rowsPrefix > 128 ? launch_prefix<D, FMT, 2>(a, ctas, st)
                                    : launch_prefix<D, FMT, 1>(a, ctas, st);
        } else {
            rc = launch_prefix<D, FMT, 1>(a, ctas, st);
        }
    } else if (plan.parts > 0) {
        a.tilesPerUnit = plan.tiles;
        rc = launch_rows<D, FMT, 1, true>(a, (long long)plan.tiles * a.Hkv, a.P, false, st);
    }
    if (rc != ROPEKV_OK)
        return rc;
    const int rows = a.S * a.G;
    if (rows <= 8)
        return launch_own<D, FMT, 1>(a, plan.parts > 0, st);
    if constexpr (D != 256) {
        if (rows > 16)
            return launch_own<D, FMT, 4>(a, plan.parts > 0, st);
    }
    return launch_own<D, FMT, 2>(a, plan.parts > 0, st);
}

template <int D>
int dispatch(const Args& a, const PrefixPlan& plan, int fmt, cudaStream_t st)
{
    switch (fmt) {
    case ROPEKV_CACHE_F16: return launch_all<D, ROPEKV_CACHE_F16>(a, plan, st);
    case ROPEKV_CACHE_E4M3: return launch_all<D, ROPEKV_CACHE_E4M3>(a, plan, st);
    default: return launch_all<D, ROPEKV_CACHE_INT8>(a, plan, st);
    }
}

int64_t workspace_size(const ropekv_attention_dims* d, const PrefixPlan& plan)
{
    const int64_t rows = (int64_t)d->batch * d->seqLen * d->numQHeads * plan.parts;
    return rows * d->headDim * 4 + (rows * 4 + 15) / 16 * 16;
}

}  // namespace

extern "C" {

int64_t paged_attention_workspace_size(const ropekv_attention_dims* dims)
{
    const int rc = check_dims(dims);
    if (rc != ROPEKV_OK)
        return rc;
    return workspace_size(dims, plan_prefix(dims));
}

int paged_attention_shared_prefix(const uint16_t* q, const void* kvCache, const float* kvScales,
                                  const int32_t* prefixTable, const int32_t* pageTable,
                                  const int32_t* kvLens, uint16_t* out, float* lse,
                                  void* workspace, int64_t workspaceBytes,
                                  const ropekv_attention_dims* dims, float smScale, void* stream)
{
    const int rc = check_dims(dims);
    if (rc != ROPEKV_OK)
        return rc;
    if (!isfinite(smScale))
        return ROPEKV_ERR_SHAPE;
    if (dims->batch == 0 || dims->seqLen == 0)
        return ROPEKV_OK;
    const PrefixPlan plan = plan_prefix(dims);
    const int64_t need = workspace_size(dims, plan);
    const bool f16 = dims->cacheFormat == ROPEKV_CACHE_F16;
    if (!q || !kvLens || !out || (!kvCache && dims->numPages > 0) ||
        (!f16 && !kvScales && dims->numPages > 0) || (!prefixTable && dims->prefixLen > 0) ||
        (!pageTable && dims->maxPagesPerSeq > 0) || (!workspace && need > 0))
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(kvCache) || !aligned16(kvScales) || !aligned16(prefixTable) ||
        !aligned16(pageTable) || !aligned16(kvLens) || !aligned16(out) || !aligned16(lse) ||
        !aligned16(workspace))
        return ROPEKV_ERR_MISALIGNED;
    if (workspaceBytes < need)
        return ROPEKV_ERR_CAPACITY;
    Args a = {};
    a.q = q;
    a.pool = (const uint8_t*)kvCache;
    a.scales = kvScales;
    a.prefixTable = prefixTable;
    a.pageTable = pageTable;
    a.kvLens = kvLens;
    a.out = out;
    a.lse = lse;
    a.scaleLog2 = smScale * 1.4426950408889634f;
    a.B = dims->batch;
    a.S = dims->seqLen;
    a.Hq = dims->numQHeads;
    a.Hkv = dims->numKVHeads;
    a.G = dims->numQHeads / dims->numKVHeads;
    a.numPages = dims->numPages;
    a.tpp = dims->tokensPerPage;
    a.mpps = dims->maxPagesPerSeq;
    a.P = dims->prefixLen;
    a.prefixPages = dims->maxPrefixPages;
    a.rowsPrefix = dims->batch * dims->seqLen * a.G;
    a.partO = (float*)workspace;
    a.partL = a.partO + (size_t)plan.parts * a.rowsPrefix * a.Hkv * dims->headDim;
    cudaStream_t st = (cudaStream_t)stream;
    switch (dims->headDim) {
    case 64: return dispatch<64>(a, plan, dims->cacheFormat, st);
    case 128: return dispatch<128>(a, plan, dims->cacheFormat, st);
    default: return dispatch<256>(a, plan, dims->cacheFormat, st);
    }
}

}  // extern "C"
