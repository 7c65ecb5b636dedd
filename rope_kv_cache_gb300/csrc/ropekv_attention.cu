// ropekv_attention.cu -- host side of paged_attention_shared_prefix: argument
// checks, the choice of launch shape and the launches
// (include/ropekv_serving.h). Nothing allocates or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "ropekv_attention_kernels.cuh"
#include "ropekv_prefix_kernel.cuh"
#include "ropekv_serving.h"

namespace {

using ropekv_attn::Args;
using ropekv_attn::make_divisor;
using ropekv_attn::PrefixConfig;
using ropekv_attn::StreamConfig;

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

// How a call is cut into launches, from its sizes alone.
struct Plan {
    int nt;             // 1, 2: row tiles of the stream kernel of 8, 16 rows
    bool tensor;        // the prefix goes to the tensor-core kernel
    int parts;          // its ranges of the prefix
    int prefixTiles;    // its row tiles per KV head
    int tilesPrefix;    // row tiles of the stream kernel's prefix unit (0: none)
    int tilesSeq;       // and of a sequence
    int pitch;
    int teams, teamSize, groups;   // stream grid: CTAs, their warps, head groups
    int64_t partRows, slots, units;
};

int stream_warps(int D, int fmt, int nt);

// KV heads that a CTA reads side by side: the largest divisor of Hkv that leaves
// at most a quarter of an SM's warps idle, else the one that leaves fewest.
int team_size(int Hkv, int perSm)
{
    int best = 1, used = perSm;
    for (int t = 1, bestUsed = 0; t <= perSm && t <= Hkv; ++t) {
        if (Hkv % t != 0)
            continue;
        used = perSm / t * t;
        if (4 * used >= 3 * perSm || used > bestUsed) {
            best = t;
            bestUsed = used;
        }
    }
    return best;
}

// Tiles of 8 rows, or of 16 where a sequence has more. A sequence of more than 16
// rows is fetched once per tile, mostly from L2: tiles of 32 rows, which leave a warp
// too few registers to overlap anything, were slower (61 sequences x 28 rows of 7 to
// 700 tokens behind 2000, FP16: 66 us with 32, 55 with 16, 81 with 8). The prefix joins
// the stream if all rows of a KV head fit into one such tile.
//
// A tensor-core prefix of p ranges takes p CTAs per row tile, one to an SM, and the
// stream's CTAs start where there is room. Either the two kernels follow one another,
// each on all SMs, or the stream gets the SMs that the prefix leaves free and runs
// beside it: the prefix's products and the stream's loads then overlap. The estimate
// below, in microseconds, chooses p and the form. The lengths lie on the device: it
// takes the form that is best over calls three quarters of which fill half of their
// tables and one quarter a twentieth, as a prefix on few SMs is long and short
// sequences do not hide it (64 of 1 to 64 tokens in tables of 8192 behind 4096: 76 us
// if only the former count, 36 us). A table much wider than that misleads it towards one
// range of the prefix, or towards the forms apart (real lengths as before, tables of 16384
// and 131072 tokens instead of exact ones): 256 sequences behind 8192, FP16: 80 us, 92,
// 92; 128 behind 4097, E4M3: 67, 79, 78; 61 x 7 rows behind 2000, INT8: 59, 73, 73; 40
// behind 3001, 2 KV heads of 256: 21, 27, 58; 64 behind 4096 + 256, 2 KV heads of 128: 19,
// 23, 46. Measured, one after the other against side by
// side: 256 sequences of 1 to 512 tokens behind 8192, FP16: 89 against 79 us; 128 of
// 1 to 2048 behind 4097, E4M3: 78 against 68; 61 x 7 rows behind 2000, INT8: 86
// against 60; 40 of 1 to 900 behind 3001, D = 256: 32 against 22. The estimate keeps
// 128 of 1 to 2048 behind 16000, E4M3, apart: 105 against 114.
Plan make_plan(const ropekv_attention_dims* d)
{
    Plan p = {};
    const long long G = d->numQHeads / d->numKVHeads, rowsSeq = d->seqLen * G, rows = d->batch * rowsSeq;
    p.nt = rowsSeq <= 8 ? 1 : 2;
    p.tilesSeq = (int)((rowsSeq + 8 * p.nt - 1) / (8 * p.nt));
    p.tensor = d->prefixLen > 0 && rows > 8 * p.nt;
    p.tilesPrefix = d->prefixLen > 0 && !p.tensor ? 1 : 0;
    const long long longest = p.tilesPrefix ? rows : rowsSeq;
    p.pitch = (int)(longest < 8 * p.nt ? longest : 8 * p.nt);
    p.units = d->batch + p.tilesPrefix;
    const int perSm = stream_warps(d->headDim, d->cacheFormat, p.nt);
    p.teamSize = team_size(d->numKVHeads, perSm);
    p.groups = d->numKVHeads / p.teamSize;
    // the table's capacity bounds the steps
    const long long own = (long long)d->maxPagesPerSeq * d->tokensPerPage - d->prefixLen;
    const long long items = (long long)d->batch * p.tilesSeq * p.groups;
    const long long steps = items * (own > 0 ? own / 16 + 2 : 0) +
                            (p.tilesPrefix ? (long long)p.groups * (d->prefixLen / 16 + 1) : 0);
    const int teamsPerSm = perSm / p.teamSize;
    long long most = (long long)kSMs * teamsPerSm;
    if (p.tensor) {
        const bool f16 = d->cacheFormat == ROPEKV_CACHE_F16;
        const int tileRows = d->headDim != 256 && rows > 128 ? 256 : 128;
        p.prefixTiles = (int)((rows + tileRows - 1) / tileRows);
        const long long units = (long long)p.prefixTiles * d->numKVHeads;
        const long long kv = ((long long)d->prefixLen + 63) / 64;
        // one prefix tile, one warp's step on an SM, one range's partial written and read
        const double tile = f16 && d->headDim != 256 ? 0.95 : 1.3;
        const double step = (p.nt > 1 ? 0.22 : f16 ? 0.16 : 0.1) * d->headDim / 128;
        const double work = (double)steps * p.teamSize * step;
        const double part = 0.1 + (double)units * tileRows * d->headDim * 8 / 5e6;
        double best = HUGE_VAL;
        for (int k = 1; k <= ropekv_attn::kMaxParts && k <= kv; ++k) {
            const long long ctas = units * k, waves = (ctas + kSMs - 1) / kSMs;
            const double prefix = (double)waves * (8.0 + tile * (double)((kv + k - 1) / k));
            for (int beside = 0; beside <= (ctas < kSMs); ++beside) {
                const double sms = (double)(beside ? kSMs - ctas : kSMs);
                double half = 8.0 + 0.5 * work / sms, few = 8.0 + 0.05 * work / sms;
                half = part * k + (beside ? std::max(prefix, half) : prefix + half);
                few = part * k + (beside ? std::max(prefix, few) : prefix + few);
                const double cost = half * half * half * few;
                if (cost < best) {
                    best = cost;
                    p.parts = k;
                    most = (beside ? kSMs - ctas : kSMs) * teamsPerSm;
                }
            }
        }
    }
    // Few long units: a share of s steps leaves n / s partials to a row, of which the join
    // takes 8192 / D at a time, in about the time of a step: s = sqrt(n D / 8192) balances
    // the two (one sequence, one KV head, 14000 prefix tokens, INT8, D = 256: 27 us with
    // s = 1, 16 with 5; two sequences, four KV heads of 128, 6000 tokens: 12.6 and 12.7).
    // That is the join of few rows; one of 4 * kSMs rows and more takes four partials at a
    // time, but so many rows have steps enough that `most` decides.
    const long long longestSteps = std::max(p.tilesPrefix ? (long long)d->prefixLen / 16 : 0LL, own > 0 ? own / 16 : 0LL);
    const long long least = std::max(1LL, (long long)(sqrt((double)longestSteps * d->headDim / 8192) + 0.5));
    most = std::min(most, (steps + least - 1) / least);
    p.teams = (int)std::max(1LL, most);
    p.slots = (items + (long long)p.tilesPrefix * p.groups + p.teams) * p.teamSize;
    p.partRows = (int64_t)p.parts * d->numKVHeads * rows;
    return p;
}

// Workspace: partO, partL, segO, segL, offsets, each on a 256-byte boundary.
struct Layout {
    int64_t partL, segO, segL, offsets, size;
};

Layout make_layout(const Plan& p, int D)
{
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    Layout w;
    w.partL = up(p.partRows * D * 4);
    w.segO = w.partL + up(p.partRows * 4);
    w.segL = w.segO + up(p.slots * p.pitch * D * 4);
    w.offsets = w.segL + up(p.slots * p.pitch * 4);
    w.size = w.offsets + up((p.units + 1) * 8);
    return w;
}

template <int D, int FMT, int MT>
int launch_prefix(const Args& a, const Plan& p, cudaStream_t st)
{
    constexpr auto kern = ropekv_attn::prefix_kernel<D, FMT, MT>;
    using C = PrefixConfig<D, FMT, MT>;
    if (!raise_smem<kern>(C::kSmem))
        return ROPEKV_ERR_LAUNCH;
    return launch(kern, (long long)p.prefixTiles * a.Hkv * p.parts, C::kThreads, C::kSmem, false, st, a);
}

template <int D, int FMT, int NT>
int launch_stream(const Args& a, const Plan& p, cudaStream_t st)
{
    constexpr auto kern = ropekv_attn::stream_kernel<D, FMT, NT>;
    using C = StreamConfig<D, FMT, NT>;
    if (!raise_smem<kern>(C::smem(C::kPerSm)))
        return ROPEKV_ERR_LAUNCH;
    return launch(kern, p.teams, p.teamSize * 32, C::smem(p.teamSize), p.tensor, st, a);
}

template <int D, int FMT>
int launch_all(const Args& a, const Plan& p, cudaStream_t st)
{
    int rc = ROPEKV_OK;
    if (p.tensor) {
        if constexpr (D != 256) {
            rc = a.rowsPrefix > 128 ? launch_prefix<D, FMT, 2>(a, p, st) : launch_prefix<D, FMT, 1>(a, p, st);
        } else {
            rc = launch_prefix<D, FMT, 1>(a, p, st);
        }
    }
    if (rc != ROPEKV_OK)
        return rc;
    rc = p.nt == 1 ? launch_stream<D, FMT, 1>(a, p, st) : launch_stream<D, FMT, 2>(a, p, st);
    if (rc != ROPEKV_OK)
        return rc;
    // few rows whose items many warps share: all groups of a CTA join one row
    const long long rows = (long long)a.B * a.S * a.Hq;
    constexpr int perCta = 2048 / D;
    const int tileShift = p.nt == 1 ? 3 : 4;
    if (rows < 4LL * kSMs)
        return launch(ropekv_attn::join_kernel<D, true>, rows, 256, 0, true, st, a, tileShift);
    return launch(ropekv_attn::join_kernel<D, false>, (rows + perCta - 1) / perCta, 256, 0, true, st, a, tileShift);
}

template <int D>
int dispatch(const Args& a, const Plan& p, int fmt, cudaStream_t st)
{
    switch (fmt) {
    case ROPEKV_CACHE_F16: return launch_all<D, ROPEKV_CACHE_F16>(a, p, st);
    case ROPEKV_CACHE_E4M3: return launch_all<D, ROPEKV_CACHE_E4M3>(a, p, st);
    default: return launch_all<D, ROPEKV_CACHE_INT8>(a, p, st);
    }
}

// Warps of an SM (both 8-bit formats have the same shape).
template <int D>
int stream_warps(bool f16, int nt)
{
    if (nt == 2)
        return f16 ? StreamConfig<D, ROPEKV_CACHE_F16, 2>::kPerSm : StreamConfig<D, ROPEKV_CACHE_E4M3, 2>::kPerSm;
    return f16 ? StreamConfig<D, ROPEKV_CACHE_F16, 1>::kPerSm : StreamConfig<D, ROPEKV_CACHE_E4M3, 1>::kPerSm;
}

int stream_warps(int D, int fmt, int nt)
{
    const bool f16 = fmt == ROPEKV_CACHE_F16;
    return D == 64 ? stream_warps<64>(f16, nt) : D == 128 ? stream_warps<128>(f16, nt) : stream_warps<256>(f16, nt);
}

}  // namespace

extern "C" {

int64_t paged_attention_workspace_size(const ropekv_attention_dims* dims)
{
    const int rc = check_dims(dims);
    if (rc != ROPEKV_OK)
        return rc;
    if (dims->batch == 0 || dims->seqLen == 0)
        return 0;
    return make_layout(make_plan(dims), dims->headDim).size;
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
    const Plan plan = make_plan(dims);
    const Layout at = make_layout(plan, dims->headDim);
    const bool f16 = dims->cacheFormat == ROPEKV_CACHE_F16;
    if (!q || !kvLens || !out || (!kvCache && dims->numPages > 0) ||
        (!f16 && !kvScales && dims->numPages > 0) || (!prefixTable && dims->prefixLen > 0) ||
        (!pageTable && dims->maxPagesPerSeq > 0) || !workspace)
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(q) || !aligned16(kvCache) || !aligned16(kvScales) || !aligned16(prefixTable) ||
        !aligned16(pageTable) || !aligned16(kvLens) || !aligned16(out) || !aligned16(lse) ||
        !aligned16(workspace))
        return ROPEKV_ERR_MISALIGNED;
    if (workspaceBytes < at.size)
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
    uint8_t* ws = (uint8_t*)workspace;
    a.partO = (float*)ws;
    a.partL = (float*)(ws + at.partL);
    a.segO = (float*)(ws + at.segO);
    a.segL = (float*)(ws + at.segL);
    a.offsets = (long long*)(ws + at.offsets);
    a.numParts = plan.parts;
    a.prefixUnit = plan.tilesPrefix;
    a.tilesPrefix = plan.tilesPrefix;
    a.tilesSeq = plan.tilesSeq;
    a.pitch = plan.pitch;
    a.teams = plan.teams;
    a.teamSize = plan.teamSize;
    a.groups = plan.groups;
    a.divTpp = make_divisor(a.tpp);
    a.divG = make_divisor(a.G);
    a.divGroups = make_divisor(a.groups);
    a.divTeam = make_divisor(a.teamSize);
    a.divS = make_divisor(a.S);
    cudaStream_t st = (cudaStream_t)stream;
    switch (dims->headDim) {
    case 64: return dispatch<64>(a, plan, dims->cacheFormat, st);
    case 128: return dispatch<128>(a, plan, dims->cacheFormat, st);
    default: return dispatch<256>(a, plan, dims->cacheFormat, st);
    }
}

}  // extern "C"
