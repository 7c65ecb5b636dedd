// ropekv_serving.cu -- cache writes with several position axes, the 8-bit
// cache with a scale per token and head, and reading a paged cache back:
// kernels and C entry points (include/ropekv_serving.h). All three are
// streaming kernels, bound by HBM, and share the item decomposition, the L2
// policies and the dependent-launch prologue of ropekv_kernels.cuh: an item is
// two 16-byte vectors of one head, D/16 consecutive lanes hold a head. All but the
// cos/sin rows comes by ordinary loads: a CTA may be resident before the grid in front of
// it has overwritten what it will read (its wait orders the two), so these are not
// constant for the life of the kernel, as the non-coherent path asks.
#include <cuda_runtime.h>

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ropekv_kernels.cuh"
#include "ropekv_serving.h"

namespace {

using namespace ropekv;

constexpr int kMaxAxes = 4;

// Token-strided Q, K, V and the slots they go to (both writes).
struct WriteArgs {
    const float* cosSin;       // [csRows, r]
    const int64_t* positions;  // [axes, T]
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int64_t* slots;      // [T]
    void* keyCache;            // [numBlocks, blockSize, Hkv, D]
    void* valueCache;
    float* keyScales;          // [numBlocks, Hkv, blockSize] (8-bit cache)
    float* valueScales;
    uint16_t* qOut;            // [T, Hq, D]
    uint16_t* kOut;            // [T, Hkv, D] or NULL
    int64_t qStride, kStride, vStride, numSlots;
    int32_t T, Hq, Hkv, r, csRows, blockSize;
    int32_t itemsPerToken;     // (Hq + 2 Hkv) * D / 16
    int32_t ctasPerToken;
    int32_t numAxes;
    uint64_t axisBits[4];      // two bits per frequency, frequency i at bit 2i
};

// ---------------------------------------------------- multi-axis positions --

__device__ __forceinline__ int64_t pick(const int64_t off[kMaxAxes], uint32_t axis)
{
    return axis == 0 ? off[0] : axis == 1 ? off[1] : axis == 2 ? off[2] : off[3];
}

__device__ __forceinline__ const uint16_t* head_row(const WriteArgs& a, int tok, int head, int D)
{
    if (head < a.Hq)
        return a.q + tok * a.qStride + (size_t)head * D;
    if (head < a.Hq + a.Hkv)
        return a.k + tok * a.kStride + (size_t)(head - a.Hq) * D;
    return a.v + tok * a.vStride + (size_t)(head - a.Hq - a.Hkv) * D;
}

// Before the wait on the previous grid: L2 prefetches of the thread's inputs
// and the token's index words, nothing into a register.
template <int D, int IPT>
__device__ __forceinline__ void prefetch_inputs(const WriteArgs& a, int tok, int item0, int va,
                                                int vb)
{
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int item = item0 + k * blockDim.x;
        if (item < a.itemsPerToken) {
            const uint16_t* p = head_row(a, tok, item / (D / 16), D);
            prefetch_l2(p + 8 * va);
            prefetch_l2(p + 8 * vb);
        }
    }
    if (threadIdx.x < a.numAxes)
        prefetch_l2(a.positions + (int64_t)threadIdx.x * a.T + tok);
    if (threadIdx.x == 0)
        prefetch_l2(a.slots + tok);
}

// Rotary positions with several axes: as the slot-mapping kernel, but each
// frequency comes from the row of its own axis. A token whose positions agree
// (text) reads one row with vector loads; for another the CTA gathers its row in
// shared memory, one thread a frequency (8192 tokens of 32 + 2 x 8 heads of 128
// dims, a quarter of them text, interleaved axes: 32.4 us, 6.35 TB/s of the bytes that
// one axis needs; 16 scalar loads in every thread instead cost 3.2 us more).
template <int D, int STYLE, int IPT, int POL>
__global__ void __launch_bounds__(256) mrope_kernel(const __grid_constant__ WriteArgs a)
{
    constexpr int kItemsPerHead = D / 16;
    const int tok = blockIdx.x / a.ctasPerToken;
    const int part = blockIdx.x - tok * a.ctasPerToken;
    const int i = threadIdx.x % kItemsPerHead;
    const int item0 = part * blockDim.x * IPT + threadIdx.x;
    int va, vb;
    item_vectors<D>(i, a.r, va, vb);
    if (POL & kPrefetch)
        prefetch_inputs<D, IPT>(a, tok, item0, va, vb);
    grid_dependency_sync<POL>();
    const L2Policies pol = make_policies<POL>();

    uint4 xa[IPT] = {}, xb[IPT] = {};
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int item = item0 + k * blockDim.x;
        if (item < a.itemsPerToken) {
            const uint16_t* p = head_row(a, tok, item / kItemsPerHead, D);
            xa[k] = load_rw<POL>(p + 8 * va, pol);
            xb[k] = load_rw<POL>(p + 8 * vb, pol);
        }
    }

    int64_t rowOff[kMaxAxes];
    const int64_t pos0 = a.positions[tok];
    bool ok = pos0 >= 0 && pos0 < a.csRows, same = true;
    rowOff[0] = pos0 * a.r;
#pragma unroll
    for (int x = 1; x < kMaxAxes; ++x) {
        rowOff[x] = rowOff[0];
        if (x < a.numAxes) {
            const int64_t p = a.positions[(int64_t)x * a.T + tok];
            ok = ok && p >= 0 && p < a.csRows;
            same = same && p == pos0;
            rowOff[x] = p * a.r;
        }
    }
    const int64_t slot = a.slots[tok];
    if (!ok)
        return;  // no cos/sin row: nothing written for the token
    const bool kvOk = slot >= 0 && slot < a.numSlots;

    float c[8], sn[8];
    const bool rotItem = i < (a.r >> 4);
    if (same) {
        if (rotItem)
            load_cos_sin<STYLE, POL>(a.cosSin + rowOff[0], i, a.r, c, sn, pol);
    } else {
        __shared__ __align__(16) float row[D];
        const int half = a.r >> 1;
        for (int f = threadIdx.x; f < half; f += blockDim.x) {
            const int64_t off = pick(rowOff, (uint32_t)(a.axisBits[f >> 5] >> (2 * (f & 31))) & 3);
            row[f] = __ldg(a.cosSin + off + f);
            row[half + f] = __ldg(a.cosSin + off + half + f);
        }
        __syncthreads();
        if (rotItem) {
            // frequencies 8i..8i+7 (NeoX), 4i..4i+3 and r/4 + 4i.. (GPT-J)
            const int f0 = STYLE == kNeox ? 8 * i : 4 * i;
            const int f1 = STYLE == kNeox ? 8 * i + 4 : 4 * i + (a.r >> 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = row[f0 + j];
                c[4 + j] = row[f1 + j];
                sn[j] = row[half + f0 + j];
                sn[4 + j] = row[half + f1 + j];
            }
        }
    }

#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int item = item0 + k * blockDim.x;
        if (item >= a.itemsPerToken)
            continue;
        const int head = item / kItemsPerHead;
        if (head >= a.Hq && !kvOk)
            continue;
        uint16_t* dst;
        if (head < a.Hq + a.Hkv) {
            if (rotItem)
                rotate_item<STYLE>(xa[k], xb[k], c, sn);
            if (head < a.Hq) {
                dst = a.qOut + ((size_t)tok * a.Hq + head) * D;
            } else {
                const int hk = head - a.Hq;
                dst = (uint16_t*)a.keyCache + ((size_t)slot * a.Hkv + hk) * D;
                if (a.kOut != nullptr) {
                    uint16_t* ko = a.kOut + ((size_t)tok * a.Hkv + hk) * D;
                    store_v<POL>(ko + 8 * va, xa[k], pol);
                    store_v<POL>(ko + 8 * vb, xb[k], pol);
                }
            }
        } else {
            dst = (uint16_t*)a.valueCache + ((size_t)slot * a.Hkv + (head - a.Hq - a.Hkv)) * D;
        }
        store_v<POL>(dst + 8 * va, xa[k], pol);
        store_v<POL>(dst + 8 * vb, xb[k], pol);
    }
}

// ------------------------------------------------------ 8-bit cache write --

// Heads whose largest magnitude is below this are stored as zeros: M / amax
// must stay finite.
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ uint2 pack8_int8(const float f[8])
{
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)  // |f| <= 127 up to its last bit: rounds into [-127, 127]
            w[h] |= ((uint32_t)__float2int_rn(f[4 * h + j]) & 0xff) << (8 * j);
    }
    return make_uint2(w[0], w[1]);
}

// Rotated K and V quantised as they are written. A head's D/16 items sit in
// D/16 consecutive lanes, so its largest magnitude is an xor-shuffle maximum
// over those lanes; the codes follow from the registers that held the head, so
// K and V cross HBM once as FP16 and once as codes. Magnitudes are compared as
// integers (the bits of non-negative floats order as they do), where an
// infinity or NaN is at least 0x7f800000 and survives the maximum. 8192 tokens of
// 32 + 2 x 8 heads of 128 dims into E4M3: 32.3 us, 5.87 TB/s; 256 tokens 3.0 us.
template <int D, int STYLE, int IPT, int POL, bool INT8>
__global__ void __launch_bounds__(256) quant_write_kernel(const __grid_constant__ WriteArgs a)
{
    constexpr int kItemsPerHead = D / 16;
    constexpr float kMaxCode = INT8 ? 127.0f : 448.0f;
    const int tok = blockIdx.x / a.ctasPerToken;
    const int part = blockIdx.x - tok * a.ctasPerToken;
    const int i = threadIdx.x % kItemsPerHead;
    const int item0 = part * blockDim.x * IPT + threadIdx.x;
    int va, vb;
    item_vectors<D>(i, a.r, va, vb);
    if (POL & kPrefetch)
        prefetch_inputs<D, IPT>(a, tok, item0, va, vb);
    grid_dependency_sync<POL>();
    const L2Policies pol = make_policies<POL>();

    uint4 xa[IPT] = {}, xb[IPT] = {};
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int item = item0 + k * blockDim.x;
        if (item < a.itemsPerToken) {
            const uint16_t* p = head_row(a, tok, item / kItemsPerHead, D);
            xa[k] = load_rw<POL>(p + 8 * va, pol);
            xb[k] = load_rw<POL>(p + 8 * vb, pol);
        }
    }
    const int64_t pos = a.positions[tok];
    const int64_t slot = a.slots[tok];
    if (pos < 0 || pos >= a.csRows)
        return;  // no cos/sin row: nothing written for the token
    const bool kvOk = slot >= 0 && slot < a.numSlots;
    const int64_t block = kvOk ? slot / a.blockSize : 0;
    const int64_t inBlock = slot - block * a.blockSize;

    float c[8], sn[8];
    const bool rotItem = i < (a.r >> 4);
    if (rotItem)
        load_cos_sin<STYLE, POL>(a.cosSin + pos * a.r, i, a.r, c, sn, pol);

#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int item = item0 + k * blockDim.x;
        // a warp's lanes stay together for the shuffles below: heads past the
        // token's last take part with zeros and store nothing
        const int head = item / kItemsPerHead;
        const bool live = item < a.itemsPerToken;
        const bool isQ = head < a.Hq;
        if (isQ) {
            if (rotItem)
                rotate_item<STYLE>(xa[k], xb[k], c, sn);
            uint16_t* dst = a.qOut + ((size_t)tok * a.Hq + head) * D;
            store_v<POL>(dst + 8 * va, xa[k], pol);
            store_v<POL>(dst + 8 * vb, xb[k], pol);
        }
        if (__all_sync(0xffffffffu, isQ || !live))
            continue;
        float fa[8], fb[8];
        unpack8(xa[k], fa);
        unpack8(xb[k], fb);
        const bool isK = head < a.Hq + a.Hkv;
        if (isK && rotItem)
            rotate_item_f32<STYLE>(fa, fb, c, sn);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, max(__float_as_uint(fa[j]) & 0x7fffffffu, __float_as_uint(fb[j]) & 0x7fffffffu));
#pragma unroll
        for (int m = 1; m < kItemsPerHead; m <<= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
        if (isQ || !live || !kvOk)
            continue;
        const float amax = __uint_as_float(top);
        const bool finite = top < 0x7f800000u;
        const bool zero = amax < kTiny;
        const bool coded = finite && !zero;
        const float mul = coded ? __fdiv_rn(kMaxCode, amax) : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            fa[j] = coded ? fa[j] * mul : 0.0f;    // +0: a negative element times 0 would be code 0x80
            fb[j] = coded ? fb[j] * mul : 0.0f;
        }
        const int hk = isK ? head - a.Hq : head - a.Hq - a.Hkv;
        uint8_t* dst = (uint8_t*)(isK ? a.keyCache : a.valueCache) + ((size_t)slot * a.Hkv + hk) * D;
        store_v8<POL>(dst + 8 * va, INT8 ? pack8_int8(fa) : pack8_e4m3(fa), pol);
        store_v8<POL>(dst + 8 * vb, INT8 ? pack8_int8(fb) : pack8_e4m3(fb), pol);
        if (i == 0)
            (isK ? a.keyScales : a.valueScales)[((size_t)block * a.Hkv + hk) * a.blockSize + inBlock] =
                !finite ? __uint_as_float(0x7fc00000u) : zero ? 0.0f : __fdiv_rn(amax, kMaxCode);
    }
}

// --------------------------------------------------------- reading back --

struct ReadArgs {
    const uint8_t* pool;       // [2, numPages, tpp, Hkv, D] in the cache's format
    const float* scales;       // [2, numPages, Hkv, tpp] (8-bit)
    const int32_t* pageTable;  // [B, 2, mpps]
    const int32_t* positions;  // [N]
    const int32_t* seqIds;     // [N]
    uint16_t* kOut;            // [N, Hkv, D]
    uint16_t* vOut;
    int32_t N, B, Hkv, numPages, mpps, tpp;
    int32_t vecsPerRow;        // 16-byte vectors of one plane's row
};

template <int FMT>
__device__ __forceinline__ float2 decode2(uint32_t two)
{
    if (FMT == ROPEKV_CACHE_E4M3) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
        return __half22float2(__half2(h));
    }
    return make_float2((float)(int8_t)(two & 0xff), (float)(int8_t)((two >> 8) & 0xff));
}

// One thread: the same 16-byte vector of a row's K and of its V. Rows of few
// vectors share a CTA. 65521 rows of 8 heads of 128 E4M3 codes: 61.1 us, 6.67 TB/s.
template <int D, int FMT>
__global__ void __launch_bounds__(256) paged_read_kernel(const __grid_constant__ ReadArgs a)
{
    constexpr int kPerVec = FMT == ROPEKV_CACHE_F16 ? 8 : 16;
    grid_dependency_sync<kPdl>();
    const L2Policies pol = make_policies<kStreamHint>();
    const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t t = g / a.vecsPerRow;
    if (t >= a.N)
        return;
    const int vec = (int)(g - t * a.vecsPerRow);
    const int pos = a.positions[t];
    const int seq = a.seqIds[t];
    if (pos < 0 || seq < 0 || seq >= a.B)
        return;
    const int lp = pos / a.tpp;
    if (lp >= a.mpps)
        return;
    const int inPage = pos - lp * a.tpp;
    const int32_t* pt = a.pageTable + (size_t)seq * 2 * a.mpps + lp;
    const int idK = pt[0];
    const int idV = pt[a.mpps];
    const bool ok[2] = {idK >= 0 && idK < a.numPages,
                        idV >= a.numPages && idV - a.numPages < a.numPages};
    const int id[2] = {idK, idV};
    const int elem = vec * kPerVec;  // within the row
    const int head = elem / D;
    const size_t rowElems = (size_t)a.Hkv * D;
    uint4 x[2] = {};
    float sc[2] = {};
#pragma unroll
    for (int p = 0; p < 2; ++p)
        if (ok[p]) {
            x[p] = load_rw<kStreamHint>(reinterpret_cast<const uint16_t*>(
                a.pool + ((size_t)id[p] * a.tpp + inPage) * rowElems * (FMT == ROPEKV_CACHE_F16 ? 2 : 1) +
                16 * (size_t)vec), pol);
            if (FMT != ROPEKV_CACHE_F16)
                sc[p] = a.scales[((size_t)id[p] * a.Hkv + head) * a.tpp + inPage];
        }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (!ok[p])
            continue;
        uint16_t* dst = (p ? a.vOut : a.kOut) + (size_t)t * rowElems + elem;
        if (FMT == ROPEKV_CACHE_F16) {
            store_v<kStreamHint>(dst, x[p], pol);
            continue;
        }
        const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
        uint4 y[2];
        uint32_t* o = reinterpret_cast<uint32_t*>(y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = decode2<FMT>((w[j >> 1] >> (16 * (j & 1))) & 0xffff);
            h2(o[j]) = __floats2half2_rn(f.x * sc[p], f.y * sc[p]);
        }
        store_v<kStreamHint>(dst, y[0], pol);
        store_v<kStreamHint>(dst + 8, y[1], pol);
    }
}

// ------------------------------------------------------------- launching --

bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <typename Args>
int launch(void (*kern)(Args), unsigned grid, int threads, cudaStream_t st, bool pdl, const Args& a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? ROPEKV_OK : ROPEKV_ERR_LAUNCH;
}

// Argument checks of both writes, in the order of rope_write_kv_slot_mapping.
int check_write(const WriteArgs& a, int32_t D, int64_t numBlocks, int32_t style)
{
    if (style != ROPEKV_NEOX && style != ROPEKV_GPTJ)
        return ROPEKV_ERR_STYLE;
    if (D != 64 && D != 128 && D != 256)
        return ROPEKV_ERR_HEAD_DIM;
    if (a.r < 16 || a.r > D || (a.r % 16) != 0)
        return ROPEKV_ERR_ROTARY_DIM;
    if (a.Hq <= 0 || a.Hkv <= 0 || a.Hq % a.Hkv != 0)
        return ROPEKV_ERR_HEADS;
    if (a.T < 0 || a.csRows < 0 || numBlocks < 0 || a.blockSize <= 0 || numBlocks > (1LL << 40) ||
        numBlocks > INT64_MAX / a.blockSize)
        return ROPEKV_ERR_SHAPE;
    if (a.qStride < (int64_t)a.Hq * D || a.kStride < (int64_t)a.Hkv * D ||
        a.vStride < (int64_t)a.Hkv * D || (a.qStride % 8) != 0 || (a.kStride % 8) != 0 ||
        (a.vStride % 8) != 0)
        return ROPEKV_ERR_SHAPE;
    if (((long long)a.Hq + 2LL * a.Hkv) * (D / 16) > (1LL << 30))
        return ROPEKV_ERR_SHAPE;
    return ROPEKV_OK;
}

int check_pointers(const WriteArgs& a, bool scales)
{
    if (!a.cosSin || !a.positions || !a.q || !a.k || !a.v || !a.slots || !a.keyCache ||
        !a.valueCache || !a.qOut || (scales && (!a.keyScales || !a.valueScales)))
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(a.cosSin) || !aligned16(a.positions) || !aligned16(a.q) || !aligned16(a.k) ||
        !aligned16(a.v) || !aligned16(a.slots) || !aligned16(a.keyCache) ||
        !aligned16(a.valueCache) || !aligned16(a.keyScales) || !aligned16(a.valueScales) ||
        !aligned16(a.qOut) || !aligned16(a.kOut))
        return ROPEKV_ERR_MISALIGNED;
    return ROPEKV_OK;
}

// Threads per CTA and CTAs per token: two items per thread, at most `perCta`
// items in a CTA, whole warps.
int shape(WriteArgs& a, int perCta, long long* grid)
{
    a.ctasPerToken = (a.itemsPerToken + perCta - 1) / perCta;
    *grid = (long long)a.T * a.ctasPerToken;
    const int per = (a.itemsPerToken + 2 * a.ctasPerToken - 1) / (2 * a.ctasPerToken);
    return ((per + 31) / 32) * 32;
}

constexpr int kPolWrite = kStreamHint | kTableKeep | kPdl | kPrefetch;

template <int D>
int launch_mrope(const WriteArgs& a, int style, unsigned grid, int threads, cudaStream_t st)
{
    return style == ROPEKV_GPTJ
               ? launch(mrope_kernel<D, kGptj, 2, kPolWrite>, grid, threads, st, true, a)
               : launch(mrope_kernel<D, kNeox, 2, kPolWrite>, grid, threads, st, true, a);
}

template <int D, bool INT8>
int launch_quant(const WriteArgs& a, int style, unsigned grid, int threads, cudaStream_t st)
{
    return style == ROPEKV_GPTJ
               ? launch(quant_write_kernel<D, kGptj, 2, kPolWrite, INT8>, grid, threads, st, true, a)
               : launch(quant_write_kernel<D, kNeox, 2, kPolWrite, INT8>, grid, threads, st, true, a);
}

template <int D>
int launch_read(const ReadArgs& a, int fmt, unsigned grid, cudaStream_t st)
{
    switch (fmt) {
    case ROPEKV_CACHE_F16: return launch(paged_read_kernel<D, ROPEKV_CACHE_F16>, grid, 256, st, true, a);
    case ROPEKV_CACHE_E4M3: return launch(paged_read_kernel<D, ROPEKV_CACHE_E4M3>, grid, 256, st, true, a);
    default: return launch(paged_read_kernel<D, ROPEKV_CACHE_INT8>, grid, 256, st, true, a);
    }
}

}  // namespace

extern "C" {

int rope_write_kv_mrope(const float* cosSin, const int64_t* positions, const int32_t* freqAxis,
                        int32_t numAxes, const uint16_t* q, int64_t qTokenStride,
                        const uint16_t* k, int64_t kTokenStride, const uint16_t* v,
                        int64_t vTokenStride, const int64_t* slotMapping, uint16_t* keyCache,
                        uint16_t* valueCache, uint16_t* qOut, uint16_t* kOut, int32_t numTokens,
                        int32_t numQHeads, int32_t numKVHeads, int32_t headDim, int32_t rotaryDim,
                        int32_t cosSinRows, int64_t numBlocks, int32_t blockSize, int32_t style,
                        void* stream)
{
    WriteArgs a = {cosSin, positions, q, k, v, slotMapping, keyCache, valueCache, nullptr, nullptr,
                   qOut, kOut, qTokenStride, kTokenStride, vTokenStride, 0, numTokens, numQHeads,
                   numKVHeads, rotaryDim, cosSinRows, blockSize, 0, 0, numAxes, {0, 0, 0, 0}};
    int rc = check_write(a, headDim, numBlocks, style);
    if (rc != ROPEKV_OK)
        return rc;
    if (numAxes < 1 || numAxes > kMaxAxes)
        return ROPEKV_ERR_SHAPE;
    if (!freqAxis)
        return ROPEKV_ERR_NULL_POINTER;
    for (int f = 0; f < rotaryDim / 2; ++f) {
        if (freqAxis[f] < 0 || freqAxis[f] >= numAxes)
            return ROPEKV_ERR_SHAPE;
        a.axisBits[f >> 5] |= (uint64_t)freqAxis[f] << (2 * (f & 31));
    }
    if (numTokens == 0)
        return ROPEKV_OK;
    rc = check_pointers(a, false);
    if (rc != ROPEKV_OK)
        return rc;
    a.numSlots = numBlocks * (int64_t)blockSize;
    a.itemsPerToken = (numQHeads + 2 * numKVHeads) * (headDim / 16);
    long long grid = 0;
    // 128 items a CTA: 32.4 us (8192 tokens, three axes) against 32.8 with 192 and 34.5 with 384
    const int threads = shape(a, 128, &grid);
    if (grid > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    cudaStream_t st = (cudaStream_t)stream;
    switch (headDim) {
    case 64: return launch_mrope<64>(a, style, (unsigned)grid, threads, st);
    case 128: return launch_mrope<128>(a, style, (unsigned)grid, threads, st);
    default: return launch_mrope<256>(a, style, (unsigned)grid, threads, st);
    }
}

int rope_write_kv_slot_mapping_quant(const float* cosSin, const int64_t* positions,
                                     const uint16_t* q, int64_t qTokenStride, const uint16_t* k,
                                     int64_t kTokenStride, const uint16_t* v, int64_t vTokenStride,
                                     const int64_t* slotMapping, uint8_t* keyCache8,
                                     uint8_t* valueCache8, float* keyScales, float* valueScales,
                                     uint16_t* qOut, int32_t numTokens, int32_t numQHeads,
                                     int32_t numKVHeads, int32_t headDim, int32_t rotaryDim,
                                     int32_t cosSinRows, int64_t numBlocks, int32_t blockSize,
                                     int32_t cacheFormat, int32_t style, void* stream)
{
    WriteArgs a = {cosSin, positions, q, k, v, slotMapping, keyCache8, valueCache8, keyScales,
                   valueScales, qOut, nullptr, qTokenStride, kTokenStride, vTokenStride, 0,
                   numTokens, numQHeads, numKVHeads, rotaryDim, cosSinRows, blockSize, 0, 0, 1,
                   {0, 0, 0, 0}};
    int rc = check_write(a, headDim, numBlocks, style);
    if (rc != ROPEKV_OK)
        return rc;
    if (cacheFormat != ROPEKV_CACHE_E4M3 && cacheFormat != ROPEKV_CACHE_INT8)
        return ROPEKV_ERR_STYLE;
    if (numTokens == 0)
        return ROPEKV_OK;
    rc = check_pointers(a, true);
    if (rc != ROPEKV_OK)
        return rc;
    a.numSlots = numBlocks * (int64_t)blockSize;
    a.itemsPerToken = (numQHeads + 2 * numKVHeads) * (headDim / 16);
    long long grid = 0;
    // 128 items a CTA: 32.3 us (8192 tokens, E4M3) against 32.9 with 192 and 34.1 with 384
    const int threads = shape(a, 128, &grid);
    if (grid > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    cudaStream_t st = (cudaStream_t)stream;
    const bool int8 = cacheFormat == ROPEKV_CACHE_INT8;
    switch (headDim) {
    case 64:
        return int8 ? launch_quant<64, true>(a, style, (unsigned)grid, threads, st)
                    : launch_quant<64, false>(a, style, (unsigned)grid, threads, st);
    case 128:
        return int8 ? launch_quant<128, true>(a, style, (unsigned)grid, threads, st)
                    : launch_quant<128, false>(a, style, (unsigned)grid, threads, st);
    default:
        return int8 ? launch_quant<256, true>(a, style, (unsigned)grid, threads, st)
                    : launch_quant<256, false>(a, style, (unsigned)grid, threads, st);
    }
}

int paged_kv_read(const void* kvCache, const float* kvScales, const int32_t* pageTable,
                  const int32_t* rowPositions, const int32_t* rowSequences, uint16_t* kOut,
                  uint16_t* vOut, int32_t numRows, int32_t batchSize, int32_t numKVHeads,
                  int32_t headDim, int32_t numPages, int32_t maxPagesPerSeq, int32_t tokensPerPage,
                  int32_t cacheFormat, void* stream)
{
    if (cacheFormat < ROPEKV_CACHE_F16 || cacheFormat > ROPEKV_CACHE_INT8)
        return ROPEKV_ERR_STYLE;
    if (headDim != 64 && headDim != 128 && headDim != 256)
        return ROPEKV_ERR_HEAD_DIM;
    if (numKVHeads <= 0)
        return ROPEKV_ERR_HEADS;
    if (numRows < 0 || batchSize < 0 || numPages < 0 || maxPagesPerSeq < 0 || tokensPerPage <= 0 ||
        2LL * numPages * tokensPerPage > 0x7FFFFFFFLL || (long long)numKVHeads * headDim > (1LL << 30))
        return ROPEKV_ERR_SHAPE;
    if (numRows == 0 || batchSize == 0)
        return ROPEKV_OK;
    const bool f16 = cacheFormat == ROPEKV_CACHE_F16;
    if (!kvCache || !pageTable || !rowPositions || !rowSequences || !kOut || !vOut ||
        (!f16 && !kvScales))
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(kvCache) || !aligned16(kvScales) || !aligned16(pageTable) ||
        !aligned16(rowPositions) || !aligned16(rowSequences) || !aligned16(kOut) ||
        !aligned16(vOut))
        return ROPEKV_ERR_MISALIGNED;
    const int vecs = numKVHeads * headDim / (f16 ? 8 : 16);
    const long long grid = ((long long)numRows * vecs + 255) / 256;
    if (grid > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    const ReadArgs a = {(const uint8_t*)kvCache, kvScales, pageTable, rowPositions, rowSequences,
                        kOut, vOut, numRows, batchSize, numKVHeads, numPages, maxPagesPerSeq,
                        tokensPerPage, vecs};
    cudaStream_t st = (cudaStream_t)stream;
    switch (headDim) {
    case 64: return launch_read<64>(a, cacheFormat, (unsigned)grid, st);
    case 128: return launch_read<128>(a, cacheFormat, (unsigned)grid, st);
    default: return launch_read<256>(a, cacheFormat, (unsigned)grid, st);
    }
}

}  // extern "C"
