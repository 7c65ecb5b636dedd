// ropekv_attention_kernels.cuh -- attention over the paged cache for a batch
// that shares a long prefix (paged_attention_shared_prefix).
//
// With q a query row, t the positions it sees and c = smScale * log2(e),
//   s_t = c * (q . k_t),  m = max s_t,  l = sum 2^(s_t - m),
//   out = sum 2^(s_t - m) v_t / l,      lse = ln 2 * (m + log2 l).
// Any split of the positions can be reduced on its own to (m, l, O) and joined
// later, which is how the parts below meet.
//
// Two parts. The prefix is the same for all sequences, so for one KV head all
// B * S * G query rows (G = Hq / Hkv) multiply the same K and V: each byte of it
// is read once per tile of rows instead of once per sequence. A sequence's own
// tokens are read by its S * G rows alone, which is bound by HBM.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ropekv_serving.h"

namespace ropekv_attn {

constexpr int kF16 = ROPEKV_CACHE_F16, kE4M3 = ROPEKV_CACHE_E4M3, kInt8 = ROPEKV_CACHE_INT8;
constexpr float kLn2 = 0.69314718055994530942f;

// n / d for 0 <= n < 2^31: a multiplication and a shift (multiplier
// ceil(2^p / d), p = 31 + ceil(log2 d): the excess n * (m d - 2^p) stays below 2^p).
struct Divisor {
    uint32_t mul, shift;
    int32_t d;
};

inline Divisor make_divisor(int32_t d)
{
    uint32_t c = 0;
    while ((1LL << c) < d)
        ++c;
    const uint64_t m = ((1ULL << (31 + c)) + (uint64_t)d - 1) / (uint64_t)d;
    return {(uint32_t)m, 31 + c, d};
}

__device__ __forceinline__ int divide(int n, const Divisor& v)
{
    return (int)(((uint64_t)(uint32_t)n * v.mul) >> v.shift);
}

struct Args {
    const uint16_t* q;           // [B, S, Hq, D]
    const uint8_t* pool;         // [2, numPages, tpp, Hkv, D]
    const float* scales;         // [2, numPages, Hkv, tpp] (8-bit)
    const int32_t* prefixTable;  // [2, prefixPages]
    const int32_t* pageTable;    // [B, 2, mpps]
    const int32_t* kvLens;       // [B]
    uint16_t* out;               // [B, S, Hq, D]
    float* lse;                  // [B, S, Hq] or NULL
    // partial results: O divided by its sum, and m + log2(l)
    float* partO;                // [numParts, Hkv, B*S*G, D]  ranges of the prefix (tensor cores)
    float* partL;                // [numParts, Hkv, B*S*G]
    float* segO;                 // [slots, pitch, D]          segments of the streamed tokens
    float* segL;                 // [slots, pitch]
    long long* offsets;          // [units + 1]: first step of each unit, their sum
    float scaleLog2;             // smScale * log2(e)
    int32_t B, S, Hq, Hkv, G, numPages, tpp, mpps, P, prefixPages;
    int32_t rowsPrefix;          // B * S * G
    int32_t numParts;            // prefix partials of the tensor cores
    // streamed units: the prefix (if it is not on the tensor cores), then the sequences
    int32_t prefixUnit;          // 1: unit 0 is the prefix
    int32_t tilesPrefix;         // row tiles of the prefix unit (0 without one)
    int32_t tilesSeq;            // row tiles of a sequence
    int32_t pitch;               // rows of a segment's slot
    int32_t teams;               // CTAs of the stream grid
    int32_t teamSize;            // their warps: KV heads that one CTA reads side by side
    int32_t groups;              // Hkv / teamSize
    Divisor divTpp, divG, divGroups, divS, divTeam;
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16-byte (4-byte) asynchronous copy; zeros where !ok (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// Whole copies of data that is read once, evict-first in L2.
__device__ __forceinline__ uint64_t stream_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void copy16_full(uint32_t dst, const void* src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "l"(policy) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool ok)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}

__device__ __forceinline__ void copy_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

__device__ __forceinline__ void copy_wait_all()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t r[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Transpose of an 8 x 8 tile of 16-bit values held one word per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], const uint32_t b[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The four 8-bit codes of a word as two pairs of FP16 values: bytes (0, 1) and
// (2, 3), or with SWAP bytes (0, 2) and (1, 3). Both formats' codes are exact in
// FP16. INT8: byte ^ 0x80 is code + 128 unsigned; as the low mantissa byte of 1024
// (0x6400) it reads 1024 + 128 + code.
template <int FMT, bool SWAP>
__device__ __forceinline__ void decode_word(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    if (FMT == kE4M3) {
        if (SWAP)
            w = __byte_perm(w, 0, 0x3120);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
        return;
    }
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, SWAP ? 0x4240 : 0x4140);
    const uint32_t b = __byte_perm(w, 0x64646464u, SWAP ? 0x4341 : 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint32_t half2_times(uint32_t x, uint32_t y)
{
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Not 0 if a word of V (two halves, four codes) holds an infinity or NaN.
template <int FMT>
__device__ __forceinline__ uint32_t non_finite(uint32_t w)
{
    if (FMT == kF16)
        return __vcmpeq2(w & 0x7c007c00u, 0x7c007c00u);
    return FMT == kE4M3 ? __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) : 0u;
}

// Shared-memory position of 16-byte chunk `c` of row `r` in a tile of rows of
// CPR chunks: eight consecutive rows of one chunk column fall into eight
// different 16-byte bank groups, as ldmatrix reads them.
template <int CPR>
__device__ __forceinline__ int swizzle(int r, int c)
{
    return (r * CPR + (CPR >= 8 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3)))) * 16;
}

// ---------------------------------------------------------- stream kernel --
//
// Few query rows against a stream of tokens: bound by HBM, so the matrix
// products only have to keep up. They are taken transposed, S^T = K Q^T and
// O^T = V^T P^T: the 16-row side of mma.m16n8k16 then holds tokens (or dims)
// and the 8-column side the rows, so that up to 8 rows (a GQA group) waste
// nothing, at half the accumulators and fragments of the other orientation.
// S^T's accumulator layout has tokens down and rows across; two movmatrix
// transposes per 16 tokens make it the B operand of the second product.
//
// Work. A unit is a sequence's own tokens (or the prefix, when few rows share
// it). A CTA is a team of warps, one for each of a group of KV heads, so that a
// page's rows, which hold all heads, are read in runs longer than one head. An
// item is one row tile and group of heads of a unit, a step 16 tokens of an item
// (steps begin at multiples of 16 positions). All steps of all items form one
// sequence, and every team takes an equal share of it, whatever the lengths:
// lengths are on the device, so each CTA sums them first. A share covers the end
// of an item, whole items, the start of another: its segments. The warps of a team
// walk the same steps but never wait for one another. A warp's ring of cp.async
// stages runs ahead across segment borders, so the loads do not drain between
// items; page ids are fetched a step before the copies that need them. Each
// segment leaves (O / l, m + log2 l) in slots item + team, which no other segment
// has, as the next segment in order has a larger item or a larger team.
//
// m follows the maximum lazily: it moves only when a score exceeds it by more
// than 8 (2^8 stays far inside FP16 and FP32), so most steps need one vote
// instead of the shuffles of a maximum and no rescaling.
//
// 8-bit caches: the codes go into the products as FP16 (exact); a token's K
// scale multiplies its scores, its V scale its weights 2^(s - m). With e_t the
// exponent of token t's V scale, m follows max(s_t + e_t) instead of max(s_t):
// weight times scale stays below 2^9, and the largest near 1, whatever the
// scales; as l and O share m nothing has to be undone at the end.
// The order of dims inside a k-step of the first product is that in which
// ldmatrix delivers bytes (lane j: codes 4j..4j+3); Q's fragments follow it.
//
// What it measured (group of 4 rows, 8 KV heads, D = 128). FP16, 256 sequences of 1 to
// 512 tokens: a call without a prefix (this kernel and the join) 51 us, 5.3 TB/s, against
// 6.78 of a plain copy; on 88 SMs beside a prefix this kernel takes 60 us, 4.5 TB/s, where
// an SM's 8 warps with three stages of 8 KB wait for loads. 8-bit, 128 sequences of 1 to
// 2048: 57 us, 5.0 TB/s: about 450 instructions a step of 4 KB and warp (decoding, the
// transposes and the softmax of 16 tokens for 4 of 8 columns) keep the ALU pipes 55 % and
// the issue slots 51 % busy; neither is a limit, so latency is the rest of it.
constexpr int kMaxParts = 32;    // prefix partials at most

// Exponent of a V scale, kept where 2^(s - m) cannot leave FP32. Up to 2^60, the largest
// finite scale that is supported, weight times scale stays below 2^9 in FP16.
__device__ __forceinline__ float scale_exponent(float scale)
{
    return (float)max(-60, min(60, (int)((__float_as_uint(scale) >> 23) & 0xff) - 127));
}

template <int D, int FMT, int NT>
struct StreamConfig {
    static constexpr int kEsize = FMT == kF16 ? 2 : 1;
    static constexpr int kRowBytes = D * kEsize;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kStages = 3;
    static constexpr int kMeta = 32 * kRowBytes;              // K, V, then 32 scales, meta
    static constexpr int kStageBytes = 32 * kRowBytes + 256;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kRows = 8 * NT;
    // warps of an SM: limited by shared memory and by registers (accumulators)
    static constexpr int kBySmem = 212 * 1024 / kWarpBytes;
    static constexpr int kByRegs = NT * D <= 128 ? 16 : 8;
    static constexpr int kPerSm = kBySmem < kByRegs ? kBySmem : kByRegs;
    static constexpr int smem(int team) { return team * kWarpBytes + (team * 32 + 1) * 8 + team * 8; }
};

// Tokens of unit u: positions [lo, hi).
__device__ __forceinline__ void unit_range(const Args& a, int u, int& lo, int& hi)
{
    if (u < a.prefixUnit) {
        lo = 0;
        hi = a.P;
    } else {
        lo = a.P;
        hi = max(a.P, min(__ldg(a.kvLens + u - a.prefixUnit), a.mpps * a.tpp));
    }
}

__device__ __forceinline__ int unit_steps(int lo, int hi)
{
    return hi > lo ? ((hi + 15) >> 4) - (lo >> 4) : 0;
}

// Steps of a team's share.
__device__ __forceinline__ long long share_of(long long total, int teams)
{
    if (total < (1LL << 31))
        return max(1u, ((uint32_t)total + (uint32_t)teams - 1) / (uint32_t)teams);
    return (total + teams - 1) / teams;
}

template <int D, int FMT, int NT>
__global__ void __launch_bounds__(StreamConfig<D, FMT, NT>::kPerSm * 32, 1)
stream_kernel(const __grid_constant__ Args a)
{
    using C = StreamConfig<D, FMT, NT>;
    constexpr int kRowBytes = C::kRowBytes, kChunks = C::kChunks, kRows = C::kRows;
    constexpr int MT = D / 16, NS = C::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, T = blockDim.x;
    const int units = a.B + a.prefixUnit;

    // ---- shares: sum of all units' steps, then this team's range
    long long* scan = reinterpret_cast<long long*>(smem + a.teamSize * C::kWarpBytes);   // [T + 1] exclusive sums
    long long* warpSum = scan + T + 1;
    const int perThread = (units + T - 1) / T;
    auto weight = [&](int u) -> long long {
        int lo, hi;
        unit_range(a, u, lo, hi);
        return (long long)unit_steps(lo, hi) * ((u < a.prefixUnit ? a.tilesPrefix : a.tilesSeq) * (long long)a.groups);
    };
    const int u0 = min(units, (int)threadIdx.x * perThread), u1 = min(units, u0 + perThread);
    long long mine = 0;
    for (int u = u0; u < u1; ++u)
        mine += weight(u);
    long long sum = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, x);
        if (lane >= x)
            sum += y;
    }
    if (lane == 31)
        warpSum[warp] = sum;
    __syncthreads();
    long long before = 0, total = 0;
    for (int x = 0; x < a.teamSize; ++x) {
        before += x < warp ? warpSum[x] : 0;
        total += warpSum[x];
    }
    scan[threadIdx.x] = before + sum - mine;
    const long long share = share_of(total, a.teams);
    if (blockIdx.x == 0) {
        long long at = before + sum - mine;
        for (int u = u0; u < u1; ++u) {
            a.offsets[u] = at;
            at += weight(u);
        }
        if (threadIdx.x == 0)
            a.offsets[units] = total;
    }
    __syncthreads();

    const long long begin = blockIdx.x * share;
    const long long count = max(0LL, min(total - begin, share));

    uint8_t* ring = smem + warp * C::kWarpBytes;
    const uint32_t ringAddr = smem_u32(ring);
    const size_t rowStride = (size_t)a.Hkv * kRowBytes;
    const bool pagesAligned = a.tpp % 16 == 0;
    const uint64_t policy = stream_policy();
    // where this lane copies from inside 16 consecutive rows, and to
    const size_t laneSrc = (size_t)(lane / kChunks) * rowStride + (lane % kChunks) * 16;

    // ---- producer: the step to issue next
    int pu = 0, pSub = 0, pStep = 0, pEnd = 0, pFirst = 0, pLo = 0, pHi = 0, pSubs = 1;
    const int32_t* table = nullptr;
    int id = -1, pGroup = 0;
    bool pNew = true;         // first step of a segment
    auto enter_unit = [&]() {
        unit_range(a, pu, pLo, pHi);
        pFirst = pLo >> 4;
        pEnd = pFirst + unit_steps(pLo, pHi);
        pSubs = (pu < a.prefixUnit ? a.tilesPrefix : a.tilesSeq) * a.groups;
        table = pu < a.prefixUnit ? a.prefixTable : a.pageTable + (size_t)(pu - a.prefixUnit) * 2 * a.mpps;
    };
    // page id of this lane's token of the step (lanes 0..15: K plane, 16..31: V plane)
    auto fetch_id = [&]() {
        const int pos = pStep * 16 + (lane & 15);
        const int stride = pu < a.prefixUnit ? a.prefixPages : a.mpps;
        id = pos >= pLo && pos < pHi ? __ldg(table + (size_t)(lane >> 4) * stride + divide(pos, a.divTpp)) : -1;
    };
    auto issue = [&](int stage, bool isLast) {
        const int plane = lane >> 4;
        const int pos = pStep * 16 + (lane & 15);
        const bool mapped = id >= plane * a.numPages && id - plane * a.numPages < a.numPages;
        const uint32_t both = __ballot_sync(0xffffffffu, mapped);
        const uint32_t ok = both & (both >> 16) & 0xffff;
        const int inPage = pos - divide(pos, a.divTpp) * a.tpp;
        const uint32_t row = mapped ? (uint32_t)id * (uint32_t)a.tpp + inPage : 0u;
        const uint32_t base = ringAddr + stage * C::kStageBytes;
        const int pHead = pGroup * a.teamSize + warp;
        const uint8_t* headBase = a.pool + (size_t)pHead * kRowBytes;
        if (pagesAligned && ok == 0xffff) {
            // 16 consecutive rows of one K page and one V page
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint8_t* src = headBase + (size_t)__shfl_sync(0xffffffffu, row, 16 * p) * rowStride + laneSrc;
#pragma unroll
                for (int i = 0; i < kChunks / 2; ++i) {
                    const int r = i * (32 / kChunks) + lane / kChunks;
                    copy16_full(base + p * 16 * kRowBytes + swizzle<kChunks>(r, lane % kChunks), src, policy);
                    src += (32 / kChunks) * rowStride;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                // 32 * kChunks chunks of 16 bytes: rows 0..15 are K, 16..31 V
                const int idx = i * 32 + lane;
                const int r = idx / kChunks, c = idx % kChunks;
                const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                copy16(base + (r >> 4) * 16 * kRowBytes + swizzle<kChunks>(r & 15, c),
                       headBase + (size_t)src * rowStride + c * 16, (ok >> (r & 15)) & 1);
            }
        }
        if (FMT != kF16) {
            const float* s = a.scales + ((size_t)(mapped ? id : 0) * a.Hkv + pHead) * a.tpp + (mapped ? inPage : 0);
            copy4(base + C::kMeta + lane * 4, s, (ok >> (lane & 15)) & 1);
        }
        if (lane == 0)
            *reinterpret_cast<int4*>(ring + stage * C::kStageBytes + C::kMeta + 128) =
                make_int4((int)ok | (pNew ? 1 << 16 : 0) | (isLast ? 1 << 17 : 0), pStep, pu, pSub);
    };
    auto advance = [&]() {
        pNew = false;
        if (++pStep < pEnd)
            return;
        pNew = true;
        ++pSub;
        pGroup = pGroup + 1 == a.groups ? 0 : pGroup + 1;
        if (pSub == pSubs) {
            pSub = 0;
            do {
                if (++pu >= units)
                    return;
                enter_unit();
            } while (pFirst == pEnd);
        }
        pStep = pFirst;
    };
    if (count > 0) {
        int chunk = 0;
        for (int x = 0; x < T; x += 32)
            chunk += __popc(__ballot_sync(0xffffffffu, scan[x + lane] <= begin));
        pu = (chunk - 1) * perThread;
        long long at = scan[chunk - 1];
        for (;; ++pu) {
            const long long n = weight(pu);
            if (at + n > begin)
                break;
            at += n;
        }
        enter_unit();
        const int n = pEnd - pFirst;
        const long long in = begin - at;
        pSub = (int)(in / n);
        pStep = pFirst + (int)(in - (long long)pSub * n);
        pGroup = pSub - divide(pSub, a.divGroups) * a.groups;
        fetch_id();
    }
    long long issued = 0;
    auto feed = [&](int stage) {
        if (issued < count) {
            issue(stage, pStep + 1 == pEnd || issued + 1 == count);
            if (++issued < count) {
                advance();
                fetch_id();
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i)
        feed(i);

    // ---- consumer
    uint32_t qf[NT][MT][2];
    float acc[NT][MT][4];
    float m[NT][2], l[NT][2];
    int last0 = 0, row0 = 0, rowsOfUnit = 0, base0 = 0, head = 0;
    int stage = 0, fill = NS - 1;
    // Last position that row n of the tile sees (-1 for rows that are not there or see nothing)
    auto last_of = [&](int n, bool prefix) {
        if (row0 + n >= rowsOfUnit)
            return -1;
        return prefix ? a.P - 1 : base0 + divide(row0 + n, a.divG);
    };
    for (long long it = 0; it < count; ++it) {
        copy_wait<NS - 2>();
        __syncwarp();
        feed(fill);
        fill = fill + 1 == NS ? 0 : fill + 1;
        const uint32_t kBase = ringAddr + stage * C::kStageBytes;
        const uint32_t vBase = kBase + 16 * kRowBytes;
        uint8_t* stagePtr = ring + stage * C::kStageBytes;
        stage = stage + 1 == NS ? 0 : stage + 1;
        const int4 meta = *reinterpret_cast<const int4*>(stagePtr + C::kMeta + 128);
        const uint32_t ok = meta.x & 0xffff;
        const int pos16 = meta.y * 16;
        const bool prefix = meta.z < a.prefixUnit;

        if (meta.x & (1 << 16)) {
            // a segment begins: its rows, Q as B fragments (column n = lane / 4,
            // k = (lane % 4) * 2 + {0, 1} (+8))
            const int t = divide(meta.w, a.divGroups);
            head = (meta.w - t * a.groups) * a.teamSize + warp;
            row0 = t * kRows;
            rowsOfUnit = prefix ? a.rowsPrefix : a.S * a.G;
            const int b = meta.z - a.prefixUnit;
            base0 = prefix ? 0 : __ldg(a.kvLens + b) - a.S;
            last0 = last_of(0, prefix);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = row0 + nt * 8 + (lane >> 2);
                const int s = divide(r, a.divG), g = r - s * a.G;
                const size_t tok = (prefix ? 0 : (size_t)b * a.S) + s;
                const uint16_t* qr = a.q + (tok * a.Hq + head * a.G + g) * D;
#pragma unroll
                for (int kk = 0; kk < MT; ++kk) {
                    const int d0 = kk * 16 + (FMT == kF16 ? (lane & 3) * 2 : (lane & 3) * 4);
                    const int d1 = d0 + (FMT == kF16 ? 8 : 2);
                    qf[nt][kk][0] = r < rowsOfUnit ? __ldg(reinterpret_cast<const uint32_t*>(qr + d0)) : 0u;
                    qf[nt][kk][1] = r < rowsOfUnit ? __ldg(reinterpret_cast<const uint32_t*>(qr + d1)) : 0u;
                    acc[nt][kk][0] = acc[nt][kk][1] = acc[nt][kk][2] = acc[nt][kk][3] = 0.0f;
                }
                m[nt][0] = m[nt][1] = -INFINITY;
                l[nt][0] = l[nt][1] = 0.0f;
            }
        }

        // S^T: rows are the step's tokens lane / 4 and lane / 4 + 8
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
        if (FMT == kF16) {
#pragma unroll
            for (int kk = 0; kk < MT; ++kk) {
                uint32_t k4[4];
                ldmatrix4(k4, kBase + swizzle<kChunks>(lane & 15, kk * 2 + (lane >> 4)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816(s[nt], k4, qf[nt][kk]);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < MT; kk += 2) {
                uint32_t x[4];
                ldmatrix4(x, kBase + swizzle<kChunks>(lane & 15, kk + (lane >> 4)));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t k4[4];
                    decode_word<FMT, false>(x[2 * u], k4[0], k4[2]);
                    decode_word<FMT, false>(x[2 * u + 1], k4[1], k4[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(s[nt], k4, qf[nt][kk + u]);
                }
            }
        }

        // scale, mask, running maximum
        const float* sc = reinterpret_cast<const float*>(stagePtr + C::kMeta);
        const int t0 = lane >> 2;
        float ks0 = a.scaleLog2, ks1 = a.scaleLog2, vs0 = 1.0f, vs1 = 1.0f, e0 = 0.0f, e1 = 0.0f;
        if (FMT != kF16) {
            ks0 *= sc[t0];
            ks1 *= sc[t0 + 8];
            vs0 = sc[16 + t0];
            vs1 = sc[16 + t0 + 8];
            e0 = scale_exponent(vs0);
            e1 = scale_exponent(vs1);
        }
        const bool masked = ok != 0xffff || pos16 + 15 > last0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[nt][j] *= ks0;
                s[nt][2 + j] *= ks1;
            }
        }
        if (masked) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int last = last_of(nt * 8 + (lane & 3) * 2 + j, prefix);
                    if (!((ok >> t0) & 1) || pos16 + t0 > last)
                        s[nt][j] = -INFINITY;
                    if (!((ok >> (t0 + 8)) & 1) || pos16 + t0 + 8 > last)
                        s[nt][2 + j] = -INFINITY;
                }
            }
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                grow = grow || fmaxf(s[nt][j] + e0, s[nt][2 + j] + e1) > m[nt][j] + 8.0f;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(s[nt][j] + e0, s[nt][2 + j] + e1);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float top = fmaxf(m[nt][j], x);
                    const float f = m[nt][j] == top ? 1.0f : exp2_fast(m[nt][j] - top);
                    m[nt][j] = top;
                    l[nt][j] *= f;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[nt][mt][j] *= f;
                        acc[nt][mt][2 + j] *= f;
                    }
                }
            }
        }

        // P^T as the B operand (columns: rows of Q; k: the step's 16 tokens)
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float mm = m[nt][j & 1] == -INFINITY ? 0.0f : m[nt][j & 1];
                p[j] = exp2_fast(s[nt][j] - mm);
                l[nt][j & 1] += p[j];
                if (FMT != kF16)
                    p[j] *= j < 2 ? vs0 : vs1;
            }
            if (FMT != kF16 && masked) {  // a token that the row does not see may have any scale
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    p[j] = s[nt][j] == -INFINITY ? 0.0f : p[j];
            }
            pf[nt][0] = transpose8(half2_bits(p[0], p[1]));
            pf[nt][1] = transpose8(half2_bits(p[2], p[3]));
        }

        // Where rows see different tokens a weight of 0 can meet an infinity or
        // NaN in V that another row sees: such values are taken out of the tile
        // and added to the rows that do see them.
        if (FMT != kInt8 && a.S > 1 && !prefix && pos16 + 15 > last0) {
            auto value = [&](int t, int d) -> float {
                const uint8_t* p = stagePtr + 16 * kRowBytes +
                    swizzle<kChunks>(t, d * C::kEsize / 16) + (d * C::kEsize) % 16;
                if (FMT == kF16)
                    return __half2float(*reinterpret_cast<const __half*>(p));
                uint32_t two, other;
                decode_word<FMT, false>(*p, two, other);
                return __half2float(__ushort_as_half((unsigned short)(two & 0xffff)));
            };
            uint32_t bad = 0;
            const uint4* v = reinterpret_cast<const uint4*>(stagePtr + 16 * kRowBytes);
#pragma unroll
            for (int x = 0; x < kChunks / 2; ++x) {
                const uint4 y = v[x * 32 + lane];
                bad |= non_finite<FMT>(y.x) | non_finite<FMT>(y.y) | non_finite<FMT>(y.z) | non_finite<FMT>(y.w);
            }
            if (__any_sync(0xffffffffu, bad != 0)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int d = mt * 16 + (FMT == kF16 ? (lane >> 2) + (j >> 1) * 8
                                                                 : (lane >> 2) * 2 + (j >> 1));
                            const int last = last_of(nt * 8 + (lane & 3) * 2 + (j & 1), prefix);
#pragma unroll 1
                            for (int t = 0; t < 16; ++t) {
                                const float v = value(t, d);
                                if (!(fabsf(v) < INFINITY) && ((ok >> t) & 1) && pos16 + t <= last)
                                    acc[nt][mt][j] += v;
                            }
                        }
                __syncwarp();
                for (int x = lane; x < 16 * D; x += 32) {
                    const int t = x / D, d = x % D;
                    if (!(fabsf(value(t, d)) < INFINITY)) {
                        uint8_t* p = stagePtr + 16 * kRowBytes +
                            swizzle<kChunks>(t, d * C::kEsize / 16) + (d * C::kEsize) % 16;
                        if (FMT == kF16)
                            *reinterpret_cast<uint16_t*>(p) = 0;
                        else
                            *p = 0;
                    }
                }
                __syncwarp();
            }
        }

        // O^T += V^T P^T
        if (FMT == kF16) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t v4[4];
                ldmatrix4_trans(v4, vBase + swizzle<kChunks>((lane & 7) + (lane >> 4) * 8,
                                                             mt * 2 + ((lane >> 3) & 1)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816(acc[nt][mt], v4, pf[nt]);
            }
        } else {
            // transposed as pairs of codes: a lane gets dims 2p, 2p + 1 of two tokens
#pragma unroll
            for (int mt = 0; mt < MT; mt += 2) {
                uint32_t x[4];
                ldmatrix4_trans(x, vBase + swizzle<kChunks>((lane & 7) + ((lane >> 3) & 1) * 8,
                                                            mt + (lane >> 4)));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t v4[4];
                    decode_word<FMT, true>(x[2 * u], v4[0], v4[1]);
                    decode_word<FMT, true>(x[2 * u + 1], v4[2], v4[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(acc[nt][mt + u], v4, pf[nt]);
                }
            }
        }

        if (meta.x & (1 << 17)) {
            // the segment ends: slots item + team
            const long long item = prefix ? meta.w :
                (a.tilesPrefix + (long long)(meta.z - a.prefixUnit) * a.tilesSeq) * a.groups + meta.w;
            const size_t slot = (size_t)((item + blockIdx.x) * a.teamSize + warp) * a.pitch;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = l[nt][j];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    const int n = nt * 8 + (lane & 3) * 2 + j;
                    if (n >= a.pitch)
                        continue;
                    const float inv = x == 0.0f ? 0.0f : 1.0f / x;
                    if (lane < 4)
                        a.segL[slot + n] = x == 0.0f ? -INFINITY : m[nt][j] + log2f(x);
                    float* dst = a.segO + (slot + n) * D;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float y0 = x == 0.0f ? 0.0f : acc[nt][mt][j] * inv;
                        const float y1 = x == 0.0f ? 0.0f : acc[nt][mt][2 + j] * inv;
                        if (FMT == kF16) {
                            dst[mt * 16 + (lane >> 2)] = y0;
                            dst[mt * 16 + (lane >> 2) + 8] = y1;
                        } else {
                            *reinterpret_cast<float2*>(dst + mt * 16 + (lane >> 2) * 2) = make_float2(y0, y1);
                        }
                    }
                }
            }
        }
        __syncwarp();  // the stage may be filled again
    }
    copy_wait<0>();
    // The next grid (the join) may start; this one ends only after the grid before it
    // (the prefix on the tensor cores) has, so that the join finds both complete.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------ join kernel --
//
// Joins the partials of every output row: the prefix's (numParts ranges, or the
// segments of the prefix unit) and the row's own segments, in that order. A group
// of D / 8 threads holds a row; SPLIT: the CTA's groups share one row's partials
// (few rows with many segments each).
//
// Bound by latency: a launch, the steps' sums, the partials. What depends on the
// lengths alone is computed before the wait for the grids before this one, and the
// partials of all kinds form one list, so that the loads of four are in flight together
// (registers for that: with 64 a thread instead of 85 a call took 0.8 us longer). From
// the last CTA before it to its own last: 3 us with few rows, 7 us for 8192 rows of 128
// with three partials each (12 MB).
// A weighted mean of FP16 values, before its rounding to FP16. The weights in O were rounded
// to FP16, those in l were not, so that a mean of values at FP16's limit of 65504 can come
// out by up to 2^-11 above it, where it would round to infinity.
__device__ __forceinline__ float within_half(float x)
{
    return fabsf(x) > 65504.0f && fabsf(x) < 65504.0f * (1.0f + 1.0f / 1024) ? copysignf(65504.0f, x) : x;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(256, 3) join_kernel(const __grid_constant__ Args a, int tileShift)
{
    constexpr int TG = D / 8, kGroups = 256 / TG;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int group = threadIdx.x / TG, d = threadIdx.x % TG * 8;
    const int hv = SPLIT ? (int)blockIdx.x : (int)blockIdx.x * kGroups + group;   // (token, q head)
    const int rows = a.B * a.S * a.Hq;
    if (!SPLIT && hv >= rows)
        return;
    const int tok = hv / a.Hq, hq = hv - tok * a.Hq;
    const int h = divide(hq, a.divG), g = hq - h * a.G;
    const int b = divide(tok, a.divS), s = tok - b * a.S;
    const bool active = __ldg(a.kvLens + b) - (long long)a.S + s >= a.P;
    const int units = a.B + a.prefixUnit, unit = b + a.prefixUnit;
    int lo, hi;
    unit_range(a, unit, lo, hi);
    const int steps = unit_steps(lo, hi);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long offset = a.offsets[unit], total = a.offsets[units];
    const long long share = share_of(total, a.teams);

    float m = -INFINITY, l = 0.0f;
    float o[8] = {};
    int count = 0;      // partials of this row
    if (active) {
        const bool small = total < (1LL << 31);
        const size_t headRow = (size_t)h * a.rowsPrefix + (size_t)tok * a.G + g;
        const size_t partStride = (size_t)a.Hkv * a.rowsPrefix;
        const int grp = divide(h, a.divTeam), member = h - grp * a.teamSize;
        const size_t slotStride = (size_t)a.teamSize * a.pitch;
        // segments of an item: the shares that its n steps, from step `at`, fall into
        auto segments = [&](int n, long long at, int row, long long itemBase, size_t& slot) -> int {
            const int t = row >> tileShift, sub = t * a.groups + grp;
            at += (long long)sub * n;
            const long long w0 = small ? (uint32_t)at / (uint32_t)share : at / share;
            const long long w1 = small ? ((uint32_t)at + n - 1) / (uint32_t)share : (at + n - 1) / share;
            slot = (size_t)((itemBase + sub + w0) * a.teamSize + member) * a.pitch + (row - (t << tileShift));
            return n == 0 ? 0 : (int)(w1 - w0) + 1;
        };
        size_t slotPrefix = 0, slotOwn = 0;
        const int nPrefix = a.prefixUnit ? segments(unit_steps(0, a.P), 0, tok * a.G + g, 0, slotPrefix) : 0;
        const int nOwn = segments(steps, offset, s * a.G + g, (a.tilesPrefix + (long long)b * a.tilesSeq) * a.groups, slotOwn);
        const int n0 = a.numParts + nPrefix;
        count = n0 + nOwn;
        for (int k = SPLIT ? 4 * group : 0; k < count; k += SPLIT ? 4 * kGroups : 4) {
            float x[4];
            float4 v[4][2];
            float top = m;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = k + j;
                const bool part = i < a.numParts;
                const size_t at = part ? i * partStride + headRow
                                : i < n0 ? slotPrefix + (i - a.numParts) * slotStride : slotOwn + (i - n0) * slotStride;
                x[j] = -INFINITY;
                v[j][0] = v[j][1] = make_float4(0, 0, 0, 0);
                if (i < count) {
                    const float* O = (part ? a.partO : a.segO) + at * D + d;
                    x[j] = (part ? a.partL : a.segL)[at];
                    v[j][0] = *reinterpret_cast<const float4*>(O);
                    v[j][1] = *reinterpret_cast<const float4*>(O + 4);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = fmaxf(top, x[j]);
            const float mm = top == -INFINITY ? 0.0f : top;
            const float f = exp2_fast(m - mm);
            m = top;
            l *= f;
#pragma unroll
            for (int y = 0; y < 8; ++y)
                o[y] *= f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2_fast(x[j] - mm);
                const float* y = reinterpret_cast<const float*>(v[j]);
                l += w;
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    o[z] += w * y[z];
            }
        }
    }
    if (SPLIT) {
        __shared__ float sm[kGroups], sl[kGroups];
        __shared__ float so[kGroups][D];
        if (d == 0) {
            sm[group] = m;
            sl[group] = l;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            so[group][d + k] = o[k];
        __syncthreads();
        if (group > 0)
            return;
        const int filled = min(kGroups, (count + 3) / 4);
        for (int k = 1; k < filled; ++k)
            m = fmaxf(m, sm[k]);
        const float mm = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o[k] = 0.0f;
        for (int x = 0; x < filled; ++x) {
            const float w = exp2_fast(sm[x] - mm);
            l += w * sl[x];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] += w * so[x][d + k];
        }
    }
    const bool none = l == 0.0f;
    const float inv = none ? 0.0f : 1.0f / l;
    uint4 y = make_uint4(0, 0, 0, 0);
    if (!none) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o[k] = within_half(o[k] * inv);
        y = make_uint4(half2_bits(o[0], o[1]), half2_bits(o[2], o[3]), half2_bits(o[4], o[5]), half2_bits(o[6], o[7]));
    }
    *reinterpret_cast<uint4*>(a.out + (size_t)hv * D + d) = y;
    if (d == 0 && a.lse != nullptr)
        a.lse[hv] = none ? -INFINITY : kLn2 * (m + log2f(l));
}

}  // namespace ropekv_attn
