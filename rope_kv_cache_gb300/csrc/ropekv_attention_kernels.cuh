// ropekv_attention_kernels.cuh -- attention over the paged cache for a batch
// that shares a long prefix (paged_attention_shared_prefix).
//
// With q a query row, t the positions it sees and c = smScale * log2(e),
//   s_t = c * (q . k_t),  m = max s_t,  l = sum 2^(s_t - m),
//   out = sum 2^(s_t - m) v_t / l,      lse = ln 2 * (m + log2 l).
// Any split of the positions can be reduced on its own to (m, l, O) and joined
// later: that is how warps, the CTAs of a cluster and the two parts below meet.
//
// Two parts. The prefix is the same for all sequences, so for one KV head all
// B * S * G query rows (G = Hq / Hkv) multiply the same K and V: each byte of it
// is read once per tile of rows instead of once per sequence. A sequence's own
// tokens are read by its S * G rows alone, which is bound by HBM.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ropekv_serving.h"

namespace ropekv_attn {

namespace cg = cooperative_groups;

constexpr int kF16 = ROPEKV_CACHE_F16, kE4M3 = ROPEKV_CACHE_E4M3, kInt8 = ROPEKV_CACHE_INT8;
constexpr float kLn2 = 0.69314718055994530942f;

struct Args {
    const uint16_t* q;           // [B, S, Hq, D]
    const uint8_t* pool;         // [2, numPages, tpp, Hkv, D]
    const float* scales;         // [2, numPages, Hkv, tpp] (8-bit)
    const int32_t* prefixTable;  // [2, prefixPages]
    const int32_t* pageTable;    // [B, 2, mpps]
    const int32_t* kvLens;       // [B]
    uint16_t* out;               // [B, S, Hq, D]
    float* lse;                  // [B, S, Hq] or NULL
    float* partO;                // [numParts, Hkv, B*S*G, D]  prefix partials, each divided by its sum
    float* partL;                // [numParts, Hkv, B*S*G]     m + log2(l) of each
    float scaleLog2;             // smScale * log2(e)
    int32_t B, S, Hq, Hkv, G, numPages, tpp, mpps, P, prefixPages;
    int32_t rowsPrefix;          // B * S * G
    int32_t numParts;            // prefix partials (0: no prefix)
    int32_t tilesPerUnit;        // row tiles of a sequence (own tokens) or of the batch (prefix)
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
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
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

// Two 8-bit codes (bytes `lo` and `hi` of w) as two FP16 values; both formats'
// codes are exact in FP16. INT8: byte ^ 0x80 is code + 128 unsigned; as the low
// mantissa byte of 1024 (0x6400) it reads 1024 + 128 + code.
template <int FMT, int SEL>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w)
{
    if (FMT == kE4M3) {
        const uint32_t two = __byte_perm(w, 0, 0x4400 | SEL);
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffff), __NV_E4M3);
        return (uint32_t)h.x | ((uint32_t)h.y << 16);
    }
    const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u,
                                   0x4040 | (SEL & 0xf) | ((SEL & 0xf0) << 4));
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Shared-memory position of 16-byte chunk `c` of row `r` in a tile of rows of
// CPR chunks: eight consecutive rows of one chunk column fall into eight
// different 16-byte bank groups, as ldmatrix reads them.
template <int CPR>
__device__ __forceinline__ int swizzle(int r, int c)
{
    return (r * CPR + (CPR >= 8 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3)))) * 16;
}

// ------------------------------------------------------------ rows kernel --
//
// Few query rows against a stream of tokens: bound by HBM, so the matrix
// products only have to keep up. They are taken transposed, S^T = K Q^T and
// O^T = V^T P^T: the 16-row side of mma.m16n8k16 then holds tokens (or dims)
// and the 8-column side the rows, so that up to 8 rows (a GQA group) waste
// nothing, at half the accumulators and fragments of the other orientation.
// S^T's accumulator layout has tokens down and rows across; two movmatrix
// transposes per 16 tokens make it the B operand of the second product.
//
// A CTA is a few warps that never meet until the end: each walks its own steps
// of 16 tokens with its own ring of cp.async stages and its own (m, l, O). The
// page ids of a step are fetched one step before its copies are issued. Steps
// begin at multiples of 16 positions. The tokens of one tile are split over the
// CTAs of a cluster (grid x = tile * cluster + rank), and the cluster's warps
// join through distributed shared memory.
//
// m follows the maximum lazily: it moves only when a score exceeds it by more
// than 8 (2^8 stays far inside FP16 and FP32), so most steps need one vote
// instead of the shuffles of a maximum and no rescaling.
//
// 8-bit caches: the codes go into the products as FP16 (exact); a token's K
// scale multiplies its scores, its V scale its weights 2^(s - m). With 2^e the
// largest V scale of a step, m follows max(s) + e instead of max(s): weight times
// scale stays below 2^9 whatever the scales, and as l and O share m nothing has
// to be undone at the end.
// The order of dims inside a k-step of the first product is that in which
// ldmatrix delivers bytes (lane j: codes 4j..4j+3); Q's fragments follow it.
constexpr int kMaxParts = 32;    // prefix partials at most
constexpr int kMaxCluster = 8;

// Exponent of the largest of a step's V scales, kept where 2^(s - m) cannot leave FP32.
__device__ __forceinline__ int scale_exponent(uint32_t bits)
{
    return max(-60, min(40, (int)(bits >> 23) - 127));
}

template <int D, int FMT, int NT>
struct RowsConfig {
    static constexpr int kEsize = FMT == kF16 ? 2 : 1;
    static constexpr int kRowBytes = D * kEsize;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kWarps = kRowBytes > 256 ? 2 : 4;
    static constexpr int kStages = 3;
    static constexpr int kStageBytes = 32 * kRowBytes + 256;  // K, V, 32 scales, mask
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;                      // floats of a partial's row
    // the warps' partials alias the stages; then (m, l) and join weights of every partial
    static constexpr int kPartBytes = kWarps * kRows * kPitch * 4;
    static constexpr int kRing = kWarps * kWarpBytes > kPartBytes ? kWarps * kWarpBytes : kPartBytes;
    static constexpr int kMaxPartials = kWarps * kMaxCluster + kMaxParts;
    static constexpr int kOffMl = kRing;
    static constexpr int kOffAll = kOffMl + kWarps * kRows * 8;
    static constexpr int kOffTotal = kOffAll + kMaxPartials * kRows * 8;
    static constexpr int kSmem = kOffTotal + kRows * 8;
};

template <int D, int FMT, int NT, bool PREFIX>
__global__ void __launch_bounds__(RowsConfig<D, FMT, NT>::kWarps * 32)
rows_kernel(const __grid_constant__ Args a)
{
    using C = RowsConfig<D, FMT, NT>;
    constexpr int kRowBytes = C::kRowBytes, kChunks = C::kChunks, kRows = C::kRows, W = C::kWarps;
    constexpr int MT = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (PREFIX)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tile = blockIdx.x / ranks;
    const int h = tile % a.Hkv;
    const int unitTile = tile / a.Hkv;
    const int unit = unitTile / a.tilesPerUnit;          // sequence (0 for the prefix)
    const int row0 = (unitTile - unit * a.tilesPerUnit) * kRows;
    const int rowsOfUnit = PREFIX ? a.rowsPrefix : a.S * a.G;

    // The token (b * S + s) of row n of the tile, or -1.
    auto token_of = [&](int n) {
        const int r = row0 + n;
        return r < rowsOfUnit ? (PREFIX ? 0 : unit * a.S) + r / a.G : -1;
    };
    // Last position that the row sees; kNoRow for rows that are not there or lie before P.
    constexpr int kNoRow = -2;
    const int tableEnd = max(a.mpps * a.tpp, a.P);
    auto last_of = [&](int n) {
        const int tok = token_of(n);
        if (tok < 0)
            return kNoRow;
        const int b = tok / a.S;
        const long long p = (long long)__ldg(a.kvLens + b) - a.S + (tok - b * a.S);
        return p < a.P ? kNoRow : (int)min(p, (long long)tableEnd - 1);
    };

    const int lo = PREFIX ? 0 : a.P;
    int hi = a.P, last0 = a.P - 1;
    if (!PREFIX) {
        hi = max(lo, last_of(min(kRows, rowsOfUnit - row0) - 1) + 1);
        last0 = last_of(0);       // the rows of the tile see different positions from here on
    }
    const int firstStep = lo >> 4;
    const int steps = hi > lo ? ((hi + 15) >> 4) - firstStep : 0;
    const int perRank = (steps + ranks - 1) / ranks;
    const int stepEnd = firstStep + min(steps, (rank + 1) * perRank);
    const int stepBegin = firstStep + rank * perRank + warp;

    const int32_t* table = PREFIX ? a.prefixTable : a.pageTable + (size_t)unit * 2 * a.mpps;
    const int planeStride = PREFIX ? a.prefixPages : a.mpps;
    const uint8_t* headBase = a.pool + (size_t)h * kRowBytes;
    const size_t rowStride = (size_t)a.Hkv * kRowBytes;

    uint8_t* ring = smem + warp * C::kWarpBytes;
    const uint32_t ringAddr = smem_u32(ring);

    // Page id of this lane's token of a step (lanes 0..15: K plane, 16..31: V plane).
    auto fetch_id = [&](int step) {
        const int pos = step * 16 + (lane & 15);
        return step < stepEnd && pos >= lo && pos < hi
                   ? __ldg(table + (size_t)(lane >> 4) * planeStride + pos / a.tpp) : -1;
    };
    auto issue = [&](int step, int stage, int id) {
        if (step >= stepEnd)
            return;
        const int pos = step * 16 + (lane & 15);
        const int plane = lane >> 4;
        const bool mapped = id >= plane * a.numPages && id - plane * a.numPages < a.numPages;
        const uint32_t both = __ballot_sync(0xffffffffu, mapped);
        const uint32_t ok = both & (both >> 16) & 0xffff;
        const int inPage = pos % a.tpp;
        const uint32_t row = mapped ? (uint32_t)id * (uint32_t)a.tpp + inPage : 0u;
        const uint32_t base = ringAddr + stage * C::kStageBytes;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            // 32 * kChunks chunks of 16 bytes: rows 0..15 are K, 16..31 V
            const int idx = i * 32 + lane;
            const int r = idx / kChunks, c = idx % kChunks;
            const uint32_t src = __shfl_sync(0xffffffffu, row, r);
            copy16(base + (r >> 4) * 16 * kRowBytes + swizzle<kChunks>(r & 15, c),
                   headBase + (size_t)src * rowStride + c * 16, (ok >> (r & 15)) & 1);
        }
        if (FMT != kF16) {
            const float* s = a.scales + ((size_t)(mapped ? id : 0) * a.Hkv + h) * a.tpp + (mapped ? inPage : 0);
            copy4(base + 32 * kRowBytes + lane * 4, s, (ok >> (lane & 15)) & 1);
        }
        if (lane == 0)
            *reinterpret_cast<uint32_t*>(ring + stage * C::kStageBytes + 32 * kRowBytes + 128) = ok;
    };

    // ---- ring: kStages - 1 steps in flight, ids one step further ahead
    int id = fetch_id(stepBegin);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
        const int next = fetch_id(stepBegin + W * (i + 1));
        issue(stepBegin + W * i, i, id);
        copy_commit();
        id = next;
    }

    // Q as B fragments: column n = lane / 4, k = (lane % 4) * 2 + {0, 1} (+8).
    uint32_t qf[NT][MT][2];
    int lastCol[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int n = nt * 8 + (lane >> 2);
        const int tok = token_of(n);
        const uint16_t* qr = tok < 0 ? nullptr
            : a.q + ((size_t)tok * a.Hq + h * a.G + (row0 + n) % a.G) * D;
#pragma unroll
        for (int kk = 0; kk < MT; ++kk) {
            const int d0 = kk * 16 + (FMT == kF16 ? (lane & 3) * 2 : (lane & 3) * 4);
            const int d1 = d0 + (FMT == kF16 ? 8 : 2);
            qf[nt][kk][0] = qr ? __ldg(reinterpret_cast<const uint32_t*>(qr + d0)) : 0u;
            qf[nt][kk][1] = qr ? __ldg(reinterpret_cast<const uint32_t*>(qr + d1)) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            lastCol[nt][j] = PREFIX ? a.P - 1 : last_of(nt * 8 + (lane & 3) * 2 + j);
    }

    float acc[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            acc[nt][mt][0] = acc[nt][mt][1] = acc[nt][mt][2] = acc[nt][mt][3] = 0.0f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
    }

    int stage = 0, fill = C::kStages - 1;
    for (int step = stepBegin; step < stepEnd; step += W) {
        copy_wait<C::kStages - 2>();
        __syncwarp();
        {
            const int ahead = step + W * (C::kStages - 1);
            const int next = fetch_id(ahead + W);
            issue(ahead, fill, id);
            copy_commit();
            id = next;
            fill = fill + 1 == C::kStages ? 0 : fill + 1;
        }
        const uint32_t kBase = ringAddr + stage * C::kStageBytes;
        const uint32_t vBase = kBase + 16 * kRowBytes;
        uint8_t* stagePtr = ring + stage * C::kStageBytes;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;

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
                uint32_t w[4];
                ldmatrix4(w, kBase + swizzle<kChunks>(lane & 15, kk + (lane >> 4)));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t k4[4] = {decode_pair<FMT, 0x10>(w[2 * u]), decode_pair<FMT, 0x10>(w[2 * u + 1]),
                                            decode_pair<FMT, 0x32>(w[2 * u]), decode_pair<FMT, 0x32>(w[2 * u + 1])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(s[nt], k4, qf[nt][kk + u]);
                }
            }
        }

        // scale, mask, running maximum
        const uint32_t ok = *reinterpret_cast<const uint32_t*>(stagePtr + 32 * kRowBytes + 128);
        const float* sc = reinterpret_cast<const float*>(stagePtr + 32 * kRowBytes);
        const int t0 = lane >> 2;
        const int pos0 = step * 16 + t0;
        const bool okA = (ok >> t0) & 1, okB = (ok >> (t0 + 8)) & 1;
        float ks0 = a.scaleLog2, ks1 = a.scaleLog2, vs0 = 1.0f, vs1 = 1.0f, e = 0.0f;
        if (FMT != kF16) {
            ks0 *= sc[t0];
            ks1 *= sc[t0 + 8];
            vs0 = sc[16 + t0];
            vs1 = sc[16 + t0 + 8];
            e = (float)scale_exponent(__reduce_max_sync(
                0xffffffffu, max(__float_as_uint(vs0) & 0x7fffffffu, __float_as_uint(vs1) & 0x7fffffffu)));
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[nt][j] = okA && pos0 <= lastCol[nt][j] ? s[nt][j] * ks0 : -INFINITY;
                s[nt][2 + j] = okB && pos0 + 8 <= lastCol[nt][j] ? s[nt][2 + j] * ks1 : -INFINITY;
                grow = grow || fmaxf(s[nt][j], s[nt][2 + j]) + e > m[nt][j] + 8.0f;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(s[nt][j], s[nt][2 + j]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float top = fmaxf(m[nt][j], x + e);
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
                if (FMT != kF16)  // a token that the row does not see may have any scale
                    p[j] = s[nt][j] == -INFINITY ? 0.0f : p[j] * (j < 2 ? vs0 : vs1);
            }
            pf[nt][0] = transpose8(half2_bits(p[0], p[1]));
            pf[nt][1] = transpose8(half2_bits(p[2], p[3]));
        }

        // Where rows see different tokens a weight of 0 can meet an infinity or
        // NaN in V that another row sees: such values are taken out of the tile
        // and added to the rows that do see them.
        if (!PREFIX && last0 + 1 < hi && step * 16 + 15 > last0) {
            auto value = [&](int t, int d) -> float {
                const uint8_t* p = stagePtr + 16 * kRowBytes +
                    swizzle<kChunks>(t, d * C::kEsize / 16) + (d * C::kEsize) % 16;
                if (FMT == kF16)
                    return __half2float(*reinterpret_cast<const __half*>(p));
                const uint32_t two = decode_pair<FMT, 0x10>(*p);
                return __half2float(__ushort_as_half((unsigned short)(two & 0xffff)));
            };
            bool bad = false;
            for (int x = lane; x < 16 * D; x += 32)
                bad = bad || !(fabsf(value(x / D, x % D)) < INFINITY);
            if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int d = mt * 16 + (FMT == kF16 ? (lane >> 2) + (j >> 1) * 8
                                                                 : (lane >> 2) * 2 + (j >> 1));
#pragma unroll 1
                            for (int t = 0; t < 16; ++t) {
                                const float v = value(t, d);
                                if (!(fabsf(v) < INFINITY) && ((ok >> t) & 1) &&
                                    step * 16 + t <= lastCol[nt][j & 1])
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
                uint32_t w[4];
                ldmatrix4_trans(w, vBase + swizzle<kChunks>((lane & 7) + ((lane >> 3) & 1) * 8,
                                                            mt + (lane >> 4)));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t v4[4] = {decode_pair<FMT, 0x20>(w[2 * u]), decode_pair<FMT, 0x31>(w[2 * u]),
                                            decode_pair<FMT, 0x20>(w[2 * u + 1]), decode_pair<FMT, 0x31>(w[2 * u + 1])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(acc[nt][mt + u], v4, pf[nt]);
                }
            }
        }
        __syncwarp();  // the stage may be filled again
    }
    copy_wait<0>();

    // ---- join: warps and ranks through (distributed) shared memory
    __syncthreads();  // every warp is done with its ring, which the partials reuse
    float* part = reinterpret_cast<float*>(smem);                           // [W][kRows][kPitch]
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);               // [W][kRows]
    float2* all = reinterpret_cast<float2*>(smem + C::kOffAll);             // [partials][kRows]: m, l, then weights
    float2* total = reinterpret_cast<float2*>(smem + C::kOffTotal);         // [kRows]: max, sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float x = l[nt][j];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (lane < 4)
                ml[warp * kRows + nt * 8 + lane * 2 + j] = make_float2(m[nt][j], x);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = nt * 8 + (lane & 3) * 2 + (j & 1);
                const int d = mt * 16 + (FMT == kF16 ? (lane >> 2) + (j >> 1) * 8
                                                     : (lane >> 2) * 2 + (j >> 1));
                part[(warp * kRows + n) * C::kPitch + d] = acc[nt][mt][j];
            }
    }
    if (!PREFIX)  // the prefix partials, and everything before them, are complete
        asm volatile("griddepcontrol.wait;" ::: "memory");
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();

    // Every partial's (m, l) of every row, the prefix's as (m + log2 l, 1)
    const int own = W * ranks, partials = own + (PREFIX ? 0 : a.numParts);
    const size_t headRow = (size_t)h * a.rowsPrefix + (PREFIX ? 0 : (size_t)unit * a.S * a.G) + row0;
    const size_t partStride = (size_t)a.Hkv * a.rowsPrefix;
    const int rowsHere = min(kRows, rowsOfUnit - row0);
    for (int i = threadIdx.x; i < partials * kRows; i += W * 32) {
        const int k = i / kRows, n = i % kRows;
        float2 v = make_float2(-INFINITY, 0.0f);
        if (k < own)
            v = (ranks > 1 ? cluster.map_shared_rank(ml, k / W) : ml)[(k % W) * kRows + n];
        else if (n < rowsHere && last_of(n) != kNoRow)
            v = make_float2(a.partL[(size_t)(k - own) * partStride + headRow + n], 1.0f);
        all[i] = v;
    }
    __syncthreads();
    for (int n = threadIdx.x; n < kRows; n += W * 32) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
        for (int k = 0; k < partials; ++k)
            top = fmaxf(top, all[k * kRows + n].x);
        const float mm = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int k = 0; k < partials; ++k) {
            const float2 v = all[k * kRows + n];
            const float w = exp2_fast(v.x - mm);
            all[k * kRows + n].x = w;
            sum += w * v.y;
        }
        total[n] = make_float2(mm, sum);
    }
    __syncthreads();

    for (int f = rank * W * 32 + (int)threadIdx.x; f < rowsHere * (D / 4); f += ranks * W * 32) {
        const int n = f / (D / 4), d = f % (D / 4) * 4;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto add = [&](float w, const float4& v) {
            o.x += w * v.x; o.y += w * v.y; o.z += w * v.z; o.w += w * v.w;
        };
        for (int k = 0; k < ranks; ++k) {
            const float* p = (ranks > 1 ? cluster.map_shared_rank(part, k) : part) + n * C::kPitch + d;
#pragma unroll
            for (int x = 0; x < W; ++x)
                add(all[(k * W + x) * kRows + n].x, *reinterpret_cast<const float4*>(p + x * kRows * C::kPitch));
        }
        const float2 t = total[n];
        const float inv = t.y == 0.0f ? 0.0f : 1.0f / t.y;
        if (PREFIX) {
            *reinterpret_cast<float4*>(a.partO + (headRow + n) * D + d) =
                t.y == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                            : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (d == 0)
                a.partL[headRow + n] = t.y == 0.0f ? -INFINITY : t.x + log2f(t.y);
        } else {
            if (last_of(n) != kNoRow) {
#pragma unroll 4
                for (int k = 0; k < a.numParts; ++k)
                    add(all[(own + k) * kRows + n].x, *reinterpret_cast<const float4*>(
                            a.partO + (k * partStride + headRow + n) * D + d));
            }
            const size_t y = (size_t)token_of(n) * a.Hq + h * a.G + (row0 + n) % a.G;
            const bool none = t.y == 0.0f;
            *reinterpret_cast<uint2*>(a.out + y * D + d) =
                none ? make_uint2(0, 0) : make_uint2(half2_bits(o.x * inv, o.y * inv), half2_bits(o.z * inv, o.w * inv));
            if (d == 0 && a.lse != nullptr)
                a.lse[y] = none ? -INFINITY : kLn2 * (t.x + log2f(t.y));
        }
    }
    if (ranks > 1)
        cluster.sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace ropekv_attn
