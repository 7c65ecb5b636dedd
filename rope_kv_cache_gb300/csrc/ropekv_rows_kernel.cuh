// ropekv_rows_kernel.cuh -- attention of rows of queries over dense keys and values on
// the 5th-generation tensor cores: prompt_attention and tree_attention
// (include/ropekv_sequence.h).
//
// With q a query row, t the keys that it sees and c = smScale * log2(e),
//   s_t = c * (q . k_t),  m = max s_t,  l = sum 2^(s_t - m),
//   out = sum 2^(s_t - m) v_t / l,      lse = ln 2 * (m + log2 l).
//
// The G = Hq / Hkv heads that share a KV head are rows beside one another: row r of a
// tile is token r / G of the tile and head r % G of the group, so that a tile of a few
// tokens still fills the 128 rows of a product and K and V are read once for the group.
// A CTA takes MT such tiles of 128 rows, which walk the same K/V tiles.
//
//   warps 0 .. 4 MT - 1   softmax: a thread owns one row, which is one TMEM lane; S
//                         comes by tcgen05.ld, the weights go back by tcgen05.st over
//                         the columns of S that they were made from
//   warp 4 MT             fetches by TMA: Q once, then a ring of K and V tiles in the
//                         order in which the products want them
//   warp 4 MT + 1         issues all products: S = Q K^T from shared memory, O += P V with
//                         P in TMEM and V as it lies in memory (N-major); V rows behind a
//                         sequence's last key it makes zeros first, whatever they hold (0
//                         times infinity or NaN would not be 0)
//   warp 4 MT + 2         allocates TMEM
//
// With two row tiles one tile's products run while the other's softmax works; with one
// the scores run ahead by kSlots tiles. The products of a CTA are issued by one thread
// and run in that order, so S may be put over weights that an earlier product reads.
//
// m moves only when a row's scores exceed it by more than 8 (2^8 stays far inside FP16
// and FP32), in which case the row's O is rescaled in TMEM; the first tile sets it.
//
// Masked scores become -infinity by selection, whatever they were. A V that is not finite
// and that some rows of a tile see and others do not (a weight of 0 times infinity) shows
// as a row of O that is not finite although its sum is: such a row is computed again
// from the tokens it sees alone.
//
// Every wait on an mbarrier is bounded. One that runs out ends its role's loop and,
// through a flag, those of the others, and the CTA writes NaN.
#pragma once

#include <cuda.h>

#include "ropekv_prefix_kernel.cuh"
#include "ropekv_sequence.h"

namespace ropekv_rows {

using namespace ropekv_attn;

struct RowsArgs {
    const uint16_t* q;         // [T, Hq, D], token stride qStride
    const uint16_t* k;         // key t of head h of sequence b: k + b * kvBatch + h * kvHead + t * kvTok
    const uint16_t* v;
    uint16_t* out;             // [T, Hq, D]
    float* lse;                // [T, Hq] or NULL
    const int32_t* qStarts;    // [B + 1] (prompt)
    const int32_t* kvStarts;
    const int32_t* endLens;    // [B] (tree)
    const int32_t* treeMask;   // [B, S, W] or NULL
    float* partO;              // [parts, T * Hq, D]
    float* partL;              // [parts, T * Hq]
    int64_t qStride, kTok, vTok, kvHead, kvBatch;
    float scaleLog2;
    int32_t T, Tk, B, S, W, cap, Hq;
    int32_t G;                 // heads of a tile (a divisor of Hq / Hkv)
    int32_t heads;             // Hq / G
    int32_t headsPerKv;        // heads / Hkv
    int32_t tokens;            // tokens of a CTA's tiles: 128 MT / G
    int32_t parts, tilesSeq;
    Divisor divG;
};

template <int D, int MT>
struct RowsConfig {
    static constexpr int kTile = D == 256 ? 64 : 128;      // keys of a K/V tile
    static constexpr int kSlots = MT == 2 ? 1 : D == 256 ? 4 : 2;   // of S per row tile
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kQBytes = MT * 128 * D * 2;
    static constexpr int kStages = (216 * 1024 - kQBytes) / kTileBytes > 8 ? 8 : (224 * 1024 - kQBytes) / kTileBytes;
    static constexpr int kSoftmax = MT * 128;
    static constexpr int kThreads = kSoftmax + 128;
    static constexpr int kColO = MT * kSlots * kTile;
    static constexpr int kCols = 512;
    // barriers: full, empty of the stages; S full, P full, O done of the slots (a wait tells
    // only the last two phases of a barrier apart, and O(j - kSlots) is done when S(j) is); O
    // free of the row tiles; Q full, Q free
    static constexpr int kBars = 2 * kStages + 3 * MT * kSlots + MT + 2;
    static constexpr int kOffRing = kQBytes;
    static constexpr int kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr int kSmem = kOffBar + kBars * 8 + 64 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kColO + MT * D <= kCols, "TMEM");
};

// One piece of work: MT row tiles of a sequence and head group, and a range of K/V tiles.
struct Segment {
    int b, head;               // sequence; head group (heads head * G ..)
    int tok0, nq;              // first token of the tiles in the sequence; its tokens
    int qRow;                  // row of its token 0 in q
    int kvRow;                 // its key 0 along the token axis of k and v
    int base;                  // keys before its token 0 (prompt: nk - nq, tree: end - S)
    int nk;                    // its keys
    int j0, j1;                // K/V tiles
    int part;
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];"
                 :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}

// Wait for a copy of the role's own, whatever has failed: nothing may land in shared memory
// after the CTA has ended.
__device__ __forceinline__ void mbar_drain(uint32_t bar, int parity)
{
    for (int i = 0; i < (1 << 20) && !mbar_try(bar, parity); ++i) {
    }
}

// Row `token` of the sequence sees its keys below this, besides what a tree mask hides.
__device__ __forceinline__ int row_limit(const RowsArgs& a, const Segment& s, int token)
{
    return a.treeMask != nullptr ? s.nk : min(s.nk, s.base + token + 1);
}

// Keys that some row of the segment's tiles sees.
__device__ __forceinline__ int tile_limit(const RowsArgs& a, int nq, int base, int nk, int tok0)
{
    return max(0, a.treeMask != nullptr ? nk : min(nk, base + min(tok0 + a.tokens, nq)));
}

// 32 bits: which of the keys t0 .. t0 + 31 the row with this limit and these mask words sees.
__device__ __forceinline__ uint32_t sees32(const RowsArgs& a, const int32_t* words, int base, int limit, int t0)
{
    const int n = limit - t0;
    uint32_t bits = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
    if (words != nullptr && t0 + 32 > base) {
        const int j = t0 - base;           // first new token of the 32
        const int w = j >> 5, sh = j & 31;
        const uint32_t lo = w >= 0 && w < a.W ? (uint32_t)__ldg(words + w) : w < 0 ? 0xffffffffu : 0u;
        const uint32_t hi = w + 1 >= 0 && w + 1 < a.W ? (uint32_t)__ldg(words + w + 1) : 0u;
        bits &= __funnelshift_r(lo, hi, sh);
    }
    return bits;
}

// A row of O / l from the segment's tokens that the row sees, in FP32 throughout.
template <int D>
__device__ __noinline__ void plain_row(const RowsArgs& a, const Segment& s, const uint16_t* q, int token, int end,
                                       float m, float l, float* o)
{
    const int kvHead = s.head / a.headsPerKv;
    const int lo = s.j0 * RowsConfig<D, 1>::kTile, limit = min(row_limit(a, s, token), end);
    const int32_t* words = a.treeMask != nullptr ? a.treeMask + ((size_t)s.b * a.S + token) * a.W : nullptr;
    const uint16_t* kBase = a.k + (size_t)s.b * a.kvBatch + (size_t)kvHead * a.kvHead;
    const uint16_t* vBase = a.v + (size_t)s.b * a.kvBatch + (size_t)kvHead * a.kvHead;
    for (int d = 0; d < D; ++d)
        o[d] = 0.0f;
    for (int t = lo; t < limit; ++t) {
        if (words != nullptr && !(sees32(a, words, s.base, limit, t) & 1))
            continue;
        const uint4* kr = reinterpret_cast<const uint4*>(kBase + (size_t)(s.kvRow + t) * a.kTok);
        const uint4* qr = reinterpret_cast<const uint4*>(q);
        float dot = 0.0f;
#pragma unroll 4
        for (int x = 0; x < D / 8; ++x) {
            uint4 kw = kr[x], qw = qr[x];
            const __half2* kh = reinterpret_cast<const __half2*>(&kw);
            const __half2* qh = reinterpret_cast<const __half2*>(&qw);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float2 f = __half22float2(kh[y]), g = __half22float2(qh[y]);
                dot = fmaf(f.x, g.x, fmaf(f.y, g.y, dot));
            }
        }
        const float p = exp2_fast(dot * a.scaleLog2 - m) / l;
        const uint4* vr = reinterpret_cast<const uint4*>(vBase + (size_t)(s.kvRow + t) * a.vTok);
        for (int x = 0; x < D / 8; ++x) {
            uint4 vw = vr[x];
            const __half2* vh = reinterpret_cast<const __half2*>(&vw);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float2 f = __half22float2(vh[y]);
                o[8 * x + 2 * y] += p * f.x;
                o[8 * x + 2 * y + 1] += p * f.y;
            }
        }
    }
}

// The work of CTA `index`, found by one warp; false where there is none.
template <int D, int MT, bool TREE>
__device__ __forceinline__ bool find_segment(const RowsArgs& a, int index, Segment& s)
{
    constexpr int TN = RowsConfig<D, MT>::kTile;
    const int lane = threadIdx.x & 31;
    s.part = index % a.parts;
    index /= a.parts;
    s.head = index % a.heads;
    int tile = index / a.heads;
    if (TREE) {
        s.b = tile / a.tilesSeq;
        tile -= s.b * a.tilesSeq;
        const int end = a.endLens[s.b];
        s.nq = a.S;
        s.qRow = s.b * a.S;
        s.kvRow = 0;
        s.base = end - a.S;
        s.nk = max(0, min(end, a.cap));
    } else {
        // prefix sums of the sequences' tiles, 32 sequences at a time
        s.b = -1;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int lo = 0, hi = 0;
            if (b < a.B) {
                lo = max(0, min(a.T, a.qStarts[b]));
                hi = max(lo, min(a.T, a.qStarts[b + 1]));
            }
            const int tiles = (hi - lo + a.tokens - 1) / a.tokens;
            int sum = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, d);
                sum += lane >= d ? y : 0;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, tile < sum);
            if (past != 0) {
                const int src = __ffs(past) - 1;
                const int before = __shfl_sync(0xffffffffu, sum - tiles, src);
                s.b = b0 + src;
                s.qRow = __shfl_sync(0xffffffffu, lo, src);
                s.nq = __shfl_sync(0xffffffffu, hi - lo, src);
                // the last tiles, which see most, first
                tile = __shfl_sync(0xffffffffu, tiles, src) - 1 - (tile - before);
                break;
            }
            tile -= __shfl_sync(0xffffffffu, sum, 31);
        }
        if (s.b < 0)
            return false;
        s.kvRow = max(0, min(a.Tk, a.kvStarts[s.b]));
        s.nk = max(0, min(a.Tk, a.kvStarts[s.b + 1]) - s.kvRow);
        s.base = s.nk - s.nq;
    }
    s.tok0 = tile * a.tokens;
    const int tiles = (tile_limit(a, s.nq, s.base, s.nk, s.tok0) + TN - 1) / TN;
    const int per = (tiles + a.parts - 1) / a.parts;
    s.j0 = min(tiles, s.part * per);
    s.j1 = min(tiles, s.j0 + per);
    return true;
}

template <int D, int MT, bool TREE>
__global__ void __launch_bounds__(RowsConfig<D, MT>::kThreads, 1)
rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ CUtensorMap mapQ,
            const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV)
{
    using C = RowsConfig<D, MT>;
    constexpr int TN = C::kTile, NS = C::kStages, SL = C::kSlots, LA = SL;
    extern __shared__ uint8_t smemRaw[];
    __shared__ Segment shared;
    __shared__ int haveWork;
    const uint32_t rawAddr = smem_u32(smemRaw);
    const uint32_t base = (rawAddr + 1023u) & ~1023u;
    uint8_t* smem = smemRaw + (base - rawAddr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kLoad = 4 * MT, kMma = kLoad + 1, kAlloc = kLoad + 2;

    const uint32_t bars = base + C::kOffBar;
    const uint32_t full = bars, empty = full + NS * 8, sFull = empty + NS * 8, pFull = sFull + MT * SL * 8,
                   oDone = pFull + MT * SL * 8, oFree = oDone + MT * SL * 8, qFull = oFree + MT * 8, qFree = qFull + 8;
    volatile int* failed = reinterpret_cast<volatile int*>(smem + C::kOffBar + C::kBars * 8);
    uint32_t* tmemSlot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kBars * 8 + 8);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < MT * SL; ++i) {
            mbar_init(sFull + 8 * i, 1);
            mbar_init(pFull + 8 * i, 128);
            mbar_init(oDone + 8 * i, 1);
        }
        for (int i = 0; i < MT; ++i)
            mbar_init(oFree + 8 * i, 128);
        mbar_init(qFull, 1);
        mbar_init(qFree, 1);
        *failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kAlloc) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmemSlot)), "n"(C::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kLoad) {
        Segment s;
        const bool found = find_segment<D, MT, TREE>(a, blockIdx.x, s);
        if (lane == 0) {
            shared = s;
            haveWork = found;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *tmemSlot;
    const Segment seg = shared;
    const bool work = haveWork != 0;
    const int J = work ? seg.j1 - seg.j0 : 0;
    const int look = min(LA, J);
    // the last tile has V rows behind the sequence's last key
    const bool tail = J > 0 && seg.j1 * TN > seg.nk;

    if (warp == kLoad) {
        // --------------------------------------------------------------- TMA
        bool ok = J > 0;
        int n = 0;                                  // loads of K and V so far
        const int kvHead = seg.head / a.headsPerKv;
        auto load = [&](const CUtensorMap* map, int j) {
            const int st = n % NS;
            ok = ok && (n < NS || mbar_wait_warp(empty + 8 * st, (n / NS - 1) & 1, failed));
            if (ok && elect_one()) {
                mbar_expect(full + 8 * st, C::kTileBytes);
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load(base + C::kOffRing + st * C::kTileBytes + x * (TN * 128), map, x * 64,
                             seg.kvRow + (seg.j0 + j) * TN, kvHead, TREE ? seg.b : 0, full + 8 * st);
            }
            __syncwarp();
            n += ok;
        };
        if (ok && elect_one()) {
            mbar_expect(qFull, (uint32_t)(a.G * a.tokens * D * 2));
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                tma_load(base + x * (MT * 128 * 128), &mapQ, x * 64, 0, seg.qRow + seg.tok0, seg.head, qFull);
        }
        __syncwarp();
        for (int j = 0; ok && j < look; ++j)
            load(&mapK, j);
        for (int j = 0; ok && j < J; ++j) {
            load(&mapV, j);
            if (j + LA < J)
                load(&mapK, j + LA);
        }
        if (J > 0)
            mbar_drain(qFull, 0);
        for (int i = n > NS ? n - NS : 0; i < n; ++i)
            mbar_drain(full + 8 * (i % NS), (i / NS) & 1);
    } else if (warp == kMma) {
        // ---------------------------------------------------------- products
        constexpr uint32_t kindS = mma_desc(TN, false), kindO = mma_desc(D, true);
        bool ok = J > 0 && mbar_wait_warp(qFull, 0, failed);
        int n = 0;
        auto acquire = [&]() -> int {
            const int st = n % NS;
            ok = ok && mbar_wait_warp(full + 8 * st, (n / NS) & 1, failed);
            ++n;
            return st;
        };
        auto scores = [&](int st, int tile, int j) {
            const int slot = tile * SL + j % SL;
            if (ok && elect_one()) {
                tmem_fence_after();
                const uint32_t qd = desc_low(base + tile * (128 * 128), 16);
                const uint32_t kd = desc_low(base + C::kOffRing + st * C::kTileBytes, 16);
                const uint32_t to = tmem + slot * TN;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(to, desc(qd + ((k >> 2) * (MT * 128 * 128) + (k & 3) * 32) / 16),
                           desc(kd + ((k >> 2) * (TN * 128) + (k & 3) * 32) / 16), kindS, k > 0);
                mma_commit(sFull + 8 * slot);
            }
            __syncwarp();
        };
        auto release = [&](int st) {
            if (ok && elect_one())
                mma_commit(empty + 8 * st);
            __syncwarp();
        };
        for (int j = 0; ok && j < look; ++j) {
            const int st = acquire();
            for (int tile = 0; tile < MT; ++tile)
                scores(st, tile, j);
            release(st);
        }
        for (int j = 0; ok && j < J; ++j) {
            const int sv = acquire();
            if (ok && tail && j == J - 1) {
                // V rows behind the sequence's last key become zeros, while its softmax works
                const int keep = seg.nk - (seg.j1 - 1) * TN;     // rows that are keys, 0 < keep < TN
                uint8_t* v = smem + C::kOffRing + sv * C::kTileBytes;
                const int perBlock = (TN - keep) * 8;
                for (int x = lane; x < (D / 64) * perBlock; x += 32) {
                    const int blk = x / perBlock, y = x - blk * perBlock;
                    *reinterpret_cast<uint4*>(v + blk * (TN * 128) + keep * 128 + y * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
            }
            int sk = 0;
            for (int tile = 0; tile < MT; ++tile) {
                const int slot = tile * SL + j % SL;
                ok = ok && mbar_wait_warp(pFull + 8 * slot, (j / SL) & 1, failed);
                if (ok && elect_one()) {
                    tmem_fence_after();
                    const uint32_t vd = desc_low(base + C::kOffRing + sv * C::kTileBytes, TN * 128);
                    const uint32_t to = tmem + C::kColO + tile * D, from = tmem + slot * TN;
#pragma unroll
                    for (int k = 0; k < TN / 16; ++k)
                        mma_ts(to, from + k * 8, desc(vd + k * (2048 / 16)), kindO, j > 0 || k > 0);
                    mma_commit(oDone + 8 * slot);
                }
                __syncwarp();
                if (tile == MT - 1)
                    release(sv);
                if (j + LA < J) {
                    if (tile == 0)
                        sk = acquire();
                    scores(sk, tile, j + LA);
                    if (tile == MT - 1)
                        release(sk);
                }
            }
        }
        // the last products' arrivals
        for (int i = n > NS ? n - NS : 0; i < n; ++i)
            mbar_wait_warp(empty + 8 * (i % NS), (i / NS) & 1, failed);
    } else if (warp < 4 * MT) {
        // ----------------------------------------------------------- softmax
        const int tile = warp >> 2;
        const uint32_t laneBase = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t oAddr = laneBase + C::kColO + tile * D;
        const int row = (int)threadIdx.x;                       // of the CTA's tiles
        const int rowTok = divide(row, a.divG), g = row - rowTok * a.G;
        const bool live = work && rowTok < a.tokens && seg.tok0 + rowTok < seg.nq;
        const int token = live ? seg.tok0 + rowTok : max(0, seg.nq - 1);
        const bool warpLive = __any_sync(0xffffffffu, live);
        const int limit = work ? row_limit(a, seg, token) : 0;
        const int32_t* words = a.treeMask != nullptr && work ? a.treeMask + ((size_t)seg.b * a.S + token) * a.W : nullptr;
        // keys below this are seen by all of the warp's rows
        int allSee = words != nullptr ? min(limit, seg.base) : limit;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            allSee = min(allSee, __shfl_xor_sync(0xffffffffu, allSee, d));
        float M = -INFINITY, l = 0.0f;
        // |c|, kept above 0 so that a masked -infinity stays one (c = 0: all scores are 0)
        const float scale = fmaxf(fabsf(a.scaleLog2), 1e-30f);
        bool ok = true;
        for (int j = 0; j < J; ++j) {
            const int slot = tile * SL + j % SL;
            const uint32_t sAddr = laneBase + slot * TN;
            ok = mbar_wait_warp(sFull + 8 * slot, (j / SL) & 1, failed);
            if (!ok)
                break;
            if (!warpLive) {
                mbar_arrive(pFull + 8 * slot);
                continue;
            }
            tmem_fence_after();
            float s[TN];
#pragma unroll
            for (int k = 0; k < TN / 32; ++k)
                tmem_load32(s + 32 * k, sAddr + 32 * k);
            tmem_wait_load();
#pragma unroll
            for (int k = 0; k < TN / 32; ++k)
                pin32(s + 32 * k);
            if (a.scaleLog2 < 0.0f) {
#pragma unroll
                for (int k = 0; k < TN; ++k)
                    s[k] = -s[k];
            }
            const int t0 = (seg.j0 + j) * TN;
            if (t0 + TN > allSee) {
#pragma unroll
                for (int w = 0; w < TN / 32; ++w) {
                    const uint32_t bits = sees32(a, words, seg.base, limit, t0 + 32 * w);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        s[32 * w + k] = (bits >> k) & 1 ? s[32 * w + k] : -INFINITY;
                }
            }
            float top4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k + 8 <= TN; k += 8)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    top4[x] = fmaxf(fmaxf(top4[x], s[k + 2 * x]), s[k + 2 * x + 1]);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                top4[x] = fmaxf(top4[x], s[TN - 4 + x]);
            float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
            top = top == -INFINITY ? top : top * scale;
            if (__any_sync(0xffffffffu, top > M + 8.0f)) {
                const float next = fmaxf(M, top);
                const float f = M == next ? 1.0f : exp2_fast(M - next);
                M = next;
                l *= f;
                if (j > 0) {
                    // O of this row tile is at rest: its last product has finished
                    ok = mbar_wait_warp(oDone + 8 * (tile * SL + (j - 1) % SL), ((j - 1) / SL) & 1, failed);
                    if (!ok)
                        break;
                    tmem_fence_after();
#pragma unroll 1
                    for (int k = 0; k < D; k += 32) {
                        float o[32];
                        tmem_load32(o, oAddr + k);
                        tmem_wait_load();
                        pin32(o);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] *= f;
                        tmem_store32(oAddr + k, reinterpret_cast<const uint32_t*>(o));
                    }
                    tmem_wait_store();
                }
            }
            const float mm = M == -INFINITY ? 0.0f : M;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < TN; k += 64) {
                uint32_t p[32];
#pragma unroll
                for (int x = 0; x < 64; x += 4) {
                    float v[4];
                    fma2(v[0], v[1], s[k + x], s[k + x + 1], scale, scale, -mm, -mm);
                    fma2(v[2], v[3], s[k + x + 2], s[k + x + 3], scale, scale, -mm, -mm);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        v[y] = exp2_fast(v[y]);
                    add2(sum[0], sum[1], v[0], v[1]);
                    add2(sum[2], sum[3], v[2], v[3]);
                    p[x / 2] = half2_bits(v[0], v[1]);
                    p[x / 2 + 1] = half2_bits(v[2], v[3]);
                }
                tmem_store32(sAddr + k / 2, p);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_store();
            tmem_fence_before();
            mbar_arrive(pFull + 8 * slot);
        }
        if (J > 0 && ok)
            ok = mbar_wait_warp(oDone + 8 * (tile * SL + (J - 1) % SL), ((J - 1) / SL) & 1, failed);
        tmem_fence_after();
        const bool none = J == 0 || l == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l;
        const float bad = *failed ? __int_as_float(0x7fc00000) : 0.0f;
        const int hq = seg.head * a.G + g;
        const size_t at = (size_t)(seg.qRow + token) * a.Hq + hq;       // row of out
        const size_t partAt = (size_t)seg.part * a.T * a.Hq + at;
        bool strange = false;
        if (warpLive) {
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                float again[D];
                if (pass == 1) {
                    if (!__any_sync(0xffffffffu, strange))
                        break;
                    if (strange)
                        plain_row<D>(a, seg, a.q + (size_t)(seg.qRow + token) * a.qStride + (size_t)hq * D, token,
                                     seg.j1 * TN, M, l, again);
                }
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    if (pass == 0) {
                        if (J > 0) {
                            tmem_load32(o, oAddr + k);
                            tmem_wait_load();
                            pin32(o);
                        }
                    } else {
                        for (int x = 0; x < 32; ++x)
                            o[x] = again[k + x];
                    }
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        if (pass == 0)
                            o[x] = none ? bad : o[x] * inv + bad;
                        strange = strange || (pass == 0 && live && !none && !(fabsf(o[x]) < INFINITY) && fabsf(l) < INFINITY && bad == 0.0f);
                    }
                    if (live && (pass == 0 || strange)) {
                        if (a.parts > 1) {
#pragma unroll
                            for (int x = 0; x < 32; x += 4)
                                *reinterpret_cast<float4*>(a.partO + partAt * D + k + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; x += 8) {
                                uint4 y;
                                uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    w[z] = half2_bits(within_half(o[x + 2 * z]), within_half(o[x + 2 * z + 1]));
                                *reinterpret_cast<uint4*>(a.out + at * D + k + x) = y;
                            }
                        }
                    }
                }
            }
            if (live) {
                if (a.parts > 1)
                    a.partL[partAt] = none ? -INFINITY + bad : M + log2f(l) + bad;
                else if (a.lse != nullptr)
                    a.lse[at] = none ? -INFINITY + bad : kLn2 * (M + log2f(l)) + bad;
            }
        }
        tmem_fence_before();
    }
    __syncthreads();
    if (warp == kAlloc) {
        __syncwarp();
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(C::kCols));
    }
}

// Joins the partial results of a row, in the order of its parts. D / 8 threads hold a row.
template <int D>
__global__ void __launch_bounds__(256) rows_join_kernel(const __grid_constant__ RowsArgs a)
{
    constexpr int TG = D / 8;
    const int64_t row = (int64_t)blockIdx.x * (256 / TG) + threadIdx.x / TG;
    const int64_t rows = (int64_t)a.T * a.Hq;
    const int d = threadIdx.x % TG * 8;
    if (row >= rows)
        return;
    float m = -INFINITY, l = 0.0f, o[8] = {};
    for (int p = 0; p < a.parts; ++p)
        m = fmaxf(m, a.partL[p * rows + row]);
    const float mm = m == -INFINITY ? 0.0f : m;
    for (int p = 0; p < a.parts; ++p) {
        const float x = a.partL[p * rows + row];
        if (x == -INFINITY)
            continue;
        const float w = exp2_fast(x - mm);
        l += w;
        const float* y = a.partO + (p * rows + row) * D + d;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o[k] += w * y[k];
    }
    const bool none = l == 0.0f;
    const float inv = none ? 0.0f : 1.0f / l;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = none ? 0u : half2_bits(within_half(o[2 * k] * inv), within_half(o[2 * k + 1] * inv));
    *reinterpret_cast<uint4*>(a.out + row * D + d) = make_uint4(w[0], w[1], w[2], w[3]);
    if (d == 0 && a.lse != nullptr)
        a.lse[row] = none ? -INFINITY : kLn2 * (m + log2f(l));
}

}  // namespace ropekv_rows
