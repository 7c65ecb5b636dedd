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
//                         the columns of S that they were made from, in two halves
//   warp 4 MT             fetches by TMA: Q once, then a ring of K and V tiles in the
//                         order in which the products want them
//   warp 4 MT + 1         issues all products: S = Q K^T from shared memory, O += P V with
//                         P in TMEM and V as it lies in memory (N-major); V rows behind a
//                         sequence's last key it makes zeros first, whatever they hold (0
//                         times infinity or NaN would not be 0)
//   warp 4 MT + 2         allocates TMEM, then cuts the CTA's share into segments
//
// With two row tiles one tile's products run while the other's softmax works; with one
// the scores run ahead by kSlots tiles, or a second CTA of the SM works. The products of a CTA are issued by one thread
// and run in that order, so S may be put over weights that an earlier product reads.
//
// Work. A unit is MT row tiles of one sequence and head group with the K/V tiles that
// they see, its steps. All steps of all units form one sequence, of which every CTA takes an
// equal share whatever the lengths, so that few rows behind long contexts and many short
// prompts fill the SMs alike (lengths are on the device, so each CTA sums them first). A share
// covers the end of a unit, whole units, the start of another: its segments. A whole unit's
// rows go to out; a piece's to a slot of the workspace (O / l, m + log2 l), which no
// other piece has: 2 c for the piece of CTA c that continues a unit, 2 c + 1 for one that
// begins it; the join kernel reads them in order. Between segments nothing drains but
// the softmax warps' own last products: K and V of the next are on their way. What such a
// change costs counts as kSwitch steps at the head of every unit. Short units are not split.
//
// m moves only when a row's scores exceed it by more than 8, in which case the row's O is rescaled in
// TMEM; the first tile sets it. The weights are 2^(s - m + 7): at most 2^15, inside FP16's range, of
// which they use what lies above 1 too. So a weight keeps FP16's 2^-11 down to 2^-21 of the largest and is
// off by 2^-32 of that below (without the 7: 2^-14, 2^-25; 3000 tokens that score 16 nats below a
// first one of small V: out off by 4e-2 to 6e-2, now 1.3e-3 to 1.8e-3). O is held in FP32, l sums the
// weights as they were before the rounding; the 7 leaves with the division.
//
// Masked scores become -infinity by selection, whatever they were. A V that is not finite and whose
// weight is 0, because a row of the tile does not see it or because FP16 does not hold the weight, shows as
// a NaN in a row of O although its sum is finite. Unless a NaN that the row sees is the reason, such an
// element is computed again from the keys that it sees, a row by a warp, in FP32, where weights stay above
// 0: an infinity that a row sees is one in out, whatever its weight. A prompt of 6000 tokens (220 us)
// takes 0.8 ms if all of V is NaN, 8.2 ms with one infinity in the middle (8.5 with a NaN token) and 31 ms
// at the end, where the rows just before it are long (a thread a row, each row in full: 68 to 100 ms).
// Looking for such values in shared memory and taking them out before the product makes that 0.5 to 2 ms, but
// cost prompts of 300 tokens 10 % (68 -> 75 us) when there are none.
//
// Bounds and figures (32 query and 8 KV heads of 128). A step of two row tiles is 2048 cycles of
// products at the tensor cores' rate, 2300 as they come here: both operands of S lie in shared
// memory, 128 bytes a cycle. It takes about 3000: a tile's own chain is the wait for its scores
// (250 cycles), their maximum (400), 128 exponentials a thread (850: a lone warp of a scheduler
// issues one in 6.5 cycles, two warps one in 4.3) and the products behind it (1150), and the
// other tile fills what it can. 12001 tokens: 785 to 830 us, 1.42 to 1.5 PFLOP/s, with the
// power limit reached at 1.65 to 1.75 GHz; with the products alone 672 us, with the softmax
// alone 632. A change of units costs 5000 cycles, half of them the rows on their way out: 24
// sequences of 1 to 1200 tokens, half behind a context, 175 us. One row tile and long contexts
// is bound by loads: 128 decoding sequences of 1 to 4000 tokens 173 us, 6.1 TB/s.
// Tried and slower: two threads a row (815 -> 1049 us: the same exponentials, more barriers),
// warps of their own to take O out (785 -> 847 us: a third stream of instructions), the first
// quarter's exponentials before the maximum is known, exponentials in two stages, scores read in
// halves (no gain), rows exchanged between lanes on their way out (no gain).
//
// Every wait on an mbarrier is bounded. One that runs out ends its role's loop and, through a flag,
// those of the others; what is in flight is waited for, and each softmax thread that has not come to the
// end of the CTA's share writes NaN to its rows in all of it: to out and lse of whole units, and to the
// sums of pieces, from where the join spreads it.
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
    float* partO;              // [2 ctas, D / 4, 128 MT, 4] pieces of units
    float* partL;              // [2 ctas, 128 MT]
    struct Joint* joints;      // [ctas] the unit that CTA c begins and others end
    int64_t qStride, kTok, vTok, kvHead, kvBatch;
    float scaleLog2;
    int32_t T, Tk, B, S, W, cap, Hq;
    int32_t G;                 // heads of a tile (a divisor of Hq / Hkv)
    int32_t heads;             // Hq / G
    int32_t headsPerKv;        // heads / Hkv
    int32_t tokens;            // tokens of a CTA's tiles: 128 MT / G
    int32_t tilesSeq;          // tree: units of a sequence and head group
    int32_t ctas;
    int32_t whole;             // no unit can be long enough to be split: there is nothing to join
    int32_t leastShare;        // steps of a share, at least
    int32_t out32;             // out is a multiple of 32 bytes, not of 16 alone
    int32_t fail;              // as if a wait had run out before the first (tests)
    Divisor divG;
};

struct Joint {
    int qRow, tok0, nq, head;
    int pieces;                // 0: nothing to join
};

// Steps that changing from one unit to the next costs.
constexpr int kSwitch = 3;

// Splitting units costs about so many steps: their pieces are written, read and joined. So
// units are left whole, and each goes to the CTA in whose share it begins, where the longest
// takes no more than that above a share (or, where shares are longer than units, about that at
// all). Whole against split, 32 query and 8 KV heads of 128: one prompt of 512 tokens 15.5
// against 19.5 us, of 1024 21.8 against 25.9, 16 of 500 62.7 against 65.1; 8 of 1000 (not left
// whole) 86.0 against 83.8; 64 decoding sequences of 100 to 200 tokens 27.4 against 29.6; one
// tree of 26 drafts behind 900 tokens (not left whole) 13.5 against 10.7.
template <int MT>
constexpr int kSplit = MT == 2 ? 8 : 4;

// A sequence as the kernel sees it.
struct Sequence {
    int b;
    int nq;                    // its query tokens
    int qRow;                  // row of its token 0 in q
    int kvRow;                 // its key 0 along the token axis of k and v
    int base;                  // keys before its token 0 (prompt: nk - nq, tree: end - S)
    int nk;                    // its keys
    int units;                 // of each head group
};

// MT row tiles of a sequence and head group, and a range of K/V tiles.
struct Segment : Sequence {
    int head;                  // head group: heads head * G ..; below 0: the end
    int tok0;                  // first token of the tiles
    int j0, j1;                // K/V tiles
    int slot;                  // of the workspace; below 0: the whole unit
};

// Where a CTA's share begins.
struct Start {
    long long at, end;         // first step and the one behind the last, of all steps
    long long share;
    long long inside;          // steps of the sequence before `at`
    long long perHead;         // steps of one of its head groups
    Sequence s;
    int found;                 // 0: no work
    int whole;                 // units are not split: each goes to the CTA in whose share it begins
};

constexpr int kSegments = 4;   // that are known ahead

constexpr float kRaise = 7.0f; // binary digits that weights are raised by

template <int D, int MT, int PER>
struct RowsConfig {
    static constexpr int kTile = D == 256 ? 64 : 128;      // keys of a K/V tile
    static constexpr int kPerSm = PER;                     // CTAs of an SM
    static_assert(PER == 1 || (PER == 2 && MT == 1 && D <= 128), "TMEM and shared memory of a half");
    static constexpr int kSlots = MT == 2 || kPerSm == 2 ? 1 : D == 256 ? 4 : 2;   // of S per row tile
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kQBytes = MT * 128 * D * 2;
    static constexpr int kFit = ((kPerSm == 2 ? 108 : 224) * 1024 - kQBytes) / kTileBytes;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSoftmax = MT * 128;
    static constexpr int kThreads = kSoftmax + 128;
    static constexpr int kColO = MT * kSlots * kTile;
    static constexpr int kCols = 512 / kPerSm;
    // barriers: full, empty of the stages; S full, the two halves of P, O done of the slots (a
    // wait tells only the last two phases of a barrier apart, and O(j - kSlots) is done when S(j)
    // is); Q full, Q free; full, free of the segments; all products done, after a failure
    static constexpr int kBars = 2 * kStages + 4 * MT * kSlots + 2 + 2 * kSegments + 1;
    static constexpr int kOffRing = kQBytes;
    static constexpr int kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr int kOffSegs = (kOffBar + kBars * 8 + 15) / 16 * 16;
    static constexpr int kOffStart = kOffSegs + kSegments * (int)sizeof(Segment);
    static constexpr int kOffSums = (kOffStart + (int)sizeof(Start) + 15) / 16 * 16;
    static constexpr int kOffFlags = kOffSums + kThreads / 32 * 16;
    static constexpr int kSmem = kOffFlags + 16;
    static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory");
    static_assert(kColO + MT * D <= kCols, "TMEM");
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

// Wait of at most 2^20 polls, each of which the hardware may suspend for a time of its own choosing (130
// ms were seen to pass within them): a step or two of the others' work. While one of them does what ends by
// itself but takes long (failed[1]: rows are mended, empty sequences passed) they start anew. LONG, for the
// segment warp, which waits for a whole segment: 2^31 polls, minutes, where 2^28 keys take 8 s; if nothing
// comes on, one of the others' waits runs out before and ends this one too. False, for the whole CTA, if it
// runs out. One poll in the code instead of one in front of the loop and one in it: 32 prompts of 300 tokens
// 68 -> 62 us, one of 8000 339 -> 343.
template <bool LONG = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, int parity, volatile int* failed)
{
    bool done = false;
    for (int i = 0; !done && i < (LONG ? 0x7fffffff : 1 << 20); ++i) {
        done = mbar_try(bar, parity);
        if ((i & 255) == 255) {
            if (*failed)
                break;
            if (failed[1])
                i = 0;
        }
    }
    if (!done)
        *failed = 1;
    return __all_sync(0xffffffffu, done);
}

// Wait for copies and products of the role's own, whatever has failed: nothing may land in shared
// memory or TMEM after the CTA has ended.
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
        const uint32_t lo = w >= 0 && w < a.W ? (uint32_t)words[w] : w < 0 ? 0xffffffffu : 0u;
        const uint32_t hi = w + 1 >= 0 && w + 1 < a.W ? (uint32_t)words[w + 1] : 0u;
        bits &= __funnelshift_r(lo, hi, sh);
    }
    return bits;
}

__device__ __forceinline__ void tmem_load16(float* f, uint32_t addr)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(addr),
           "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_load(float* f, uint32_t addr)
{
#pragma unroll
    for (int k = 0; k < N; k += 32)
        tmem_load32(f + k, addr + k);
}

template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* r)
{
    if constexpr (N == 16)
        tmem_store16(addr, r);
    else
        tmem_store8(addr, r);
}

// Ties values to this point, behind a wait: nothing that uses them can be scheduled before it.
template <int N>
__device__ __forceinline__ void pin(float* f)
{
#pragma unroll
    for (int k = 0; k < N; k += 8)
        asm volatile("" : "+f"(f[k]), "+f"(f[k + 1]), "+f"(f[k + 2]), "+f"(f[k + 3]), "+f"(f[k + 4]), "+f"(f[k + 5]),
                          "+f"(f[k + 6]), "+f"(f[k + 7]));
}

// 32 bytes, in one piece if the address is a multiple of that.
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t* r, bool whole)
{
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     :: "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4*>(p + 8) = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

// Halves of a word that are NaN: bits 0 and 1.
__device__ __forceinline__ uint32_t nan2(uint32_t w)
{
    return ((w & 0x7fffu) > 0x7c00u ? 1u : 0u) | ((w >> 16 & 0x7fffu) > 0x7c00u ? 2u : 0u);
}

// A weight that FP32 does not hold, but which is above 0 (so an infinity of such a weight stays one; the
// product with a finite value is nothing beside FP16's least).
__device__ __forceinline__ float above_zero(float w)
{
    return w < 1e-37f ? 1e-37f : w;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const uint16_t* p)
{
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Rows (`mine`, one a lane) of which an element of O / l is not finite although the sum is. Out has
// held infinities as +-65504: it gets them. Then, row by row with the whole warp, a NaN element whose
// column has no NaN in a key of the segment that the row sees is computed again from those keys alone:
// a value that is not finite met a weight of 0, of a key that the row does not see, or of one whose
// weight FP16 does not hold (or that was scaled by 0 when m rose). Weights of the latter are kept above 0
// here, as they are in truth, so that an infinity is one in out whatever its weight.
template <int D, int MT>
__device__ __noinline__ void mend_rows(const RowsArgs& a, const Segment& s, uint32_t oAddr, bool mine, float m, float l)
{
    constexpr int TN = RowsConfig<D, MT, 1>::kTile, kWords = D / 64;
    constexpr int kLanes = D / 8, kKeys = 32 / kLanes;         // a key of K by kLanes lanes, a row of V by all
    constexpr int kBatch = D == 256 ? 16 : 32;                 // rows of V on their way at once
    const int lane = threadIdx.x & 31, row = threadIdx.x;
    const int rowTok = divide(row, a.divG), token = s.tok0 + rowTok;
    const int at = (s.qRow + token) * a.Hq + s.head * a.G + row - rowTok * a.G;
    uint32_t lost[D / 32];                                     // the lane's row: its NaN elements
#pragma unroll
    for (int k = 0; k < D; k += 16) {
        float o[16];
        tmem_load16(o, oAddr + k);
        tmem_wait_load();
        pin<16>(o);
        uint32_t bits = 0;
#pragma unroll
        for (int x = 0; x < 16; x += 2) {
            bits |= (o[x] != o[x] ? 1u : 0u) << x | (o[x + 1] != o[x + 1] ? 2u : 0u) << x;
            if (mine && s.slot < 0)
                *reinterpret_cast<uint32_t*>(a.out + (size_t)at * D + k + x) =
                    half2_bits(within_half(o[x] / l), within_half(o[x + 1] / l));
        }
        lost[k / 32] = k % 32 == 0 ? bits : lost[k / 32] | bits << 16;
    }
    tmem_fence_before();
    __syncwarp();
    const size_t kv = (size_t)s.b * a.kvBatch + (size_t)(s.head / a.headsPerKv) * a.kvHead;
    const uint16_t* kBase = a.k + kv + (size_t)s.kvRow * a.kTok + (lane % kLanes) * 8;
    const uint16_t* vBase = a.v + kv + (size_t)s.kvRow * a.vTok + lane * (2 * kWords);
    const int first = s.j0 * TN, end = min(s.nk, s.j1 * TN);
    // the lane's columns of a row's D bits
    auto columns = [&](const uint32_t (&row)[D / 32]) -> uint32_t {
        uint32_t bits = 0;
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
            bits = w == lane * (2 * kWords) / 32 ? row[w] >> lane * (2 * kWords) % 32 & ((1u << 2 * kWords) - 1) : bits;
        return bits;
    };
    // those with a NaN in one of the keys t0 .. t0 + 31 that are seen
    auto nan_columns = [&](int t0, uint32_t seen) -> uint32_t {
        uint32_t found = 0;
#pragma unroll 1
        for (int y0 = 0; y0 < 32; y0 += kBatch) {
            uint32_t w[kBatch][kWords];
#pragma unroll
            for (int y = 0; y < kBatch; ++y)
                load_words<kWords>(w[y], vBase + (size_t)min(t0 + y0 + y, end - 1) * a.vTok);
#pragma unroll
            for (int y = 0; y < kBatch; ++y)
#pragma unroll
                for (int x = 0; x < kWords; ++x)
                    found |= seen >> (y0 + y) & 1 ? nan2(w[y][x]) << 2 * x : 0u;
        }
        return found;
    };
    // first of the keys that all the rows see, for all of them at once
    const int limitAll = a.treeMask != nullptr ? min(s.nk, s.base) : row_limit(a, s, token);
    const int common = max(first, __reduce_min_sync(0xffffffffu, mine ? min(limitAll, end) : end) & ~31);
    uint32_t any[D / 32], knownAll = 0;
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
        any[w] = __reduce_or_sync(0xffffffffu, mine ? lost[w] : 0u);
    const uint32_t wanted = columns(any);
#pragma unroll 1
    for (int t0 = first; t0 < common && __any_sync(0xffffffffu, wanted & ~knownAll); t0 += 32)
        knownAll |= nan_columns(t0, 0xffffffffu);
#pragma unroll 1
    for (uint32_t left = __ballot_sync(0xffffffffu, mine); left != 0; left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int tok = __shfl_sync(0xffffffffu, token, src), atRow = __shfl_sync(0xffffffffu, at, src);
        const int partRow = __shfl_sync(0xffffffffu, row, src);
        const float mRow = __shfl_sync(0xffffffffu, m, src), lRow = __shfl_sync(0xffffffffu, l, src);
        const int limit = min(row_limit(a, s, tok), end);
        const int32_t* words = a.treeMask != nullptr ? a.treeMask + ((size_t)s.b * a.S + tok) * a.W : nullptr;
        uint32_t rowLost[D / 32], known = knownAll;
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
            rowLost[w] = __shfl_sync(0xffffffffu, lost[w], src);
        const uint32_t bits = columns(rowLost);
#pragma unroll 1
        for (int t0 = common; t0 < limit && __any_sync(0xffffffffu, bits & ~known); t0 += 32)
            known |= nan_columns(t0, sees32(a, words, s.base, limit, t0));
        const uint32_t again = bits & ~known;
        if (!__any_sync(0xffffffffu, again))
            continue;
        float q[8], o[2 * kWords];
        const uint4 qw = *reinterpret_cast<const uint4*>(
            a.q + (size_t)(s.qRow + tok) * a.qStride + (size_t)(atRow % a.Hq) * D + (lane % kLanes) * 8);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float2 f = __half22float2(reinterpret_cast<const __half2*>(&qw)[x]);
            q[2 * x] = f.x, q[2 * x + 1] = f.y;
        }
#pragma unroll
        for (int x = 0; x < 2 * kWords; ++x)
            o[x] = 0.0f;
#pragma unroll 1
        for (int t0 = first; t0 < limit; t0 += 32) {
            const uint32_t seen = sees32(a, words, s.base, limit, t0);
            if (seen == 0)
                continue;
            float score = 0.0f;
#pragma unroll 1
            for (int x0 = 0; x0 < kLanes; x0 += 8) {
                uint4 kw[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    kw[x] = *reinterpret_cast<const uint4*>(
                        kBase + (size_t)min(t0 + (x0 + x) * kKeys + lane / kLanes, end - 1) * a.kTok);
                float dot[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    dot[x] = 0.0f;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float2 f = __half22float2(reinterpret_cast<const __half2*>(kw + x)[y]);
                        dot[x] = fmaf(f.x, q[2 * y], fmaf(f.y, q[2 * y + 1], dot[x]));
                    }
                }
#pragma unroll
                for (int y = 1; y < kLanes; y *= 2)
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        dot[x] += __shfl_xor_sync(0xffffffffu, dot[x], y);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float d = __shfl_sync(0xffffffffu, dot[x], lane % kKeys * kLanes);
                    score = lane / kKeys == x0 + x ? d : score;
                }
            }
            const float e = score * a.scaleLog2 - mRow;
            const float p = seen >> lane & 1 && e > -INFINITY ? above_zero(exp2_fast(e) / lRow) : 0.0f;
#pragma unroll 1
            for (int y0 = 0; y0 < 32; y0 += kBatch) {
                uint32_t w[kBatch][kWords];
#pragma unroll
                for (int y = 0; y < kBatch; ++y)
                    load_words<kWords>(w[y], vBase + (size_t)min(t0 + y0 + y, end - 1) * a.vTok);
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                    const float weight = __shfl_sync(0xffffffffu, p, y0 + y);
                    const uint32_t keep = seen >> (y0 + y) & 1 ? 0xffffffffu : 0u;
#pragma unroll
                    for (int x = 0; x < kWords; ++x) {
                        const uint32_t bits = w[y][x] & keep;
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&bits));
                        o[2 * x] = fmaf(weight, f.x, o[2 * x]);
                        o[2 * x + 1] = fmaf(weight, f.y, o[2 * x + 1]);
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2 * kWords; ++x) {
            const int d = lane * (2 * kWords) + x;
            if (again >> x & 1) {
                if (s.slot >= 0)
                    a.partO[(((size_t)s.slot * (D / 4) + d / 4) * (MT * 128) + partRow) * 4 + d % 4] = o[x];
                else
                    a.out[(size_t)atRow * D + d] = (uint16_t)half2_bits(within_half(o[x]), 0.0f);
            }
        }
    }
    __syncwarp();
}

template <bool TREE>
__device__ __forceinline__ Sequence sequence(const RowsArgs& a, int b)
{
    Sequence s;
    s.b = b;
    if (TREE) {
        const int end = a.endLens[b];
        s.nq = a.S;
        s.qRow = b * a.S;
        s.kvRow = 0;
        s.base = end < -(1 << 30) ? -(1 << 30) : end - a.S;
        s.nk = max(0, min(end, a.cap));
        s.units = a.tilesSeq;
    } else {
        s.qRow = max(0, min(a.T, a.qStarts[b]));
        s.nq = max(0, min(a.T, a.qStarts[b + 1]) - s.qRow);
        s.kvRow = max(0, min(a.Tk, a.kvStarts[b]));
        s.nk = max(0, min(a.Tk, a.kvStarts[b + 1]) - s.kvRow);
        s.base = s.nk - s.nq;
        s.units = (s.nq + a.tokens - 1) / a.tokens;
    }
    return s;
}

// K/V tiles that the sequence's unit u sees.
template <int TN>
__device__ __forceinline__ int tiles_of(const RowsArgs& a, const Sequence& s, int u)
{
    return (tile_limit(a, s.nq, s.base, s.nk, u * a.tokens) + TN - 1) / TN;
}

// Sum of floor((a i + b) / m) over 0 <= i < n, all non-negative, by Euclid's steps on (a, m).
template <typename U>
__device__ __forceinline__ long long floor_sum(U n, U m, U a, U b)
{
    long long sum = 0;
    while (n > 0) {
        const U qa = a / m, qb = b / m;
        sum += (long long)((uint64_t)n * (n - 1) / 2 * qa + (uint64_t)n * qb);
        a -= qa * m;
        b -= qb * m;
        const U y = a * n + b;
        n = y / m;
        b = y - n * m;
        const U t = m;
        m = a;
        a = t;
    }
    return sum;
}

// x / y, by 32 bits where they do (a tenth of the time).
__device__ __forceinline__ long long quotient(long long x, long long y)
{
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// Steps of a head group's units before unit u, with their changes; a unit has one at least.
template <int TN, bool TREE>
__device__ __forceinline__ long long steps_before(const RowsArgs& a, const Sequence& s, int u)
{
    if (TREE && a.treeMask != nullptr)
        return (long long)u * (kSwitch + max(1, tiles_of<TN>(a, s, 0)));
    // all but the last unit see base + (i + 1) tokens keys (at most nk of a tree's): one step as
    // long as that is at most TN, then its quotient rounded up
    if (u <= 0)
        return 0;
    const int last = s.units - 1, n = min(u, last);
    long long sum = (long long)u * kSwitch + (u > last ? max(1, tiles_of<TN>(a, s, last)) : 0);
    if (n <= 0)
        return sum;
    const long long first = (long long)s.base + a.tokens + TN - 1;        // floor(first / TN) tiles of unit 0
    int ones = first >= 2 * TN ? 0 : min(n, ((int)(2 * TN - first) + a.tokens - 1) / a.tokens);
    // a tree's units behind the cache's end see nk
    int full = n;
    if (TREE && (long long)s.base + (long long)n * a.tokens > s.nk) {
        full = s.nk <= s.base ? 0 : min(n, (s.nk - s.base) / a.tokens);
        ones = min(ones, full);
        sum += (long long)(n - full) * max(1, (s.nk + TN - 1) / TN);
    }
    const long long from = first + (long long)ones * a.tokens;
    const int rest = full - ones;
    if (rest <= 0)
        return sum + ones;
    if (from + (long long)rest * a.tokens < (1LL << 31))
        return sum + ones + floor_sum<uint32_t>(rest, TN, a.tokens, (uint32_t)from);
    return sum + ones + floor_sum<uint64_t>(rest, TN, a.tokens, from);
}

template <int D, int MT, int PER, bool TREE>
__device__ __forceinline__ void find_start(const RowsArgs& a, long long* sums, Start* out)
{
    constexpr int TN = RowsConfig<D, MT, PER>::kTile, kThreads = RowsConfig<D, MT, PER>::kThreads, kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    Sequence q;
    long long perHead = 0;
    auto work = [&](int b) -> long long {
        q = sequence<TREE>(a, b);
        perHead = steps_before<TN, TREE>(a, q, q.units);
        return a.heads * perHead;
    };
    long long mine = 0;
    int longest = 0;
    for (int b = b0; b < b1; ++b) {
        mine += work(b);
        longest = max(longest, q.units > 0 ? q.nk : 0);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, d);
        sum += lane >= d ? y : 0;
    }
    if (lane == 31) {
        sums[2 * warp] = sum;
        sums[2 * warp + 1] = longest;
    }
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? sums[2 * w] : 0;
        total += sums[2 * w];
        longest = max(longest, (int)sums[2 * w + 1]);
    }
    before += sum - mine;
    const long long share = max((long long)a.leastShare, quotient(total + a.ctas - 1, a.ctas));
    longest = (longest + TN - 1) / TN + kSwitch;
    const int whole = a.whole || longest <= (share >= longest ? 2 : share) + kSplit<MT>;
    const long long at = share * blockIdx.x;
    if (threadIdx.x == 0 && at >= total)
        out->found = 0;
    if (mine > 0 && at >= before && at < before + mine) {
        if (per > 1) {
            int b = b0;
            long long n = work(b);
            while (at >= before + n) {
                before += n;
                n = work(++b);
            }
        }
        *out = {at, min(total, at + share), share, at - before, perHead, q, 1, whole};
    }
}

// The segments of a CTA's share, in order, each given to f. Returns the unit that the share begins
// and others end, if there is one. For a whole warp.
template <int TN, bool TREE, typename F>
__device__ __forceinline__ Joint each_segment(const RowsArgs& a, const Start& start, volatile int* failed, F&& f)
{
    Joint joint = {};
    if (!start.found)
        return joint;
    const int lane = threadIdx.x & 31;
    Segment s;
    long long at = start.at;
    const long long end = start.end, share = start.share;
    static_cast<Sequence&>(s) = start.s;
    s.head = (int)quotient(start.inside, start.perHead);
    long long inside = start.inside - s.head * start.perHead;      // steps of the head group before `at`
    // the unit: the last with no more steps before it, by 32 guesses at a time
    int lo = 0, hi = s.units;
    long long skip = 0;
    while (hi - lo > 1) {
        const int width = (hi - lo + 31) / 32, u = min(hi, lo + lane * width);
        const long long n = steps_before<TN, TREE>(a, s, u);
        const uint32_t fits = __ballot_sync(0xffffffffu, u < hi && n <= inside);
        const int best = 31 - __clz(fits);
        skip = __shfl_sync(0xffffffffu, n, best);
        lo += best * width;
        hi = min(hi, lo + width);
    }
    inside -= skip;
    int unit = lo;
    while (at < end) {
        const int tiles = tiles_of<TN>(a, s, unit), len = kSwitch + max(1, tiles);
        const long long first = at - inside + kSwitch;       // of the unit's real steps, among all
        long long take = min((long long)len - inside, end - at);
        if (start.whole)
            take = len - inside;                             // nothing of a unit that began before
        const int r0 = max(0, (int)inside - kSwitch), r1 = max(0, (int)(inside + take) - kSwitch);
        if (start.whole ? inside == 0 : r1 > r0) {
            s.tok0 = unit * a.tokens;
            s.j0 = min(r0, tiles);
            s.j1 = min(r1, tiles);
            const bool all = r0 == 0 && r1 == len - kSwitch;
            s.slot = all ? -1 : 2 * (int)blockIdx.x + (r0 == 0);
            if (r0 == 0 && !all)
                joint = {s.qRow, s.tok0, s.nq, s.head, (int)(quotient(first + (len - kSwitch) - 1, share) - quotient(first, share)) + 1};
            f(s);
        }
        at += take;
        inside = 0;
        if (++unit == s.units) {
            unit = 0;
            if (++s.head == a.heads) {
                s.head = 0;
                int b = s.b + 1;
                if (at >= end || b == a.B)
                    return joint;
                static_cast<Sequence&>(s) = sequence<TREE>(a, b);
                if (s.units == 0) {
                    if (lane == 0)
                        atomicAdd(const_cast<int*>(failed) + 1, 1);
                    while (s.units == 0 && ++b < a.B)
                        static_cast<Sequence&>(s) = sequence<TREE>(a, b);
                    if (lane == 0)
                        atomicSub(const_cast<int*>(failed) + 1, 1);
                    if (b == a.B)
                        return joint;
                }
            }
        }
    }
    return joint;
}

// A wait has run out: the thread's rows in every segment of the share become NaN, those too that had
// been finished.
template <int D, int MT, int PER, bool TREE>
__device__ __noinline__ void spoil_rows(const RowsArgs& a, const Start& start, volatile int* failed)
{
    const int row = threadIdx.x, rowTok = divide(row, a.divG);
    const float nan = __int_as_float(0x7fc00000);
    each_segment<RowsConfig<D, MT, PER>::kTile, TREE>(a, start, failed, [&](const Segment& s) {
        if (rowTok >= a.tokens || s.tok0 + rowTok >= s.nq)
            return;
        if (s.slot >= 0) {
            a.partL[(size_t)s.slot * (MT * 128) + row] = nan;
            return;
        }
        const int at = (s.qRow + s.tok0 + rowTok) * a.Hq + s.head * a.G + row - rowTok * a.G;
#pragma unroll 1
        for (int d = 0; d < D; d += 8)
            *reinterpret_cast<uint4*>(a.out + (size_t)at * D + d) = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
        if (a.lse != nullptr)
            a.lse[at] = nan;
    });
}

// The softmax warps, which hold kTile scores a thread, take registers of the others: 256 x 208 +
// 128 x 88 are the 384 x 168 of the launch with two row tiles, 128 x 200 + 128 x 56 the 256 x 128
// of one of two CTAs on an SM (200 and 56 spill nothing, 184 and 72 60 words a thread: 200 prompts of 30
// tokens 38 against 45 us).
template <typename C>
__device__ __forceinline__ void few_registers()
{
    if constexpr (C::kThreads == 384)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    else if constexpr (C::kPerSm == 2)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

template <typename C>
__device__ __forceinline__ void more_registers()
{
    if constexpr (C::kThreads == 384)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    else if constexpr (C::kPerSm == 2)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// d = a * b of two values; FP16 of two, infinities and values past its range as +-65504.
__device__ __forceinline__ void mul2(float& d0, float& d1, float b)
{
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1) : "f"(b));
}

__device__ __forceinline__ uint32_t half2_sat(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <int D, int MT, int PER, bool TREE>
__global__ void __launch_bounds__(RowsConfig<D, MT, PER>::kThreads, RowsConfig<D, MT, PER>::kPerSm)
rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ CUtensorMap mapQ,
            const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV)
{
    using C = RowsConfig<D, MT, PER>;
    constexpr int TN = C::kTile, NS = C::kStages, SL = C::kSlots, LA = SL;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    Segment* ring = reinterpret_cast<Segment*>(smem + C::kOffSegs);
    Start& start = *reinterpret_cast<Start*>(smem + C::kOffStart);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kLoad = 4 * MT, kMma = kLoad + 1, kAlloc = kLoad + 2;

    const uint32_t bars = base + C::kOffBar;
    const uint32_t full = bars, empty = full + NS * 8, sFull = empty + NS * 8, pFull = sFull + MT * SL * 8,
                   oDone = pFull + 2 * MT * SL * 8, qFull = oDone + MT * SL * 8, qFree = qFull + 8, segFull = qFree + 8,
                   segFree = segFull + kSegments * 8, drained = segFree + kSegments * 8;
    volatile int* failed = reinterpret_cast<volatile int*>(smem + C::kOffFlags);
    uint32_t* tmemSlot = reinterpret_cast<uint32_t*>(smem + C::kOffFlags + 8);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < MT * SL; ++i) {
            mbar_init(sFull + 8 * i, 1);
            mbar_init(pFull + 16 * i, 4);
            mbar_init(pFull + 16 * i + 8, 4);
            mbar_init(oDone + 8 * i, 1);
        }
        mbar_init(qFull, 1);
        mbar_init(qFree, 1);
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(segFull + 8 * i, 1);
            mbar_init(segFree + 8 * i, 4 * MT + 2);
        }
        mbar_init(drained, 1);
        *failed = (base & 1023) | a.fail;      // tiles of 1024 bytes: 0
        failed[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kLoad && lane < 3) {
        const CUtensorMap* map = lane == 0 ? &mapQ : lane == 1 ? &mapK : &mapV;
        asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // TMEM is taken only now: a CTA that held some while it waits for a grid in front, one of whose own
    // CTAs has yet to take its share on this SM, would wait for ever
    if (warp == kAlloc) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmemSlot)), "n"(C::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    find_start<D, MT, PER, TREE>(a, reinterpret_cast<long long*>(smem + C::kOffSums), &start);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *tmemSlot;
    bool ok = true;
    // The segments, in order, for every warp that works on them; false at the end.
    int segments = 0;
    auto next = [&](Segment& s) -> bool {
        const int i = segments % kSegments;
        if (!wait_warp(segFull + 8 * i, (segments / kSegments) & 1, failed))
            return false;
        s = ring[i];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(segFree + 8 * i);
        ++segments;
        return s.head >= 0;
    };

    if (warp == kLoad) {
        // --------------------------------------------------------------- TMA
        few_registers<C>();
        int n = 0, nq = 0;                          // loads of K and V, of Q so far
        Segment seg;
        while (ok && next(seg)) {
            const int J = seg.j1 - seg.j0, look = min(LA, J), kvHead = seg.head / a.headsPerKv;
            if (J == 0)
                continue;
            auto load = [&](const CUtensorMap* map, int j) {
                const int st = n % NS;
                ok = ok && (n < NS || wait_warp(empty + 8 * st, (n / NS - 1) & 1, failed));
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
            // the scores of the segment before have read its Q
            ok = nq == 0 || wait_warp(qFree, (nq - 1) & 1, failed);
            if (ok && elect_one()) {
                mbar_expect(qFull, (uint32_t)(a.G * a.tokens * D * 2));
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load(base + x * (MT * 128 * 128), &mapQ, x * 64, 0, seg.qRow + seg.tok0, seg.head, qFull);
            }
            __syncwarp();
            nq += ok;
            for (int j = 0; ok && j < look; ++j)
                load(&mapK, j);
            for (int j = 0; ok && j < J; ++j) {
                load(&mapV, j);
                if (j + LA < J)
                    load(&mapK, j + LA);
            }
        }
        if (nq > 0)
            mbar_drain(qFull, (nq - 1) & 1);
        for (int i = n > NS ? n - NS : 0; i < n; ++i)
            mbar_drain(full + 8 * (i % NS), (i / NS) & 1);
    } else if (warp == kMma) {
        // ---------------------------------------------------------- products
        few_registers<C>();
        // a negative smScale: -Q K^T (bit 13 negates A), scaled by |smScale|
        const uint32_t kindS = mma_desc(TN, false) | (a.scaleLog2 < 0.0f ? 1u << 13 : 0u);
        constexpr uint32_t kindO = mma_desc(D, true);
        int n = 0, nq = 0, items = 0;               // loads taken, Q taken, items of a row tile before this segment
        auto acquire = [&]() -> int {
            const int st = n % NS;
            ok = ok && wait_warp(full + 8 * st, (n / NS) & 1, failed);
            ++n;
            return st;
        };
        auto scores = [&](int st, int tile, int item) {
            const int slot = tile * SL + item % SL;
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
        auto commit = [&](uint32_t bar) {
            if (ok && elect_one())
                mma_commit(bar);
            __syncwarp();
        };
        Segment seg;
        while (ok && next(seg)) {
            const int J = seg.j1 - seg.j0, look = min(LA, J);
            if (J == 0)
                continue;
            ok = wait_warp(qFull, nq & 1, failed);
            ++nq;
            for (int j = 0; ok && j < look; ++j) {
                const int st = acquire();
                for (int tile = 0; tile < MT; ++tile)
                    scores(st, tile, items + j);
                commit(empty + 8 * st);
            }
            if (look == J)
                commit(qFree);
            for (int j = 0; ok && j < J; ++j) {
                const int sv = acquire(), item = items + j;
                if (ok && j == J - 1 && seg.j1 * TN > seg.nk) {
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
                    // the weights; with them the rows of the segment before have left O
                    const int slot = tile * SL + item % SL;
                    const uint32_t vd = desc_low(base + C::kOffRing + sv * C::kTileBytes, TN * 128);
                    const uint32_t to = tmem + C::kColO + tile * D, from = tmem + slot * TN;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && wait_warp(pFull + 16 * slot + 8 * h, (item / SL) & 1, failed);
                        if (ok && elect_one()) {
                            tmem_fence_after();
#pragma unroll
                            for (int k = h * TN / 32; k < (h + 1) * TN / 32; ++k)
                                mma_ts(to, from + k * 8, desc(vd + k * (2048 / 16)), kindO, j > 0 || k > 0);
                            if (h == 1)
                                mma_commit(oDone + 8 * slot);
                        }
                        __syncwarp();
                    }
                    if (tile == MT - 1)
                        commit(empty + 8 * sv);
                    if (j + LA < J) {
                        if (tile == 0)
                            sk = acquire();
                        scores(sk, tile, item + LA);
                        if (tile == MT - 1) {
                            commit(empty + 8 * sk);
                            if (j + LA == J - 1)
                                commit(qFree);
                        }
                    }
                }
            }
            items += J;
        }
        // the last products' arrivals
        for (int i = n > NS ? n - NS : 0; ok && i < n; ++i)
            ok = wait_warp(empty + 8 * (i % NS), (i / NS) & 1, failed);
        ok = ok && (nq == 0 || wait_warp(qFree, (nq - 1) & 1, failed));
        if (!ok) {
            if (elect_one())
                mma_commit(drained);
            __syncwarp();
            mbar_drain(drained, 0);
        }
    } else if (warp == kAlloc) {
        // ---------------------------------------------------------- segments
        few_registers<C>();
        ok = a.fail == 0;                           // without segments nothing begins
        int n = 0;
        auto publish = [&](const Segment& s) {
            const int i = n % kSegments;
            ok = ok && (n < kSegments || wait_warp<true>(segFree + 8 * i, (n / kSegments - 1) & 1, failed));
            if (ok && lane == 0) {
                ring[i] = s;
                mbar_arrive(segFull + 8 * i);
            }
            __syncwarp();
            ++n;
        };
        const Joint joint = each_segment<TN, TREE>(a, start, failed, publish);
        Segment s;
        s.head = -1;
        publish(s);
        if (lane == 0 && !a.whole)
            a.joints[blockIdx.x] = joint;
    } else if (warp < 4 * MT) {
        // ----------------------------------------------------------- softmax
        more_registers<C>();
        const int tile = warp >> 2;
        const int row = (int)threadIdx.x;                       // of the CTA's tiles
        const uint32_t laneBase = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t oAddr = laneBase + C::kColO + tile * D;
        const int rowTok = divide(row, a.divG), g = row - rowTok * a.G;
        // |c|, kept above 0 so that a masked -infinity stays one (c = 0: all scores are 0)
        const float scale = fmaxf(fabsf(a.scaleLog2), 1e-30f);
        int items = 0;
        for (; ok; ++segments) {
            const int at4 = segments % kSegments;
            ok = wait_warp(segFull + 8 * at4, (segments / kSegments) & 1, failed);
            const Segment& seg = ring[at4];                     // given back when its rows have left
            if (!ok || seg.head < 0)
                break;
            const int J = seg.j1 - seg.j0;
            const bool live = rowTok < a.tokens && seg.tok0 + rowTok < seg.nq;
            const int token = live ? seg.tok0 + rowTok : seg.nq - 1;
            const bool warpLive = __any_sync(0xffffffffu, live);
            const int limit = row_limit(a, seg, token);
            const int32_t* words = a.treeMask != nullptr ? a.treeMask + ((size_t)seg.b * a.S + token) * a.W : nullptr;
            // keys below this are seen by all of the warp's rows (limits do not fall from row to row)
            const int least = __shfl_sync(0xffffffffu, limit, 0);
            const int allSee = words != nullptr ? min(least, seg.base) : least;
            float M = -INFINITY, l = 0.0f;
            for (int j = 0; ok && j < J; ++j) {
                const int item = items + j, slot = tile * SL + item % SL;
                const uint32_t sAddr = laneBase + slot * TN;
                ok = wait_warp(sFull + 8 * slot, (item / SL) & 1, failed);
                if (!ok)
                    break;
                if (!warpLive) {
                    if (lane == 0) {
                        mbar_arrive(pFull + 16 * slot);
                        mbar_arrive(pFull + 16 * slot + 8);
                    }
                    continue;
                }
                tmem_fence_after();
                float s[TN];
                tmem_load<TN>(s, sAddr);
                tmem_wait_load();
                pin<TN>(s);
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
                        top4[x] = max3(top4[x], s[k + 2 * x], s[k + 2 * x + 1]);
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
                        ok = wait_warp(oDone + 8 * (tile * SL + (item - 1) % SL), ((item - 1) / SL) & 1, failed);
                        if (!ok)
                            break;
                        tmem_fence_after();
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            float o[16];
                            tmem_load16(o, oAddr + k);
                            tmem_wait_load();
                            pin<16>(o);
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                o[x] *= f;
                            tmem_store16(oAddr + k, reinterpret_cast<const uint32_t*>(o));
                        }
                    }
                }
                const float mm = (M == -INFINITY ? 0.0f : M) - kRaise;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < TN; k += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
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
                    tmem_store16(sAddr + k / 2, p);
                    if (k + 32 == TN / 2 || k + 32 == TN) {
                        // this half's products may start
                        tmem_wait_store();
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(pFull + 16 * slot + (k + 32 == TN ? 8 : 0));
                    }
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            if (!ok)
                break;
            items += J;
            if (J > 0)
                ok = wait_warp(oDone + 8 * (tile * SL + (items - 1) % SL), ((items - 1) / SL) & 1, failed);
            if (!ok)
                break;
            if (!warpLive) {
                if (lane == 0)
                    mbar_arrive(segFree + 8 * at4);
                continue;
            }
            tmem_fence_after();
            const bool none = J == 0 || l == 0.0f;
            const float inv = none ? 0.0f : 1.0f / l;
            const int at = (seg.qRow + token) * a.Hq + seg.head * a.G + g;      // row of out
            const int slot = seg.slot;
            const bool plain = __all_sync(0xffffffffu, !none);
            float nan0 = 0.0f, nan1 = 0.0f;                                     // NaN if an element is not finite
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
                float o[32];
                if (J > 0) {
                    tmem_load<32>(o, oAddr + k);
                    tmem_wait_load();
                    pin<32>(o);
                }
                if (!plain) {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        o[x] = none ? 0.0f : o[x];
                }
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    mul2(o[x], o[x + 1], inv);
                    fma2(nan0, nan1, o[x], o[x + 1], 0.0f, 0.0f, nan0, nan1);
                }
                if (slot >= 0) {
                    // in quarters of 16 bytes, each of all rows
                    float4* to = reinterpret_cast<float4*>(a.partO) + ((size_t)slot * (D / 4) + k / 4) * (MT * 128) + row;
                    if (live) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            to[(x / 4) * (MT * 128)] = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    }
                    continue;
                }
                uint32_t c[16];
#pragma unroll
                for (int z = 0; z < 16; ++z)
                    c[z] = half2_sat(o[2 * z], o[2 * z + 1]);
                if (live) {
                    uint16_t* to = a.out + (size_t)at * D + k;
                    store32(to, c, a.out32);
                    store32(to + 16, c + 8, a.out32);
                }
            }
            tmem_fence_before();
            if (live) {
                if (slot >= 0)
                    a.partL[(size_t)slot * (MT * 128) + row] = none ? -INFINITY : (M - kRaise) + log2f(l);
                else if (a.lse != nullptr)
                    a.lse[at] = none ? -INFINITY : kLn2 * ((M - kRaise) + log2f(l));
            }
            const bool strange = live && !none && fabsf(l) < INFINITY && !(nan0 + nan1 == 0.0f);
            if (__any_sync(0xffffffffu, strange)) {
                __syncwarp();
                if (lane == 0)
                    atomicAdd(const_cast<int*>(failed) + 1, 1);
                mend_rows<D, MT>(a, seg, oAddr, strange, M - kRaise, l);
                if (lane == 0)
                    atomicSub(const_cast<int*>(failed) + 1, 1);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(segFree + 8 * at4);
        }
        if (__any_sync(0xffffffffu, !ok || *failed != 0))
            spoil_rows<D, MT, PER, TREE>(a, start, failed);
    } else {
        few_registers<C>();
    }
    // the join may start; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    if (warp == kAlloc) {
        __syncwarp();
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(C::kCols));
    }
}

// Joins the pieces of a unit, in the order of its steps: CTA c's piece, which begins it, then
// those of the CTAs behind. A warp takes 8 rows x 32 dims, a thread 8 dims of a row; four
// pieces' loads are in flight together.
template <int D, int MT>
__global__ void __launch_bounds__(256) rows_join_kernel(const __grid_constant__ RowsArgs a)
{
    constexpr int kChunks = MT * 16 * (D / 32) / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x / kChunks, warp = (blockIdx.x - c * kChunks) * 8 + (threadIdx.x >> 5);
    const Joint joint = a.joints[c];
    const int row = warp / (D / 32) * 8 + (threadIdx.x >> 2 & 7), d = warp % (D / 32) * 32 + (threadIdx.x & 3) * 8;
    const int rowTok = divide(row, a.divG), g = row - rowTok * a.G;
    if (joint.pieces == 0 || rowTok >= a.tokens || joint.tok0 + rowTok >= joint.nq)
        return;
    float m = -INFINITY, l = 0.0f, o[8] = {};
    for (int k = 0; k < joint.pieces; k += 4) {
        float x[4];
        float4 v[4][2];
        float top = m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = k + j, slot = i == 0 ? 2 * c + 1 : 2 * (c + i);
            x[j] = -INFINITY;
            v[j][0] = v[j][1] = make_float4(0, 0, 0, 0);
            if (i < joint.pieces) {
                const size_t at = (size_t)slot * (MT * 128) + row;
                x[j] = a.partL[at];
                const float4* from = reinterpret_cast<const float4*>(a.partO) + ((size_t)slot * (D / 4) + d / 4) * (MT * 128) + row;
                v[j][0] = from[0];
                v[j][1] = from[MT * 128];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top = fmaxf(top, x[j]);
        const float mm = top == -INFINITY ? 0.0f : top;
        const float f = above_zero(exp2_fast(m - mm));
        m = top;
        l *= f;
#pragma unroll
        for (int y = 0; y < 8; ++y)
            o[y] *= f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float w = above_zero(exp2_fast(x[j] - mm));
            const float* y = reinterpret_cast<const float*>(v[j]);
            if (x[j] != -INFINITY) {
                l += w;
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    o[z] += w * y[z];
            }
        }
    }
    const bool none = l == 0.0f;
    const float inv = none ? 0.0f : 1.0f / l;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = none ? 0u : half2_bits(within_half(o[2 * k] * inv), within_half(o[2 * k + 1] * inv));
    const size_t at = (size_t)(joint.qRow + joint.tok0 + rowTok) * a.Hq + joint.head * a.G + g;
    *reinterpret_cast<uint4*>(a.out + at * D + d) = make_uint4(w[0], w[1], w[2], w[3]);
    if (d == 0 && a.lse != nullptr)
        a.lse[at] = none ? -INFINITY : kLn2 * (m + log2f(l));
}

}  // namespace ropekv_rows
