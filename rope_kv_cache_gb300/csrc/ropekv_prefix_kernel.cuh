// ropekv_prefix_kernel.cuh -- the shared prefix of
// paged_attention_shared_prefix on the 5th-generation tensor cores.
//
// For one KV head the B * S * G query rows of the batch form a matrix Q, the
// prefix matrices K and V: S = Q K^T, P = 2^(c S - M), O += P V, with M and the
// row sums kept per row. One CTA takes MT tiles of 128 rows and one range of the
// prefix, and leaves (O / l, M + log2 l) of every row in the workspace.
//
//   warps 0-3 (and 4-7 with MT = 2)  softmax: a thread owns one row, which is
//                     one TMEM lane; S comes by tcgen05.ld, P goes back by
//                     tcgen05.st over the columns of S that it was made from
//   warp 8            issues the products S (both operands K-major in shared memory)
//   warp 9            issues the products O (P in TMEM, V from shared memory, N-major:
//                     V is stored as it lies in the cache)
//   warps 10-15 (and 4-7 with MT = 1)  fetch pages: a ring of tiles K0, V0, K1, V1,
//                     ... of 64 tokens in shared memory, 128-byte swizzled rows of 64
//                     dims. FP16 rows come by cp.async, 8-bit rows are decoded to FP16
//                     (exact) on the way, which paces it with D = 256 (166 rows of 8, E4M3,
//                     2248 tokens: 127 us with six warps, 91 with ten)
//
// Items i = 0, 1, ... take the SL TMEM slots for S in turn. With two row tiles item
// i is (tile i & 1, K/V tile i >> 1), with one it is K/V tile i. S(i + SL) overwrites
// its slot after O(i) has read the P in it; the slots keep the next scores of a row
// tile ready while its softmax works. With a single slot per row tile (128 tokens
// wide) the chain product - softmax - product of one tile, 2500 cycles of latencies
// even without any arithmetic, set the pace; with one warp issuing both products its
// waits, fences and commits did (about 100 cycles each, 1150 per item).
//
// M moves only when a row's scores exceed it by more than 8, in which case the
// row's O is rescaled in TMEM; the first tile sets it. 8-bit caches: with ks and vs
// a token's scales, x = ks c s + log2(vs) and P = 2^(x - M) is weight times V scale
// in one exponential, near [0, 2^8] whatever the scales; the row sum adds P / vs.
// (A V row whose scale is below 2^-40 in magnitude is fetched as zeros with vs = 2^-40,
// one with a negative scale as its negative. The codes of such a row are worth less than
// 2^-31 each, nothing beside an FP16 result's last place of 2^-24; 1 / vs of a smaller
// scale would push the sum P / vs out of FP32, and P itself below it, while a larger vs
// would lift M, and with it the FP16 weights of rows whose values are small would lose
// their last bits; beside the largest supported scale, 2^60, a token with 2^-40 is still
// summed down to 2^-26 of the other's share. A row whose scale is not finite is fetched
// as NaN with vs = 2^-40: it belongs to the sum of the softmax like any other.)
//
// Bound by the chain of products and exponentials of an item: 256 sequences x 4 rows,
// 8 KV heads of 128, 8192 tokens, FP16: 64 CTAs walk 64 tiles each in 68 us, of which 3.4
// until the first scores and 3 to write the partials; a tile of two items takes 0.98 us,
// against 0.68 us of tensor-core time at the measured 1.88 PFLOP/s and 0.53 us of
// exponentials at 16 a cycle. On all SMs (four ranges) 41 us. 8-bit caches take 1.2 to
// 1.4 us a tile: the fetch warps' decoding comes on top.
//
// Every wait on an mbarrier is bounded. One that runs out ends its role's loop and,
// through a flag, those of the others, and the CTA writes NaN; no role goes on past
// a wait that was not satisfied, so no barrier gets an arrival too many.
#pragma once

#include "ropekv_attention_kernels.cuh"

namespace ropekv_attn {

// V scales of smaller magnitude count as 0.
constexpr float kSmallestScale = 9.094947017729282e-13f;   // 2^-40

template <int D, int FMT, int MT>
struct PrefixConfig {
    static constexpr int kTile = 64;                       // tokens of a K/V tile
    static constexpr int kSlots = D == 256 ? 2 : 4;        // of S in TMEM
    static constexpr int kTileBytes = kTile * D * 2;
    // a ring as wide as the products look ahead: V of item i to K of item i + kSlots
    static constexpr int kStages = 2 * kSlots;
    static constexpr int kMeta = 8;                        // tiles whose scales are kept
    static constexpr int kQBytes = MT * 128 * D * 2;
    static constexpr int kGroups = kTile / 32;             // 32 rows of a tile: one warp's copy
    static constexpr int kFetchers = MT == 1 ? 10 : 6;     // warps 10-15, and 4-7 if no softmax needs them
    static constexpr int kThreads = 16 * 32;
    // arrivals that complete a tile: per group of rows one of each lane's copies and one of
    // the warp (FP16), or the warp's alone
    static constexpr int kArrivals = kGroups * (FMT == kF16 ? 33 : 1);
    // TMEM columns: S slots, then O of each row tile
    static constexpr int kColO = kSlots * kTile;
    static constexpr int kCols = 512;
    static constexpr int kBars = 3 * kStages + 3 * kSlots + 1;
    static constexpr int kOffRing = kQBytes;
    static constexpr int kOffKs = kOffRing + kStages * kTileBytes;
    static constexpr int kOffVs = kOffKs + kMeta * kTile * 4;
    static constexpr int kOffRv = kOffVs + kMeta * kTile * 4;
    static constexpr int kOffMask = kOffRv + kMeta * kTile * 4;
    static constexpr int kOffBar = kOffMask + kMeta * 16;
    // 8-bit, D = 128: one more group per fetch warp on its way, raw
    static constexpr int kOffStage = (kOffBar + kBars * 8 + 16 + 15) / 16 * 16;
    static constexpr int kUsed = kOffStage + (FMT != kF16 && D == 128 ? kFetchers * 32 * D : 0);
    // one CTA per SM (each takes all of TMEM)
    static constexpr int kSmem = (kUsed > 120 * 1024 ? kUsed : 120 * 1024) + 1024;
};

__device__ __forceinline__ void mbar_init(uint32_t bar, int count)
{
    asm volatile("mbarrier.init.shared.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, int parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Wait of at most 2^20 polls, each of which the hardware may suspend for a time of its own
// choosing; false, for the whole CTA, if it runs out.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, int parity, volatile int* failed)
{
    if (mbar_try(bar, parity))
        return true;
    for (int i = 0; i < (1 << 20); ++i) {
        if (mbar_try(bar, parity))
            return true;
        if ((i & 255) == 255 && *failed)
            return false;
    }
    *failed = 1;
    return false;
}

// The same by a whole warp, with one answer.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, int parity, volatile int* failed)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, failed));
}

__device__ __forceinline__ void fence_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_load32(float* f, uint32_t addr)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(addr),
           "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
           "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
           "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_load()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Ties 32 loaded values to this point, behind the wait: nothing that uses them
// can be scheduled before it.
__device__ __forceinline__ void pin32(float* f)
{
    asm volatile(""
        : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]),
          "+f"(f[8]), "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15]),
          "+f"(f[16]), "+f"(f[17]), "+f"(f[18]), "+f"(f[19]), "+f"(f[20]), "+f"(f[21]), "+f"(f[22]), "+f"(f[23]),
          "+f"(f[24]), "+f"(f[25]), "+f"(f[26]), "+f"(f[27]), "+f"(f[28]), "+f"(f[29]), "+f"(f[30]), "+f"(f[31]));
}

__device__ __forceinline__ void tmem_wait_store()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}

// D[128 x N] (+)= A[128 x 16] B[16 x N], A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}

// The same with A in TMEM (FP16, two per column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}

// Two FP32 operations in one instruction: d = a * b + c, d += a.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1)
{
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1)
{
    asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
        "add.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}

// Shared-memory matrix descriptor, 128-byte swizzle: the upper word holds the
// stride of 1024 bytes between groups of eight rows, the version and the swizzle;
// the lower word the address and the leading offset, both in units of 16 bytes.
// Operands further on in the same tile differ by an addition to the lower word.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t leading)
{
    return (addr >> 4) | ((leading >> 4) << 16);
}

__device__ __forceinline__ uint64_t desc(uint32_t low)
{
    return ((uint64_t)kDescHigh << 32) | low;
}

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Instruction descriptor: FP16 x FP16 -> FP32, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool bIsNMajor)
{
    return (1u << 4) | ((bIsNMajor ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// Position of 16-byte chunk c (8 dims) of row r in a tile of `rows` rows: blocks
// of 64 dims, rows of 128 bytes, chunks permuted by the row within eight.
__device__ __forceinline__ uint32_t tile_pos(int rows, int r, int c)
{
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(PrefixConfig<D, FMT, MT>::kThreads, 1) prefix_kernel(const __grid_constant__ Args a)
{
    using C = PrefixConfig<D, FMT, MT>;
    constexpr int TN = C::kTile, NS = C::kStages, GP = C::kGroups, SL = C::kSlots;
    constexpr int kEsize = FMT == kF16 ? 2 : 1;
    extern __shared__ uint8_t smemRaw[];
    const uint32_t rawAddr = smem_u32(smemRaw);
    const uint32_t base = (rawAddr + 1023u) & ~1023u;
    uint8_t* smem = smemRaw + (base - rawAddr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t bars = base + C::kOffBar;
    const uint32_t kvFull = bars, kvEmpty = bars + NS * 8, sFull = bars + 3 * NS * 8,
                   pFull = sFull + SL * 8, oDone = pFull + SL * 8, qFull = oDone + SL * 8;
    volatile int* failed = reinterpret_cast<volatile int*>(smem + C::kOffBar + C::kBars * 8);
    uint32_t* tmemSlot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kBars * 8 + 8);

    // blockIdx.x = (row tile * Hkv + head) * parts + part
    const int part = blockIdx.x % a.numParts;
    const int unit = blockIdx.x / a.numParts;
    const int h = unit % a.Hkv;
    const int row0 = (unit / a.Hkv) * (MT * 128);
    const int tilesAll = (a.P + TN - 1) / TN;
    const int perPart = (tilesAll + a.numParts - 1) / a.numParts;
    const int tile0 = part * perPart;
    const int J = max(0, min(tilesAll, tile0 + perPart) - tile0);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(kvFull + 8 * i, C::kArrivals);
            mbar_init(kvEmpty + 8 * i, 1);
            mbar_init(kvEmpty + 8 * (NS + i), 1);
        }
        for (int i = 0; i < SL; ++i) {
            mbar_init(sFull + 8 * i, 1);
            mbar_init(pFull + 8 * i, 128);
            mbar_init(oDone + 8 * i, 1);
        }
        mbar_init(qFull, MT * 128);
        *failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmemSlot)), "n"(C::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *tmemSlot;
    const int items = MT * J;

    if (warp == 8) {
        // ------------------------------------------------ products S = Q K^T
        // The whole warp walks the loop, so that addresses and descriptors stay in uniform
        // registers; one elected lane issues (from a lone lane's registers every product
        // cost 55 cycles to issue, about what it takes to run).
        constexpr uint32_t kind = mma_desc(TN, false);
        bool ok = items > 0 && mbar_wait_warp(qFull, 0, failed);
        for (int i = 0; ok && i < items; ++i) {
            const int j = MT == 2 ? i >> 1 : i, tile = MT == 2 ? i & 1 : 0;
            const int t = 2 * j, st = t % NS;
            if (tile == 0)
                ok = mbar_wait_warp(kvFull + 8 * st, (t / NS) & 1, failed);
            // the slot's P was read by O(i - SL)
            if (ok && i >= SL)
                ok = mbar_wait_warp(oDone + 8 * (i % SL), (i / SL - 1) & 1, failed);
            if (ok && elect_one()) {
                if ((FMT == kF16 && tile == 0) || i == 0)
                    fence_async_smem();  // the copies landed in the generic proxy
                tmem_fence_after();
                const uint32_t qd = desc_low(base + tile * (128 * D * 2), 16);
                const uint32_t kd = desc_low(base + C::kOffRing + st * C::kTileBytes, 16);
                const uint32_t to = tmem + (i % SL) * TN;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(to, desc(qd + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16),
                           desc(kd + ((k >> 2) * (TN * 128) + (k & 3) * 32) / 16), kind, k > 0);
                mma_commit(sFull + 8 * (i % SL));
                if (tile == MT - 1 && t + NS < 2 * J)  // the stage will be filled again
                    mma_commit(kvEmpty + 8 * (t % (2 * NS)));
            }
            __syncwarp();
        }
    } else if (warp == 9) {
        // ------------------------------------------------- products O += P V
        constexpr uint32_t kind = mma_desc(D, true);
        bool ok = true;
        for (int i = 0; ok && i < items; ++i) {
            const int j = MT == 2 ? i >> 1 : i, tile = MT == 2 ? i & 1 : 0;
            const int t = 2 * j + 1, st = t % NS;
            if (tile == 0)
                ok = mbar_wait_warp(kvFull + 8 * st, (t / NS) & 1, failed);
            ok = ok && mbar_wait_warp(pFull + 8 * (i % SL), (i / SL) & 1, failed);
            if (ok && elect_one()) {
                if (FMT == kF16 && tile == 0)
                    fence_async_smem();
                tmem_fence_after();
                const uint32_t vd = desc_low(base + C::kOffRing + st * C::kTileBytes, TN * 128);
                const uint32_t to = tmem + C::kColO + tile * D, from = tmem + (i % SL) * TN;
#pragma unroll
                for (int k = 0; k < TN / 16; ++k)
                    mma_ts(to, from + k * 8, desc(vd + k * (2048 / 16)), kind, j > 0 || k > 0);
                mma_commit(oDone + 8 * (i % SL));
                if (tile == MT - 1 && t + NS < 2 * J)
                    mma_commit(kvEmpty + 8 * (t % (2 * NS)));
            }
            __syncwarp();
        }
    } else if (warp > 9 || (MT == 1 && warp >= 4)) {
        // ------------------------------------------------------- page fetch
        const int me = warp > 9 ? warp - 10 : warp + 2;
        const int groups = 2 * J * GP;
        const size_t rowStride = (size_t)a.Hkv * D * kEsize;
        const uint8_t* headBase = a.pool + (size_t)h * D * kEsize;
        constexpr int kVecs = D * kEsize / 16;         // 16-byte vectors of a row
        constexpr int kPerLane = kVecs;                // 32 rows of kVecs vectors over 32 lanes
        // 8-bit: groups of a warp in flight; D = 128 keeps every other one in shared memory (two
        // in registers spill, one alone cannot cover the latency beside a busy stream)
        constexpr int kDepth = kVecs > 8 ? 1 : 2;
        constexpr bool kStaged = kVecs == 8;

        // page ids of this lane's row of the next kIds groups: an id is a round trip to L2
        // ahead of the copies that need it
        constexpr int kIds = 4;
        int idsK[kIds], idsV[kIds];
        auto fetch_ids = [&](int u, int& idK, int& idV) {
            idK = idV = -1;
            const int pos = (tile0 + (u / GP >> 1)) * TN + (u % GP) * 32 + lane;
            if (u < groups && pos < a.P) {
                const int lp = divide(pos, a.divTpp);
                idK = __ldg(a.prefixTable + lp);
                idV = __ldg(a.prefixTable + a.prefixPages + lp);
            }
        };
        // Row of the pool for this lane's token and the mask of mapped tokens
        auto locate = [&](int u, int idK, int idV, uint32_t& mask) -> uint32_t {
            const int t = u / GP, g = u % GP;
            const int pos = (tile0 + (t >> 1)) * TN + g * 32 + lane;
            const bool ok = idK >= 0 && idK < a.numPages && idV >= a.numPages &&
                            idV - a.numPages < a.numPages;
            mask = __ballot_sync(0xffffffffu, ok);
            const int inPage = pos - divide(pos, a.divTpp) * a.tpp;
            return ok ? (uint32_t)((t & 1) ? idV : idK) * (uint32_t)a.tpp + inPage : 0u;
        };
        // Waits until tile t - NS, which had tile t's stage, is consumed. Barriers of two
        // laps of the ring: a barrier's parity tells only its last two phases apart, and a
        // warp visits only every d-th tile, d = kFetchers / GP. With barrier (t - NS) % 2 NS
        // the phase before the one waited for is tile t - 3 NS, which is consumed: the warp
        // waited for tile t - d - NS, and with a tile all up to NS - 1 before it are consumed.
        // The phase after is tile t + NS, for which tile t would be needed.
        static_assert(C::kFetchers % GP == 0 && C::kFetchers / GP <= NS + 1, "see above");
        auto stage_free = [&](int t) -> bool {
            const int old = t - NS;
            return old < 0 || mbar_wait_warp(kvEmpty + 8 * (old % (2 * NS)), (old / (2 * NS)) & 1, failed);
        };
        // what the softmax needs of a K group's tokens: the mask and (8-bit) the K scale
        // times c, log2 and reciprocal of the V scale's magnitude
        auto write_meta = [&](int u, uint32_t mask, float ks, float vs) {
            const int j = (u / GP) >> 1, g = u % GP, slot = j % C::kMeta;
            if (FMT != kF16) {
                const int at = slot * TN + g * 32 + lane;
                const float v = fabsf(vs) >= kSmallestScale && fabsf(vs) < INFINITY ? fabsf(vs) : kSmallestScale;
                reinterpret_cast<float*>(smem + C::kOffKs)[at] = ks * a.scaleLog2;
                reinterpret_cast<float*>(smem + C::kOffVs)[at] = log2f(v);
                reinterpret_cast<float*>(smem + C::kOffRv)[at] = 1.0f / v;
            }
            if (lane == 0)
                reinterpret_cast<uint32_t*>(smem + C::kOffMask)[slot * 4 + g] = mask;
        };
        constexpr int kStep = C::kFetchers;
#pragma unroll
        for (int x = 0; x < kIds; ++x)
            fetch_ids(me + kStep * x, idsK[x], idsV[x]);
        if (FMT == kF16) {
            // the copies arrive at the tile's barrier by themselves when they land
            for (int v = me; v < groups; v += kStep * kIds) {
#pragma unroll
            for (int x = 0; x < kIds; ++x) {
                const int u = v + kStep * x;
                if (u >= groups)
                    break;
                uint32_t mask;
                const uint32_t row = locate(u, idsK[x], idsV[x], mask);
                fetch_ids(u + kStep * kIds, idsK[x], idsV[x]);
                const int t = u / GP;
                if (!stage_free(t)) {
                    v = groups;
                    break;
                }
                const uint32_t dst = base + C::kOffRing + (t % NS) * C::kTileBytes;
                const int r0 = (u % GP) * 32;
                if (mask == 0xffffffffu) {
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i) {
                        const int idx = i * 32 + lane, r = idx / kVecs, c = idx % kVecs;
                        const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                        copy16(dst + tile_pos(TN, r0 + r, c), headBase + (size_t)src * rowStride + c * 16);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i) {
                        const int idx = i * 32 + lane, r = idx / kVecs, c = idx % kVecs;
                        const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                        copy16(dst + tile_pos(TN, r0 + r, c), headBase + (size_t)src * rowStride + c * 16,
                               (mask >> r) & 1);
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];"
                             :: "r"(kvFull + 8 * (t % NS)) : "memory");
                if (!(t & 1))
                    write_meta(u, mask, 0.0f, 0.0f);
                if (lane == 0)
                    mbar_arrive(kvFull + 8 * (t % NS));
            }
            }
            copy_wait_all();
        } else {
            // registers of kDepth groups in flight
            auto publish = [&](int u) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(kvFull + 8 * ((u / GP) % NS));
            };
            uint4 buf[kStaged ? 1 : kDepth][kPerLane];
            const uint32_t staging = base + C::kOffStage + me * (32 * kVecs * 16) + lane * 16;
            float ks[kDepth], vs[kDepth];
            uint32_t mask[kDepth];
            auto load = [&](int u, int k, int& idK, int& idV) {
                const uint32_t row = locate(u, idK, idV, mask[k]);
                ks[k] = vs[k] = 0.0f;
                if ((mask[k] >> lane) & 1) {
                    const int pos = (tile0 + (u / GP >> 1)) * TN + (u % GP) * 32 + lane;
                    const int inPage = pos - divide(pos, a.divTpp) * a.tpp;
                    ks[k] = __ldg(a.scales + ((size_t)idK * a.Hkv + h) * a.tpp + inPage);
                    vs[k] = __ldg(a.scales + ((size_t)idV * a.Hkv + h) * a.tpp + inPage);
                }
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) {
                    const int idx = i * 32 + lane, r = idx / kVecs, c = idx % kVecs;
                    const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                    if (kStaged && k == 1) {
                        copy16(staging + i * 512, headBase + (size_t)src * rowStride + c * 16, (mask[k] >> r) & 1);
                        continue;
                    }
                    buf[kStaged ? 0 : k][i] = make_uint4(0, 0, 0, 0);
                    if ((mask[k] >> r) & 1)
                        buf[kStaged ? 0 : k][i] = __ldg(reinterpret_cast<const uint4*>(headBase + (size_t)src * rowStride + c * 16));
                }
                fetch_ids(u + kStep * kIds, idK, idV);
            };
#pragma unroll
            for (int k = 0; k < kDepth; ++k)
                if (me + kStep * k < groups)
                    load(me + kStep * k, k, idsK[k], idsV[k]);
            for (int v = me; v < groups; v += kStep * kIds) {
#pragma unroll
                for (int y = 0; y < kIds; ++y) {
                    const int u = v + kStep * y, k = y % kDepth, ahead = (y + kDepth) % kIds;
                    if (u >= groups)
                        break;
                    const int t = u / GP;
                    if (!stage_free(t)) {
                        v = groups;
                        break;
                    }
                    uint8_t* dst = smem + C::kOffRing + (t % NS) * C::kTileBytes;
                    const int r0 = (u % GP) * 32;
                    // V rows are taken times 1, -1 (negative scale), 0 (small scale, unmapped token) or
                    // NaN (scale not finite); unmapped K rows are zeros as loaded
                    const uint32_t factor = fabsf(vs[k]) < kSmallestScale ? 0u : !(fabsf(vs[k]) < INFINITY) ? 0x7fff7fffu
                                            : vs[k] < 0.0f ? 0xbc00bc00u : 0x3c003c00u;
                    const bool plain = !(t & 1) || __all_sync(0xffffffffu, factor == 0x3c003c00u);
                    if (kStaged && k == 1)
                        copy_wait_all();       // each lane reads what it copied
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i) {
                        const int idx = i * 32 + lane, r = idx / kVecs, c = idx % kVecs;
                        const uint4 raw = kStaged && k == 1
                            ? *reinterpret_cast<const uint4*>(smem + (staging - base) + i * 512) : buf[kStaged ? 0 : k][i];
                        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
                        uint32_t o[8];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            decode_word<FMT, false>(w[x], o[2 * x], o[2 * x + 1]);
                        if (!plain) {
                            const uint32_t f = __shfl_sync(0xffffffffu, factor, r);
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                o[x] = half2_times(o[x], f);
                        }
                        *reinterpret_cast<uint4*>(dst + tile_pos(TN, r0 + r, 2 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(dst + tile_pos(TN, r0 + r, 2 * c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    if (!(t & 1))
                        write_meta(u, mask[k], ks[k], vs[k]);
                    publish(u);
                    if (u + kStep * kDepth < groups)
                        load(u + kStep * kDepth, k, idsK[ahead], idsV[ahead]);
                }
            }
            copy_wait_all();
        }
    } else {
        // ----------------------------------------------------------- softmax
        // first of all Q, zeros past the last row, while the first pages come
        for (int i = threadIdx.x; i < MT * 128 * (D / 8); i += MT * 128) {
            const int r = i / (D / 8), c = i % (D / 8);
            const int row = row0 + r;
            const bool ok = row < a.rowsPrefix;
            const size_t tok = ok ? divide(row, a.divG) : 0;
            const int g = ok ? row - (int)tok * a.G : 0;
            copy16(base + (r >> 7) * (128 * D * 2) + tile_pos(128, r & 127, c),
                   a.q + (tok * a.Hq + h * a.G + g) * D + c * 8, ok);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(qFull) : "memory");
        const int tile = warp >> 2;
        const uint32_t laneBase = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t oAddr = laneBase + C::kColO + tile * D;
        float M = -INFINITY, l = 0.0f;
        // |c|, kept above 0 so that a masked -infinity stays one (c = 0: all scores are 0)
        const float scale = fmaxf(fabsf(a.scaleLog2), 1e-30f);
        for (int j = 0; j < J; ++j) {
            const int i = MT == 2 ? 2 * j + tile : j;
            const int slot = i % SL;
            const uint32_t sAddr = laneBase + slot * TN;
            if (!mbar_wait_warp(sFull + 8 * slot, (i / SL) & 1, failed))
                break;
            tmem_fence_after();
            float s[TN];
#pragma unroll
            for (int k = 0; k < TN / 32; ++k)
                tmem_load32(s + 32 * k, sAddr + 32 * k);
            const int meta = j % C::kMeta;
            const uint32_t* mask = reinterpret_cast<const uint32_t*>(smem + C::kOffMask) + meta * 4;
            const float* ks = reinterpret_cast<const float*>(smem + C::kOffKs) + meta * TN;
            const float* lv = reinterpret_cast<const float*>(smem + C::kOffVs) + meta * TN;
            const float* rv = reinterpret_cast<const float*>(smem + C::kOffRv) + meta * TN;
            uint32_t all = 0xffffffffu;
#pragma unroll
            for (int g = 0; g < GP; ++g)
                all &= mask[g];
            tmem_wait_load();
#pragma unroll
            for (int k = 0; k < TN / 32; ++k)
                pin32(s + 32 * k);
            if (FMT != kF16) {
#pragma unroll
                for (int k = 0; k < TN; k += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(ks + k);
                    const float4 v = *reinterpret_cast<const float4*>(lv + k);
                    fma2(s[k], s[k + 1], s[k], s[k + 1], f.x, f.y, v.x, v.y);
                    fma2(s[k + 2], s[k + 3], s[k + 2], s[k + 3], f.z, f.w, v.z, v.w);
                }
            } else if (a.scaleLog2 < 0.0f) {
#pragma unroll
                for (int k = 0; k < TN; ++k)
                    s[k] = -s[k];
            }
            if (all != 0xffffffffu) {
#pragma unroll
                for (int k = 0; k < TN; ++k)
                    s[k] = (mask[k >> 5] >> (k & 31)) & 1 ? s[k] : -INFINITY;
            }
            // FP16: s is unscaled until the exponential takes c s - M
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
            if (FMT == kF16)
                top = top == -INFINITY ? top : top * scale;
            if (__any_sync(0xffffffffu, top > M + 8.0f)) {
                const float next = fmaxf(M, top);
                const float f = M == next ? 1.0f : exp2_fast(M - next);
                M = next;
                l *= f;
                if (j > 0) {
                    // O of this row tile is at rest: its last product has finished
                    const int before = i - MT;
                    if (!mbar_wait_warp(oDone + 8 * (before % SL), (before / SL) & 1, failed))
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
            const float mul = FMT == kF16 ? scale : 1.0f;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < TN; k += 64) {
                uint32_t p[32];
#pragma unroll
                for (int x = 0; x < 64; x += 4) {
                    float v[4];
                    fma2(v[0], v[1], s[k + x], s[k + x + 1], mul, mul, -mm, -mm);
                    fma2(v[2], v[3], s[k + x + 2], s[k + x + 3], mul, mul, -mm, -mm);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        v[y] = exp2_fast(v[y]);
                    if (FMT == kF16) {
                        add2(sum[0], sum[1], v[0], v[1]);
                        add2(sum[2], sum[3], v[2], v[3]);
                    } else {
                        const float4 f = *reinterpret_cast<const float4*>(rv + k + x);
                        fma2(sum[0], sum[1], v[0], v[1], f.x, f.y, sum[0], sum[1]);
                        fma2(sum[2], sum[3], v[2], v[3], f.z, f.w, sum[2], sum[3]);
                    }
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
        copy_wait_all();   // Q, should no product have waited for it
        // the last products of this row tile
        if (J > 0) {
            const int last = MT == 2 ? 2 * (J - 1) + tile : J - 1;
            mbar_wait_warp(oDone + 8 * (last % SL), (last / SL) & 1, failed);
        }
        tmem_fence_after();
        const int row = row0 + (int)threadIdx.x;       // threads 0..127: tile 0, 128..255: tile 1
        const bool live = row < a.rowsPrefix;
        const size_t r = ((size_t)part * a.Hkv + h) * a.rowsPrefix + row;
        const bool none = J == 0 || l == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l;
        const float bad = *failed ? __int_as_float(0x7fc00000) : 0.0f;
        // 32 columns at a time through shared memory (this tile's Q: its products have
        // finished), so that eight lanes write 128 bytes of one row
        float* mine = reinterpret_cast<float*>(smem + tile * (128 * D * 2)) + (warp & 3) * (32 * 32);
        const int warpRow = row - lane;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
            float o[32];
            if (J > 0) {
                tmem_load32(o, oAddr + k);
                tmem_wait_load();
                pin32(o);
            }
#pragma unroll
            for (int x = 0; x < 32; x += 4)
                *reinterpret_cast<float4*>(mine + lane * 32 + (((x >> 2) ^ (lane & 7)) << 2)) =
                    none ? make_float4(bad, bad, bad, bad)
                         : make_float4(o[x] * inv + bad, o[x + 1] * inv + bad, o[x + 2] * inv + bad, o[x + 3] * inv + bad);
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int n = x * 4 + (lane >> 3);
                if (warpRow + n < a.rowsPrefix)
                    *reinterpret_cast<float4*>(a.partO + (r - lane + n) * D + k + (lane & 7) * 4) =
                        *reinterpret_cast<const float4*>(mine + n * 32 + (((lane & 7) ^ (n & 7)) << 2));
            }
            __syncwarp();
        }
        if (live)
            a.partL[r] = none ? -INFINITY + bad : M + log2f(l) + bad;
        tmem_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "n"(C::kCols));
    }
}

}  // namespace ropekv_attn
