// ropekv_pages.cu -- rows and pages of the caches moved, shared and given up:
// kv_accept_drafts, paged_kv_accept_drafts, paged_kv_copy_pages, paged_kv_fork and
// paged_kv_free (include/ropekv_sequence.h), kernels and C entry points. Nothing is
// computed: copies are bound by HBM, the rest by the latency of a launch and of a few
// loads that depend on one another. All are dependent launches that wait for the grid in
// front of them before they touch anything, and read what it may have written by ordinary
// loads.
#include <cuda_runtime.h>

#include <stdint.h>

#include "ropekv_sequence.h"

namespace {

bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <typename Kern, typename Args>
int launch(Kern kern, long long grid, int threads, int smem, cudaStream_t st, const Args& a)
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
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? ROPEKV_OK : ROPEKV_ERR_LAUNCH;
}

// Lets the next grid begin to launch, then waits until the one before has completed.
__device__ __forceinline__ void dependency_sync()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Copied data is touched once: past L1, evict-first in L2.
__device__ __forceinline__ uint64_t stream_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ uint4 load16(const uint8_t* p, uint64_t policy)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "l"(policy) : "memory");
    return v;
}

__device__ __forceinline__ void store16(uint8_t* p, const uint4& v, uint64_t policy)
{
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;"
                 :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "l"(policy) : "memory");
}

// ------------------------------------------------------- accepted drafts --

struct AcceptArgs {
    uint8_t* cache;            // [B, 2, Hkv, cap, D] FP16, or [2, P, tpp, Hkv, D]
    float* scales;             // [2, P, Hkv, tpp] or NULL
    const int32_t* pageTable;  // [B, 2, M] (paged)
    const int32_t* lens;       // [B]
    const int32_t* accepted;   // [B, A]
    const int32_t* acceptedLens;
    int32_t* lensOut;          // [B] or NULL
    int32_t S, A, Hkv, rowVecs;    // 16-byte vectors of one head's row
    int32_t cap;               // slots (contiguous), positions (paged: M * tpp)
    int32_t numPages, M, tpp;
};

// One CTA per sequence. Entries are taken in order, eight at a time: one warp finds their rows,
// then a thread moves one 16-byte column (of either plane and any head), all sources read
// before the first of the eight is written. Entry j's source is at least j, every
// destination before it is smaller, so nothing is overwritten that is still to move, and a
// column has the same thread throughout. Scales are further columns of 4 bytes. Bound by
// latency: lengths and entries, page ids, rows, one after the other (128 sequences, up to 8 of 61
// drafts, INT8: 3.9 us, 5.7 with every thread looking its rows up itself; 4 sequences of a
// contiguous cache 2.5 us, about what any dependent launch takes).
template <bool PAGED>
__global__ void __launch_bounds__(512) accept_kernel(const __grid_constant__ AcceptArgs a)
{
    constexpr int kBatch = 8;
    // rows of the plane (paged: page * tpp + place), below 0 where nothing moves
    __shared__ int rows[2][2][kBatch];
    dependency_sync();
    const int b = blockIdx.x;
    const int len = a.lens[b];
    const int n = max(0, min(a.acceptedLens[b], min(a.A, a.S)));
    const int64_t base = (int64_t)len - a.S;
    const int vecs = 2 * a.Hkv * a.rowVecs;
    const int items = vecs + (PAGED && a.scales != nullptr ? 2 * a.Hkv : 0);
    for (int j0 = 0; j0 < n; j0 += kBatch) {
        if (threadIdx.x < 32) {
            const int plane = threadIdx.x >> 4, to = (threadIdx.x >> 3) & 1, j = j0 + (threadIdx.x & 7);
            const int node = j < n ? a.accepted[(size_t)b * a.A + j] : -1;
            const int64_t src = base + node, dst = base + j, pos = to ? dst : src;
            int row = node > j && node < a.S && dst >= 0 && src < a.cap ? (int)pos : -1;   // node == j stays where it is
            if (PAGED && row >= 0) {
                const int lp = row / a.tpp;
                const int64_t id = (int64_t)a.pageTable[((size_t)b * 2 + plane) * a.M + lp] - (int64_t)plane * a.numPages;
                row = id >= 0 && id < a.numPages ? (int)id * a.tpp + (row - lp * a.tpp) : -1;
            }
            // both or neither
            if (__shfl_xor_sync(0xffffffffu, row, 8) < 0)
                row = -1;
            rows[plane][to][threadIdx.x & 7] = row;
        }
        __syncthreads();
        for (int item = threadIdx.x; item < items; item += blockDim.x) {
            const bool scale = item >= vecs;
            const int ph = scale ? item - vecs : item / a.rowVecs;      // plane * Hkv + head
            const int vec = scale ? 0 : item - ph * a.rowVecs;
            const int plane = ph >= a.Hkv, h = ph - plane * a.Hkv;
            auto at = [&](int row) -> uint8_t* {
                if (!PAGED)
                    return a.cache + ((((size_t)b * 2 + plane) * a.Hkv + h) * a.cap + row) * a.rowVecs * 16 + vec * 16;
                if (scale) {
                    const int page = row / a.tpp;
                    return reinterpret_cast<uint8_t*>(
                        a.scales + (((size_t)plane * a.numPages + page) * a.Hkv + h) * a.tpp + (row - page * a.tpp));
                }
                return a.cache + (((size_t)plane * a.numPages * a.tpp + row) * a.Hkv + h) * a.rowVecs * 16 + vec * 16;
            };
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int row = rows[plane][0][k];
                if (row < 0)
                    continue;
                if (scale)
                    x[k].x = *reinterpret_cast<const uint32_t*>(at(row));
                else
                    x[k] = *reinterpret_cast<const uint4*>(at(row));
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int row = rows[plane][1][k];
                if (row < 0)
                    continue;
                if (scale)
                    *reinterpret_cast<uint32_t*>(at(row)) = x[k].x;
                else
                    *reinterpret_cast<uint4*>(at(row)) = x[k];
            }
        }
        __syncthreads();
    }
    __syncthreads();   // lensOut may be lens
    if (threadIdx.x == 0 && a.lensOut != nullptr && len >= a.S)
        a.lensOut[b] = len - a.S + n;
}

int check_accept(const AcceptArgs& a, int32_t batch, int32_t D)
{
    if (D != 64 && D != 128 && D != 256)
        return ROPEKV_ERR_HEAD_DIM;
    if (a.Hkv <= 0)
        return ROPEKV_ERR_HEADS;
    if (batch < 0 || a.S < 0 || a.A < 0 || a.S > (1 << 15) || a.A > (1 << 15) || (long long)a.Hkv * D > (1LL << 24))
        return ROPEKV_ERR_SHAPE;
    return ROPEKV_OK;
}

int run_accept(const AcceptArgs& a, int32_t batch, bool paged, cudaStream_t st)
{
    const int items = 2 * a.Hkv * a.rowVecs + (a.scales != nullptr ? 2 * a.Hkv : 0);
    const int threads = items < 512 ? (items + 31) / 32 * 32 : 512;
    return paged ? launch(accept_kernel<true>, batch, threads, 0, st, a) : launch(accept_kernel<false>, batch, threads, 0, st, a);
}

// ------------------------------------------------------------ page copies --

struct CopyArgs {
    uint8_t* cache;            // [2, P, tpp, Hkv, D]
    float* scales;             // [2, P, Hkv, tpp] or NULL
    const int32_t* src;        // [N]
    const int32_t* dst;
    int32_t N, numPages, tpp, Hkv, chunks;
    int64_t pageVecs;          // 16-byte vectors of one plane's page
};

constexpr int kCopyUnroll = 4;

// A CTA copies one run of one plane of one pair: four vectors a thread, all loaded before
// the first is stored; the first run's CTA takes the page's scales along. 1200 pages of 32 tokens x 8
// heads of 128, FP16: 47.5 us, 6.6 TB/s read and written, 97 % of a plain copy; 6 small pages 2.9 us.
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ CopyArgs a)
{
    dependency_sync();
    const uint64_t pol = stream_policy();
    const int chunk = blockIdx.x % a.chunks, pair = blockIdx.x / a.chunks;
    const int plane = pair & 1, i = pair >> 1;
    const int src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.numPages || dst < 0 || dst >= a.numPages || src == dst)
        return;
    const size_t from = (size_t)plane * a.numPages + src, to = (size_t)plane * a.numPages + dst;
    const int64_t v0 = (int64_t)chunk * blockDim.x * kCopyUnroll + threadIdx.x;
    const uint8_t* s = a.cache + from * a.pageVecs * 16;
    uint8_t* d = a.cache + to * a.pageVecs * 16;
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
        if (v0 + k * blockDim.x < a.pageVecs)
            x[k] = load16(s + (v0 + k * blockDim.x) * 16, pol);
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k)
        if (v0 + k * blockDim.x < a.pageVecs)
            store16(d + (v0 + k * blockDim.x) * 16, x[k], pol);
    if (a.scales != nullptr && chunk == 0) {
        const size_t row = (size_t)a.Hkv * a.tpp;
        for (size_t k = threadIdx.x; k < row; k += blockDim.x)
            a.scales[to * row + k] = a.scales[from * row + k];
    }
}

// ----------------------------------------------------------------- forks --

struct ForkArgs {
    uint8_t* cache;            // [2, P, tpp, Hkv, D]
    float* scales;             // [2, P, Hkv, tpp] or NULL
    int32_t* pageTable;        // [B, 2, M]
    int32_t* kvLens;           // [B]
    int32_t* refCounts;        // [P]
    const int32_t* parents;    // [N]
    const int32_t* children;
    struct Fork* forks;        // [N] workspace: what the plan decided
    int32_t* found;            // [1] workspace: free pages found, at most the number needed
    int32_t* fresh;            // [N] workspace: the free pages, ascending
    int32_t N, B, numPages, M, tpp, Hkv, chunks;
    int64_t rowVecs;           // 16-byte vectors of one plane's row (all heads)
};

constexpr int kNoPage = -1, kSkipped = -2;

struct __align__(16) Fork {
    int rank;                  // among the forks that need a page, or one of the above
    int parent, child;
    int length;                // of the parent
    int tail;                  // its partly filled page
};
static_assert(sizeof(Fork) == 32, "workspace");

__device__ __forceinline__ int fork_length(const ForkArgs& a, int parent)
{
    return (int)min((long long)max(0, a.kvLens[parent]), (long long)a.M * a.tpp);
}

// Exclusive sum over the CTA's 1024 threads; the total in `sum`.
__device__ __forceinline__ int scan1024(int x, int& sum, int* shared)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        v += lane >= d ? y : 0;
    }
    __syncthreads();           // the last scan's sums have been read
    if (lane == 31)
        shared[warp] = v;
    __syncthreads();
    int w = shared[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, d);
        w += lane >= d ? y : 0;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return v - x + (warp > 0 ? before : 0);
}

// One CTA decides for all forks, so that free pages go out in the order of the forks,
// lowest first, without atomics whose order could change it. Sequences named as parent, as
// child and as child twice are bits in shared memory. The reference counts are read 16
// pages a thread until there are enough free ones; those of the first round, and of the first
// 1024 forks all that depends on memory alone, are on their way before the bits are known
// (192 forks over 1000 pages: 5 us as a launch of its own, four loads after one another).
__global__ void __launch_bounds__(1024) fork_plan_kernel(const __grid_constant__ ForkArgs a)
{
    extern __shared__ uint32_t bits[];
    __shared__ int sums[32];
    const int words = (a.B + 31) / 32;
    uint32_t *isParent = bits, *isChild = bits + words, *isTwice = bits + 2 * words;
    for (int i = threadIdx.x; i < 3 * words; i += 1024)
        bits[i] = 0;
    dependency_sync();
    auto free_pages = [&](int p) -> uint32_t {
        uint32_t freeBits = 0;
        if (p + 16 <= a.numPages) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int4 r = *reinterpret_cast<const int4*>(a.refCounts + p + 4 * k);
                freeBits |= ((r.x <= 0) | (r.y <= 0) << 1 | (r.z <= 0) << 2 | (r.w <= 0) << 3) << (4 * k);
            }
        } else {
            for (int k = 0; k < 16 && p + k < a.numPages; ++k)
                freeBits |= (uint32_t)(a.refCounts[p + k] <= 0) << k;
        }
        return freeBits;
    };
    // a fork as far as memory says: rank kSkipped, kNoPage, or 0 where a page is needed
    auto read_fork = [&](int i) -> Fork {
        Fork f = {kSkipped, -1, -1, 0, -1};
        if (i >= a.N)
            return f;
        f.parent = a.parents[i];
        f.child = a.children[i];
        if (f.parent < 0 || f.parent >= a.B || f.child < 0 || f.child >= a.B) {
            f.parent = f.child = -1;
            return f;
        }
        f.length = fork_length(a, f.parent);
        if (a.kvLens[f.child] > 0)
            return f;
        f.rank = kNoPage;
        const int whole = f.length / a.tpp;
        if (f.length - whole * a.tpp > 0) {
            f.tail = a.pageTable[(size_t)f.parent * 2 * a.M + whole];
            if (f.tail >= 0 && f.tail < a.numPages)
                f.rank = 0;
        }
        return f;
    };
    const Fork mine = read_fork(threadIdx.x);
    const uint32_t firstFree = free_pages(16 * threadIdx.x);
    __syncthreads();
    for (int i = threadIdx.x; i < a.N; i += 1024) {
        const Fork f = i < 1024 ? mine : read_fork(i);
        if (f.child < 0)
            continue;
        atomicOr(isParent + (f.parent >> 5), 1u << (f.parent & 31));
        const uint32_t bit = 1u << (f.child & 31);
        if (atomicOr(isChild + (f.child >> 5), bit) & bit)
            atomicOr(isTwice + (f.child >> 5), bit);
    }
    __syncthreads();
    int needed = 0;
    for (int i0 = 0; i0 < a.N; i0 += 1024) {
        const int i = i0 + threadIdx.x;
        Fork f = i0 == 0 ? mine : read_fork(i);
        if (f.child >= 0 && (((isTwice[f.child >> 5] | isParent[f.child >> 5]) >> (f.child & 31)) & 1))
            f.rank = kSkipped;
        int sum;
        const int before = scan1024(f.rank == 0, sum, sums);
        if (f.rank == 0)
            f.rank = needed + before;
        if (i < a.N)
            a.forks[i] = f;
        needed += sum;
    }
    int found = 0;
    for (int p0 = 0; p0 < a.numPages && found < needed; p0 += 16 * 1024) {
        const int p = p0 + 16 * threadIdx.x;
        uint32_t freeBits = p0 == 0 ? firstFree : free_pages(p);
        int sum;
        int at = found + scan1024(__popc(freeBits), sum, sums);
        for (; freeBits != 0 && at < needed; freeBits &= freeBits - 1, ++at)
            a.fresh[at] = p + __ffs(freeBits) - 1;
        found += sum;
    }
    if (threadIdx.x == 0)
        *a.found = min(found, needed);
}

// CTAs of one fork: runs of the partly filled page's rows (four vectors a thread); the
// first also writes the child's row of the table, the counts and the length. Children
// are no parents, so nothing that is read here is written here. 192 children given up and forked
// anew from 64 sequences of up to 2000 tokens (pages of 64, 8 heads of 128, FP16; 50 MB): 14.6 us in three
// launches, of which the copy takes about 8; four children 8.7 us.
__global__ void __launch_bounds__(256) fork_copy_kernel(const __grid_constant__ ForkArgs a)
{
    dependency_sync();
    const uint64_t pol = stream_policy();
    const int chunk = blockIdx.x % a.chunks, i = blockIdx.x / a.chunks;
    const Fork f = a.forks[i];
    if (f.rank == kSkipped)
        return;
    const int whole = f.length / a.tpp, rest = f.length - whole * a.tpp;
    // the source's rows need not wait for the destination
    const int64_t vecs = f.rank >= 0 ? (int64_t)rest * a.rowVecs : 0, page = (int64_t)a.tpp * a.rowVecs;
    const int64_t v0 = (int64_t)chunk * blockDim.x * kCopyUnroll + threadIdx.x;
    uint4 x[2][kCopyUnroll];
#pragma unroll
    for (int plane = 0; plane < 2; ++plane)
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k)
            if (v0 + k * blockDim.x < vecs)
                x[plane][k] = load16(a.cache + (((int64_t)plane * a.numPages + f.tail) * page + v0 + k * blockDim.x) * 16, pol);
    const int fresh = f.rank >= 0 && f.rank < *a.found ? a.fresh[f.rank] : -1;
    if (chunk == 0) {
        const int32_t* from = a.pageTable + (size_t)f.parent * 2 * a.M;
        int32_t* to = a.pageTable + (size_t)f.child * 2 * a.M;
        for (int k = threadIdx.x; k < a.M; k += blockDim.x) {
            const int id = k < whole ? from[k] : -1;
            const int old = to[k];               // an empty child may still name pages: it gives them up
            const bool mapped = id >= 0 && id < a.numPages;
            if (mapped)
                atomicAdd(a.refCounts + id, 1);
            if (old >= 0 && old < a.numPages)
                atomicSub(a.refCounts + old, 1);
            const int mine = mapped ? id : k == whole ? fresh : -1;
            to[k] = mine;
            to[a.M + k] = mine >= 0 ? mine + a.numPages : -1;
        }
        if (threadIdx.x == 0) {
            a.kvLens[f.child] = fresh >= 0 || rest == 0 ? f.length : whole * a.tpp;
            if (fresh >= 0)
                a.refCounts[fresh] = 1;
        }
    }
    if (fresh < 0)
        return;
#pragma unroll
    for (int plane = 0; plane < 2; ++plane)
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k)
            if (v0 + k * blockDim.x < vecs)
                store16(a.cache + (((int64_t)plane * a.numPages + fresh) * page + v0 + k * blockDim.x) * 16, x[plane][k], pol);
    if (a.scales != nullptr) {
        const int64_t row = (int64_t)a.Hkv * rest, all = 2 * row;
        for (int64_t k = (int64_t)chunk * blockDim.x + threadIdx.x; k < all; k += (int64_t)a.chunks * blockDim.x) {
            const int plane = k >= row, h = (int)((k - plane * row) / rest), t = (int)((k - plane * row) - (int64_t)h * rest);
            const size_t at = ((size_t)plane * a.numPages * a.Hkv + h) * a.tpp + t, step = (size_t)a.Hkv * a.tpp;
            a.scales[at + fresh * step] = a.scales[at + f.tail * step];
        }
    }
}

// ------------------------------------------------------------------- free --

struct FreeArgs {
    int32_t* pageTable;        // [B, 2, M]
    int32_t* kvLens;           // [B]
    int32_t* refCounts;        // [P]
    const int32_t* sequences;  // [N]
    const int32_t* keep;       // [N] or NULL
    int32_t B, numPages, M, tpp, chunks;
};

// A thread takes one column of one sequence. Entries are claimed by an exchange, so that
// a sequence named twice gives up each page once; sums of the counts do not depend on
// their order.
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ FreeArgs a)
{
    dependency_sync();
    const int chunk = blockIdx.x % a.chunks, i = blockIdx.x / a.chunks;
    const int s = a.sequences[i];
    if (s < 0 || s >= a.B)
        return;
    const int keep = a.keep != nullptr ? max(0, a.keep[i]) : 0;
    const int k = chunk * blockDim.x + threadIdx.x;
    if (chunk == 0 && threadIdx.x == 0)
        atomicMin(a.kvLens + s, keep);
    if (k >= a.M || (long long)k * a.tpp < keep)
        return;
    int32_t* entry = a.pageTable + (size_t)s * 2 * a.M + k;
    entry[a.M] = -1;
    if (*entry == -1)
        return;
    const int id = atomicExch(entry, -1);
    if (id >= 0 && id < a.numPages)
        atomicSub(a.refCounts + id, 1);
}

int check_pool(int32_t D, int32_t Hkv, int32_t numPages, int32_t tpp, int32_t fmt)
{
    if (fmt < ROPEKV_CACHE_F16 || fmt > ROPEKV_CACHE_INT8)
        return ROPEKV_ERR_STYLE;
    if (D != 64 && D != 128 && D != 256)
        return ROPEKV_ERR_HEAD_DIM;
    if (Hkv <= 0)
        return ROPEKV_ERR_HEADS;
    if (numPages < 0 || tpp <= 0 || 2LL * numPages * tpp > 0x7FFFFFFFLL || (long long)Hkv * D > (1LL << 24))
        return ROPEKV_ERR_SHAPE;
    return ROPEKV_OK;
}

int check_table(int32_t batch, int32_t M, int32_t tpp)
{
    return batch < 0 || M < 0 || tpp <= 0 || (long long)M * tpp > (1LL << 30) ? ROPEKV_ERR_SHAPE : ROPEKV_OK;
}

constexpr int32_t kMostSequences = 1 << 18;

// Shared memory of the plan of forks: three bits a sequence.
int fork_smem(int32_t batch)
{
    return 3 * ((batch + 31) / 32) * 4;
}

int64_t up16(int64_t n)
{
    return (n + 15) / 16 * 16;
}

}  // namespace

extern "C" {

int kv_accept_drafts(uint16_t* kvCache, const int32_t* kvCacheEndLens, const int32_t* accepted,
                     const int32_t* acceptedLens, int32_t* endLensOut, int32_t batch,
                     int32_t seqLen, int32_t maxAccepted, int32_t numKVHeads, int32_t headDim,
                     int32_t kvCapacity, void* stream)
{
    const AcceptArgs a = {(uint8_t*)kvCache, nullptr, nullptr, kvCacheEndLens, accepted, acceptedLens,
                          endLensOut, seqLen, maxAccepted, numKVHeads, headDim / 8, kvCapacity, 0, 0, 1};
    const int rc = check_accept(a, batch, headDim);
    if (rc != ROPEKV_OK)
        return rc;
    if (kvCapacity < 0)
        return ROPEKV_ERR_SHAPE;
    if (batch == 0)
        return ROPEKV_OK;
    if (!kvCache || !kvCacheEndLens || (!accepted && maxAccepted > 0) || !acceptedLens)
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(kvCache) || !aligned16(kvCacheEndLens) || !aligned16(accepted) ||
        !aligned16(acceptedLens) || !aligned16(endLensOut))
        return ROPEKV_ERR_MISALIGNED;
    return run_accept(a, batch, false, (cudaStream_t)stream);
}

int paged_kv_accept_drafts(void* kvCache, float* kvScales, const int32_t* pageTable,
                           const int32_t* kvLens, const int32_t* accepted,
                           const int32_t* acceptedLens, int32_t* kvLensOut, int32_t batch,
                           int32_t seqLen, int32_t maxAccepted, int32_t numKVHeads,
                           int32_t headDim, int32_t numPages, int32_t maxPagesPerSeq,
                           int32_t tokensPerPage, int32_t cacheFormat, void* stream)
{
    int rc = check_pool(headDim, numKVHeads, numPages, tokensPerPage, cacheFormat);
    if (rc == ROPEKV_OK)
        rc = check_table(batch, maxPagesPerSeq, tokensPerPage);
    if (rc != ROPEKV_OK)
        return rc;
    const bool f16 = cacheFormat == ROPEKV_CACHE_F16;
    const AcceptArgs a = {(uint8_t*)kvCache, f16 ? nullptr : kvScales, pageTable, kvLens, accepted, acceptedLens,
                          kvLensOut, seqLen, maxAccepted, numKVHeads, headDim / (f16 ? 8 : 16),
                          maxPagesPerSeq * tokensPerPage, numPages, maxPagesPerSeq, tokensPerPage};
    rc = check_accept(a, batch, headDim);
    if (rc != ROPEKV_OK)
        return rc;
    if (batch == 0)
        return ROPEKV_OK;
    if ((!kvCache && numPages > 0) || (!f16 && !kvScales && numPages > 0) || (!pageTable && maxPagesPerSeq > 0) ||
        !kvLens || (!accepted && maxAccepted > 0) || !acceptedLens)
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(kvCache) || !aligned16(kvScales) || !aligned16(pageTable) || !aligned16(kvLens) ||
        !aligned16(accepted) || !aligned16(acceptedLens) || !aligned16(kvLensOut))
        return ROPEKV_ERR_MISALIGNED;
    return run_accept(a, batch, true, (cudaStream_t)stream);
}

int paged_kv_copy_pages(void* kvCache, float* kvScales, const int32_t* srcPages,
                        const int32_t* dstPages, int32_t numCopies, int32_t numKVHeads,
                        int32_t headDim, int32_t numPages, int32_t tokensPerPage,
                        int32_t cacheFormat, void* stream)
{
    const int rc = check_pool(headDim, numKVHeads, numPages, tokensPerPage, cacheFormat);
    if (rc != ROPEKV_OK)
        return rc;
    if (numCopies < 0)
        return ROPEKV_ERR_SHAPE;
    if (numCopies == 0)
        return ROPEKV_OK;
    const bool f16 = cacheFormat == ROPEKV_CACHE_F16;
    if ((!kvCache && numPages > 0) || (!f16 && !kvScales && numPages > 0) || !srcPages || !dstPages)
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(kvCache) || !aligned16(kvScales) || !aligned16(srcPages) || !aligned16(dstPages))
        return ROPEKV_ERR_MISALIGNED;
    const int64_t vecs = (int64_t)tokensPerPage * numKVHeads * headDim / (f16 ? 8 : 16);
    const int64_t per = (vecs + kCopyUnroll - 1) / kCopyUnroll;
    const int threads = per < 256 ? (int)((per + 31) / 32 * 32) : 256;
    const int64_t chunks = (vecs + (int64_t)threads * kCopyUnroll - 1) / ((int64_t)threads * kCopyUnroll);
    if (chunks * 2 * numCopies > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    const CopyArgs a = {(uint8_t*)kvCache, f16 ? nullptr : kvScales, srcPages, dstPages, numCopies, numPages,
                        tokensPerPage, numKVHeads, (int32_t)chunks, vecs};
    return launch(copy_pages_kernel, chunks * 2 * numCopies, threads, 0, (cudaStream_t)stream, a);
}

int64_t paged_kv_fork_workspace_size(int32_t numForks, int32_t batch)
{
    if (numForks < 0 || numForks > (1 << 20) || batch < 0 || batch > kMostSequences)
        return ROPEKV_ERR_SHAPE;
    return 16 + (int64_t)sizeof(Fork) * numForks + up16(4LL * numForks);
}

int paged_kv_fork(void* kvCache, float* kvScales, int32_t* pageTable, int32_t* kvLens,
                  int32_t* refCounts, const int32_t* parents, const int32_t* children,
                  void* workspace, int64_t workspaceBytes, int32_t numForks, int32_t batch,
                  int32_t numKVHeads, int32_t headDim, int32_t numPages, int32_t maxPagesPerSeq,
                  int32_t tokensPerPage, int32_t cacheFormat, void* stream)
{
    int rc = check_pool(headDim, numKVHeads, numPages, tokensPerPage, cacheFormat);
    if (rc == ROPEKV_OK)
        rc = check_table(batch, maxPagesPerSeq, tokensPerPage);
    if (rc != ROPEKV_OK)
        return rc;
    const int64_t size = paged_kv_fork_workspace_size(numForks, batch);
    if (size < 0)
        return (int)size;
    if (numForks == 0 || batch == 0)
        return ROPEKV_OK;
    const bool f16 = cacheFormat == ROPEKV_CACHE_F16;
    if ((numPages > 0 && (!kvCache || !refCounts || (!f16 && !kvScales))) || (!pageTable && maxPagesPerSeq > 0) ||
        !kvLens || !parents || !children || !workspace)
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(kvCache) || !aligned16(kvScales) || !aligned16(pageTable) || !aligned16(kvLens) ||
        !aligned16(refCounts) || !aligned16(parents) || !aligned16(children) || !aligned16(workspace))
        return ROPEKV_ERR_MISALIGNED;
    if (workspaceBytes < size)
        return ROPEKV_ERR_CAPACITY;
    uint8_t* ws = (uint8_t*)workspace;
    ForkArgs a = {(uint8_t*)kvCache, f16 ? nullptr : kvScales, pageTable, kvLens, refCounts, parents, children,
                  (Fork*)(ws + 16), (int32_t*)ws, (int32_t*)(ws + 16 + sizeof(Fork) * (size_t)numForks), numForks, batch,
                  numPages, maxPagesPerSeq, tokensPerPage, numKVHeads, 0,
                  (int64_t)numKVHeads * headDim / (f16 ? 8 : 16)};
    const int64_t vecs = tokensPerPage * a.rowVecs, chunks = (vecs + 256 * kCopyUnroll - 1) / (256 * kCopyUnroll);
    if (chunks * numForks > 0x7FFFFFFFLL)
        return ROPEKV_ERR_SHAPE;
    a.chunks = (int32_t)chunks;
    // the limit belongs to the kernel, not to the call: always the same, as calls may overlap
    const int smem = fork_smem(batch);
    if (smem > 48 * 1024 && cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 fork_smem(kMostSequences)) != cudaSuccess)
        return ROPEKV_ERR_LAUNCH;
    rc = launch(fork_plan_kernel, 1, 1024, smem, (cudaStream_t)stream, a);
    return rc != ROPEKV_OK ? rc : launch(fork_copy_kernel, chunks * numForks, 256, 0, (cudaStream_t)stream, a);
}

int paged_kv_free(int32_t* pageTable, int32_t* kvLens, int32_t* refCounts, const int32_t* sequences,
                  const int32_t* keepLens, int32_t numSequences, int32_t batch, int32_t numPages,
                  int32_t maxPagesPerSeq, int32_t tokensPerPage, void* stream)
{
    const int rc = check_table(batch, maxPagesPerSeq, tokensPerPage);
    if (rc != ROPEKV_OK)
        return rc;
    if (numSequences < 0 || numPages < 0)
        return ROPEKV_ERR_SHAPE;
    if (numSequences == 0 || batch == 0)
        return ROPEKV_OK;
    if ((!pageTable && maxPagesPerSeq > 0) || !kvLens || (!refCounts && numPages > 0) || !sequences)
        return ROPEKV_ERR_NULL_POINTER;
    if (!aligned16(pageTable) || !aligned16(kvLens) || !aligned16(refCounts) || !aligned16(sequences) ||
        !aligned16(keepLens))
        return ROPEKV_ERR_MISALIGNED;
    const int chunks = maxPagesPerSeq > 0 ? (maxPagesPerSeq + 255) / 256 : 1;
    const FreeArgs a = {pageTable, kvLens, refCounts, sequences, keepLens, batch, numPages, maxPagesPerSeq,
                        tokensPerPage, chunks};
    const int threads = maxPagesPerSeq < 256 ? (maxPagesPerSeq + 32) / 32 * 32 : 256;
    return launch(free_kernel, (long long)chunks * numSequences, threads, 0, (cudaStream_t)stream, a);
}

}  // extern "C"
