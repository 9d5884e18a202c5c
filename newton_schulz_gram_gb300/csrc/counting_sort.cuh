// A stable counting sort by digits of 0 .. G, without atomics: a function of the
// digits alone.
//
// A warp owns a run of consecutive slots and walks it 32 at a time:
// __match_any_sync groups the lanes of one digit, a lane's rank in its group
// is the popcount of the lanes before it, and the warp's running count of
// the digit (its own column of shared memory, so no atomics) gives the rest.
// Up to `alone` slots a single block does it all. Beyond, a first kernel
// stores each block's counts and the second one's blocks sum, each for
// itself, the counts of all blocks and of those before it: nblocks * (G + 1)
// loads that stay in L2, which is less than the round trip of a third launch
// for up to kMaxBlocks blocks.
//
// A source says what is sorted: key(s), read for slot s, and its digit(key); begin(),
// called by a block's threads before its slots; note(key), called for every slot by each
// kernel; value(s), read for slot s and handed with it to place(s, key, value, at), called
// once for every slot with its place; start(d, at), called once for every digit with the
// place of its first slot; extra(b), called by the b-th of the blocks that a launch has
// beside the sort's, which is bound by latency and leaves most of the GPU free for them.
#pragma once

#include <algorithm>

#include "blockops.cuh"
#include "ptx.cuh"

namespace gns {

constexpr int kSortWarps = 16;
constexpr int kSortThreads = 32 * kSortWarps;
constexpr int kMaxBlocks = 152;
constexpr int kMaxDigit = 1024;

// How n slots are shared out: one block up to `alone` of them, else blocks of at least `tile`.
struct SortPlan {
    long long n;
    int G;
    long long alone, tile;
};

// Dynamic shared memory that a launch gets without asking: 48 KB less what the kernels and
// their sources have statically, 64 bytes and the embedding's 4096.
constexpr size_t kSortShared = 40 << 10;

inline size_t sort_smem(int G) { return sizeof(int) * static_cast<size_t>(G + 1) * (kSortWarps + 1); }

inline long long sort_blocks(const SortPlan& p) {
    if (p.n <= p.alone) return 1;
    return std::min<long long>(kMaxBlocks, (p.n + p.tile - 1) / p.tile);
}

// Slots per block, a multiple of 32 per warp.
inline long long sort_span(const SortPlan& p) {
    const long long per = (p.n + sort_blocks(p) - 1) / sort_blocks(p);
    return (per + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// Bytes of the blocks' counts, 0 where one block does it all.
inline size_t sort_scratch(const SortPlan& p) {
    const long long b = sort_blocks(p);
    return b > 1 ? sizeof(int) * static_cast<size_t>(b) * (p.G + 1) : 0;
}

constexpr int kSortTurns = 4;  // times 32 slots whose loads a warp issues together

// The keys of slots s0 .., -1 from `end` on.
template <typename Source>
__device__ __forceinline__ void load_keys(const Source& src, long long s0, long long end, int lane, int (&key)[kSortTurns]) {
#pragma unroll
    for (int u = 0; u < kSortTurns; ++u) {
        const long long s = s0 + 32 * u + lane;
        key[u] = s < end ? src.key(s) : -1;
    }
}

// Counts of this warp's run of slots into its column cnt[0 .. G].
template <typename Source>
__device__ __forceinline__ void count_run(const Source& src, long long beg, long long end, int* cnt, int lane) {
    for (long long s0 = beg; s0 < end; s0 += 32 * kSortTurns) {
        int key[kSortTurns];
        load_keys(src, s0, end, lane, key);
#pragma unroll
        for (int u = 0; u < kSortTurns; ++u) {
            if (s0 + 32 * u >= end) break;
            const int e = key[u] < 0 ? -1 : src.digit(key[u]);
            const unsigned peers = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && (peers & ((1u << lane) - 1)) == 0) cnt[e] += __popc(peers);
            if (e >= 0) src.note(key[u]);
            __syncwarp();
        }
    }
}

template <typename Source>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(Source src, long long n, int G, long long span,
                                                                  int blocks, int* hist) {
    extern __shared__ int smem[];
    if (static_cast<int>(blockIdx.x) >= blocks) {
        grid_dependency_wait();
        grid_launch_dependents();
        src.extra(blockIdx.x - blocks);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (G + 1) * kSortWarps; i += kSortThreads) smem[i] = 0;
    src.begin();
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    const long long run = span / kSortWarps;
    const long long beg = blockIdx.x * span + warp * run;
    count_run(src, beg, min(beg + run, n), smem + warp * (G + 1), lane);
    __syncthreads();
    for (int e = threadIdx.x; e <= G; e += kSortThreads) {
        int c = 0;
        for (int w = 0; w < kSortWarps; ++w) c += smem[w * (G + 1) + e];
        hist[static_cast<long long>(blockIdx.x) * (G + 1) + e] = c;
    }
}

// hist null: the grid is one block and its own counts are all there are.
template <typename Source>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(Source src, long long n, int G, long long span,
                                                                  int blocks, const int* hist) {
    extern __shared__ int smem[];
    __shared__ int warp_sum[kSortWarps];
    if (static_cast<int>(blockIdx.x) >= blocks) {
        grid_dependency_wait();
        grid_launch_dependents();
        src.extra(blockIdx.x - blocks);
        return;
    }
    int* first = smem + (G + 1) * kSortWarps;  // first place of this block's slots of each digit
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (G + 1) * kSortWarps; i += kSortThreads) smem[i] = 0;
    src.begin();
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    const long long run = span / kSortWarps;
    const long long beg = blockIdx.x * span + warp * run;
    const long long end = min(beg + run, n);
    int* cnt = smem + warp * (G + 1);
    count_run(src, beg, end, cnt, lane);
    __syncthreads();

    // Totals of all blocks, scanned over the digits: thread t owns digits
    // t * per .. t * per + per - 1.
    constexpr int kPer = (kMaxDigit + 1 + kSortThreads - 1) / kSortThreads;
    const int per = (G + kSortThreads) / kSortThreads;  // ceil((G + 1) / threads)
    int total[kPer], before[kPer];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * per + i;
        total[i] = before[i] = 0;
        if (i >= per || e > G) continue;
        if (hist) {
#pragma unroll 8
            for (int b = 0; b < blocks; ++b) {
                const int c = hist[static_cast<long long>(b) * (G + 1) + e];
                total[i] += c;
                if (b < static_cast<int>(blockIdx.x)) before[i] += c;
            }
        } else {
            for (int w = 0; w < kSortWarps; ++w) total[i] += smem[w * (G + 1) + e];
        }
        mine += total[i];
    }
    int scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int start = scan - mine;
    for (int w = 0; w < warp; ++w) start += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * per + i;
        if (i >= per || e > G) continue;
        first[e] = start + before[i];
        if (blockIdx.x == 0) src.start(e, start);
        start += total[i];
    }
    __syncthreads();
    // Each warp's first place per digit: the block's, plus the warps before it.
    for (int e = threadIdx.x; e <= G; e += kSortThreads) {
        int at = first[e];
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = smem[w * (G + 1) + e];
            smem[w * (G + 1) + e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (long long s0 = beg; s0 < end; s0 += 32 * kSortTurns) {
        int key[kSortTurns], value[kSortTurns];
        load_keys(src, s0, end, lane, key);
#pragma unroll
        for (int u = 0; u < kSortTurns; ++u) {
            const long long s = s0 + 32 * u + lane;
            value[u] = s < end ? src.value(s) : 0;
        }
#pragma unroll
        for (int u = 0; u < kSortTurns; ++u) {
            if (s0 + 32 * u >= end) break;
            const int e = key[u] < 0 ? -1 : src.digit(key[u]);
            const unsigned peers = __match_any_sync(0xffffffffu, e);
            const int rank = __popc(peers & ((1u << lane) - 1));
            if (e >= 0) src.place(s0 + 32 * u + lane, key[u], value[u], cnt[e] + rank);
            __syncwarp();
            if (e >= 0 && rank == 0) cnt[e] += __popc(peers);
            __syncwarp();
        }
    }
}

template <typename... KArgs, typename... Args>
int sort_step(void (*kernel)(KArgs...), const SortPlan& p, unsigned extra, cudaStream_t s, Args... args) {
    const size_t smem = sort_smem(p.G);
    if (smem > kSortShared) {
        // The same for every call: another thread's call must not lower it before this launch.
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sort_smem(kMaxDigit)));
        if (e != cudaSuccess) return e;
    }
    return launch_after(kernel, dim3(static_cast<unsigned>(sort_blocks(p)) + extra), dim3(kSortThreads), smem, s, args...);
}

// The two kernels; the first is left out where sort_scratch() is 0 (hist null).
template <typename Source>
int launch_sort_count(const Source& src, const SortPlan& p, int* hist, cudaStream_t s, unsigned extra = 0) {
    return sort_step(sort_count_kernel<Source>, p, extra, s, src, p.n, p.G, sort_span(p), static_cast<int>(sort_blocks(p)), hist);
}

template <typename Source>
int launch_sort_place(const Source& src, const SortPlan& p, const int* hist, cudaStream_t s, unsigned extra = 0) {
    return sort_step(sort_place_kernel<Source>, p, extra, s, src, p.n, p.G, sort_span(p), static_cast<int>(sort_blocks(p)), hist);
}

}  // namespace gns
