// Routing of tokens to experts and back: a stable counting sort of the slots
// by expert, the copy of each token's row to its places, the weighted sum of
// a token's rows, and the gradients of both.
//
// Everything is a function of the inputs alone: the sort (counting_sort.cuh) ranks
// slots by counting (no atomics), a token's rows are summed in slot order in fp32 and
// rounded once, and the weights' gradients are summed in a fixed order.
//
// Bound: HBM for the moves, a token's row once and its topk rows once each way.
// 16384 tokens of 2048 bf16 values, 8 of 256 experts: gather 91 us (6.7 TB/s),
// combine 103 (5.9), its gradient 180 (6.3), the gather's gradient 96 (6.3); the
// sort, latency, 14. One token: 2 to 3 us each.
#include <algorithm>

#include "blockops.cuh"
#include "counting_sort.cuh"
#include "moe.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// ------------------------------------------------------------------ the sort

// The slots by expert; ids outside 0 .. G - 1 have digit G.
template <typename I>
struct ExpertSlots {
    const I* ids;
    int G;
    int *offsets, *rows, *slots;
    __device__ __forceinline__ int key(long long s) const {
        const I v = ids[s];
        return v >= 0 && v < static_cast<I>(G) ? static_cast<int>(v) : G;
    }
    __device__ __forceinline__ int digit(int key) const { return key; }
    __device__ __forceinline__ int value(long long) const { return 0; }
    __device__ __forceinline__ void begin() const {}
    __device__ __forceinline__ void note(int) const {}
    __device__ __forceinline__ void extra(unsigned) const {}
    __device__ __forceinline__ void place(long long s, int, int, int at) const {
        rows[s] = at;
        slots[at] = static_cast<int>(s);
    }
    __device__ __forceinline__ void start(int e, int at) const { offsets[e] = at; }  // offsets[G]: the slots with an expert
};

SortPlan plan_of(long long n, int G) { return {n, G, 4096, 2048}; }

template <typename I>
ExpertSlots<I> slots_of(const SortJob& j) {
    return {static_cast<const I*>(j.ids), j.G, j.offsets, j.rows, j.slots};
}

// --------------------------------------------------------- moves over tokens
//
// All three walk the tokens, not the sorted rows: a token's own row is read
// (or written) once and stays in registers while its topk places are visited,
// so HBM sees each byte once. A thread owns one 16-byte piece of a token's
// row and issues the loads of up to kJ places before it uses the first. Where
// rows are not 16-byte aligned a piece is kLoose elements 32 apart, the
// neighbouring lanes' next to them: single accesses, but whole lines per warp
// and the piece's bookkeeping shared (4093 tokens of 1021 fp32 values, 3
// places each: single elements took 18, 31, 33 and 27 us for gather, combine, its gradient and
// the gather's, pieces 9, 12, 22 and 10).

constexpr int kThreads = 256;
constexpr int kJ = 8;  // places handled together

struct Walk {
    unsigned long long pieces;  // tokens * per_row
    unsigned per_row;           // pieces of a row
    int topk, H;
    const int* offsets_end;     // &offsets[G]
    const int* rows;
};

__device__ __forceinline__ void token_piece(const Walk& w, unsigned long long i, int& t, unsigned& v) {
    if (w.pieces <= 0xffffffffULL) {
        const unsigned q = static_cast<unsigned>(i) / w.per_row;
        t = static_cast<int>(q);
        v = static_cast<unsigned>(i) - q * w.per_row;
    } else {
        const unsigned long long q = i / w.per_row;
        t = static_cast<int>(q);
        v = static_cast<unsigned>(i - q * w.per_row);
    }
}

template <typename T, typename Piece>
__global__ void __launch_bounds__(kThreads) moe_gather_kernel(Walk w, const T* x, long long ldx, T* y, long long ldy) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int live = *w.offsets_end;
    const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * kThreads;
    for (unsigned long long i = static_cast<unsigned long long>(blockIdx.x) * kThreads + threadIdx.x; i < w.pieces;
         i += step) {
        int t;
        unsigned v;
        token_piece(w, i, t, v);
        Piece p, zero;
        p.load(x + t * ldx, v, w.H);
        zero.clear();
        const int* at = w.rows + static_cast<long long>(t) * w.topk;
        for (int j = 0; j < w.topk; ++j) {
            const int r = at[j];
            (r < live ? p : zero).store(y + r * ldy, v, w.H);
        }
    }
}

template <typename T, typename Piece, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(Walk w, const T* y, long long ldy, const float* weights,
                                                               T* out, long long ldo) {
    constexpr int N = Piece::kSize;
    grid_dependency_wait();
    grid_launch_dependents();
    const int live = *w.offsets_end;
    const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * kThreads;
    for (unsigned long long i = static_cast<unsigned long long>(blockIdx.x) * kThreads + threadIdx.x; i < w.pieces;
         i += step) {
        int t;
        unsigned v;
        token_piece(w, i, t, v);
        const long long s0 = static_cast<long long>(t) * w.topk;
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        for (int j0 = 0; j0 < w.topk; j0 += kJ) {
            int r[kJ];
            Piece p[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) r[j] = j0 + j < w.topk ? w.rows[s0 + j0 + j] : 0x7fffffff;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
                if (r[j] < live) p[j].load_stream(y + r[j] * ldy, v, w.H);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                if (r[j] < live) {
                    float f[N];
                    p[j].get(f);
                    const float g = WEIGHTS ? weights[s0 + j0 + j] : 1.0f;
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] = fmaf(g, f[e], acc[e]);
                }
            }
        }
        Piece o;
        o.set(acc);
        o.store(out + t * ldo, v, w.H);
    }
}

// WPT warps share a token: one when there are tokens enough to fill the
// machine, a whole block otherwise.
template <typename T, typename Piece, int WPT, bool DOTS>
__global__ void __launch_bounds__(kThreads) moe_combine_backward_kernel(Walk w, int tokens, const T* dout,
                                                                        long long lddo, const T* y, long long ldy,
                                                                        const float* weights, T* dy, long long lddy,
                                                                        float* dweights) {
    constexpr int kWarps = kThreads / 32;
    constexpr int N = Piece::kSize;
    __shared__ float part[kJ][kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int live = *w.offsets_end;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = WPT == 1 ? static_cast<int>(blockIdx.x) * kWarps + warp : static_cast<int>(blockIdx.x);
    if (WPT == 1 && t >= tokens) return;
    const long long s0 = static_cast<long long>(t) * w.topk;
    for (int j0 = 0; j0 < w.topk; j0 += kJ) {
        int r[kJ];
        float g[kJ], dot[kJ];
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const bool in = j0 + j < w.topk;
            r[j] = in ? w.rows[s0 + j0 + j] : -1;
            g[j] = in ? weights[s0 + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (unsigned v = WPT == 1 ? lane : threadIdx.x; v < w.per_row; v += 32 * WPT) {
            Piece pd, py[kJ];
            pd.load(dout + t * lddo, v, w.H);
            if (DOTS) {
#pragma unroll
                for (int j = 0; j < kJ; ++j)
                    if (r[j] >= 0 && r[j] < live) py[j].load_stream(y + r[j] * ldy, v, w.H);
            }
            float d[N];
            pd.get(d);
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                if (r[j] < 0) continue;
                Piece o;
                if (r[j] < live) {
                    float f[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) f[e] = g[j] * d[e];
                    o.set(f);
                    if (DOTS) {
                        py[j].get(f);
#pragma unroll
                        for (int e = 0; e < N; ++e) dot[j] = fmaf(d[e], f[e], dot[j]);
                    }
                } else {
                    o.clear();
                }
                o.store(dy + r[j] * lddy, v, w.H);
            }
        }
        if (DOTS) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], m);
            }
            if (WPT == 1) {
#pragma unroll
                for (int j = 0; j < kJ; ++j)
                    if (lane == j && j0 + j < w.topk) dweights[s0 + j0 + j] = dot[j];
            } else {
#pragma unroll
                for (int j = 0; j < kJ; ++j)
                    if (lane == 0) part[j][warp] = dot[j];
                __syncthreads();
                if (threadIdx.x < kJ && j0 + threadIdx.x < w.topk) {
                    float sum = 0.0f;
                    for (int k = 0; k < kWarps; ++k) sum += part[threadIdx.x][k];
                    dweights[s0 + j0 + threadIdx.x] = sum;
                }
                __syncthreads();
            }
        }
    }
}

Walk make_walk(const RouteJob& j, bool vec) {
    Walk w;
    const int n = 16 / elem_bytes(j.dtype), loose = 32 * kLoose;
    w.per_row = static_cast<unsigned>(vec ? j.H / n : (j.H + loose - 1) / loose * 32);
    w.H = j.H;
    w.pieces = static_cast<unsigned long long>(j.tokens) * w.per_row;
    w.topk = j.topk;
    w.offsets_end = j.offsets + j.G;
    w.rows = j.rows;
    return w;
}

dim3 walk_grid(const Walk& w) {
    const unsigned long long b = (w.pieces + kThreads - 1) / kThreads;
    return dim3(static_cast<unsigned>(std::min<unsigned long long>(b, 0x7fffffffULL)));
}

}  // namespace

size_t moe_sort_scratch(long long n, int G) { return sort_scratch(plan_of(n, G)); }

int launch_moe_count(const SortJob& j, cudaStream_t s) {
    return j.id_bytes == 8 ? launch_sort_count(slots_of<long long>(j), plan_of(j.n, j.G), j.hist, s)
                           : launch_sort_count(slots_of<int>(j), plan_of(j.n, j.G), j.hist, s);
}

int launch_moe_place(const SortJob& j, cudaStream_t s) {
    return j.id_bytes == 8 ? launch_sort_place(slots_of<long long>(j), plan_of(j.n, j.G), j.hist, s)
                           : launch_sort_place(slots_of<int>(j), plan_of(j.n, j.G), j.hist, s);
}

int launch_moe_gather(const RouteJob& j, const void* x, long long ldx, void* y, long long ldy, cudaStream_t s) {
    const int es = elem_bytes(j.dtype), n = 16 / es;
    const bool vec = j.H % n == 0 && rows_aligned(x, ldx, j.tokens, es) &&
                     rows_aligned(y, ldy, static_cast<long long>(j.tokens) * j.topk, es);
    const Walk w = make_walk(j, vec);
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        auto k = vec ? moe_gather_kernel<T, Wide<T, 16 / sizeof(T)>> : moe_gather_kernel<T, Loose<T>>;
        return static_cast<int>(launch_after(k, walk_grid(w), dim3(kThreads), 0, s, w, static_cast<const T*>(x), ldx,
                                             static_cast<T*>(y), ldy));
    });
}

int launch_moe_combine(const RouteJob& j, const void* y, long long ldy, const float* weights, void* out, long long ldo,
                       cudaStream_t s) {
    const int es = elem_bytes(j.dtype), n = 16 / es;
    const bool vec = j.H % n == 0 && rows_aligned(y, ldy, static_cast<long long>(j.tokens) * j.topk, es) &&
                     rows_aligned(out, ldo, j.tokens, es);
    const Walk w = make_walk(j, vec);
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        using W = Wide<T, 16 / sizeof(T)>;
        using L = Loose<T>;
        auto k = weights ? (vec ? moe_combine_kernel<T, W, true> : moe_combine_kernel<T, L, true>)
                         : (vec ? moe_combine_kernel<T, W, false> : moe_combine_kernel<T, L, false>);
        return static_cast<int>(launch_after(k, walk_grid(w), dim3(kThreads), 0, s, w, static_cast<const T*>(y), ldy,
                                             weights, static_cast<T*>(out), ldo));
    });
}

int launch_moe_combine_backward(const RouteJob& j, const void* dout, long long lddo, const void* y, long long ldy,
                                const float* weights, void* dy, long long lddy, float* dweights, cudaStream_t s) {
    const int es = elem_bytes(j.dtype), n = 16 / es;
    const long long slots = static_cast<long long>(j.tokens) * j.topk;
    const bool vec = j.H % n == 0 && rows_aligned(dout, lddo, j.tokens, es) && rows_aligned(dy, lddy, slots, es) &&
                     (!dweights || rows_aligned(y, ldy, slots, es));
    const Walk w = make_walk(j, vec);
    constexpr int kWarps = kThreads / 32;
    const bool wide = j.tokens < 152 * kWarps;  // fewer tokens than one round of warps: a block per token
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        auto run = [&](auto kernel) {
            const unsigned blocks = static_cast<unsigned>(wide ? j.tokens : (j.tokens + kWarps - 1) / kWarps);
            return static_cast<int>(launch_after(kernel, dim3(blocks), dim3(kThreads), 0, s, w, j.tokens,
                                                 static_cast<const T*>(dout), lddo, static_cast<const T*>(y), ldy,
                                                 weights, static_cast<T*>(dy), lddy, dweights));
        };
        using W = Wide<T, 16 / sizeof(T)>;
        using L = Loose<T>;
        if (dweights)
            return vec ? run(wide ? moe_combine_backward_kernel<T, W, kWarps, true> : moe_combine_backward_kernel<T, W, 1, true>)
                       : run(wide ? moe_combine_backward_kernel<T, L, kWarps, true> : moe_combine_backward_kernel<T, L, 1, true>);
        return vec ? run(wide ? moe_combine_backward_kernel<T, W, kWarps, false> : moe_combine_backward_kernel<T, W, 1, false>)
                   : run(wide ? moe_combine_backward_kernel<T, L, kWarps, false> : moe_combine_backward_kernel<T, L, 1, false>);
    });
}

}  // namespace gns
