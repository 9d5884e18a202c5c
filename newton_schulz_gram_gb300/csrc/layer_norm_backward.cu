// Layer norm, backward: with h = (x - mean) rstd and g = weight dy,
//   dx = residual + rstd (g - mean(g) - h mean(g h))   (mean(g) only where the mean was taken off)
//   dweight = sum over the rows of dy h,  dbias = sum over the rows of dy.
//
// One pass over x and dy: a thread keeps its columns from row to row and sums
// their dweight and dbias in registers, a block writes the sums of its rows, and a
// second kernel adds the blocks' in their order. Which rows a block takes follows
// from the sizes and the number of SMs alone, so results repeat.
//
// Bound: HBM, x, dy (and the residual) read and dx written once.
#include <algorithm>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// A block's sums of one piece's columns: the groups of a warp, then the warps, in
// shared memory where several rows share the block.
template <typename Piece, int N>
__device__ __forceinline__ void store_sums(float (&acc)[N], const Piece& p, const NormJob& j, unsigned v, int at, float* part,
                                           float* smem) {
    if (j.tpr <= 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        for (int m = j.tpr; m < 32; m <<= 1) {
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], m);
        }
        __syncthreads();
        if (lane < j.tpr) {
#pragma unroll
            for (int e = 0; e < N; ++e) smem[(warp * 32 + lane) * N + e] = acc[e];
        }
        __syncthreads();
        if (warp > 0 || lane >= j.tpr) return;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float sum = 0.0f;
            for (int w = 0; w < warps; ++w) sum += smem[(w * 32 + lane) * N + e];
            acc[e] = sum;
        }
    }
    if (v >= j.per_row) return;
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (piece_has(p, v, e, j.cols)) part[piece_column(p, v, e)] = acc[e];
}

// A row that a block's registers hold: up to kMostPieces pieces of each of
// kMostThreads threads. (Four pieces of 16-bit values with their sums spill 40
// registers: rows of 8193 to 16384 such columns.)
constexpr int kMostPieces = 4, kMostThreads = 512;

template <typename T, typename Piece, int V, bool SUMS>
__global__ void __launch_bounds__(kMostThreads) layer_norm_backward_kernel(NormJob j) {
    constexpr int N = Piece::kSize;
    __shared__ float2 red[2][32];
    __shared__ float smem[SUMS ? 8 * 32 * N : 1];
    int phase = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const int at = j.tpr <= 32 ? threadIdx.x & (j.tpr - 1) : threadIdx.x;
    const int group = j.tpr <= 32 ? threadIdx.x / j.tpr : 0;
    const int groups = blockDim.x / j.tpr;
    const float n = static_cast<float>(j.cols);
    const T* x = static_cast<const T*>(j.x);
    const T* dy = static_cast<const T*>(j.dy);
    const T* res = static_cast<const T*>(j.residual);
    T* dx = static_cast<T*>(j.dx);
    float dw[V][N], db[V][N];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = db[i][e] = 0.0f;
    for (long long r0 = static_cast<long long>(blockIdx.x) * groups; r0 < j.rows; r0 += static_cast<long long>(gridDim.x) * groups) {
        const long long r = r0 + group;
        const bool live = r < j.rows;
        Piece px[V], pd[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned v = at + i * j.tpr;
            if (live && v < j.per_row) {
                px[i].load_stream(x + r * j.ldx, v, j.cols);
                pd[i].load_stream(dy + r * j.lddy, v, j.cols);
            } else {
                px[i].clear();
                pd[i].clear();
            }
        }
        const float mean = live ? j.stats[2 * r] : 0.0f, rstd = live ? j.stats[2 * r + 1] : 0.0f;
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned v = at + i * j.tpr;
            float f[N], d[N], w[N];
            px[i].get(f);
            pd[i].get(d);
            if (j.weight && v < j.per_row) {
                piece_weights(px[i], j.weight, j.wf32, v, j.cols, w);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) w[e] = 1.0f;
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float h = (f[e] - mean) * rstd, g = d[e] * w[e];
                c1 += g;
                c2 = fmaf(g, h, c2);
                if (SUMS) {
                    dw[i][e] = fmaf(d[e], h, dw[i][e]);
                    db[i][e] += d[e];
                }
            }
        }
        row_sum2(c1, c2, j.tpr, red[phase ^= 1]);
        c1 = j.rms ? 0.0f : c1 / n;
        c2 /= n;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned v = at + i * j.tpr;
            if (!live || v >= j.per_row) continue;
            float f[N], d[N], w[N];
            px[i].get(f);
            pd[i].get(d);
            if (j.weight) {
                piece_weights(px[i], j.weight, j.wf32, v, j.cols, w);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) w[e] = 1.0f;
            }
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = (d[e] * w[e] - c1 - (f[e] - mean) * rstd * c2) * rstd;
            if (res) {
                Piece pr;
                pr.load_stream(res + r * j.ldr, v, j.cols);
                pr.get(d);
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] += d[e];
            }
            Piece o;
            o.set(f);
            o.store(dx + r * j.lddx, v, j.cols);
        }
    }
    if (SUMS) {
        float* part = j.part + static_cast<long long>(blockIdx.x) * j.cols;
        const long long all = static_cast<long long>(gridDim.x) * j.cols;
        const Piece p{};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            store_sums(dw[i], p, j, at + i * j.tpr, at, part, smem);
            if (j.dbias) store_sums(db[i], p, j, at + i * j.tpr, at, part + all, smem);
        }
    }
}

// Rows beyond a block's registers: the same in two passes over the row, the second
// from L2, and the columns' sums in a kernel of their own.
constexpr int kLongThreads = 512;

template <typename T, typename Piece>
__global__ void __launch_bounds__(kLongThreads) layer_norm_backward_long_kernel(NormJob j) {
    constexpr int N = Piece::kSize;
    __shared__ float2 red[2][32];
    int phase = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const float n = static_cast<float>(j.cols);
    for (long long r = blockIdx.x; r < j.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(j.x) + r * j.ldx;
        const T* dy = static_cast<const T*>(j.dy) + r * j.lddy;
        const float mean = j.stats[2 * r], rstd = j.stats[2 * r + 1];
        float c1 = 0.0f, c2 = 0.0f;
        for (int pass = 0; pass < 2; ++pass) {
            for (unsigned v = threadIdx.x; v < j.per_row; v += kLongThreads) {
                Piece px, pd;
                px.load(x, v, j.cols);
                pd.load(dy, v, j.cols);
                float f[N], d[N], w[N];
                px.get(f);
                pd.get(d);
                if (j.weight) {
                    piece_weights(px, j.weight, j.wf32, v, j.cols, w);
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e) w[e] = 1.0f;
                }
                if (pass == 0) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float g = d[e] * w[e];
                        c1 += g;
                        c2 = fmaf(g, (f[e] - mean) * rstd, c2);
                    }
                    continue;
                }
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] = (d[e] * w[e] - c1 - (f[e] - mean) * rstd * c2) * rstd;
                if (j.residual) {
                    pd.load_stream(static_cast<const T*>(j.residual) + r * j.ldr, v, j.cols);
                    pd.get(d);
#pragma unroll
                    for (int e = 0; e < N; ++e) f[e] += d[e];
                }
                px.set(f);
                px.store(static_cast<T*>(j.dx) + r * j.lddx, v, j.cols);
            }
            if (pass == 0) {
                row_sum2(c1, c2, kLongThreads, red[phase ^= 1]);
                c1 = j.rms ? 0.0f : c1 / n;
                c2 /= n;
            }
        }
    }
}

// A thread owns a piece of the columns, a block's part of the grid's y a run of rows.
template <typename T, typename Piece>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(NormJob j) {
    constexpr int N = Piece::kSize;
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned v = blockIdx.x * 256 + threadIdx.x;
    if (v >= j.per_row) return;
    float dw[N], db[N];
#pragma unroll
    for (int e = 0; e < N; ++e) dw[e] = db[e] = 0.0f;
    for (long long r = blockIdx.y; r < j.rows; r += gridDim.y) {
        Piece px, pd;
        px.load_stream(static_cast<const T*>(j.x) + r * j.ldx, v, j.cols);
        pd.load_stream(static_cast<const T*>(j.dy) + r * j.lddy, v, j.cols);
        const float mean = j.stats[2 * r], rstd = j.stats[2 * r + 1];
        float f[N], d[N];
        px.get(f);
        pd.get(d);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            dw[e] = fmaf(d[e], (f[e] - mean) * rstd, dw[e]);
            db[e] += d[e];
        }
    }
    const Piece p{};
    float* part = j.part + static_cast<long long>(blockIdx.y) * j.cols;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (!piece_has(p, v, e, j.cols)) continue;
        part[piece_column(p, v, e)] = dw[e];
        if (j.dbias) part[static_cast<long long>(gridDim.y) * j.cols + piece_column(p, v, e)] = db[e];
    }
}

// The blocks' sums of 32 columns, each warp every 32nd block's, then the warps'.
__global__ void __launch_bounds__(1024) layer_norm_join_kernel(const float* part, int parts, int cols, void* dweight,
                                                               void* dbias, int dtype) {
    __shared__ float sums[32][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    void* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    part += static_cast<long long>(blockIdx.y) * parts * cols;
    float sum = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int b = warp; b < parts; b += 32) sum += part[static_cast<long long>(b) * cols + c];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    sum = sums[lane][warp];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    const int o = blockIdx.x * 32 + warp;
    if (lane == 0 && o < cols) {
        by_dtype_device(dtype, [&](auto t) {
            using W = decltype(t);
            static_cast<W*>(out)[o] = from_f32<W>(sum);
        });
    }
}

struct Shape {
    bool vec, fits;
    int V, threads, tpr, per_row;
    unsigned blocks, strips;  // strips: the column kernel's
    int parts;
};

Shape shape_of(const NormJob& j, int num_sms) {
    Shape c{};
    c.vec = norm_vec(j, true);
    const int p = c.per_row = norm_pieces(j, c.vec);
    c.V = p <= 32 ? 1 : p <= 1024 ? 2 : kMostPieces;
    c.fits = p <= kMostPieces * kMostThreads;
    if (!c.fits) {
        c.blocks = static_cast<unsigned>(std::min<long long>(j.rows, 4LL * num_sms));
        c.strips = static_cast<unsigned>((p + 255) / 256);
        c.parts = static_cast<int>(std::min<long long>(j.rows, std::max(1u, 8u * num_sms / c.strips)));
        return c;
    }
    if (p <= 32) {
        c.threads = 256;
        c.tpr = next_pow2(p);
    } else if (p <= 64) {
        c.threads = 256;
        c.tpr = 32;
    } else {
        c.threads = c.tpr = (p + 32 * c.V - 1) / (32 * c.V) * 32;
    }
    const long long groups = c.threads / c.tpr;
    c.blocks = static_cast<unsigned>(std::min<long long>((j.rows + groups - 1) / groups,
                                                         static_cast<long long>(num_sms) * std::max(1, 768 / c.threads)));
    c.parts = static_cast<int>(c.blocks);
    return c;
}

}  // namespace

size_t norm_backward_scratch(const NormJob& j, int num_sms) {
    if (!j.dweight && !j.dbias) return 0;
    return sizeof(float) * 2 * static_cast<size_t>(shape_of(j, num_sms).parts) * j.cols;
}

int launch_layer_norm_backward(NormJob j, int num_sms, cudaStream_t s) {
    const Shape c = shape_of(j, num_sms);
    j.per_row = c.per_row;
    j.tpr = c.tpr;
    const bool sums = j.dweight || j.dbias;
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        using W = Wide<T, 16 / sizeof(T)>;
        using L = Loose<T>;
        if (!c.fits)
            return static_cast<int>(launch_after(c.vec ? layer_norm_backward_long_kernel<T, W> : layer_norm_backward_long_kernel<T, L>,
                                                 dim3(c.blocks), dim3(kLongThreads), 0, s, j));
        auto run = [&](auto k) { return static_cast<int>(launch_after(k, dim3(c.blocks), dim3(c.threads), 0, s, j)); };
        if (sums)
            return c.vec ? run(c.V == 1 ? layer_norm_backward_kernel<T, W, 1, true> : c.V == 2 ? layer_norm_backward_kernel<T, W, 2, true> : layer_norm_backward_kernel<T, W, 4, true>)
                         : run(c.V == 1 ? layer_norm_backward_kernel<T, L, 1, true> : c.V == 2 ? layer_norm_backward_kernel<T, L, 2, true> : layer_norm_backward_kernel<T, L, 4, true>);
        return c.vec ? run(c.V == 1 ? layer_norm_backward_kernel<T, W, 1, false> : c.V == 2 ? layer_norm_backward_kernel<T, W, 2, false> : layer_norm_backward_kernel<T, W, 4, false>)
                     : run(c.V == 1 ? layer_norm_backward_kernel<T, L, 1, false> : c.V == 2 ? layer_norm_backward_kernel<T, L, 2, false> : layer_norm_backward_kernel<T, L, 4, false>);
    });
}

bool layer_norm_columns_apart(const NormJob& j) { return !shape_of(j, 1).fits; }

int launch_layer_norm_columns(NormJob j, int num_sms, cudaStream_t s) {
    const Shape c = shape_of(j, num_sms);
    j.per_row = c.per_row;
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return static_cast<int>(launch_after(c.vec ? layer_norm_columns_kernel<T, Wide<T, 16 / sizeof(T)>> : layer_norm_columns_kernel<T, Loose<T>>,
                                             dim3(c.strips, static_cast<unsigned>(c.parts)), dim3(256), 0, s, j));
    });
}

int launch_layer_norm_join(NormJob j, int num_sms, cudaStream_t s) {
    const Shape c = shape_of(j, num_sms);
    const int dtype = j.wf32 ? static_cast<int>(GNS_FP32) : j.dtype;
    return static_cast<int>(launch_after(layer_norm_join_kernel, dim3(static_cast<unsigned>((j.cols + 31) / 32), 2), dim3(1024), 0, s,
                                         static_cast<const float*>(j.part), c.parts, j.cols, j.dweight, j.dbias, dtype));
}

}  // namespace gns
