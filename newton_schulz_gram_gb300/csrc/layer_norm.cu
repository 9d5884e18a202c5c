// Layer norm, forward: mean and variance of each row, and the scaled row.
//
// A row stays in the registers of the threads that share it: `tpr` neighbouring
// lanes for short rows (several rows a warp), a block for long ones. The mean is
// found first, then the deviations from it and their squares in one sum: the
// squares of the centred values lose nothing to cancellation, and the mean of the
// deviations, which is what rounding left of the first mean, is taken off them
// (a constant row of any size gives 0).
//
// Bound: HBM, x read and y written once.
#include <algorithm>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// Pieces a thread keeps: four of a warp's row in blocks of 256, two of a block's.
constexpr int kWarpPieces = 4, kBlockPieces = 2;

template <typename T, typename Piece, int V>
__global__ void __launch_bounds__(V == kBlockPieces ? 1024 : 256) layer_norm_kernel(NormJob j) {
    constexpr int N = Piece::kSize;
    __shared__ float2 red[2][32];
    int phase = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const int at = j.tpr <= 32 ? threadIdx.x & (j.tpr - 1) : threadIdx.x;
    const int group = j.tpr <= 32 ? threadIdx.x / j.tpr : 0;
    const int groups = blockDim.x / j.tpr;
    const float n = static_cast<float>(j.cols);
    const T* x = static_cast<const T*>(j.x);
    T* y = static_cast<T*>(j.y);
    for (long long r0 = static_cast<long long>(blockIdx.x) * groups; r0 < j.rows; r0 += static_cast<long long>(gridDim.x) * groups) {
        const long long r = r0 + group;
        const bool live = r < j.rows;
        Piece p[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned v = at + i * j.tpr;
            if (live && v < j.per_row)
                p[i].load_stream(x + r * j.ldx, v, j.cols);
            else
                p[i].clear();
        }
        float mean = 0.0f, none = 0.0f;
        if (!j.rms) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[N];
                p[i].get(f);
#pragma unroll
                for (int e = 0; e < N; ++e) mean += f[e];
            }
            row_sum2(mean, none, j.tpr, red[phase ^= 1]);
            mean /= n;
        }
        float dev = 0.0f, squares = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned v = at + i * j.tpr;
            float f[N];
            p[i].get(f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = v < j.per_row && piece_has(p[i], v, e, j.cols) ? f[e] - mean : 0.0f;
                dev += d;
                squares = fmaf(d, d, squares);
            }
        }
        row_sum2(dev, squares, j.tpr, red[phase ^= 1]);
        dev = j.rms ? 0.0f : dev / n;
        const float var = fmaxf(squares / n - dev * dev, 0.0f);
        // fmaxf drops a NaN; the sum of squares carries it.
        const float rstd = 1.0f / sqrtf((squares == squares ? var : squares) + j.eps);
        if (live && at == 0) {
            j.stats[2 * r] = mean + dev;
            j.stats[2 * r + 1] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned v = at + i * j.tpr;
            if (!live || v >= j.per_row) continue;
            float f[N];
            p[i].get(f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = ((f[e] - mean) - dev) * rstd;
            if (j.weight) {
                float w[N];
                piece_weights(p[i], j.weight, j.wf32, v, j.cols, w);
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] *= w[e];
            }
            if (j.bias) {
                float b[N];
                piece_weights(p[i], j.bias, j.wf32, v, j.cols, b);
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] += b[e];
            }
            Piece o;
            o.set(f);
            o.store(y + r * j.ldy, v, j.cols);
        }
    }
}

// Rows beyond the registers of a block: read three times, the later ones from L2.
constexpr int kLongThreads = 1024;

template <typename T, typename Piece>
__global__ void __launch_bounds__(kLongThreads) layer_norm_long_kernel(NormJob j) {
    constexpr int N = Piece::kSize;
    __shared__ float2 red[2][32];
    int phase = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const float n = static_cast<float>(j.cols);
    for (long long r = blockIdx.x; r < j.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(j.x) + r * j.ldx;
        T* y = static_cast<T*>(j.y) + r * j.ldy;
        float mean = 0.0f, none = 0.0f;
        if (!j.rms) {
            for (unsigned v = threadIdx.x; v < j.per_row; v += kLongThreads) {
                Piece p;
                p.load(x, v, j.cols);
                float f[N];
                p.get(f);
#pragma unroll
                for (int e = 0; e < N; ++e) mean += f[e];
            }
            row_sum2(mean, none, kLongThreads, red[phase ^= 1]);
            mean /= n;
        }
        float dev = 0.0f, squares = 0.0f;
        for (unsigned v = threadIdx.x; v < j.per_row; v += kLongThreads) {
            Piece p;
            p.load(x, v, j.cols);
            float f[N];
            p.get(f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = piece_has(p, v, e, j.cols) ? f[e] - mean : 0.0f;
                dev += d;
                squares = fmaf(d, d, squares);
            }
        }
        row_sum2(dev, squares, kLongThreads, red[phase ^= 1]);
        dev = j.rms ? 0.0f : dev / n;
        const float var = fmaxf(squares / n - dev * dev, 0.0f);
        const float rstd = 1.0f / sqrtf((squares == squares ? var : squares) + j.eps);
        if (threadIdx.x == 0) {
            j.stats[2 * r] = mean + dev;
            j.stats[2 * r + 1] = rstd;
        }
        for (unsigned v = threadIdx.x; v < j.per_row; v += kLongThreads) {
            Piece p;
            p.load(x, v, j.cols);
            float f[N];
            p.get(f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = ((f[e] - mean) - dev) * rstd;
            if (j.weight) {
                float w[N];
                piece_weights(p, j.weight, j.wf32, v, j.cols, w);
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] *= w[e];
            }
            if (j.bias) {
                float b[N];
                piece_weights(p, j.bias, j.wf32, v, j.cols, b);
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] += b[e];
            }
            p.set(f);
            p.store(y, v, j.cols);
        }
    }
}

}  // namespace

int launch_layer_norm(NormJob j, int num_sms, cudaStream_t s) {
    const bool vec = norm_vec(j, false);
    j.per_row = norm_pieces(j, vec);
    const int p = j.per_row;
    const bool fits = p <= kBlockPieces * 1024;
    const int V = p <= 32 ? 1 : p <= 64 || p > 32 * kWarpPieces ? kBlockPieces : kWarpPieces;
    int threads = 256;
    if (p <= 32 * kWarpPieces) {
        j.tpr = std::min(32, next_pow2(p));
    } else {
        threads = j.tpr = (p + 32 * V - 1) / (32 * V) * 32;
    }
    const long long groups = threads / (fits ? j.tpr : threads);
    const long long most = (j.rows + groups - 1) / groups;
    const unsigned blocks = static_cast<unsigned>(std::min<long long>(most, static_cast<long long>(num_sms) * std::max(1, 2048 / threads)));
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        using W = Wide<T, 16 / sizeof(T)>;
        using L = Loose<T>;
        if (!fits) {
            const unsigned b = static_cast<unsigned>(std::min<long long>(j.rows, 2LL * num_sms));
            return static_cast<int>(launch_after(vec ? layer_norm_long_kernel<T, W> : layer_norm_long_kernel<T, L>, dim3(b),
                                                 dim3(kLongThreads), 0, s, j));
        }
        auto k = vec ? (V == 1 ? layer_norm_kernel<T, W, 1> : V == 2 ? layer_norm_kernel<T, W, 2> : layer_norm_kernel<T, W, 4>)
                     : (V == 1 ? layer_norm_kernel<T, L, 1> : V == 2 ? layer_norm_kernel<T, L, 2> : layer_norm_kernel<T, L, 4>);
        return static_cast<int>(launch_after(k, dim3(blocks), dim3(threads), 0, s, j));
    });
}

}  // namespace gns
