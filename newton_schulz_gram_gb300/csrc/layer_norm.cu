// Layer norm, forward: mean and variance of each row, and the scaled row.
//
// The mean is found first, then the deviations from it and their squares in one sum:
// the squares of the centred values lose nothing to cancellation, and the mean of the
// deviations, which is what rounding left of the first mean, is taken off them (a
// constant row of any size gives 0, and 4096 +- 1 in fp32 keeps its digits).
//
// Bound: HBM, x read and y written once; but the instructions of a row's 4096 values and
// its two sums take about as long. Rows go through shared memory ahead of their use, as
// 16-byte pieces or, unaligned, as the words that hold them; rows beyond that are read
// three times. 16384 x 4096 bf16 with fp32 weights: 52 us (5.1 TB/s; issue slots 65%
// busy with 16 warps a processor: 24, by one row at a time instead of two, took 53);
// 262144 x 128: 20 (6.6); 4096 x 14336 by two CTAs a row: 69 (3.4); 65536 x 257: 24;
// one row: 2.4 (from registers alone 2.9; 304 rows 2.9 and 5.0).
#include <algorithm>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// From the mean of the squared deviations and of the deviations. fmaxf drops a NaN;
// the squares carry it.
__device__ __forceinline__ float norm_rstd(float squares, float dev, float eps) {
    const float var = fmaxf(squares - dev * dev, 0.0f);
    return rsqrtf((squares == squares ? var : squares) + eps);
}

// ------------------------------------------------------------- aligned rows
//
// A thread keeps its columns, and their weights, from row to row: read for every row,
// 4096 fp32 weights and biases are four times the row and were what a warp a row was
// bound by (72 us for 16384 x 4096, 92 a block a row). It copies its pieces of rows to
// come to shared memory (cp.async) while it works on R rows in registers, so a copy
// needs no barrier, and the R rows' sums share a reduction. The ring lies on a 128-byte
// boundary: 16 bytes off cost 20%. FULL: every thread has all its pieces.
//
// CLUSTER: rows of more columns than a CTA's registers have weights for are shared by the
// CTAs of a cluster, which exchange the sums.

template <typename T, int V, bool FULL, bool CLUSTER>
__global__ void __launch_bounds__(kRingThreads) layer_norm_ring_kernel(NormJob j) {
    constexpr int N = 16 / sizeof(T), P = N / 2, R = 2;
    extern __shared__ __align__(128) uint4 ring[];  // [stage][row][piece][thread]
    __shared__ __align__(128) RowSums<2 * R> red;
    int use = 0;
    bool dead = false;
    if (CLUSTER) {
        if (threadIdx.x < 2) mbar_init(smem_u32(&red.full[threadIdx.x]), 1);
        fence_mbar_init();
        cluster_sync();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const int at = j.tpr <= 32 ? threadIdx.x & (j.tpr - 1) : threadIdx.x;
    const int group = j.tpr <= 32 ? threadIdx.x / j.tpr : 0;
    const int groups = blockDim.x / j.tpr, threads = blockDim.x;
    const int rank = CLUSTER ? cluster_ctarank() : 0;
    const int piece = rank * j.per_cta + at, pieces = min(j.per_row, (rank + 1) * j.per_cta);  // this thread's first, the CTA's end
    const unsigned cluster = CLUSTER ? blockIdx.x / j.ctas : blockIdx.x, clusters = CLUSTER ? gridDim.x / j.ctas : gridDim.x;
    const float inv = 1.0f / static_cast<float>(j.cols);
    const unsigned rows = static_cast<unsigned>(j.rows), batch = groups * R, step = clusters * batch;
    const unsigned first = cluster * batch + group;
    const T* x = static_cast<const T*>(j.x) + first * j.ldx + piece * N;  // of the rows fetched next
    T* y = static_cast<T*>(j.y) + first * j.ldy + piece * N;
    const long long x_step = step * j.ldx, y_step = step * j.ldy, x_row = groups * j.ldx, y_row = groups * j.ldy;
    const int apart = j.tpr * N;  // from one piece to the next
    const uint4* mine = ring + threadIdx.x;
    const uint32_t slots = smem_u32(mine);
    auto has = [&](int i) { return FULL || piece + i * j.tpr < pieces; };
    unsigned ahead = first;
    auto fetch = [&](int stage) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (ahead + r * groups >= rows) break;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (has(i)) copy16(slots + 16 * ((stage * R + r) * V + i) * threads, x + r * x_row + i * apart);
        }
        copies_commit();
        x += x_step;
        ahead += step;
    };
    float2 w[V][P], b[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[N];
        const Wide<T, N> p{};
#pragma unroll
        for (int e = 0; e < P; ++e) w[i][e] = both(1.0f), b[i][e] = both(0.0f);
        if (j.weight && has(i)) {
            piece_weights(p, j.weight, j.wf32, piece + i * j.tpr, j.cols, f);
#pragma unroll
            for (int e = 0; e < P; ++e) w[i][e] = make_float2(f[2 * e], f[2 * e + 1]);
        }
        if (j.bias && has(i)) {
            piece_weights(p, j.bias, j.wf32, piece + i * j.tpr, j.cols, f);
#pragma unroll
            for (int e = 0; e < P; ++e) b[i][e] = make_float2(f[2 * e], f[2 * e + 1]);
        }
    }
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k);
    int stage = 0;
    for (unsigned row = first; row - group < rows; row += step, y += y_step) {
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        copies_wait<kStages - 1>();
        float2 f[R][V][P];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (has(i) && row + r * groups < rows) v = mine[((stage * R + r) * V + i) * threads];
                unpack<T, N>(v, f[r][i]);
            }
        float mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = 0.0f;
        if (!j.rms) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 sum = both(0.0f);
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < P; ++e) sum = add2(sum, f[r][i][e]);
                mean[r] = sum.x + sum.y;
            }
            row_sums<R, CLUSTER>(mean, j, red, use, dead);
        }
        float c[2 * R];  // sums of the deviations and of their squares
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv;
            float2 dev = both(0.0f), squares = both(0.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!has(i)) continue;
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    f[r][i][e] = add2(f[r][i][e], both(-mean[r]));
                    dev = add2(dev, f[r][i][e]);
                    squares = fma2(f[r][i][e], f[r][i][e], squares);
                }
            }
            c[2 * r] = dev.x + dev.y;
            c[2 * r + 1] = squares.x + squares.y;
        }
        row_sums<2 * R, CLUSTER>(c, j, red, use, dead);
        float dev[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            dev[r] = j.rms ? 0.0f : c[2 * r] * inv;
            rstd[r] = norm_rstd(c[2 * r + 1] * inv, dev[r], j.eps);
            const unsigned o = row + r * groups;
            if (piece == 0 && o < rows) {
                j.stats[2LL * o] = mean[r] + dev[r];
                j.stats[2LL * o + 1] = rstd[r];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!has(i)) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (row + r * groups >= rows) break;
                float2 o[P];
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    o[e] = fma2(f[r][i][e], both(rstd[r]), both(-dev[r] * rstd[r]));
                    o[e] = fma2(o[e], w[i][e], b[i][e]);
                }
                *reinterpret_cast<uint4*>(y + r * y_row + i * apart) = pack<T>(o);
            }
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
    if (CLUSTER) cluster_sync();  // no CTA ends while another may send to it
}

// ----------------------------------------------------------- unaligned rows
//
// The same with the row's words in shared memory and neighbouring lanes reading and
// writing neighbouring elements. NARROW: rows of less than a warp.

template <typename T, bool NARROW>
__global__ void __launch_bounds__(kRingThreads) layer_norm_loose_kernel(NormJob j) {
    constexpr int R = 2, P = kLoosePairs;
    extern __shared__ __align__(128) uint4 ring[];  // [stage][row][group][window]
    __shared__ __align__(128) RowSums<2 * R> red;
    int use = 0;
    bool dead = false;
    grid_dependency_wait();
    grid_launch_dependents();
    const int at = j.tpr <= 32 ? threadIdx.x & (j.tpr - 1) : threadIdx.x;
    const int group = j.tpr <= 32 ? threadIdx.x / j.tpr : 0;
    const int groups = blockDim.x / j.tpr, tpr = j.tpr, window = window_bytes(j.cols * static_cast<int>(sizeof(T)));
    const float inv = 1.0f / static_cast<float>(j.cols);
    const unsigned rows = static_cast<unsigned>(j.rows), batch = groups * R, step = gridDim.x * batch;
    const unsigned first = blockIdx.x * batch + group;
    const T* x = static_cast<const T*>(j.x) + first * j.ldx;  // of the rows worked on
    const T* x_ahead = x;                                     // of those fetched next
    T* y = static_cast<T*>(j.y) + first * j.ldy;
    const long long x_step = step * j.ldx, y_step = step * j.ldy, x_row = groups * j.ldx, y_row = groups * j.ldy;
    const char* slots = reinterpret_cast<const char*>(ring) + group * window;
    auto slot = [&](int stage, int r) { return slots + (stage * R + r) * groups * window; };
    unsigned ahead = first;
    auto fetch = [&](int stage) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (ahead + r * groups < rows) copy_window(smem_u32(slot(stage, r)), x_ahead + r * x_row, j.cols, at, tpr);
        copies_commit();
        x_ahead += x_step;
        ahead += step;
    };
    const LooseColumns k = loose_columns<NARROW>(j, at);
    const int stride = NARROW ? tpr : 32;
    auto pairs = [&](auto&& fn) { loose_pairs<NARROW>(k, tpr, fn); };
    auto weight = [&](const void* v, int c) { return j.wf32 ? static_cast<const float*>(v)[k.first + c] : to_f32<T>(static_cast<const T*>(v)[k.first + c]); };
    float2 w[P], b[P];
    pairs([&](int q, int c, bool has0, bool has1) {
        w[q] = both(1.0f), b[q] = both(0.0f);
        if (j.weight && has0) w[q].x = weight(j.weight, c);
        if (j.weight && has1) w[q].y = weight(j.weight, c + stride);
        if (j.bias && has0) b[q].x = weight(j.bias, c);
        if (j.bias && has1) b[q].y = weight(j.bias, c + stride);
    });
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    int stage = 0;
    for (unsigned row = first; row - group < rows; row += step, x += x_step, y += y_step) {
        copies_wait<kStages - 2>();
        row_barrier(tpr);
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        float2 f[R][P];
        float mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // Behind the last row its slot's bytes are whatever they are, and not used.
            const T* in = in_window(slot(stage, r), x + r * x_row) + k.first;
            float2 sum = both(0.0f);
            pairs([&](int q, int c, bool has0, bool has1) {
                f[r][q] = make_float2(has0 ? to_f32<T>(in[c]) : 0.0f, has1 ? to_f32<T>(in[c + stride]) : 0.0f);
                sum = add2(sum, f[r][q]);
            });
            mean[r] = sum.x + sum.y;
        }
        if (j.rms) {
#pragma unroll
            for (int r = 0; r < R; ++r) mean[r] = 0.0f;
        } else {
            row_sums<R, false>(mean, j, red, use, dead);
        }
        float c[2 * R];  // sums of the deviations and of their squares
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv;
            float2 dev = both(0.0f), squares = both(0.0f);
            pairs([&](int q, int, bool has0, bool has1) {
                f[r][q] = add2(f[r][q], both(-mean[r]));
                if (!has0) f[r][q].x = 0.0f;
                if (!has1) f[r][q].y = 0.0f;
                dev = add2(dev, f[r][q]);
                squares = fma2(f[r][q], f[r][q], squares);
            });
            c[2 * r] = dev.x + dev.y;
            c[2 * r + 1] = squares.x + squares.y;
        }
        row_sums<2 * R, false>(c, j, red, use, dead);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const unsigned o = row + r * groups;
            if (o >= rows) break;
            const float dev = j.rms ? 0.0f : c[2 * r] * inv, rstd = norm_rstd(c[2 * r + 1] * inv, dev, j.eps);
            if (at == 0) {
                j.stats[2LL * o] = mean[r] + dev;
                j.stats[2LL * o + 1] = rstd;
            }
            T* to = y + r * y_row + k.first;
            pairs([&](int q, int c, bool has0, bool has1) {
                const float2 v = fma2(fma2(f[r][q], both(rstd), both(-dev * rstd)), w[q], b[q]);
                if (has0) to[c] = from_f32<T>(v.x);
                if (has1) to[c + stride] = from_f32<T>(v.y);
            });
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
}

// Rows that do not fit: read three times, the later ones from L2.
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
        const float rstd = norm_rstd(squares / n, dev, j.eps);
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
    const int p = j.per_row = norm_pieces(j, vec);
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int n = 16 / sizeof(T), few = 16 / n;
        RingShape c;
        if (vec ? ring_shape(p, n, 2 * kStages, &c) : loose_shape(j.cols, &c)) {
            j.tpr = c.tpr;
            j.ctas = c.ctas;
            j.per_cta = c.per_cta;
            const long long batch = 2LL * (c.threads / c.tpr);  // rows
            const size_t smem = kStages * (vec ? sizeof(uint4) * 2 * c.V * c.threads : static_cast<size_t>(batch) * window_bytes(j.cols * static_cast<int>(sizeof(T))));
            if (smem <= kRingBytes) {
                const unsigned clusters = ring_clusters(c, (j.rows + batch - 1) / batch, num_sms, smem);
                const bool full = p == c.V * c.tpr * c.ctas;
                const auto run = [&](auto k) { return launch_ring(k, c, clusters, smem, s, j); };
                if (!vec) return run(c.tpr < 32 ? layer_norm_loose_kernel<T, true> : layer_norm_loose_kernel<T, false>);
                if (c.ctas > 1) return run(full ? layer_norm_ring_kernel<T, few, true, true> : layer_norm_ring_kernel<T, few, false, true>);
                if (c.V == 1) return run(full ? layer_norm_ring_kernel<T, 1, true, false> : layer_norm_ring_kernel<T, 1, false, false>);
                return run(full ? layer_norm_ring_kernel<T, few, true, false> : layer_norm_ring_kernel<T, few, false, false>);
            }
        }
        const unsigned blocks = static_cast<unsigned>(std::min<long long>(j.rows, 2LL * num_sms));
        return static_cast<int>(launch_after(vec ? layer_norm_long_kernel<T, Wide<T, n>> : layer_norm_long_kernel<T, Loose<T>>, dim3(blocks),
                                             dim3(kLongThreads), 0, s, j));
    });
}

}  // namespace gns
