// Layer norm, forward: mean and variance of each row, and the scaled row.
//
// The mean is found first, then the deviations from it and their squares in one sum:
// the squares of the centred values lose nothing to cancellation, and the mean of the
// deviations, which is what rounding left of the first mean, is taken off them (4096 +- 1
// in fp32 keeps its digits). Where a row has next to no spread beside its mean, its squares
// are mostly those of that remainder, and their difference is what rounding leaves: such
// rows are made anew at the block's end (a constant row of any size gives 0).
//
// Bound: HBM, x read and y written once; but the instructions of a row's 4096 values and
// its two sums take about as long. Rows go through shared memory ahead of their use, as
// 16-byte pieces or, unaligned, as the words that hold them; rows beyond that are read
// three times. 16384 x 4096 bf16 with fp32 weights: 51 us (5.3 TB/s; issue slots 68%
// busy with 16 warps a processor: 24, by one row at a time instead of two, took 53);
// 262144 x 128: 21 (6.3); by two CTAs a row 8192 x 5120: 39 (4.3) and 4096 x 14336: 71 (3.3);
// unaligned 65536 x 257: 24 (2.8) and 16384 x 4093: 70 (3.9); one row: 2.4 (from registers
// alone 2.9; 304 rows 2.9 and 5.0). Rows made anew take a block 4 us each at 4000 columns:
// 16384 x 4000 fp32 takes 93 us, 940 if all of it is 123456.789.
#include <algorithm>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// Like fmaxf and fminf, but NaN where one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}

// From the mean of the squared deviations and of the deviations.
__device__ __forceinline__ float norm_rstd(float squares, float dev, float eps) { return rsqrtf(max_nan(squares - dev * dev, 0.0f) + eps); }

// A row's rstd as the kernels below first write it: below 0 where the mean that was taken off
// first lies more than a deviation (with eps) from the row's. Such rows are made anew at the
// block's end, as are those whose rstd is 0, since their squares overflow, or NaN. (Of the
// others, whose sums are off by up to 160 half steps, 2^-16.7 of themselves, the squares are no
// more than twice the variance and eps: it is off by 2^-14 of them at worst, 2^-22 as measured.)
__device__ __forceinline__ float rstd_or_again(float dev, float rstd) {
    const float beyond = fmaf(fabsf(dev), rstd, -1.0f);
    return __uint_as_float(__float_as_uint(rstd) ^ (~__float_as_uint(beyond) & 0x80000000u));
}

// Such a row by `threads` threads (a warp or the block), whose own sums row_sum2 joins: from the
// differences to its first element, which lose nothing in a row of next to no spread.
template <typename T>
__device__ __noinline__ void norm_row_again(const NormJob& j, long long row, int threads, float2* red0, float2* red1) {
    const T* x = static_cast<const T*>(j.x) + row * j.ldx;
    T* y = static_cast<T*>(j.y) + row * j.ldy;
    const int at = threads == 32 ? threadIdx.x & 31 : threadIdx.x;
    const float n = static_cast<float>(j.cols), first = j.rms ? 0.0f : to_f32<T>(x[0]);
    float mean = 0.0f, none = 0.0f, dev = 0.0f, squares = 0.0f;  // of the differences
#pragma unroll 4
    for (int c = at; c < j.cols; c += threads) mean += to_f32<T>(x[c]) - first;
    row_sum2(mean, none, threads, red0);
    mean = j.rms ? 0.0f : mean / n;
#pragma unroll 4
    for (int c = at; c < j.cols; c += threads) {
        const float d = to_f32<T>(x[c]) - first - mean;
        dev += d;
        squares = fmaf(d, d, squares);
    }
    row_sum2(dev, squares, threads, red1);
    dev = j.rms ? 0.0f : dev / n;
    const float rstd = norm_rstd(squares / n, dev, j.eps);
    const auto value = [&](const void* v, int c) { return j.wf32 ? static_cast<const float*>(v)[c] : to_f32<T>(static_cast<const T*>(v)[c]); };
#pragma unroll 4
    for (int c = at; c < j.cols; c += threads) {
        float o = (to_f32<T>(x[c]) - first - mean - dev) * rstd;
        if (j.weight) o *= value(j.weight, c);
        if (j.bias) o += value(j.bias, c);
        y[c] = from_f32<T>(o);
    }
    if (at == 0) {
        j.stats[2 * row] = first + (mean + dev);
        j.stats[2 * row + 1] = rstd;
    }
}

// Those of a block's rows, which are base .. base + batch - 1, those `step` further, and so on,
// a warp each or one after the other. After a barrier behind all that the block has written.
template <typename T, typename Red>
__device__ __forceinline__ void norm_rows_again(const NormJob& j, unsigned base, unsigned batch, unsigned step, Red& red) {
    const int threads = j.tpr <= 32 ? 32 : blockDim.x, workers = blockDim.x / threads;
    float2 *red0 = reinterpret_cast<float2*>(red.sums[0]), *red1 = reinterpret_cast<float2*>(red.sums[1]);
    for (unsigned b = base; b < j.rows; b += step)
        for (unsigned r = b + threadIdx.x / threads; r < b + batch && r < j.rows; r += workers) {
            float* rstd = j.stats + 2LL * r + 1;
            if (*rstd > 0.0f) continue;
            if (j.again) {
                norm_row_again<T>(j, r, threads, red0, red1);
            } else {
                row_barrier(threads);  // all have read it
                if (threadIdx.x % threads == 0) *rstd = fabsf(*rstd);
            }
        }
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
__global__ void __launch_bounds__(kRingThreads) layer_norm_ring_kernel(const __grid_constant__ NormJob j) {
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
    float least = 1.0f;  // rstd_or_again of the rows whose stats this thread writes
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
                const float kept = rstd_or_again(dev[r], rstd[r]);
                j.stats[2LL * o + 1] = kept;
                least = min_nan(least, kept);
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
    if (rank == 0 && __syncthreads_or(!(least > 0.0f))) norm_rows_again<T>(j, cluster * batch, batch, step, red);
    if (CLUSTER) cluster_sync();  // no CTA ends while another may send to it
}

// ----------------------------------------------------------- unaligned rows
//
// The same with the row's words in shared memory and neighbouring lanes reading and
// writing neighbouring elements. NARROW: rows of less than a warp.

template <typename T, bool NARROW>
__global__ void __launch_bounds__(kRingThreads) layer_norm_loose_kernel(const __grid_constant__ NormJob j) {
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
    float least = 1.0f;  // as above
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
            const float kept = rstd_or_again(dev, rstd);
            least = min_nan(least, kept);
            if (at == 0) {
                j.stats[2LL * o] = mean[r] + dev;
                j.stats[2LL * o + 1] = kept;
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
    if (__builtin_expect(__syncthreads_or(!(least > 0.0f)), 0)) norm_rows_again<T>(j, blockIdx.x * batch, batch, step, red);
}

// Rows that do not fit: read three times, the later ones from L2. The mean is made of the
// differences to the first element, which costs nothing here and leaves no row to make anew.
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
            const float first = to_f32<T>(x[0]);
            for (unsigned v = threadIdx.x; v < j.per_row; v += kLongThreads) {
                Piece p;
                p.load(x, v, j.cols);
                float f[N];
                p.get(f);
#pragma unroll
                for (int e = 0; e < N; ++e) mean += piece_has(p, v, e, j.cols) ? f[e] - first : 0.0f;
            }
            row_sum2(mean, none, kLongThreads, red[phase ^= 1]);
            mean = first + mean / n;
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
