// Layer norm, backward: with h = (x - mean) rstd and g = weight dy,
//   dx = residual + rstd (g - mean(g) - h mean(g h))   (mean(g) only where the mean was taken off)
//   dweight = sum over the rows of dy h,  dbias = sum over the rows of dy.
//
// One pass over x and dy: a thread keeps its columns from row to row and sums
// their dweight and dbias in registers, a block writes the sums of its rows, and a
// second kernel adds the blocks' in their order. Which rows a block takes follows
// from the sizes and the number of SMs alone, so results repeat.
//
// Bound: HBM, x, dy (and the residual) read and dx written once. Without a residual
// 16384 x 4096 bf16 with fp32 weights: 73 us (5.5 TB/s), of which the second kernel is 6;
// 262144 x 128: 37 (5.5); unaligned 65536 x 257: 56 (1.8). With one 16384 x 4096: 89 (6.1);
// by two CTAs a row 8192 x 5120: 68 (4.9) and 4096 x 14336: 107 (4.4); unaligned 16384 x
// 4093: 162 (3.3), by instructions (single elements to and from shared memory, 60 for
// each of the row).
#include <algorithm>
#include <type_traits>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// A block's sums of N of a thread's columns, col(e) or -1: the groups of a warp, then the
// warps, in shared memory, where several rows share the block.
template <int N, typename Col>
__device__ __forceinline__ void store_sums(float (&acc)[N], const NormJob& j, float* part, float* smem, Col&& col) {
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
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int c = col(e);
        if (c >= 0) part[c] = acc[e];
    }
}

// ------------------------------------------------------------- aligned rows
//
// The same with the rows copied to shared memory ahead of their use (cp.async): a
// thread copies, and later reads, the pieces of its own columns alone, so the copies
// need no barrier and hold no registers (loaded to registers instead, 160 us for
// 16384 x 4096). FULL: every thread has all its pieces.
// CLUSTER: rows of more columns than a CTA's registers have sums for are shared by the CTAs
// of a cluster, which exchange the row's sums.

template <typename T, int V, bool SUMS, bool FULL, bool CLUSTER>
__global__ void __launch_bounds__(kRingThreads) layer_norm_backward_ring_kernel(NormJob j) {
    constexpr int N = 16 / sizeof(T), P = N / 2;
    extern __shared__ __align__(128) uint4 ring[];  // [stage][x, dy, residual][piece][thread]
    __shared__ __align__(128) RowSums<2> red;
    __shared__ float smem[SUMS ? 8 * 32 * N : 1];
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
    const unsigned rows = static_cast<unsigned>(j.rows), step = clusters * groups, first = cluster * groups + group;
    const T* x = static_cast<const T*>(j.x) + first * j.ldx + piece * N;  // of the row fetched next
    const T* dy = static_cast<const T*>(j.dy) + first * j.lddy + piece * N;
    const T* res = static_cast<const T*>(j.residual) + (j.residual ? first * j.ldr + piece * N : 0);
    T* dx = static_cast<T*>(j.dx) + first * j.lddx + piece * N;
    const float* stats = j.stats + 2LL * first;
    const long long x_step = step * j.ldx, dy_step = step * j.lddy, res_step = step * j.ldr, dx_step = step * j.lddx;
    const int apart = j.tpr * N, kinds = j.residual ? 3 : 2;
    const uint4* mine = ring + threadIdx.x;
    const uint32_t slots = smem_u32(mine);
    auto has = [&](int i) { return FULL || piece + i * j.tpr < pieces; };
    unsigned ahead = first;
    auto fetch = [&](int stage) {
        float2 st = both(0.0f);
        if (ahead < rows) {
            st = make_float2(stats[0], stats[1]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!has(i)) continue;
                const uint32_t to = slots + 16 * (stage * kinds * V + i) * threads;
                copy16(to, x + i * apart);
                copy16(to + 16 * V * threads, dy + i * apart);
                if (kinds == 3) copy16(to + 32 * V * threads, res + i * apart);
            }
        }
        copies_commit();
        x += x_step, dy += dy_step, res += res_step, stats += 2LL * step, ahead += step;
        return st;
    };
    float2 dw[V][P], db[V][P], w[V][P];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < P; ++e) w[i][e] = both(1.0f), dw[i][e] = db[i][e] = both(0.0f);
        if (j.weight && has(i)) {
            float f[N];
            const Wide<T, N> p{};
            piece_weights(p, j.weight, j.wf32, piece + i * j.tpr, j.cols, f);
#pragma unroll
            for (int e = 0; e < P; ++e) w[i][e] = make_float2(f[2 * e], f[2 * e + 1]);
        }
    }
    float2 st[kStages];  // mean and rstd of the rows in flight, the next one's first
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) st[k] = fetch(k);
    int stage = 0;
    for (unsigned row = first; row - group < rows; row += step, dx += dx_step) {
        st[kStages - 1] = fetch(stage == 0 ? kStages - 1 : stage - 1);
        copies_wait<kStages - 1>();
        const bool live = row < rows;
        const float rstd = st[0].y;
        float2 h[V][P], g[V][P], c1 = both(0.0f), c2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint4 u = make_uint4(0, 0, 0, 0), d = u;
            if (has(i) && live) {
                u = mine[(stage * kinds * V + i) * threads];
                d = mine[((stage * kinds + 1) * V + i) * threads];
            }
            unpack<T, N>(u, h[i]);
            unpack<T, N>(d, g[i]);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                h[i][e] = mul2(add2(h[i][e], both(-st[0].x)), both(rstd));
                if (SUMS) {
                    dw[i][e] = fma2(g[i][e], h[i][e], dw[i][e]);
                    db[i][e] = add2(db[i][e], g[i][e]);
                }
                g[i][e] = mul2(g[i][e], w[i][e]);
                c1 = add2(c1, g[i][e]);
                c2 = fma2(g[i][e], h[i][e], c2);
            }
        }
        float c[2] = {c1.x + c1.y, c2.x + c2.y};
        row_sums<2, CLUSTER>(c, j, red, use, dead);
        if (live) {
            const float2 minus = both(j.rms ? 0.0f : -c[0] * inv), by = both(-c[1] * inv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!has(i)) continue;
                float2 r[P];
#pragma unroll
                for (int e = 0; e < P; ++e) r[e] = both(0.0f);
                if (j.residual) unpack<T, N>(mine[((stage * kinds + 2) * V + i) * threads], r);
#pragma unroll
                for (int e = 0; e < P; ++e) r[e] = fma2(add2(fma2(h[i][e], by, g[i][e]), minus), both(rstd), r[e]);
                *reinterpret_cast<uint4*>(dx + i * apart) = pack<T>(r);
            }
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) st[k] = st[k + 1];
    }
    copies_wait<0>();
    if (SUMS) {
        float* part = j.part + static_cast<long long>(cluster) * j.cols;
        const long long all = static_cast<long long>(clusters) * j.cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = piece + i * j.tpr;
            const auto col = [&](int e) { return v < pieces ? v * N + e : -1; };
            float sum[N];
#pragma unroll
            for (int e = 0; e < P; ++e) sum[2 * e] = dw[i][e].x, sum[2 * e + 1] = dw[i][e].y;
            store_sums(sum, j, part, smem, col);
            if (!j.dbias) continue;
#pragma unroll
            for (int e = 0; e < P; ++e) sum[2 * e] = db[i][e].x, sum[2 * e + 1] = db[i][e].y;
            store_sums(sum, j, part + all, smem, col);
        }
    }
    if (CLUSTER) cluster_sync();  // no CTA ends while another may send to it
}

// ----------------------------------------------------------- unaligned rows
//
// The same with the row's words in shared memory and neighbouring lanes reading and
// writing neighbouring elements. NARROW: rows of less than a warp.

template <typename T, bool SUMS, bool NARROW>
__global__ void __launch_bounds__(kRingThreads) layer_norm_backward_loose_kernel(NormJob j) {
    constexpr int P = kLoosePairs;
    extern __shared__ __align__(128) uint4 ring[];  // [stage][x, dy, residual][group][window]
    __shared__ __align__(128) RowSums<2> red;
    __shared__ float smem[SUMS ? 8 * 32 * P : 1];
    int use = 0;
    bool dead = false;
    grid_dependency_wait();
    grid_launch_dependents();
    const int at = j.tpr <= 32 ? threadIdx.x & (j.tpr - 1) : threadIdx.x;
    const int group = j.tpr <= 32 ? threadIdx.x / j.tpr : 0;
    const int groups = blockDim.x / j.tpr, tpr = j.tpr, window = window_bytes(j.cols * static_cast<int>(sizeof(T)));
    const float inv = 1.0f / static_cast<float>(j.cols);
    const unsigned rows = static_cast<unsigned>(j.rows), step = gridDim.x * groups, first = blockIdx.x * groups + group;
    const T* x = static_cast<const T*>(j.x) + first * j.ldx;  // of the row worked on
    const T* dy = static_cast<const T*>(j.dy) + first * j.lddy;
    const T* res = static_cast<const T*>(j.residual) + (j.residual ? first * j.ldr : 0);
    const T *x_ahead = x, *dy_ahead = dy, *res_ahead = res;  // of the row fetched next
    T* dx = static_cast<T*>(j.dx) + first * j.lddx;
    const float* stats = j.stats + 2LL * first;
    const long long x_step = step * j.ldx, dy_step = step * j.lddy, res_step = step * j.ldr, dx_step = step * j.lddx;
    const int kinds = j.residual ? 3 : 2;
    const char* slots = reinterpret_cast<const char*>(ring) + group * window;
    auto slot = [&](int stage, int kind) { return slots + (stage * kinds + kind) * groups * window; };
    unsigned ahead = first;
    auto fetch = [&](int stage) {
        float2 st = both(0.0f);
        if (ahead < rows) {
            st = make_float2(stats[0], stats[1]);
            copy_window(smem_u32(slot(stage, 0)), x_ahead, j.cols, at, tpr);
            copy_window(smem_u32(slot(stage, 1)), dy_ahead, j.cols, at, tpr);
            if (kinds == 3) copy_window(smem_u32(slot(stage, 2)), res_ahead, j.cols, at, tpr);
        }
        copies_commit();
        x_ahead += x_step, dy_ahead += dy_step, res_ahead += res_step, stats += 2LL * step, ahead += step;
        return st;
    };
    const LooseColumns k = loose_columns<NARROW>(j, at);
    const int stride = NARROW ? tpr : 32;
    auto pairs = [&](auto&& fn) { loose_pairs<NARROW>(k, tpr, fn); };
    auto weight = [&](int c) { return j.wf32 ? static_cast<const float*>(j.weight)[k.first + c] : to_f32<T>(static_cast<const T*>(j.weight)[k.first + c]); };
    float2 dw[P], db[P], w[P];
#pragma unroll
    for (int q = 0; q < P; ++q) w[q] = both(1.0f), dw[q] = db[q] = both(0.0f);
    pairs([&](int q, int c, bool has0, bool has1) {
        if (j.weight && has0) w[q].x = weight(c);
        if (j.weight && has1) w[q].y = weight(c + stride);
    });
    const bool deep = j.stages == 3;
    float2 st[3];  // mean and rstd of the rows in flight, the next one's first
    st[0] = fetch(0);
    if (deep) st[1] = fetch(1);
    int stage = 0;
    for (unsigned row = first; row - group < rows; row += step, x += x_step, dy += dy_step, res += res_step, dx += dx_step) {
        if (deep)
            copies_wait<1>();
        else
            copies_wait<0>();
        row_barrier(tpr);
        if (deep)
            st[2] = fetch(stage == 0 ? 2 : stage - 1);
        else
            st[1] = fetch(stage ^ 1);
        const float mean = st[0].x, rstd = st[0].y;
        float2 h[P], g[P], c1 = both(0.0f), c2 = both(0.0f);
        const T* xs = in_window(slot(stage, 0), x) + k.first;
        const T* ds = in_window(slot(stage, 1), dy) + k.first;
        const bool live = row < rows;
        if (live) {
            pairs([&](int q, int c, bool has0, bool has1) {
                // A column that is not there has dy = 0 and x = mean.
                h[q] = make_float2(has0 ? to_f32<T>(xs[c]) : mean, has1 ? to_f32<T>(xs[c + stride]) : mean);
                g[q] = make_float2(has0 ? to_f32<T>(ds[c]) : 0.0f, has1 ? to_f32<T>(ds[c + stride]) : 0.0f);
                h[q] = mul2(add2(h[q], both(-mean)), both(rstd));
                if (SUMS) {
                    dw[q] = fma2(g[q], h[q], dw[q]);
                    db[q] = add2(db[q], g[q]);
                }
                g[q] = mul2(g[q], w[q]);
                c1 = add2(c1, g[q]);
                c2 = fma2(g[q], h[q], c2);
            });
        }
        float c[2] = {c1.x + c1.y, c2.x + c2.y};
        row_sums<2, false>(c, j, red, use, dead);
        if (live) {
            const float2 minus = both(j.rms ? 0.0f : -c[0] * inv), by = both(-c[1] * inv);
            const T* rs = in_window(slot(stage, kinds - 1), res) + k.first;
            T* to = dx + k.first;
            pairs([&](int q, int c, bool has0, bool has1) {
                float2 r = both(0.0f);
                if (kinds == 3) r = make_float2(has0 ? to_f32<T>(rs[c]) : 0.0f, has1 ? to_f32<T>(rs[c + stride]) : 0.0f);
                r = fma2(add2(fma2(h[q], by, g[q]), minus), both(rstd), r);
                if (has0) to[c] = from_f32<T>(r.x);
                if (has1) to[c + stride] = from_f32<T>(r.y);
            });
        }
        stage = stage == j.stages - 1 ? 0 : stage + 1;
        st[0] = st[1], st[1] = st[2];
    }
    copies_wait<0>();
    if (SUMS) {
        float* part = j.part + static_cast<long long>(blockIdx.x) * j.cols;
        const long long all = static_cast<long long>(gridDim.x) * j.cols;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const auto col = [&](int q) {
                if (q == P - 1) return (half ? k.hi : k.lo) ? k.first + k.last + half * stride : -1;
                return q < k.whole ? k.first + (2 * q + half) * stride : -1;
            };
            float sum[P];
#pragma unroll
            for (int q = 0; q < P; ++q) sum[q] = half ? dw[q].y : dw[q].x;
            store_sums(sum, j, part, smem, col);
            if (!j.dbias) continue;
#pragma unroll
            for (int q = 0; q < P; ++q) sum[q] = half ? db[q].y : db[q].x;
            store_sums(sum, j, part + all, smem, col);
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
    RingShape ring;
    size_t smem;
    unsigned blocks, strips;  // blocks: of clusters; strips: the column kernel's
    int per_row, parts, stages;
};

Shape shape_of(const NormJob& j, int num_sms) {
    Shape c{};
    const int es = elem_bytes(j.dtype), kinds = j.residual ? 3 : 2;
    c.vec = norm_vec(j, true);
    c.per_row = norm_pieces(j, c.vec);
    c.fits = c.vec ? ring_shape(c.per_row, 16 / es, kStages * kinds, &c.ring) : loose_shape(j.cols, &c.ring);
    if (c.fits) {
        const long long groups = c.ring.threads / c.ring.tpr;
        const size_t stage = static_cast<size_t>(kinds) * (c.vec ? sizeof(uint4) * c.ring.V * c.ring.threads : groups * window_bytes(j.cols * es));
        // Two unaligned rows in flight rather than three where that lets more blocks share a
        // processor. (Aligned ones: the branch costs more, 100 us instead of 89 for 16384 x 4096.)
        c.stages = !c.vec && kRingBytes / (kStages * stage) * c.ring.threads < 512 ? kStages - 1 : kStages;
        c.smem = c.stages * stage;
        // Each block's sums are written and read again: four rows to each, once every
        // processor has one (300 x 4096: 12 us instead of 16, and 64 rows 9 instead of 11).
        const long long batches = (j.rows + groups - 1) / groups;
        const long long most = j.dweight || j.dbias ? std::max<long long>(num_sms / c.ring.ctas, (batches + 3) / 4) : batches;
        c.blocks = ring_clusters(c.ring, std::min(batches, std::max(1LL, most)), num_sms, c.smem);
        c.parts = static_cast<int>(c.blocks);
        c.fits = c.smem <= kRingBytes;
    }
    if (!c.fits) {
        c.blocks = static_cast<unsigned>(std::min<long long>(j.rows, 4LL * num_sms));
        c.strips = static_cast<unsigned>((c.per_row + 255) / 256);
        c.parts = static_cast<int>(std::min<long long>(j.rows, std::max(1u, 8u * num_sms / c.strips)));
    }
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
    j.tpr = c.ring.tpr;
    j.ctas = c.ring.ctas;
    j.per_cta = c.ring.per_cta;
    j.stages = c.stages;
    const bool sums = j.dweight || j.dbias;
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        using W = Wide<T, 16 / sizeof(T)>;
        using L = Loose<T>;
        if (!c.fits)
            return static_cast<int>(launch_after(c.vec ? layer_norm_backward_long_kernel<T, W> : layer_norm_backward_long_kernel<T, L>,
                                                 dim3(c.blocks), dim3(kLongThreads), 0, s, j));
        const auto run = [&](auto k) { return launch_ring(k, c.ring, c.blocks, c.smem, s, j); };
        if (!c.vec) {
            if (c.ring.tpr < 32) return sums ? run(layer_norm_backward_loose_kernel<T, true, true>) : run(layer_norm_backward_loose_kernel<T, false, true>);
            return sums ? run(layer_norm_backward_loose_kernel<T, true, false>) : run(layer_norm_backward_loose_kernel<T, false, false>);
        }
        constexpr int few = 16 / (16 / sizeof(T));
        const bool full = c.per_row == c.ring.V * c.ring.tpr * c.ring.ctas;
        const auto pick = [&](auto v, auto shared) {
            constexpr int V = decltype(v)::value;
            constexpr bool CLUSTER = decltype(shared)::value;
            if (sums) return run(full ? layer_norm_backward_ring_kernel<T, V, true, true, CLUSTER> : layer_norm_backward_ring_kernel<T, V, true, false, CLUSTER>);
            return run(full ? layer_norm_backward_ring_kernel<T, V, false, true, CLUSTER> : layer_norm_backward_ring_kernel<T, V, false, false, CLUSTER>);
        };
        if (c.ring.ctas > 1) return pick(std::integral_constant<int, few>{}, std::true_type{});
        return c.ring.V == 1 ? pick(std::integral_constant<int, 1>{}, std::false_type{}) : pick(std::integral_constant<int, few>{}, std::false_type{});
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
