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
#include <type_traits>

#include "layer_norm.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

// A block's sums of one piece's columns: the groups of a warp, then the warps, in
// shared memory where several rows share the block.
template <typename Piece, int N>
__device__ __forceinline__ void store_sums(float (&acc)[N], const Piece& p, const NormJob& j, unsigned v, unsigned end,
                                           float* part, float* smem) {
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
    if (v >= end) return;
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (piece_has(p, v, e, j.cols)) part[piece_column(p, v, e)] = acc[e];
}

// A row that a block's registers hold: up to kMostPieces pieces of each of
// kMostThreads threads.
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
            store_sums(dw[i], p, j, at + i * j.tpr, j.per_row, part, smem);
            if (j.dbias) store_sums(db[i], p, j, at + i * j.tpr, j.per_row, part + all, smem);
        }
    }
}

// ------------------------------------------------------------- aligned rows
//
// The same with the rows copied to shared memory ahead of their use (cp.async): a
// thread copies, and later reads, the pieces of its own columns alone, so the copies
// need no barrier and hold no registers. FULL: every thread has all its pieces.
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
            const float2 minus = both(j.rms ? 0.0f : -c[0] * inv * rstd), by = both(-c[1] * inv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!has(i)) continue;
                float2 r[P];
                if (j.residual) {
                    unpack<T, N>(mine[((stage * kinds + 2) * V + i) * threads], r);
#pragma unroll
                    for (int e = 0; e < P; ++e) r[e] = add2(r[e], minus);
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e) r[e] = minus;
                }
#pragma unroll
                for (int e = 0; e < P; ++e) r[e] = fma2(fma2(h[i][e], by, g[i][e]), both(rstd), r[e]);
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
        const Wide<T, N> p{};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float sum[N];
#pragma unroll
            for (int e = 0; e < P; ++e) sum[2 * e] = dw[i][e].x, sum[2 * e + 1] = dw[i][e].y;
            store_sums(sum, p, j, piece + i * j.tpr, pieces, part, smem);
            if (!j.dbias) continue;
#pragma unroll
            for (int e = 0; e < P; ++e) sum[2 * e] = db[i][e].x, sum[2 * e + 1] = db[i][e].y;
            store_sums(sum, p, j, piece + i * j.tpr, pieces, part + all, smem);
        }
    }
    if (CLUSTER) cluster_sync();  // no CTA ends while another may send to it
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
    int V, threads, tpr, per_row;
    size_t smem;  // of the ring, 0 where the rows go through registers
    unsigned blocks, strips;  // strips: the column kernel's
    int parts;
};

Shape shape_of(const NormJob& j, int num_sms) {
    Shape c{};
    c.vec = norm_vec(j, true);
    const int p = c.per_row = norm_pieces(j, c.vec);
    c.fits = c.vec ? ring_shape(p, 16 / elem_bytes(j.dtype), kStages * (j.residual ? 3 : 2), &c.ring) : p <= kMostPieces * kMostThreads;
    if (!c.fits) {
        c.blocks = static_cast<unsigned>(std::min<long long>(j.rows, 4LL * num_sms));
        c.strips = static_cast<unsigned>((p + 255) / 256);
        c.parts = static_cast<int>(std::min<long long>(j.rows, std::max(1u, 8u * num_sms / c.strips)));
        return c;
    }
    if (c.vec) {
        c.threads = c.ring.threads;
        c.tpr = c.ring.tpr;
        c.smem = sizeof(uint4) * kStages * (j.residual ? 3 : 2) * c.ring.V * c.threads;
        const long long groups = c.threads / c.tpr;
        c.blocks = ring_clusters(c.ring, (j.rows + groups - 1) / groups, num_sms, c.smem);
    } else {
        c.V = p <= 32 ? 1 : p <= 1024 ? 2 : kMostPieces;
        c.threads = c.tpr = (p + 32 * c.V - 1) / (32 * c.V) * 32;
        if (c.tpr == 32) c.threads = 256;
        const long long groups = c.threads / c.tpr;
        c.blocks = static_cast<unsigned>(std::min<long long>((j.rows + groups - 1) / groups, static_cast<long long>(num_sms) * std::max(1, 768 / c.threads)));
    }
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
        if (c.vec) {
            constexpr int few = 16 / (16 / sizeof(T));
            const bool full = c.per_row == c.ring.V * c.tpr * c.ring.ctas;
            j.ctas = c.ring.ctas;
            j.per_cta = c.ring.per_cta;
            const auto pick = [&](auto v, auto shared) {
                constexpr int V = decltype(v)::value;
                constexpr bool CLUSTER = decltype(shared)::value;
                const auto run = [&](auto k) { return launch_ring(k, c.ring, c.blocks, c.smem, s, j); };
                if (sums) return run(full ? layer_norm_backward_ring_kernel<T, V, true, true, CLUSTER> : layer_norm_backward_ring_kernel<T, V, true, false, CLUSTER>);
                return run(full ? layer_norm_backward_ring_kernel<T, V, false, true, CLUSTER> : layer_norm_backward_ring_kernel<T, V, false, false, CLUSTER>);
            };
            if (c.ring.ctas > 1) return pick(std::integral_constant<int, few>{}, std::true_type{});
            return c.ring.V == 1 ? pick(std::integral_constant<int, 1>{}, std::false_type{}) : pick(std::integral_constant<int, few>{}, std::false_type{});
        }
        auto run = [&](auto k) { return static_cast<int>(launch_after(k, dim3(c.blocks), dim3(c.threads), 0, s, j)); };
        if (sums)
            return run(c.V == 1 ? layer_norm_backward_kernel<T, L, 1, true> : c.V == 2 ? layer_norm_backward_kernel<T, L, 2, true> : layer_norm_backward_kernel<T, L, 4, true>);
        return run(c.V == 1 ? layer_norm_backward_kernel<T, L, 1, false> : c.V == 2 ? layer_norm_backward_kernel<T, L, 2, false> : layer_norm_backward_kernel<T, L, 4, false>);
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
