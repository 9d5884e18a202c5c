// Embedding: rows of a table looked up by token and scaled, and the gradient of the
// table.
//
// The gradient sorts the tokens by id (stable counting sorts by digits, lowest
// first) and sums the rows of dy that share an id in token order, so it is a
// function of the inputs alone, and every row of the table is written once:
// - runs: a warp takes `chunk` consecutive sorted tokens and a strip of 32 pieces of
//   the row, adds up rows in fp32 registers while the id stays the same and writes
//   a sum when it changes. Sums of an id that lies within the chunk are the table's
//   row; those that began before it or go on behind it are parts. However often one
//   token occurs, the work is spread evenly.
// - rows: the parts of an id that spans chunks are added in order, and the rows of
//   the ids that do not occur are set to zero.
//
// Bound: HBM. Forward the rows and y; backward dy read and the table written once.
#include <algorithm>
#include <type_traits>

#include "blockops.cuh"
#include "counting_sort.cuh"
#include "embedding.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename I>
__device__ __forceinline__ int row_of(const I* ids, long long t, int vocab) {
    const I v = ids[t];
    return v >= 0 && v < static_cast<I>(vocab) ? static_cast<int>(v) : vocab;
}

// ------------------------------------------------------------------ forward

template <typename T, typename Piece, typename I>
__global__ void __launch_bounds__(kThreads) embedding_kernel(EmbeddingJob j, unsigned per_row) {
    constexpr int N = Piece::kSize;
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned long long pieces = static_cast<unsigned long long>(j.tokens) * per_row;
    const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * kThreads;
    for (unsigned long long i = static_cast<unsigned long long>(blockIdx.x) * kThreads + threadIdx.x; i < pieces; i += step) {
        const long long t = pieces <= 0xffffffffULL ? static_cast<unsigned>(i) / per_row : i / per_row;
        const unsigned v = static_cast<unsigned>(i - t * per_row);
        const int r = row_of(static_cast<const I*>(j.ids), t, j.vocab);
        Piece p;
        p.clear();
        if (r < j.vocab) {
            p.load(static_cast<const T*>(j.table) + r * j.ldt, v, j.cols);
            float f[N];
            p.get(f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] *= j.scale;
            p.set(f);
        }
        p.store(static_cast<T*>(j.y) + t * j.ldy, v, j.cols);
    }
}

// ----------------------------------------------------------------- backward

// The tokens by one digit of their id (vocab for those without a row, which are last).
template <typename I>
struct TokenDigits {
    const I* ids;                // the first pass reads these,
    const int *keys_in, *order_in;  // later ones what the pass before wrote
    int vocab, shift, mask;
    int *keys_out, *order_out;
    __device__ __forceinline__ int key(long long s) const { return keys_in ? keys_in[s] : row_of(ids, s, vocab); }
    __device__ __forceinline__ int digit(long long s) const { return (key(s) >> shift) & mask; }
    __device__ __forceinline__ void place(long long s, int at) const {
        keys_out[at] = key(s);
        order_out[at] = order_in ? order_in[s] : static_cast<int>(s);
    }
    __device__ __forceinline__ void start(int, int) const {}
};

// A sum as elements of the table's gradient.
template <typename O, int N>
__device__ __forceinline__ void store_row(O* row, unsigned v, int, const float (&f)[N], std::true_type) {
    O* at = row + static_cast<long long>(v) * N;
    if constexpr (N * sizeof(O) >= 16) {
        Pack<O, N> p;
        p.set(f);
        p.store(at);
    } else {  // four 16-bit values of a row of fp32 ones
        uint2 u;
        O* e = reinterpret_cast<O*>(&u);
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_f32<O>(f[i]);
        *reinterpret_cast<uint2*>(at) = u;
    }
}
template <typename O, int N>
__device__ __forceinline__ void store_row(O* row, unsigned v, int H, const float (&f)[N], std::false_type) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = Loose<O>::column(v, i);
        if (c < H) row[c] = from_f32<O>(f[i]);
    }
}

// The parts of chunk c: [c][0] of an id that began before it, [c][1] of one that
// began in it and goes on behind it.
__device__ __forceinline__ float* part_at(float* part, long long c, int which, unsigned per_row, unsigned v, int N) {
    return part + ((c * 2 + which) * per_row + v) * N;
}

constexpr int kAhead = 8;  // rows whose loads are issued together

// Blocks from run_blocks on find where each id's tokens start in the sorted order.
template <typename T, typename Piece, typename O, bool WIDE>
__global__ void __launch_bounds__(kThreads) embedding_runs_kernel(EmbeddingJob j, const int* keys, const int* order, float* part,
                                                                  int* starts, int chunk, int chunks, unsigned per_row,
                                                                  unsigned strips, unsigned run_blocks) {
    constexpr int N = Piece::kSize;
    using Wideness = std::integral_constant<bool, WIDE>;
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= run_blocks) {
        const long long v = static_cast<long long>(blockIdx.x - run_blocks) * kThreads + threadIdx.x;
        if (v > j.vocab) return;
        int lo = 0, hi = j.tokens;
        while (lo < hi) {
            const int mid = lo + ((hi - lo) >> 1);
            if (keys[mid] < v)
                lo = mid + 1;
            else
                hi = mid;
        }
        starts[v] = lo;
        return;
    }
    const int lane = threadIdx.x & 31;
    const unsigned long long item = static_cast<unsigned long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long c = static_cast<long long>(item / strips);
    if (c >= chunks) return;
    const unsigned v = static_cast<unsigned>(item - c * strips) * 32 + lane;
    const bool mine = v < per_row;
    const long long beg = c * chunk, end = min(beg + chunk, static_cast<long long>(j.tokens));
    const T* dy = static_cast<const T*>(j.dy);
    O* out = static_cast<O*>(j.dtable);
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    int current = keys[beg];
    bool before = beg > 0 && keys[beg - 1] == current;  // the id began in an earlier chunk
    auto flush = [&](bool behind) {
        if (current < j.vocab && mine) {
            if (before || behind) {
                float* p = part_at(part, c, before ? 0 : 1, per_row, v, N);
#pragma unroll
                for (int e = 0; e < N; e += 4) *reinterpret_cast<float4*>(p + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
            } else {
                float f[N];
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] = acc[e] * j.scale;
                store_row<O, N>(out + current * j.lddt, v, j.cols, f, Wideness{});
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        before = false;
    };
    for (long long s0 = beg; s0 < end; s0 += 32) {
        const bool in = s0 + lane < end;
        const int my_key = in ? keys[s0 + lane] : j.vocab, my_token = in ? order[s0 + lane] : 0;
        const int count = static_cast<int>(min(32LL, end - s0));
        for (int k0 = 0; k0 < count; k0 += kAhead) {
            Piece p[kAhead];
            int key[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                key[k] = __shfl_sync(0xffffffffu, my_key, k0 + k);
                const int t = __shfl_sync(0xffffffffu, my_token, k0 + k);
                if (mine && key[k] < j.vocab)
                    p[k].load_stream(dy + t * j.lddy, v, j.cols);
                else
                    p[k].clear();
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (k0 + k >= count) break;
                if (key[k] != current) {
                    flush(false);
                    current = key[k];
                }
                float f[N];
                p[k].get(f);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += f[e];
            }
        }
    }
    flush(end < j.tokens && keys[end] == current);
}

// Blocks up to join_blocks add the parts of the id that begins in a chunk and goes on
// behind it, a warp a strip, or the whole block one strip after the other where there
// are many; the others set the rows of ids that do not occur to zero, a warp a row.
constexpr int kManyParts = 32;

template <typename Piece, typename O, bool WIDE>
__global__ void __launch_bounds__(kThreads) embedding_rows_kernel(EmbeddingJob j, const int* keys, const float* part,
                                                                  const int* starts, int chunk, int chunks, unsigned per_row,
                                                                  unsigned strips, unsigned join_blocks) {
    constexpr int N = Piece::kSize;
    using Wideness = std::integral_constant<bool, WIDE>;
    __shared__ float sums[kWarps][32][N + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    O* out = static_cast<O*>(j.dtable);
    if (blockIdx.x >= join_blocks) {
        const long long r = static_cast<long long>(blockIdx.x - join_blocks) * kWarps + warp;
        if (r >= j.vocab || starts[r] != starts[r + 1]) return;
        float zero[N];
#pragma unroll
        for (int e = 0; e < N; ++e) zero[e] = 0.0f;
        for (unsigned v = lane; v < per_row; v += 32) store_row<O, N>(out + r * j.lddt, v, j.cols, zero, Wideness{});
        return;
    }
    const unsigned per_chunk = (strips + kWarps - 1) / kWarps;  // blocks
    const long long c = blockIdx.x / per_chunk;
    const unsigned strip0 = (blockIdx.x - static_cast<unsigned>(c) * per_chunk) * kWarps;
    const long long end = (c + 1) * chunk;
    if (end >= j.tokens) return;
    const int id = keys[end];
    if (id >= j.vocab || keys[end - 1] != id) return;             // nothing goes on behind this chunk
    if (starts[id] < c * chunk) return;                           // it began in an earlier one, which adds it up
    const long long last = (starts[id + 1] - 1) / chunk;
    const long long parts = last - c;                             // of the chunks behind this one
    auto add = [&](float (&acc)[N], const float* p) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + e);
            acc[e] += f.x, acc[e + 1] += f.y, acc[e + 2] += f.z, acc[e + 3] += f.w;
        }
    };
    if (parts <= kManyParts) {
        const unsigned v = (strip0 + warp) * 32 + lane;
        if (v >= per_row) return;
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        add(acc, part_at(const_cast<float*>(part), c, 1, per_row, v, N));
#pragma unroll 4
        for (long long k = c + 1; k <= last; ++k) add(acc, part_at(const_cast<float*>(part), k, 0, per_row, v, N));
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= j.scale;
        store_row<O, N>(out + id * j.lddt, v, j.cols, acc, Wideness{});
        return;
    }
    const long long each = (parts + kWarps - 1) / kWarps;
    for (unsigned strip = strip0; strip < min(strip0 + kWarps, strips); ++strip) {
        const unsigned v = strip * 32 + lane;
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        if (v < per_row) {
            if (warp == 0) add(acc, part_at(const_cast<float*>(part), c, 1, per_row, v, N));
            const long long k1 = min(c + (warp + 1) * each, last);
#pragma unroll 8
            for (long long k = c + 1 + warp * each; k <= k1; ++k) add(acc, part_at(const_cast<float*>(part), k, 0, per_row, v, N));
        }
#pragma unroll
        for (int e = 0; e < N; ++e) sums[warp][lane][e] = acc[e];
        __syncthreads();
        if (warp == 0 && v < per_row) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                for (int w = 1; w < kWarps; ++w) acc[e] += sums[w][lane][e];
                acc[e] *= j.scale;
            }
            store_row<O, N>(out + id * j.lddt, v, j.cols, acc, Wideness{});
        }
        __syncthreads();
    }
}

unsigned pieces_of(int cols, int n, bool vec) {
    const int loose = 32 * kLoose;
    return static_cast<unsigned>(vec ? cols / n : (static_cast<long long>(cols) + loose - 1) / loose * 32);
}

bool backward_vec(const EmbeddingJob& j) {
    const int es = elem_bytes(j.dtype), n = 16 / es, eo = elem_bytes(j.out_dtype);
    const int align = std::min(16, n * eo);  // of a piece of the output
    return j.cols % n == 0 && rows_aligned(j.dy, j.lddy, j.tokens, es) &&
           (reinterpret_cast<uintptr_t>(j.dtable) & (align - 1)) == 0 && j.lddt * eo % align == 0;
}

template <typename I>
TokenDigits<I> digits_of(const EmbeddingJob& j, const EmbeddingPlan& p, int pass) {
    const bool first = pass == 0;
    return {static_cast<const I*>(j.ids), first ? nullptr : p.keys[pass & 1], first ? nullptr : p.order[pass & 1], j.vocab,
            pass * p.bits, (1 << p.bits) - 1, p.keys[(pass + 1) & 1], p.order[(pass + 1) & 1]};
}

}  // namespace

int launch_embedding(const EmbeddingJob& j, cudaStream_t s) {
    const int es = elem_bytes(j.dtype), n = 16 / es;
    const bool vec = j.cols % n == 0 && rows_aligned(j.table, j.ldt, j.vocab, es) && rows_aligned(j.y, j.ldy, j.tokens, es);
    const unsigned per_row = pieces_of(j.cols, n, vec);
    const unsigned long long blocks = (static_cast<unsigned long long>(j.tokens) * per_row + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(std::min<unsigned long long>(blocks, 0x7fffffffULL)));
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        using W = Wide<T, 16 / sizeof(T)>;
        using L = Loose<T>;
        auto k = j.id_bytes == 8 ? (vec ? embedding_kernel<T, W, long long> : embedding_kernel<T, L, long long>)
                                 : (vec ? embedding_kernel<T, W, int> : embedding_kernel<T, L, int>);
        return static_cast<int>(launch_after(k, grid, dim3(kThreads), 0, s, j, per_row));
    });
}

EmbeddingPlan embedding_plan(const EmbeddingJob& j, char* scratch) {
    EmbeddingPlan p{};
    int bits = 1;
    while ((static_cast<long long>(j.vocab) >> bits) != 0) ++bits;  // ids 0 .. vocab
    p.passes = (bits + 9) / 10;
    p.bits = (bits + p.passes - 1) / p.passes;
    const size_t hist = sort_scratch(j.tokens, (1 << p.bits) - 1);
    p.counts = hist != 0;
    p.chunk = 32;
    while (static_cast<long long>(p.chunk) * 2048 < j.tokens) p.chunk *= 2;
    p.chunks = (j.tokens + p.chunk - 1) / p.chunk;
    const bool vec = backward_vec(j);
    const int n = 16 / elem_bytes(j.dtype);
    const size_t row = sizeof(float) * pieces_of(j.cols, n, vec) * (vec ? n : kLoose);
    auto take = [&](size_t bytes) {
        char* at = scratch + p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    const size_t tokens = sizeof(int) * static_cast<size_t>(j.tokens);
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = reinterpret_cast<int*>(take(tokens));
        p.order[i] = reinterpret_cast<int*>(take(tokens));
    }
    p.hist = reinterpret_cast<int*>(take(hist));
    p.starts = reinterpret_cast<int*>(take(sizeof(int) * (static_cast<size_t>(j.vocab) + 1)));
    p.part = reinterpret_cast<float*>(take(p.chunks > 1 ? 2 * row * p.chunks : 0));
    return p;
}

int launch_embedding_count(const EmbeddingJob& j, const EmbeddingPlan& p, int pass, cudaStream_t s) {
    const int G = (1 << p.bits) - 1;
    return j.id_bytes == 8 ? launch_sort_count(digits_of<long long>(j, p, pass), j.tokens, G, p.hist, s)
                           : launch_sort_count(digits_of<int>(j, p, pass), j.tokens, G, p.hist, s);
}

int launch_embedding_place(const EmbeddingJob& j, const EmbeddingPlan& p, int pass, cudaStream_t s) {
    const int G = (1 << p.bits) - 1;
    const int* hist = p.counts ? p.hist : nullptr;
    return j.id_bytes == 8 ? launch_sort_place(digits_of<long long>(j, p, pass), j.tokens, G, hist, s)
                           : launch_sort_place(digits_of<int>(j, p, pass), j.tokens, G, hist, s);
}

int launch_embedding_runs(const EmbeddingJob& j, const EmbeddingPlan& p, cudaStream_t s) {
    const bool vec = backward_vec(j);
    const unsigned per_row = pieces_of(j.cols, 16 / elem_bytes(j.dtype), vec), strips = (per_row + 31) / 32;
    const unsigned long long runs = (static_cast<unsigned long long>(p.chunks) * strips + kWarps - 1) / kWarps;
    const unsigned long long finds = (static_cast<unsigned long long>(j.vocab) + kThreads) / kThreads;
    const int* keys = p.keys[p.passes & 1];
    const int* order = p.order[p.passes & 1];
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_dtype(j.out_dtype, [&](auto o) {
            using O = decltype(o);
            auto k = vec ? embedding_runs_kernel<T, Wide<T, 16 / sizeof(T)>, O, true> : embedding_runs_kernel<T, Loose<T>, O, false>;
            return static_cast<int>(launch_after(k, dim3(static_cast<unsigned>(runs + finds)), dim3(kThreads), 0, s, j, keys, order,
                                                 p.part, p.starts, p.chunk, p.chunks, per_row, strips, static_cast<unsigned>(runs)));
        });
    });
}

int launch_embedding_rows(const EmbeddingJob& j, const EmbeddingPlan& p, cudaStream_t s) {
    const bool vec = backward_vec(j);
    const unsigned per_row = pieces_of(j.cols, 16 / elem_bytes(j.dtype), vec), strips = (per_row + 31) / 32;
    const unsigned joins = p.chunks > 1 ? static_cast<unsigned>(p.chunks) * ((strips + kWarps - 1) / kWarps) : 0;
    const unsigned zeros = (static_cast<unsigned>(j.vocab) + kWarps - 1) / kWarps;
    const int* keys = p.keys[p.passes & 1];
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_dtype(j.out_dtype, [&](auto o) {
            using O = decltype(o);
            auto k = vec ? embedding_rows_kernel<Wide<T, 16 / sizeof(T)>, O, true> : embedding_rows_kernel<Loose<T>, O, false>;
            return static_cast<int>(launch_after(k, dim3(joins + zeros), dim3(kThreads), 0, s, j, keys, static_cast<const float*>(p.part),
                                                 static_cast<const int*>(p.starts), p.chunk, p.chunks, per_row, strips, joins));
        });
    });
}

}  // namespace gns
