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
// - joins: the parts of an id that spans chunks are added in order.
// The rows of ids that do not occur are set to zero beside the sort, whose few blocks
// wait for latency: its first kernel marks the ids that do, and every later one has
// blocks for a share of the rows.
//
// Bound: HBM. Forward the rows and y; backward dy read and the table written once.
// 16384 tokens of 4096 bf16 values: forward 42 us (6.5 TB/s); backward, of 32768 rows, 83
// (4.8 TB/s of dy and the table): the sort with the empty rows about 45, the runs 30,
// which is their share of HBM, the joins 5. 131072 tokens of 2048, a third of them one id,
// to 131072 rows in fp32: 272 (5.9). A single token: the table, 43 (6.3).
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

// Rows of the table's gradient to set to zero: those of [begin, end) without a mark.
struct Zeros {
    const unsigned char* marks;
    long long begin, end;
    char* table;
    long long ld;  // bytes, as the others
    int row, element;
    int rows, share, lanes;  // that a block looks after, and warps of it, or lanes, for each
};

// z.share warps a row, or LANES lanes (0: z.lanes), in 16-byte stores but for a row's ends.
template <int LANES>
__device__ __forceinline__ void set_zero(const Zeros& z, unsigned block) {
    const int lanes = LANES ? LANES : z.lanes;
    const int worker = threadIdx.x / lanes, lane = threadIdx.x & (lanes - 1), part = worker % z.share;
    const long long r0 = z.begin + static_cast<long long>(block) * z.rows, r1 = min(r0 + z.rows, z.end);
    for (long long r = r0 + worker / z.share; r < r1; r += blockDim.x / lanes / z.share) {
        if (z.marks[r]) continue;
        char* at = z.table + r * z.ld;
        const int head = min(static_cast<int>(-reinterpret_cast<intptr_t>(at) & 15), z.row), body = (z.row - head) >> 4;
        uint4* wide = reinterpret_cast<uint4*>(at + head);
#pragma unroll 4
        for (int i = lanes * part + lane; i < body; i += lanes * z.share) wide[i] = make_uint4(0, 0, 0, 0);
        if (part > 0) continue;
        for (int b = lane * z.element; b < z.row - 16 * body; b += lanes * z.element) {  // the ends' elements
            char* e = at + (b < head ? b : b + 16 * body);
            if (z.element == 4)
                *reinterpret_cast<unsigned*>(e) = 0;
            else
                *reinterpret_cast<unsigned short*>(e) = 0;
        }
    }
}

// (65536 tokens of 3000000 x 16 bf16: 320 us with a warp a row, 87 with two lanes.)
__device__ __forceinline__ void set_zero(const Zeros& z, unsigned block) {
    if (z.lanes == 32)
        set_zero<32>(z, block);
    else
        set_zero<0>(z, block);
}

// The tokens by one digit of their id (vocab for those without a row, which are last).
template <typename I>
struct TokenDigits {
    const I* ids;                // the first pass reads these,
    const int *keys_in, *order_in;  // later ones what the pass before wrote
    int vocab, shift, mask;
    int *keys_out, *order_out;
    unsigned char* marks;  // where the ids are to be marked, or null
    Zeros zeros;
    __device__ __forceinline__ int key(long long s) const { return keys_in ? keys_in[s] : row_of(ids, s, vocab); }
    __device__ __forceinline__ int digit(int key) const { return (key >> shift) & mask; }
    __device__ __forceinline__ int value(long long s) const { return order_in ? order_in[s] : static_cast<int>(s); }
    __device__ __forceinline__ void place(long long, int key, int value, int at) const {
        keys_out[at] = key;
        order_out[at] = value;
    }
    __device__ __forceinline__ void start(int, int) const {}
    // Ids that a block has marked lately, so that frequent ones are not written over and
    // over (262144 tokens of 32768 ids, log-uniform: 31 us, 22 so).
    static constexpr int kSeen = 1024;
    __device__ static __forceinline__ int* seen() {
        __shared__ int ids[kSeen];
        return ids;
    }
    __device__ __forceinline__ void begin() const {
        if (!marks) return;
        for (int i = threadIdx.x; i < kSeen; i += blockDim.x) seen()[i] = -1;
    }
    __device__ __forceinline__ void note(int key) const {
        if (!marks || key >= vocab) return;
        int* last = seen() + (key & (kSeen - 1));
        if (*last == key) return;
        *last = key;
        marks[key] = 1;
    }
    __device__ __forceinline__ void extra(unsigned block) const { set_zero(zeros, block); }
};

// The parts of chunk c: [c][0] of an id that began before it, [c][1] of one that
// began in it and goes on behind it.
__device__ __forceinline__ float* part_at(float* part, long long c, int which, unsigned per_row, unsigned v, int N) {
    return part + ((c * 2 + which) * per_row + v) * N;
}

constexpr int kAhead = 8;  // rows in flight with the one that is added

struct Runs {
    const int *keys, *order;  // sorted
    float* part;
    int chunk, chunks;
    unsigned per_row, strips;  // pieces of a row, in strips of 32
    unsigned blocks;
    unsigned* ready;  // blocks that have added their share of an id's parts, at first: 0
};

// Blocks beyond w.blocks set rows to zero (where no kernel of the sort could).
template <typename T, typename Piece, typename O, bool WIDE>
__global__ void __launch_bounds__(kThreads) embedding_runs_kernel(EmbeddingJob j, Runs w, Zeros z) {
    constexpr int N = Piece::kSize;
    using Wideness = std::integral_constant<bool, WIDE>;
    __shared__ __align__(128) uint4 ring[WIDE ? kAhead * kThreads : 1];  // [row][thread]
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= w.blocks) {
        set_zero(z, blockIdx.x - w.blocks);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned long long item = static_cast<unsigned long long>(blockIdx.x) * kWarps + warp;
    const long long c = static_cast<long long>(item / w.strips);
    if (c >= w.chunks) return;
    const unsigned v = static_cast<unsigned>(item - c * w.strips) * 32 + lane;
    const bool mine = v < w.per_row;
    const int beg = static_cast<int>(c * w.chunk), count = min(w.chunk, j.tokens - beg);
    const T* dy = static_cast<const T*>(j.dy);
    O* out = static_cast<O*>(j.dtable);
    // The keys of 32 sorted places and their tokens, -1 for one without a row, and those of
    // the next 32.
    auto places = [&](int at, int& key, int& token) {
        const bool in = at + lane < count;
        key = in ? w.keys[beg + at + lane] : j.vocab;
        token = in && key < j.vocab ? w.order[beg + at + lane] : -1;
    };
    int key, token, next_key, next_token;
    places(0, key, token);
    places(32, next_key, next_token);
    const int key_before = beg > 0 ? w.keys[beg - 1] : -1, key_behind = beg + count < j.tokens ? w.keys[beg + count] : -1;
    // The row of place `at`, which is among the 32 from base on or among the next; nothing
    // is fetched, and what is there is not used, where it has none.
    auto row_at = [&](int at, int base) -> const T* {
        const int t = __shfl_sync(0xffffffffu, at - base < 32 ? token : next_token, at & 31);
        return mine && t >= 0 ? dy + t * j.lddy : nullptr;
    };
    const uint4* slots = ring + threadIdx.x;
    auto fetch = [&](int at, int base) {
        const T* row = row_at(at, base);
        if (row) copy16(smem_u32(slots + (at % kAhead) * kThreads), row + static_cast<long long>(v) * N);
        copies_commit();
    };
    constexpr int kTurn = 4;  // places that a turn of the loop takes
    Piece held[WIDE ? 1 : kTurn];
    float2 acc[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) acc[e] = both(0.0f);
    int current = __shfl_sync(0xffffffffu, key, 0);
    bool before = key_before == current;  // the id began in an earlier chunk
    auto flush = [&](bool behind) {
        if (current < j.vocab && mine) {
            if (before || behind) {
                float* p = part_at(w.part, c, before ? 0 : 1, w.per_row, v, N);
#pragma unroll
                for (int e = 0; e < N / 2; e += 2) *reinterpret_cast<float4*>(p + 2 * e) = make_float4(acc[e].x, acc[e].y, acc[e + 1].x, acc[e + 1].y);
            } else {
                float f[N];
#pragma unroll
                for (int e = 0; e < N / 2; ++e) {
                    const float2 s = mul2(acc[e], both(j.scale));
                    f[2 * e] = s.x, f[2 * e + 1] = s.y;
                }
                store_row<O, N>(out + current * j.lddt, v, j.cols, f, Wideness{});
            }
        }
#pragma unroll
        for (int e = 0; e < N / 2; ++e) acc[e] = both(0.0f);
        before = false;
    };
    if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < kAhead - 1; ++k) fetch(k, 0);
    } else {
#pragma unroll
        for (int k = 0; k < kTurn; ++k) {
            held[k].clear();
            if (const T* row = row_at(k, 0)) held[k].load_stream(row, v, j.cols);
        }
    }
    for (int at0 = 0; at0 < count; at0 += kTurn) {
        if (at0 > 0 && at0 % 32 == 0) {
            key = next_key, token = next_token;
            places(at0 + 32, next_key, next_token);
        }
#pragma unroll
        for (int u = 0; u < kTurn; ++u) {
            const int at = at0 + u;
            if (at >= count) break;
            const int k = __shfl_sync(0xffffffffu, key, at & 31);
            float f[N];
            if constexpr (WIDE) {
                fetch(at + kAhead - 1, at0 & ~31);
                copies_wait<kAhead - 1>();
                Piece p;
                p.p.p[0] = slots[(at % kAhead) * kThreads];
                p.get(f);
            } else {
                held[u].get(f);
                held[u].clear();
                if (const T* row = row_at(at + kTurn, at0 & ~31)) held[u].load_stream(row, v, j.cols);
            }
            if (k != current) {
                flush(false);
                current = k;
            }
#pragma unroll
            for (int e = 0; e < N / 2; ++e) acc[e] = add2(acc[e], make_float2(f[2 * e], f[2 * e + 1]));
        }
    }
    copies_wait<0>();
    flush(key_behind == current);
}

// A block for each chunk and 16 strips adds the parts of the id that begins in the chunk
// and goes on behind it, a warp a strip. The parts of an id that spans many chunks are
// shared: the blocks of its first 16 chunks take a strip each, every warp a part of the
// chunks; beyond kMostParts eight blocks share a strip, and the one that is ready last
// adds their sums, in order. (One block reads 55 GB/s: 680 parts of 2048 columns took
// it 20 us.)
constexpr int kManyParts = 32, kMostParts = 128, kJoinWarps = 16, kShare = 8;

template <typename Piece, typename O, bool WIDE>
__global__ void __launch_bounds__(32 * kJoinWarps) embedding_joins_kernel(EmbeddingJob j, Runs w) {
    constexpr int N = Piece::kSize;
    using Wideness = std::integral_constant<bool, WIDE>;
    __shared__ float sums[kJoinWarps][32][N + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned groups = (w.strips + kJoinWarps - 1) / kJoinWarps;  // blocks of a chunk
    const long long c = blockIdx.x / groups;
    const unsigned strip0 = (blockIdx.x - static_cast<unsigned>(c) * groups) * kJoinWarps;
    const long long end = (c + 1) * w.chunk;
    if (end >= j.tokens) return;
    const int id = w.keys[end];
    if (id >= j.vocab || w.keys[end - 1] != id) return;  // nothing goes on behind this chunk
    // How far the id reaches, in chunks: lane l looks at the border l chunks ahead and
    // l chunks back; beyond 32 ahead a search finds its end.
    const long long ahead_at = (c + 2 + lane) * w.chunk, back_at = (c - lane) * w.chunk - 1;
    const unsigned ahead = __ballot_sync(0xffffffffu, ahead_at < j.tokens && w.keys[min(ahead_at, static_cast<long long>(j.tokens) - 1)] == id);
    const unsigned back = __ballot_sync(0xffffffffu, back_at >= 0 && w.keys[max(back_at, 0LL)] == id);
    int before = back == 0xffffffffu ? 32 : __ffs(~back) - 1;
    for (int more = 32; before == more && more < kJoinWarps * kShare; more += 32) {
        const long long at = (c - more - lane) * w.chunk - 1;
        const unsigned b = __ballot_sync(0xffffffffu, at >= 0 && w.keys[max(at, 0LL)] == id);
        before += b == 0xffffffffu ? 32 : __ffs(~b) - 1;
    }
    const bool began = before > 0;  // in an earlier chunk
    const long long first = c - before;
    if (before >= kJoinWarps * kShare) return;
    long long last = c + __ffs(~ahead);
    if (ahead == 0xffffffffu) {  // from chunk c + 32 on: in steps of 64 chunks, two and one, of 2048 at most
        last = c + 32;
        for (int step = 64; step > 0; step = step == 64 ? 2 : step - 1) {
            const long long at = (last + static_cast<long long>(lane) * step) * w.chunk;
            last += static_cast<long long>(step) * (__popc(__ballot_sync(0xffffffffu, at < j.tokens && w.keys[min(at, static_cast<long long>(j.tokens) - 1)] == id)) - 1);
        }
    }
    const long long parts = last - first;  // of the chunks behind the first
    O* out = static_cast<O*>(j.dtable) + id * j.lddt;
    auto add = [&](float (&acc)[N], const float* p) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + e);
            acc[e] += f.x, acc[e + 1] += f.y, acc[e + 2] += f.z, acc[e + 3] += f.w;
        }
    };
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    if (parts <= kManyParts) {
        const unsigned v = (strip0 + warp) * 32 + lane;
        if (began || v >= w.per_row) return;
        add(acc, part_at(w.part, first, 1, w.per_row, v, N));
#pragma unroll 4
        for (long long k = first + 1; k <= last; ++k) add(acc, part_at(w.part, k, 0, w.per_row, v, N));
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= j.scale;
        store_row<O, N>(out, v, j.cols, acc, Wideness{});
        return;
    }
    const int share = parts > kMostParts ? kShare : 1, turn = static_cast<int>(c - first) % share;
    const unsigned strip = strip0 + static_cast<unsigned>(c - first) / share;
    if (c - first >= kJoinWarps * share || strip >= w.strips) return;
    const unsigned v = strip * 32 + lane;
    // This block's chunks, (from, to], and the warp's of them.
    const long long from = first + parts * turn / share, to = first + parts * (turn + 1) / share;
    const long long each = (to - from + kJoinWarps - 1) / kJoinWarps;
    if (v < w.per_row) {
        if (warp == 0 && turn == 0) add(acc, part_at(w.part, first, 1, w.per_row, v, N));
        const long long k1 = min(from + (warp + 1) * each, to);
#pragma unroll 8
        for (long long k = from + 1 + warp * each; k <= k1; ++k) add(acc, part_at(w.part, k, 0, w.per_row, v, N));
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sums[warp][lane][e] = acc[e];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int e = 0; e < N; ++e)
        for (int k = 1; k < kJoinWarps; ++k) acc[e] += sums[k][lane][e];
    if (share > 1) {
        // The sum goes where the block's first part was, which nobody else reads.
        float* mine = part_at(w.part, from + 1, 0, w.per_row, v, N);
        if (v < w.per_row) {
#pragma unroll
            for (int e = 0; e < N; e += 4) *reinterpret_cast<float4*>(mine + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        }
        __threadfence();
        __syncwarp();
        unsigned ready = 0;
        if (lane == 0) ready = atomicAdd(w.ready + first / kMostParts * w.strips + strip, 1u);
        if (__shfl_sync(0xffffffffu, ready, 0) != kShare - 1) return;
        __threadfence();
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        if (v < w.per_row) {
#pragma unroll
            for (int k = 0; k < kShare; ++k) {
                const float* p = part_at(w.part, first + parts * k / kShare + 1, 0, w.per_row, v, N);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += __ldcg(p + e);
            }
        }
    }
    if (v >= w.per_row) return;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] *= j.scale;
    store_row<O, N>(out, v, j.cols, acc, Wideness{});
}

int next_pow2(int v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
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

// A warp of the sort takes 32 tokens at a time and its rounds wait for one another, so
// many blocks of a round or two each are better than few; but each block reads the counts
// of all.
constexpr long long kMostCounts = 32768;
SortPlan sort_plan(const EmbeddingJob& j, const EmbeddingPlan& p) {
    return {j.tokens, (1 << p.bits) - 1, 1024, std::max(512LL, (static_cast<long long>(j.tokens) << p.bits) / kMostCounts)};
}

Runs runs_of(const EmbeddingJob& j, const EmbeddingPlan& p, bool vec) {
    Runs w{};
    w.keys = p.keys[p.passes & 1];
    w.order = p.order[p.passes & 1];
    w.part = p.part;
    w.ready = p.ready;
    w.chunk = p.chunk;
    w.chunks = p.chunks;
    w.per_row = pieces_of(j.cols, 16 / elem_bytes(j.dtype), vec);
    w.strips = (w.per_row + 31) / 32;
    w.blocks = static_cast<unsigned>((static_cast<unsigned long long>(p.chunks) * w.strips + kWarps - 1) / kWarps);
    return w;
}

// The rows that the h-th of p.hosts kernels sets to zero, and the blocks it has for them.
Zeros zeros_of(const EmbeddingJob& j, const EmbeddingPlan& p, int h, unsigned* blocks) {
    Zeros z{};
    *blocks = 0;
    if (h < 0 || h >= p.hosts) return z;
    const int eo = elem_bytes(j.out_dtype);
    z.marks = p.marks;
    z.begin = static_cast<long long>(j.vocab) * h / p.hosts;
    z.end = static_cast<long long>(j.vocab) * (h + 1) / p.hosts;
    z.table = static_cast<char*>(j.dtable);
    z.ld = j.lddt * eo;
    z.row = j.cols * eo;
    z.element = eo;
    z.share = z.row <= 4096 ? 1 : z.row <= 8192 ? 2 : 4;
    z.lanes = std::min(32, next_pow2((z.row + 15) / 16));
    z.rows = std::max(kWarps / z.share, (32 << 10) / z.row);
    *blocks = static_cast<unsigned>((z.end - z.begin + z.rows - 1) / z.rows);
    return z;
}

// step: the kernel's number in the sort. The first marks, the others set rows to zero.
template <typename I>
TokenDigits<I> digits_of(const EmbeddingJob& j, const EmbeddingPlan& p, int pass, int step, unsigned* extra) {
    const bool first = pass == 0;
    return {static_cast<const I*>(j.ids), first ? nullptr : p.keys[pass & 1], first ? nullptr : p.order[pass & 1], j.vocab,
            pass * p.bits, (1 << p.bits) - 1, p.keys[(pass + 1) & 1], p.order[(pass + 1) & 1], step == 0 ? p.marks : nullptr,
            zeros_of(j, p, step - 1, extra)};
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

// 27 warps a processor (4093 tokens of 1021 fp32 values: 60 us with runs of 32, 48 of 8).
constexpr long long kLeastRuns = 4096;

EmbeddingPlan embedding_plan(const EmbeddingJob& j, char* scratch) {
    EmbeddingPlan p{};
    int bits = 1;
    while ((static_cast<long long>(j.vocab) >> bits) != 0) ++bits;  // ids 0 .. vocab
    p.passes = (bits + 9) / 10;
    p.bits = (bits + p.passes - 1) / p.passes;
    const size_t hist = sort_scratch(sort_plan(j, p));
    p.counts = hist != 0;
    const bool vec = backward_vec(j);
    const int n = 16 / elem_bytes(j.dtype);
    const long long strips = (pieces_of(j.cols, n, vec) + 31) / 32;
    // Few tokens: short runs, so that there are warps for every processor. Else runs whose
    // parts are few bytes beside dy (65536 tokens of 1024 x 2048 bf16: 95 us by 32, 87 by 64).
    p.chunk = 64;
    while (p.chunk > 8 && strips * j.tokens < kLeastRuns * p.chunk) p.chunk /= 2;
    while (static_cast<long long>(p.chunk) * 2048 < j.tokens) p.chunk *= 2;
    p.chunks = static_cast<int>((static_cast<long long>(j.tokens) + p.chunk - 1) / p.chunk);
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
    p.hosts = std::max(1, p.passes * (p.counts ? 2 : 1) - 1);
    p.ready = reinterpret_cast<unsigned*>(take(sizeof(unsigned) * strips * (p.chunks / kMostParts + 1)));
    p.marks = reinterpret_cast<unsigned char*>(take(j.vocab));
    p.cleared = p.marks + j.vocab - reinterpret_cast<unsigned char*>(p.ready);
    p.part = reinterpret_cast<float*>(take(p.chunks > 1 ? 2 * row * p.chunks : 0));
    return p;
}

int launch_embedding_count(const EmbeddingJob& j, const EmbeddingPlan& p, int pass, cudaStream_t s) {
    unsigned extra;
    const auto run = [&](const auto& src) { return launch_sort_count(src, sort_plan(j, p), p.hist, s, extra); };
    if (j.id_bytes == 8) return run(digits_of<long long>(j, p, pass, 2 * pass, &extra));
    return run(digits_of<int>(j, p, pass, 2 * pass, &extra));
}

int launch_embedding_place(const EmbeddingJob& j, const EmbeddingPlan& p, int pass, cudaStream_t s) {
    unsigned extra;
    const int step = p.counts ? 2 * pass + 1 : pass;
    const auto run = [&](const auto& src) { return launch_sort_place(src, sort_plan(j, p), p.counts ? p.hist : nullptr, s, extra); };
    if (j.id_bytes == 8) return run(digits_of<long long>(j, p, pass, step, &extra));
    return run(digits_of<int>(j, p, pass, step, &extra));
}

int launch_embedding_runs(const EmbeddingJob& j, const EmbeddingPlan& p, cudaStream_t s) {
    const bool vec = backward_vec(j);
    const Runs w = runs_of(j, p, vec);
    unsigned extra;  // the only host where the sort is a single kernel
    const Zeros z = zeros_of(j, p, p.passes * (p.counts ? 2 : 1) == 1 ? 0 : -1, &extra);
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_dtype(j.out_dtype, [&](auto o) {
            using O = decltype(o);
            auto k = vec ? embedding_runs_kernel<T, Wide<T, 16 / sizeof(T)>, O, true> : embedding_runs_kernel<T, Loose<T>, O, false>;
            return static_cast<int>(launch_after(k, dim3(w.blocks + extra), dim3(kThreads), 0, s, j, w, z));
        });
    });
}

int launch_embedding_joins(const EmbeddingJob& j, const EmbeddingPlan& p, cudaStream_t s) {
    const bool vec = backward_vec(j);
    const Runs w = runs_of(j, p, vec);
    const unsigned blocks = static_cast<unsigned>(p.chunks) * ((w.strips + kJoinWarps - 1) / kJoinWarps);
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_dtype(j.out_dtype, [&](auto o) {
            using O = decltype(o);
            auto k = vec ? embedding_joins_kernel<Wide<T, 16 / sizeof(T)>, O, true> : embedding_joins_kernel<Loose<T>, O, false>;
            return static_cast<int>(launch_after(k, dim3(blocks), dim3(32 * kJoinWarps), 0, s, j, w));
        });
    });
}

}  // namespace gns
