// Launchers of layer norm and its gradients (layer_norm.cu, layer_norm_backward.cu).
//
// y = (x - mean) * rstd * weight + bias over each row of `cols` elements, rstd =
// 1 / sqrt(var + eps), var the mean of the squares of x - mean; with rms the mean
// is taken as 0.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "blockops.cuh"
#include "ptx.cuh"

namespace gns {

struct NormJob {
    const void* x;
    long long ldx;
    long long rows;
    int cols, dtype;
    const void* weight;  // fp32 where wf32, else of dtype; null for 1
    const void* bias;    // forward; null for 0
    int wf32, rms;
    int again;  // forward: rows may be read again after y is written
    float eps;
    void* y;  // forward
    long long ldy;
    float* stats;  // [rows][2]: mean, rstd; written forward, read backward
    // backward
    const void* dy;
    long long lddy;
    const void* residual;  // null for 0
    long long ldr;
    void* dx;
    long long lddx;
    void* dweight;  // typed as weight; either may be null
    void* dbias;
    float* part;    // norm_backward_scratch() bytes
    DevStatus st;   // of waits among the CTAs of a row
    int tpr, per_row;  // set by the launchers
    int ctas, per_cta;  // of the ring kernels: CTAs that share a row, and pieces of each (unaligned: columns of a thread)
    int stages;         // of unaligned rows, backward: rows in flight with the one that is worked on, 2 or 3
};

int launch_layer_norm(NormJob job, int num_sms, cudaStream_t s);

// One kernel; where a weight's or bias' gradient is asked for a second one joins
// the blocks' sums, and rows beyond a block's registers take a kernel of their own
// for those sums.
size_t norm_backward_scratch(const NormJob& job, int num_sms);
int launch_layer_norm_backward(NormJob job, int num_sms, cudaStream_t s);
bool layer_norm_columns_apart(const NormJob& job);
int launch_layer_norm_columns(NormJob job, int num_sms, cudaStream_t s);
int launch_layer_norm_join(NormJob job, int num_sms, cudaStream_t s);

// ------------------------------------------------- pieces of weights and rows

// The weights of a piece as fp32 values, 0 beyond the row.
template <typename T, int N>
__device__ __forceinline__ void piece_weights(const Wide<T, N>&, const void* w, bool f32, unsigned v, int, float (&f)[N]) {
    if (f32) {
        Pack<float, N> p;
        p.load(static_cast<const float*>(w) + static_cast<long long>(v) * N);
        p.get(f);
    } else {
        Pack<T, N> p;
        p.load(static_cast<const T*>(w) + static_cast<long long>(v) * N);
        p.get(f);
    }
}
template <typename T>
__device__ __forceinline__ void piece_weights(const Loose<T>&, const void* w, bool f32, unsigned v, int H, float (&f)[kLoose]) {
#pragma unroll
    for (int i = 0; i < kLoose; ++i) {
        const int c = Loose<T>::column(v, i);
        f[i] = c >= H ? 0.0f : f32 ? static_cast<const float*>(w)[c] : to_f32<T>(static_cast<const T*>(w)[c]);
    }
}

// Whether element i of piece v lies in the row.
template <typename T, int N>
__device__ __forceinline__ bool piece_has(const Wide<T, N>&, unsigned, int, int) {
    return true;
}
template <typename T>
__device__ __forceinline__ bool piece_has(const Loose<T>&, unsigned v, int i, int H) {
    return Loose<T>::column(v, i) < H;
}

template <typename T, int N>
__device__ __forceinline__ int piece_column(const Wide<T, N>&, unsigned v, int i) {
    return static_cast<int>(v) * N + i;
}
template <typename T>
__device__ __forceinline__ int piece_column(const Loose<T>&, unsigned v, int i) {
    return Loose<T>::column(v, i);
}

// Sums of a and b over the threads of a row: `tpr` neighbouring lanes (a power of
// two) or, beyond 32, the whole block. `red` is shared memory of a pair per warp; a
// block's next call takes the other one of two, so one barrier does.
__device__ __forceinline__ void row_sum2(float& a, float& b, int tpr, float2* red) {
    for (int m = (tpr < 32 ? tpr : 32) >> 1; m > 0; m >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, m);
        b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, warps = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
        const float2 t = red[w];
        a += t.x;
        b += t.y;
    }
}

// The 16 bytes of a piece as pairs and back.
template <typename T, int N>
__device__ __forceinline__ void unpack(const uint4& u, float2 (&f)[N / 2]) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) f[i] = make_float2(to_f32<T>(e[2 * i]), to_f32<T>(e[2 * i + 1]));
}
__device__ __forceinline__ unsigned pack2(float2 a, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a.x, a.y);
    return *reinterpret_cast<const unsigned*>(&v);
}
__device__ __forceinline__ unsigned pack2(float2 a, __half) {
    const __half2 v = __floats2half2_rn(a.x, a.y);
    return *reinterpret_cast<const unsigned*>(&v);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
    return make_uint4(pack2(f[0], T{}), pack2(f[1], T{}), pack2(f[2], T{}), pack2(f[3], T{}));
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
}

// What the CTAs of a cluster that share a row exchange their sums through: every warp
// writes its sums into all of them (st.async), where they count on a barrier. A CTA can
// be one reduction ahead of another at most, so two buffers in turn are enough, and a
// count that comes before the barrier is armed for it is not lost.
constexpr int kMaxCtas = 8, kMostWarps = 16;  // of a row
template <int K>
struct __align__(128) RowSums {
    float4 sums[2][kMaxCtas * kMostWarps * K / 4 + 1];
    uint64_t full[2];
};

template <int K>
__device__ __forceinline__ void send_sums(uint32_t to, uint32_t bar, const float (&a)[K]) {
    static_assert(K == 2 || K == 4, "8 or 16 bytes");
    if (K == 2)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%2, %3}, [%1];" ::"r"(to), "r"(bar),
                     "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1]))
                     : "memory");
    else
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(to), "r"(bar),
                     "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2 % K])), "r"(__float_as_uint(a[3 % K]))
                     : "memory");
}

// Sums of K = 2 or 4 values over the threads of a row: `tpr` neighbouring lanes, the
// block (one barrier; its next call takes the other buffer of two), or, CLUSTER, the
// CTAs of the cluster. Across a whole warp the values part on the way: half the lanes go
// on with half of them, so that four cost 12 shuffles' and adds' worth instead of 40.
// use: reductions done so far.
template <int K, bool CLUSTER, int KS>
__device__ __forceinline__ void row_sums(float (&a)[K], const NormJob& j, RowSums<KS>& red, int& use, bool& dead) {
    const int tpr = j.tpr;
    if (tpr < 32) {
        for (int m = tpr >> 1; m > 0; m >>= 1) {
#pragma unroll
            for (int k = 0; k < K; ++k) a[k] += __shfl_xor_sync(0xffffffffu, a[k], m);
        }
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float v;
    if (K == 4) {
        const bool up = lane & 16;
        const float p = (up ? a[2 % K] : a[0]) + __shfl_xor_sync(0xffffffffu, up ? a[0] : a[2 % K], 16);
        const float q = (up ? a[3 % K] : a[1]) + __shfl_xor_sync(0xffffffffu, up ? a[1] : a[3 % K], 16);
        const bool odd = lane & 8;
        v = (odd ? q : p) + __shfl_xor_sync(0xffffffffu, odd ? p : q, 8);
    } else {
        const bool up = lane & 16;
        v = (up ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, up ? a[0] : a[1], 16);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
    }
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    constexpr int kSpan = 32 / K;  // lanes that hold the same sum
    const int buf = use & 1, warps = tpr >> 5;
    float* sums = reinterpret_cast<float*>(red.sums[buf]);
    if (tpr == 32 || CLUSTER) {
#pragma unroll
        for (int k = 0; k < K; ++k) a[k] = __shfl_sync(0xffffffffu, v, k * kSpan);
        if (!CLUSTER) return;
        const uint32_t bar = smem_u32(&red.full[buf]);
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(j.ctas * warps * K * sizeof(float)));
        if (lane < j.ctas) {  // lane l sends to CTA l
            const uint32_t to = smem_u32(sums + (cluster_ctarank() * warps + warp) * K);
            send_sums(map_to_rank(to, lane), map_to_rank(bar, lane), a);
        }
        if (!dead && !mbar_wait_cluster(bar, (use >> 1) & 1, j.st)) dead = true;
    } else {
        if (lane % kSpan == 0) sums[warp * K + lane / kSpan] = v;
        __syncthreads();
    }
    ++use;
    const int parts = CLUSTER ? warps * j.ctas : warps;
    if (K == 4) {
        float2 p = both(0.0f), q = both(0.0f);
#pragma unroll 4
        for (int w = 0; w < parts; ++w) {
            const float4 t = reinterpret_cast<const float4*>(sums)[w];
            p = add2(p, make_float2(t.x, t.y));
            q = add2(q, make_float2(t.z, t.w));
        }
        a[0] = p.x, a[1] = p.y, a[2 % K] = q.x, a[3 % K] = q.y;
    } else {
        float2 p = both(0.0f);
#pragma unroll 4
        for (int w = 0; w < parts; ++w) p = add2(p, reinterpret_cast<const float2*>(sums)[w]);
        a[0] = p.x, a[1] = p.y;
    }
}

// Pieces of a row, and whether they are 16 bytes wide.
inline bool norm_vec(const NormJob& j, bool backward) {
    const int es = elem_bytes(j.dtype);
    if (j.cols % (16 / es) || !rows_aligned(j.x, j.ldx, j.rows, es)) return false;
    if (j.weight && !rows_aligned(j.weight, 0, 1, 1)) return false;
    if (!backward) return rows_aligned(j.y, j.ldy, j.rows, es) && (!j.bias || rows_aligned(j.bias, 0, 1, 1));
    return rows_aligned(j.dy, j.lddy, j.rows, es) && rows_aligned(j.dx, j.lddx, j.rows, es) &&
           (!j.residual || rows_aligned(j.residual, j.ldr, j.rows, es));
}

inline int norm_pieces(const NormJob& j, bool vec) {
    const int n = 16 / elem_bytes(j.dtype), loose = 32 * kLoose;
    return vec ? j.cols / n : static_cast<int>((static_cast<long long>(j.cols) + loose - 1) / loose * 32);
}

// How the ring kernels share out rows of p pieces: V pieces, 16 elements (one piece of
// very short rows), for each of tpr threads of each of `ctas` CTAs.
constexpr int kRingThreads = 32 * kMostWarps;
constexpr int kStages = 3;                // batches of rows in flight, with the one that is worked on
constexpr size_t kRingBytes = 204 << 10;  // of shared memory, at most
struct RingShape {
    int V, threads, tpr, ctas, per_cta, resident;  // resident: threads of a processor
};

inline int next_pow2(int v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// n: elements of a piece; copies: pieces in flight for each of a row.
inline bool ring_shape(int p, int n, int copies, RingShape* s) {
    const int few = 16 / n;
    const int most = std::min(kRingThreads, static_cast<int>(kRingBytes / (sizeof(uint4) * copies * few)) / 32 * 32);
    s->threads = 256;
    s->V = p <= 4 ? 1 : few;
    s->ctas = 1;
    while (s->ctas < kMaxCtas && p > s->ctas * few * most) s->ctas *= 2;
    // A block of nine to eleven warps would leave the processor's other half idle, which
    // costs more than the exchange (8192 rows of 5120 bf16 values: 47 us, 39 by two CTAs).
    // One of twelve does not (5760: 44 us forward and 69 backward, 52 and 77 by two CTAs;
    // fp32 60 and 93, 64 and 90).
    if (s->ctas == 1 && p > 256 * few && p <= 352 * few) s->ctas = 2;
    s->per_cta = (p + s->ctas - 1) / s->ctas;
    // fp32 rows that would leave a quarter or more of the pieces of 64 threads' sixteen
    // elements empty: single pieces, which need half the registers (65536 x 640: 61 and 82
    // us instead of 70 and 107, 768: 78 and 98 instead of 79 and 118; bf16 gains nothing; rows
    // of less than a warp, whose lanes are a power of two, were not tried).
    const bool single = few == 4 && p > 128 && p <= 192;
    s->resident = single ? 1024 : 512;
    if (single) s->V = 1;
    if (p <= 32 * few)
        s->tpr = next_pow2((p + s->V - 1) / s->V);
    else
        s->threads = s->tpr = (s->per_cta + 32 * s->V - 1) / (32 * s->V) * 32;
    return s->tpr <= most;
}

// Clusters (or blocks) that walk the rows, `resident` CTAs a processor. Not every
// processor has its place in a cluster of four or eight (74 of 76 fours fitted), and one
// that has to wait for the others to end would double the time.
inline unsigned ring_clusters(const RingShape& c, long long batches, int num_sms, size_t smem) {
    const int resident = std::max(1, std::min(c.resident / c.threads, static_cast<int>(kRingBytes / smem)));
    long long fit = static_cast<long long>(num_sms) * resident / c.ctas;
    if (c.ctas > 2) fit = fit * 15 / 16;
    return static_cast<unsigned>(std::min(batches, std::max(1LL, fit)));
}

// Rows that are not 16-byte aligned are copied as the aligned 16-byte words that hold
// them, by the threads of a row together, to a slot that has room for one word more.
// The bytes of its first word before a row come along and are never used; those behind
// its end are not read.
//
// A thread has pairs of columns, `stride` apart: of rows of less than a warp the number
// of its lanes, else 32, a warp then having consecutive columns, so that every access
// of a thread lies at a known offset from its first (16384 x 4093 bf16: 69 us forward and
// 162 backward with a residual; 73 and 165 with columns a block's threads apart, whose offsets
// are sums).
constexpr int kLoosePairs = 8;

struct LooseColumns {
    int first;      // the thread's first column
    int whole;      // pairs that lie in the row for all threads of the row or warp
    int last;       // what the pair after those is from the first column on
    bool lo, hi;    // which of that pair's columns there are
};
template <bool NARROW>
__device__ __forceinline__ LooseColumns loose_columns(const NormJob& j, int at) {
    const int stride = NARROW ? j.tpr : 32, lane = NARROW ? at : at & 31;
    const int base = NARROW ? 0 : (at >> 5) * 32 * j.per_cta;
    const int len = NARROW ? j.cols : min(32 * j.per_cta, j.cols - base);  // columns of the row or warp
    const int whole = (len - 1) / (2 * stride), last = 2 * stride * whole;
    return {base + lane, whole, last, lane + last < len, lane + last + stride < len};
}
// Calls fn with each pair of the thread, its place from the first column on and which of the two there are.
template <bool NARROW, typename F>
__device__ __forceinline__ void loose_pairs(const LooseColumns& k, int tpr, F&& fn) {
#pragma unroll
    for (int q = 0; q < kLoosePairs - 1; ++q)
        if (q < k.whole) fn(q, 2 * q * (NARROW ? tpr : 32), true, true);
    fn(kLoosePairs - 1, k.last, k.lo, k.hi);
}

__host__ __device__ __forceinline__ int window_bytes(int row_bytes) { return (row_bytes + 15) / 16 * 16 + 16; }

template <typename T>
__device__ __forceinline__ void copy_window(uint32_t slot, const T* row, int cols, int at, int tpr) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row);
    const char* base = reinterpret_cast<const char*>(a & ~static_cast<uintptr_t>(15));
    const int bytes = static_cast<int>(a & 15) + cols * static_cast<int>(sizeof(T));
    for (int w = at; 16 * w < bytes; w += tpr) copy16(slot + 16 * w, base + 16 * w, min(16, bytes - 16 * w));
}

// The row's first element in its slot.
template <typename T>
__device__ __forceinline__ const T* in_window(const char* slot, const T* row) {
    return reinterpret_cast<const T*>(slot + (reinterpret_cast<uintptr_t>(row) & 15));
}

// After a thread's own copies have come: those of the others of its row, too, and the
// others are done with the rows before.
__device__ __forceinline__ void row_barrier(int tpr) {
    if (tpr <= 32)
        __syncwarp();
    else
        __syncthreads();
}

inline bool loose_shape(int cols, RingShape* s) {
    constexpr int each = 2 * kLoosePairs;
    s->V = 1;
    s->ctas = 1;
    s->threads = 256;
    s->resident = 512;
    if (cols <= 32 * each)
        s->tpr = next_pow2((cols + each - 1) / each);
    else
        s->threads = s->tpr = (cols + 32 * each - 1) / (32 * each) * 32;
    s->per_cta = (cols + s->tpr - 1) / s->tpr;  // columns of a thread
    return s->tpr <= kRingThreads;
}

// Launches a ring kernel on the clusters that share its rows.
template <typename... KArgs>
int launch_ring(void (*kernel)(KArgs...), const RingShape& c, unsigned clusters, size_t smem, cudaStream_t s, const NormJob& j) {
    // The same for every call: another thread's call must not lower it before this launch.
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * c.ctas);
    cfg.blockDim = dim3(c.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c.ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, j);
}

}  // namespace gns
