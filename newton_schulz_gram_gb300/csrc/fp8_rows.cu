// The block-scaled 8-bit linear layer for up to eight rows (a decode step), in
// one launch: D[r][n] = x_r . w[g(r)][n] with x cast to 8 bits on the way.
//
// Bound: HBM, the weights once, N K bytes per group that has rows. A block of
// threads takes 32 weight rows; its eight warps split the contraction (k block
// b belongs to warp b mod 8), so even a 512 x 2048 expert puts every byte in
// flight at once. The rows of x are the 8 columns of mma.sync m16n8k32: a
// lane's 16-byte loads of two weight rows are two A fragments as they are,
// because the order of k within a block is free as long as x uses the same
// one, and x's fragment is cast in the registers that hold it (the block's
// maximum is shared by four lanes). Tensor throughput does not matter at 8
// columns; tcgen05 would add a TMA ring, TMEM and their set-up to a kernel
// that lives for a few microseconds. The warps' sums are joined in a fixed
// order.
#include "blockops.cuh"
#include "fp8.cuh"
#include "fp8_convert.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerBlock = 32;
constexpr int kUnroll = 2;  // k blocks whose loads are issued together

template <bool E5M2>
__device__ __forceinline__ void mma_16832(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    if constexpr (E5M2)
        asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The bytes of a 16-byte piece that lie inside the row (left of them).
__device__ __forceinline__ uint4 clip(uint4 v, int left) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        if (n < 4) w[i] = n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1);
    }
    return v;
}

// 16 values of a row of x from column k (K columns in all) as fp32.
template <typename T>
__device__ __forceinline__ void load_x(const T* row, int k, int K, bool vec, float (&v)[16]) {
    if (vec && k + 16 <= K) {
        Pack<T, 16> p;
        p.load(row + k);
        p.get(v);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = k + i < K ? to_f32<T>(row[k + i]) : 0.0f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_rows_kernel(Fp8RowsJob j, bool vec) {
    __shared__ float sums[kWarps][kRowsPerBlock][kFp8FewRows + 1];
    __shared__ int found[3];  // group, its first row, its row count
    grid_dependency_wait();
    grid_launch_dependents();
    const int n0 = blockIdx.x * kRowsPerBlock;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int g = 0, r0 = 0, count = j.rows;
    if (j.offsets) {
        // Row blockIdx.y stands for its group if it is the group's first.
        const int r = blockIdx.y;
        if (threadIdx.x == 0) found[0] = -1;
        __syncthreads();
        for (int i = threadIdx.x; i < j.G; i += kThreads) {
            const int beg = j.offsets[i], end = j.offsets[i + 1];
            if (beg <= r && r < end) {
                found[0] = i;
                found[1] = beg;
                found[2] = end - beg;
            }
        }
        __syncthreads();
        g = found[0];
        r0 = found[1];
        count = found[2];
        if (g < 0) {  // a row of no group: zero
            const int n = n0 + static_cast<int>(threadIdx.x);
            if (threadIdx.x < kRowsPerBlock && n < j.N)
                by_dtype_device(j.out_dtype, [&](auto t) {
                    using O = decltype(t);
                    static_cast<O*>(j.D)[static_cast<long long>(r) * j.ldd + n] = from_f32<O>(0.0f);
                });
            return;
        }
        if (r != r0) return;
    }
    const int gq = lane >> 2, t = lane & 3;
    const uint8_t* wg = j.w + g * j.stride_w;
    const int nkb = (j.K + kFp8Block - 1) / kFp8Block;
    const uint8_t* sw = j.sw + (static_cast<long long>(g) * ((j.N + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block) * nkb;
    const T* xrow = nullptr;  // the row of x of this lane's column
    if (gq < count) {
        const int r = r0 + gq;
        xrow = static_cast<const T*>(j.x) + static_cast<long long>(j.slots ? j.slots[r] / j.topk : r) * j.ldx;
    }
    float acc[2][4] = {};
    for (int kb0 = warp; kb0 < nkb; kb0 += kWarps * kUnroll) {
        uint4 a[kUnroll][2][2][2];  // [k block][16-row tile][row g, g + 8][64-byte half]
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = n0 + 16 * m + 8 * h + gq;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int k = (kb0 + u * kWarps) * kFp8Block + 64 * c + 16 * t;
                        a[u][m][h][c] = n < j.N && k < j.K ? load_once(wg + n * j.ldw + k) : make_uint4(0, 0, 0, 0);
                        if (k + 16 > j.K) a[u][m][h][c] = clip(a[u][m][h][c], j.K - k);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int kb = kb0 + u * kWarps;
            if (kb >= nkb) break;  // the same for the whole warp
            float v[2][16];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (xrow) {
                    load_x(xrow, kb * kFp8Block + 64 * c + 16 * t, j.K, vec, v[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[c][i] = 0.0f;
                }
            }
            float amax = 0.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(v[c][i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const uint32_t e = scale_exponent(amax, 8);
            const float inv = exp_inverse(e);
            const float s = exp_value(sw[kb]) * exp_value(e);  // of this lane's column
            uint32_t b[2][4];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[c][i] = cast_pair<false>(no_infinity(v[c][4 * i]) * inv, no_infinity(v[c][4 * i + 1]) * inv) |
                              (cast_pair<false>(no_infinity(v[c][4 * i + 2]) * inv, no_infinity(v[c][4 * i + 3]) * inv)
                               << 16);
            const float s0 = __shfl_sync(0xffffffffu, s, 8 * t);      // column 2 t
            const float s1 = __shfl_sync(0xffffffffu, s, 8 * t + 4);  // column 2 t + 1
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 lo = a[u][m][0][c], hi = a[u][m][1][c];
                    if (j.fmt_w == GNS_E5M2) {
                        mma_16832<true>(part, lo.x, hi.x, lo.y, hi.y, b[c][0], b[c][1]);
                        mma_16832<true>(part, lo.z, hi.z, lo.w, hi.w, b[c][2], b[c][3]);
                    } else {
                        mma_16832<false>(part, lo.x, hi.x, lo.y, hi.y, b[c][0], b[c][1]);
                        mma_16832<false>(part, lo.z, hi.z, lo.w, hi.w, b[c][2], b[c][3]);
                    }
                }
                acc[m][0] = fmaf(part[0], s0, acc[m][0]);
                acc[m][1] = fmaf(part[1], s1, acc[m][1]);
                acc[m][2] = fmaf(part[2], s0, acc[m][2]);
                acc[m][3] = fmaf(part[3], s1, acc[m][3]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        sums[warp][16 * m + gq][2 * t] = acc[m][0];
        sums[warp][16 * m + gq][2 * t + 1] = acc[m][1];
        sums[warp][16 * m + 8 + gq][2 * t] = acc[m][2];
        sums[warp][16 * m + 8 + gq][2 * t + 1] = acc[m][3];
    }
    __syncthreads();
    const int r = warp, n = n0 + lane;  // one warp per row of D
    if (r < count && n < j.N) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += sums[k][lane][r];
        by_dtype_device(j.out_dtype, [&](auto o) {
            using O = decltype(o);
            static_cast<O*>(j.D)[static_cast<long long>(r0 + r) * j.ldd + n] = from_f32<O>(v);
        });
    }
}

static_assert(kWarps == kFp8FewRows, "one warp stores each row");

}  // namespace

int launch_fp8_rows(const Fp8RowsJob& j, cudaStream_t s) {
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        const bool vec = (reinterpret_cast<uintptr_t>(j.x) & 15) == 0 && j.ldx * static_cast<int>(sizeof(T)) % 16 == 0;
        const dim3 grid((j.N + kRowsPerBlock - 1) / kRowsPerBlock, j.offsets ? j.rows : 1);
        return static_cast<int>(launch_after(fp8_rows_kernel<T>, grid, dim3(kThreads), 0, s, j, vec));
    });
}

}  // namespace gns
