// Inverted dropout from a counter-based generator, with the residual added.
//
//   y_i = r_i + (u_i >= t ? x_i * 65536 / (65536 - t) : 0),  t = round(65536 p)
//
// u_i is the 16-bit draw of the element's global index g = base + row * cols +
// col: Philox4x32-10 with key (seed low, seed high) and counter (g >> 3 low,
// g >> 3 high, step low, step high | 2^31); the eight elements of a block
// share one output, as in the stochastic rounding of the weight update, whose
// counters have that top bit clear, so the two never share a draw. The mask is
// a function of (seed, step, g) alone: the backward pass recomputes it and
// nothing is stored. The scale is that of the rounded probability t / 65536,
// so the expectation is exact. A dropped element contributes 0 whatever its
// value (a NaN in x is dropped too).
//
// Bound: HBM, 2 (3 with the residual) elements moved per element; about nine
// integer instructions of Philox per element stay below that at 2 bytes. 2^26
// bf16 elements: 59 us with the residual (6.8 TB/s), 48 without (5.6); 1021 x
// 4093 unaligned fp32 ones 8.0 (4.2 TB/s, from L2).
#include "blockops.cuh"
#include "dropout.cuh"
#include "philox.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int kThreads = 256;
// Blocks of eight elements per thread on the vector path. With and without the
// residual, as above: one 70 and 58 us, two 67 and 47, four 59 and 48, eight 68 and 46.
constexpr int kUnroll = 4;

struct Draw {
    uint32_t k0, k1, step_lo, step_hi, threshold;
    float inv;
};

__device__ __forceinline__ void draws_of(const Draw& d, unsigned long long block, uint32_t (&c)[4]) {
    c[0] = static_cast<uint32_t>(block);
    c[1] = static_cast<uint32_t>(block >> 32);
    c[2] = d.step_lo;
    c[3] = d.step_hi;
    philox4x32_10(c, d.k0, d.k1);
}

__device__ __forceinline__ float apply(const Draw& d, float x, uint32_t u16) {
    return u16 >= d.threshold ? __fmul_rn(x, d.inv) : 0.0f;
}

// Every row starts on a 16-byte boundary with its first index a multiple of 8:
// a thread owns whole Philox blocks and moves them as 16-byte pieces.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(const T* x, const T* res, T* y, long long rows,
                                                               long long cols, long long ldx, long long ldr,
                                                               long long ldy, unsigned long long base, Draw d) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long c0 = (static_cast<long long>(blockIdx.x) * kUnroll * kThreads + threadIdx.x) * 8;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
        const T* xr = x + r * ldx;
        const T* rr = RES ? res + r * ldr : nullptr;
        T* yr = y + r * ldy;
        const unsigned long long g0 = base + static_cast<unsigned long long>(r) * cols;
        Pack<T, 8> px[kUnroll], pr[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long c = c0 + 8LL * kThreads * u;
            if (c + 8 <= cols) {
                px[u].load_stream(xr + c);
                if (RES) pr[u].load_stream(rr + c);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long c = c0 + 8LL * kThreads * u;
            if (c >= cols) continue;
            uint32_t w[4];
            draws_of(d, (g0 + c) >> 3, w);
            if (c + 8 <= cols) {
                float f[8], a[8];
                px[u].get(f);
                if (RES) pr[u].get(a);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] = apply(d, f[e], sr_draw(w, e));
                    if (RES) f[e] = __fadd_rn(a[e], f[e]);
                }
                px[u].set(f);
                px[u].store(yr + c);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (c + e < cols) {
                        float f = apply(d, to_f32<T>(xr[c + e]), sr_draw(w, e));
                        if (RES) f = __fadd_rn(to_f32<T>(rr[c + e]), f);
                        yr[c + e] = from_f32<T>(f);
                    }
                }
            }
        }
    }
}

// Any alignment: each warp covers 32 Philox blocks (256 indices from a
// multiple of 8), shares their draws through shared memory and moves single
// elements, neighbouring lanes neighbouring elements.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(const T* x, const T* res, T* y, long long rows,
                                                               long long cols, long long ldx, long long ldr,
                                                               long long ldy, unsigned long long base, Draw d) {
    __shared__ __align__(16) uint16_t draws[kThreads / 32][256];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long span = (static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp) * 256;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
        const unsigned long long g0 = base + static_cast<unsigned long long>(r) * cols;
        const long long first = span - static_cast<long long>(g0 & 7);  // column of the span's first index
        if (first >= cols) continue;                                     // the whole warp
        const T* xr = x + r * ldx;
        const T* rr = RES ? res + r * ldr : nullptr;
        T* yr = y + r * ldy;
        float f[8], a[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const long long c = first + 32 * e + lane;
            const bool in = c >= 0 && c < cols;
            f[e] = in ? to_f32<T>(xr[c]) : 0.0f;
            a[e] = RES && in ? to_f32<T>(rr[c]) : 0.0f;
        }
        uint32_t w[4];
        draws_of(d, ((g0 & ~7ULL) + static_cast<unsigned long long>(span)) / 8 + lane, w);
        *reinterpret_cast<uint4*>(&draws[warp][8 * lane]) = make_uint4(w[0], w[1], w[2], w[3]);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const long long c = first + 32 * e + lane;
            if (c < 0 || c >= cols) continue;
            float v = apply(d, f[e], draws[warp][32 * e + lane]);
            if (RES) v = __fadd_rn(a[e], v);
            yr[c] = from_f32<T>(v);
        }
        __syncwarp();  // the draws are read before the next row's replace them
    }
}

template <typename T>
int launch_typed(const DropoutJob& j, cudaStream_t s) {
    const Draw d{static_cast<uint32_t>(j.seed), static_cast<uint32_t>(j.seed >> 32), static_cast<uint32_t>(j.step),
                 static_cast<uint32_t>(j.step >> 32) | 0x80000000u, j.threshold, j.inv};
    const T* x = static_cast<const T*>(j.x);
    const T* r = static_cast<const T*>(j.residual);
    T* y = static_cast<T*>(j.y);
    auto aligned = [&](const void* p, long long ld) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (j.rows == 1 || ld * sizeof(T) % 16 == 0);
    };
    const bool vec = aligned(j.x, j.ldx) && aligned(j.y, j.ldy) && (!r || aligned(r, j.ldr)) && j.base % 8 == 0 &&
                     (j.rows == 1 || j.cols % 8 == 0);
    // The unaligned kernel's spans start at most 7 indices before the row.
    const long long per = vec ? 8LL * kThreads * kUnroll : 8LL * kThreads;
    const long long blocks = (j.cols + (vec ? 0 : 7) + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(j.rows < 65535 ? j.rows : 65535));
    const dim3 block(kThreads);
    if (vec)
        return r ? launch_after(dropout_vec_kernel<T, true>, grid, block, 0, s, x, r, y, j.rows, j.cols, j.ldx, j.ldr,
                                j.ldy, j.base, d)
                 : launch_after(dropout_vec_kernel<T, false>, grid, block, 0, s, x, r, y, j.rows, j.cols, j.ldx, j.ldr,
                                j.ldy, j.base, d);
    return r ? launch_after(dropout_any_kernel<T, true>, grid, block, 0, s, x, r, y, j.rows, j.cols, j.ldx, j.ldr,
                            j.ldy, j.base, d)
             : launch_after(dropout_any_kernel<T, false>, grid, block, 0, s, x, r, y, j.rows, j.cols, j.ldx, j.ldr,
                            j.ldy, j.base, d);
}

}  // namespace

int launch_dropout(DropoutJob j, cudaStream_t s) {
    // Rows that follow one another without gaps are one long row.
    if (j.ldx == j.cols && j.ldy == j.cols && (!j.residual || j.ldr == j.cols)) {
        j.cols *= j.rows;
        j.rows = 1;
    }
    return by_dtype(j.dtype, [&](auto t) { return static_cast<int>(launch_typed<decltype(t)>(j, s)); });
}

}  // namespace gns
