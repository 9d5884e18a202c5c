// Launchers of layer norm and its gradients (layer_norm.cu, layer_norm_backward.cu).
//
// y = (x - mean) * rstd * weight + bias over each row of `cols` elements, rstd =
// 1 / sqrt(var + eps), var the mean of the squares of x - mean; with rms the mean
// is taken as 0.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "blockops.cuh"

namespace gns {

struct NormJob {
    const void* x;
    long long ldx;
    long long rows;
    int cols, dtype;
    const void* weight;  // fp32 where wf32, else of dtype; null for 1
    const void* bias;    // forward; null for 0
    int wf32, rms;
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
    int tpr, per_row;  // set by the launchers
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

// The weights of a piece as fp32 values, `fill` beyond the row.
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

inline int next_pow2(int v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

}  // namespace gns
