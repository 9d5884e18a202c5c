// Small pieces shared by the training-block operators: element types, 16-byte
// vectors of them as fp32 values, and launches with programmatic dependent
// launch.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gns.h"

namespace gns {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
    return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Pairs of fp32 values. (With the paired instructions, add.rn.f32x2 and the like, layer
// norm took the same time: 16384 x 4096 52.2 us forward and 89.4 backward, 52.1 and 88.5
// without.)
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// N consecutive elements as they lie in memory, in 16-byte pieces; they start on
// a 16-byte boundary.
template <typename T, int N>
struct Pack {
    static constexpr int kPieces = N * static_cast<int>(sizeof(T)) / 16;
    uint4 p[kPieces];

    __device__ __forceinline__ void load(const T* a) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) p[i] = reinterpret_cast<const uint4*>(a)[i];
    }
    __device__ __forceinline__ void load_stream(const T* a) {  // read once: not kept in L1
#pragma unroll
        for (int i = 0; i < kPieces; ++i) p[i] = __ldcs(reinterpret_cast<const uint4*>(a) + i);
    }
    __device__ __forceinline__ void store(T* a) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) reinterpret_cast<uint4*>(a)[i] = p[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) p[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&f)[N]) const {
        const T* e = reinterpret_cast<const T*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32<T>(e[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[N]) {
        T* e = reinterpret_cast<T*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_f32<T>(f[i]);
    }
};

// Pieces: what a thread owns of a row of H elements, 16 bytes of it where rows are
// 16-byte aligned. Where they are not a piece is kLoose elements 32 apart, the
// neighbouring lanes' next to them: single accesses, but whole lines per warp and
// the piece's bookkeeping shared.
constexpr int kLoose = 4;

// Piece v of a row of H elements.
template <typename T, int N>
struct Wide {
    static constexpr int kSize = N;
    Pack<T, N> p;
    __device__ __forceinline__ void load(const T* row, unsigned v, int) { p.load(row + static_cast<long long>(v) * N); }
    __device__ __forceinline__ void load_stream(const T* row, unsigned v, int) {
        p.load_stream(row + static_cast<long long>(v) * N);
    }
    __device__ __forceinline__ void store(T* row, unsigned v, int) const { p.store(row + static_cast<long long>(v) * N); }
    __device__ __forceinline__ void clear() { p.clear(); }
    __device__ __forceinline__ void get(float (&f)[N]) const { p.get(f); }
    __device__ __forceinline__ void set(const float (&f)[N]) { p.set(f); }
};

template <typename T>
struct Loose {
    static constexpr int kSize = kLoose;
    T e[kLoose];
    static __device__ __forceinline__ int column(unsigned v, int i) {
        return static_cast<int>((v >> 5) * (32 * kLoose) + (v & 31) + 32 * i);
    }
    __device__ __forceinline__ void load(const T* row, unsigned v, int H) {
#pragma unroll
        for (int i = 0; i < kLoose; ++i) e[i] = column(v, i) < H ? row[column(v, i)] : from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void load_stream(const T* row, unsigned v, int H) { load(row, v, H); }
    __device__ __forceinline__ void store(T* row, unsigned v, int H) const {
#pragma unroll
        for (int i = 0; i < kLoose; ++i)
            if (column(v, i) < H) row[column(v, i)] = e[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kLoose; ++i) e[i] = from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void get(float (&f)[kLoose]) const {
#pragma unroll
        for (int i = 0; i < kLoose; ++i) f[i] = to_f32<T>(e[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[kLoose]) {
#pragma unroll
        for (int i = 0; i < kLoose; ++i) e[i] = from_f32<T>(f[i]);
    }
};

// Copies to shared memory that the thread waits for itself.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// The first `bytes` of 16, zeros for the others, which are not read.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Launch with the programmatic-dependent-launch attribute: the kernel calls
// grid_dependency_wait() before it reads what an earlier grid wrote or
// writes what an earlier grid may still read.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

inline bool rows_aligned(const void* p, long long ld, long long rows, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || ld * es % 16 == 0);
}

inline int elem_bytes(int dtype) { return dtype == GNS_FP32 ? 4 : 2; }

// Calls fn with a value of the element type of `dtype`.
template <typename F>
int by_dtype(int dtype, F&& fn) {
    switch (dtype) {
        case GNS_BF16: return fn(__nv_bfloat16{});
        case GNS_FP16: return fn(__half{});
        default: return fn(float{});
    }
}

template <typename F>
__device__ __forceinline__ void by_dtype_device(int dtype, F&& fn) {
    if (dtype == GNS_BF16)
        fn(__nv_bfloat16{});
    else if (dtype == GNS_FP16)
        fn(__half{});
    else
        fn(float{});
}

}  // namespace gns
