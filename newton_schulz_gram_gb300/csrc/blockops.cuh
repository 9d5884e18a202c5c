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
