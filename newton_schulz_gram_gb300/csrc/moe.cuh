// Launchers of the expert routing operators (moe.cu).
//
// n = tokens * topk slots; slot s belongs to token s / topk. The sort gives
// every slot a place: rows[s] in 0 .. n - 1, experts ascending, slots of one
// expert in slot order, slots without an expert (an id outside 0 .. G - 1)
// last. slots is the inverse. Expert e owns the places offsets[e] ..
// offsets[e + 1] - 1; places from offsets[G] on belong to no expert.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gns {

constexpr int kMaxExperts = 1024;

struct SortJob {
    const void* ids;
    int id_bytes;  // 4 or 8
    long long n;
    int G;
    int* offsets;
    int* rows;
    int* slots;
    int* hist;  // moe_sort_scratch() bytes, or null where that is 0
};

size_t moe_sort_scratch(long long n, int G);
// Two kernels where there is scratch, the counts and the places, else the latter alone.
int launch_moe_count(const SortJob& job, cudaStream_t s);
int launch_moe_place(const SortJob& job, cudaStream_t s);

struct RouteJob {
    int tokens, topk, G, H;
    const int* offsets;
    const int* rows;
    int dtype;
};

// y[rows[s]] = x[s / topk] for the slots with an expert, 0 for the others.
int launch_moe_gather(const RouteJob& job, const void* x, long long ldx, void* y, long long ldy, cudaStream_t s);

// out[t] = sum over t's slots with an expert, in slot order, of weight * y[rows[slot]] (weight 1 when weights is null).
int launch_moe_combine(const RouteJob& job, const void* y, long long ldy, const float* weights, void* out,
                       long long ldo, cudaStream_t s);

// dy[rows[s]] = weights[s] * dout[s / topk] and dweights[s] = <dout[s / topk], y[rows[s]]>; 0 for slots without an
// expert. dweights (and y) may be null.
int launch_moe_combine_backward(const RouteJob& job, const void* dout, long long lddo, const void* y, long long ldy,
                                const float* weights, void* dy, long long lddy, float* dweights, cudaStream_t s);

}  // namespace gns
