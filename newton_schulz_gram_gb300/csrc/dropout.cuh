// Launcher of the counter-based dropout (dropout.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace gns {

// y = residual + keep ? x inv : 0 over rows x cols elements; see gns_dropout.
struct DropoutJob {
    const void* x;
    const void* residual;  // or null
    void* y;
    long long rows, cols, ldx, ldr, ldy;
    int dtype;
    uint32_t threshold;  // an element is kept when its 16-bit draw is at least this (0 .. 65536)
    float inv;
    uint64_t seed, step;
    unsigned long long base;
};

int launch_dropout(DropoutJob job, cudaStream_t s);

}  // namespace gns
