// Launchers of the router's gates, balance loss and their gradients (moe_gate.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe.cuh"

namespace gns {

constexpr int kMaxTopk = 32;  // a lane holds a choice

struct GateJob {
    const void* logits;  // [tokens][ld >= experts]
    long long ld;
    int tokens, experts, topk, dtype;
    int normalize;
    const long long* ids;  // [tokens][topk]
    const float* weights;
    const float* lse;      // [tokens]
};

// The gates, written through the three pointers above.
int launch_moe_gate(const GateJob& job, cudaStream_t s);

struct BalanceJob {
    float balance, z;
    float* loss;    // [1]
    int* counts;    // [experts + 1]
    float* probs;   // [experts]
    float* part;    // moe_balance_scratch() bytes
};

size_t moe_balance_scratch(const GateJob& job, int num_sms);
// Two kernels: each block's sums, and their sums with the loss.
int launch_moe_balance(const GateJob& job, const BalanceJob& b, int num_sms, cudaStream_t s);
int launch_moe_balance_join(const GateJob& job, const BalanceJob& b, int num_sms, cudaStream_t s);

struct GateGradJob {
    const float* dweights;  // [tokens][topk]
    const int* counts;      // as written above, null without the loss
    float balance, z;
    const float* dloss;     // device, null for 1
    void* dlogits;          // of the logits' type
    long long ldd;
};

int launch_moe_gate_backward(const GateJob& job, const GateGradJob& g, cudaStream_t s);

}  // namespace gns
