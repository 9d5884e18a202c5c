// The router: each token's top-k experts with their weights, the loss that keeps
// the experts' loads level, and the gradient of both with respect to the logits.
//
// A warp owns a token; lane l holds the logits of the experts l, l + 32, ... in
// registers. The choice is topk rounds of a warp-wide maximum over order-preserving
// integer keys: a lane keeps its own best, so a round is two warp reductions (the
// key, then the lowest expert that has it) and one lane's search for its next best.
//
// Bound: latency. 16384 tokens of 256 fp32 logits are 17 MB, 2.5 us of HBM.
#include <algorithm>
#include <type_traits>

#include "blockops.cuh"
#include "moe_gate.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

constexpr float kInf = __builtin_huge_valf();

// Keys that compare as the values do: NaN above all, -0 like 0, 0 for nothing.
// Values of -inf have kNoKey, the least of all; they are never chosen.
constexpr unsigned kNoKey = 0x007fffffu;
__device__ __forceinline__ unsigned key_of(float v) {
    if (v != v) return 0xffffffffu;
    const unsigned b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// A token's logits, -inf beyond the last expert.
template <typename T, int NV>
__device__ __forceinline__ void load_logits(const GateJob& j, long long t, int lane, float (&l)[NV]) {
    const T* row = static_cast<const T*>(j.logits) + t * j.ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = lane + 32 * i < j.experts ? to_f32<T>(row[lane + 32 * i]) : -kInf;
}

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) moe_gate_kernel(GateJob j, long long* ids, float* weights, float* lse) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < j.tokens; t += static_cast<long long>(gridDim.x) * kWarps) {
        float l[NV];
        load_logits<T>(j, t, lane, l);
        unsigned key[NV], best = 0;
        int at = 0;  // this lane's best: its key and the first of its values that has it
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            key[i] = lane + 32 * i < j.experts ? key_of(l[i]) : 0;
            if (key[i] > best) best = key[i], at = i;
        }
        float most = 0.0f, total = 0.0f, chosen = -kInf;
        int id = -1;
        for (int r = 0; r < j.topk; ++r) {
            const unsigned top = __reduce_max_sync(0xffffffffu, best);
            if (top <= kNoKey) break;  // nothing is left
            const int e = __reduce_min_sync(0xffffffffu, best == top ? lane + 32 * at : 0x7fffffff);
            const float v = __uint_as_float(top == 0xffffffffu ? 0x7fc00000u : top & 0x80000000u ? top & 0x7fffffffu : ~top);
            if (r == 0) most = v;
            if (lane == r) id = e, chosen = v;
            if (lane == (e & 31)) {
                best = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (lane + 32 * i == e) key[i] = 0;
                    if (key[i] > best) best = key[i], at = i;
                }
            }
        }
        const bool left = __shfl_sync(0xffffffffu, id, 0) >= 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += expf(l[i] - most);
        total = warp_sum(total);
        const float all = left ? most + logf(total) : -kInf;
        float w = id >= 0 ? expf(chosen - most) : 0.0f;
        const float divisor = j.normalize ? warp_sum(w) : total;
        if (id >= 0) w = w / divisor;
        if (lane < j.topk) {
            ids[t * j.topk + lane] = id;
            weights[t * j.topk + lane] = w;
        }
        if (lane == 0) lse[t] = all;
    }
}

// ------------------------------------------------------------ the balance loss
//
// Each block sums, over its tokens, the experts' probabilities and the squares of
// lse, and counts the slots; a second kernel, one block, adds the blocks' sums in
// their order and computes the loss.

constexpr int kBalanceWarps = 16;
constexpr int kBalanceThreads = 32 * kBalanceWarps;

int balance_blocks(const GateJob& j, int num_sms) {
    return std::max(1, std::min(num_sms, (j.tokens + kBalanceWarps - 1) / kBalanceWarps));
}

template <typename T, int NV>
__global__ void __launch_bounds__(kBalanceThreads) moe_balance_kernel(GateJob j, float* part, int* part_counts) {
    __shared__ int count[kMaxExperts + 1];
    __shared__ float sum[kMaxExperts + 1];
    for (int e = threadIdx.x; e <= j.experts; e += kBalanceThreads) count[e] = 0, sum[e] = 0.0f;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float p[NV], squares = 0.0f;
    int rows = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = 0.0f;
    for (long long t = static_cast<long long>(blockIdx.x) * kBalanceWarps + warp; t < j.tokens;
         t += static_cast<long long>(gridDim.x) * kBalanceWarps) {
        const float z = j.lse[t];
        const long long id = lane < j.topk ? j.ids[t * j.topk + lane] : -1;
        float l[NV];
        load_logits<T>(j, t, lane, l);
        if (id >= 0 && id < j.experts) atomicAdd(&count[id], 1);
        if (z == -kInf) continue;
        ++rows;
        squares = fmaf(z, z, squares);
#pragma unroll
        for (int i = 0; i < NV; ++i) p[i] += expf(l[i] - z);
    }
    for (int w = 0; w < kBalanceWarps; ++w) {  // one warp after the other: the order of the sums is fixed
        if (w == warp) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane + 32 * i < j.experts) sum[lane + 32 * i] += p[i];
            if (lane == 0) sum[j.experts] += squares, count[j.experts] += rows;
        }
        __syncthreads();
    }
    const long long base = static_cast<long long>(blockIdx.x) * (j.experts + 1);
    for (int e = threadIdx.x; e <= j.experts; e += kBalanceThreads) {
        part[base + e] = sum[e];
        part_counts[base + e] = count[e];
    }
}

__global__ void __launch_bounds__(1024) moe_balance_join_kernel(const float* part, const int* part_counts, int blocks,
                                                                GateJob j, BalanceJob b) {
    __shared__ float sum[1024 + 1];
    __shared__ int count[1024 + 1];
    __shared__ float terms[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int cols = j.experts + 1, groups = max(1, 1024 / cols);  // threads that share a column
    for (int i = threadIdx.x; i < cols * groups; i += 1024) {
        const int g = i / cols, e = i - g * cols;
        float s = 0.0f;
        int c = 0;
#pragma unroll 4
        for (int k = g; k < blocks; k += groups) {
            s += part[static_cast<long long>(k) * cols + e];
            c += part_counts[static_cast<long long>(k) * cols + e];
        }
        sum[i] = s;
        count[i] = c;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < cols; e += 1024) {
        float s = sum[e];
        int c = count[e];
        for (int g = 1; g < groups; ++g) s += sum[g * cols + e], c += count[g * cols + e];
        sum[e] = s;
        count[e] = c;
    }
    __syncthreads();
    const float n = static_cast<float>(max(1, count[j.experts]));
    float dot = 0.0f;
    for (int e = threadIdx.x; e < cols; e += 1024) {
        b.counts[e] = count[e];
        if (e == j.experts) continue;
        const float mean = sum[e] / n;
        b.probs[e] = mean;
        dot = fmaf(static_cast<float>(count[e]), mean, dot);
    }
    dot = warp_sum(dot);
    if ((threadIdx.x & 31) == 0) terms[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x < 32) {
        dot = warp_sum(terms[threadIdx.x]);
        if (threadIdx.x == 0) {
            const float level = b.balance * (static_cast<float>(j.experts) / (n * static_cast<float>(j.topk))) * dot;
            // Squares beyond fp32 (|lse| > 1.8e19) matter only where they are asked for.
            *b.loss = b.z != 0.0f ? level + b.z * (sum[j.experts] / n) : level;
        }
    }
}

// ------------------------------------------------------------------- backward

// PROBS: the gradient has terms in the probabilities (the loss, or weights over all experts).
template <typename T, int NV, bool PROBS>
__global__ void __launch_bounds__(kThreads) moe_gate_backward_kernel(GateJob j, GateGradJob g) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float c[NV], by_count = 0.0f, by_lse = 0.0f;  // the counts times their factor, and the factor of lse
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = 0.0f;
    if (PROBS && g.counts) {
        const float scale = g.dloss ? *g.dloss : 1.0f, n = static_cast<float>(max(1, g.counts[j.experts]));
        by_count = scale * g.balance * static_cast<float>(j.experts) / (n * static_cast<float>(j.topk)) / n;
        by_lse = scale * g.z * 2.0f / n;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < j.experts) c[i] = static_cast<float>(g.counts[lane + 32 * i]);
    }
    T* out = static_cast<T*>(g.dlogits);
    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < j.tokens; t += static_cast<long long>(gridDim.x) * kWarps) {
        const long long slot = t * j.topk + lane;
        const bool mine = lane < j.topk;
        const long long chosen = mine ? j.ids[slot] : -1;
        const int id = chosen >= 0 && chosen < j.experts ? static_cast<int>(chosen) : -1;
        const float w = id >= 0 ? j.weights[slot] : 0.0f, dw = id >= 0 ? g.dweights[slot] : 0.0f;
        const float inner = warp_sum(w * dw);
        const float term = j.normalize ? w * (dw - inner) : w * dw;
        float d[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = 0.0f;
        if (PROBS) {
            const float z = j.lse[t];
            if (z != -kInf) {
                float p[NV], level = 0.0f;
                load_logits<T>(j, t, lane, p);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    p[i] = expf(p[i] - z);
                    level = fmaf(p[i], c[i], level);
                }
                level = warp_sum(level);
                const float all = by_lse * z - (j.normalize ? 0.0f : inner);
#pragma unroll
                for (int i = 0; i < NV; ++i) d[i] = p[i] * (by_count * (c[i] - level) + all);
            }
        }
        for (int r = 0; r < j.topk; ++r) {
            const int e = __shfl_sync(0xffffffffu, id, r);
            const float v = __shfl_sync(0xffffffffu, term, r);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane + 32 * i == e) d[i] += v;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < j.experts) out[t * g.ldd + lane + 32 * i] = from_f32<T>(d[i]);
    }
}

// Calls fn with the number of logits a lane holds.
template <typename F>
int by_experts(int experts, F&& fn) {
    if (experts <= 32) return fn(std::integral_constant<int, 1>{});
    if (experts <= 64) return fn(std::integral_constant<int, 2>{});
    if (experts <= 128) return fn(std::integral_constant<int, 4>{});
    if (experts <= 256) return fn(std::integral_constant<int, 8>{});
    if (experts <= 512) return fn(std::integral_constant<int, 16>{});
    return fn(std::integral_constant<int, 32>{});
}

dim3 token_grid(int tokens, int num_sms_times) {
    return dim3(static_cast<unsigned>(std::min((tokens + kWarps - 1) / kWarps, num_sms_times)));
}

}  // namespace

int launch_moe_gate(const GateJob& j, cudaStream_t s) {
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_experts(j.experts, [&](auto nv) {
            return static_cast<int>(launch_after(moe_gate_kernel<T, decltype(nv)::value>, token_grid(j.tokens, 0x7fffffff), dim3(kThreads),
                                                 0, s, j, const_cast<long long*>(j.ids), const_cast<float*>(j.weights),
                                                 const_cast<float*>(j.lse)));
        });
    });
}

size_t moe_balance_scratch(const GateJob& j, int num_sms) {
    return (sizeof(float) + sizeof(int)) * static_cast<size_t>(balance_blocks(j, num_sms)) * (j.experts + 1);
}

int launch_moe_balance(const GateJob& j, const BalanceJob& b, int num_sms, cudaStream_t s) {
    const int blocks = balance_blocks(j, num_sms);
    int* counts = reinterpret_cast<int*>(b.part + static_cast<size_t>(blocks) * (j.experts + 1));
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_experts(j.experts, [&](auto nv) {
            return static_cast<int>(launch_after(moe_balance_kernel<T, decltype(nv)::value>, dim3(blocks), dim3(kBalanceThreads), 0, s, j,
                                                 b.part, counts));
        });
    });
}

int launch_moe_balance_join(const GateJob& j, const BalanceJob& b, int num_sms, cudaStream_t s) {
    const int blocks = balance_blocks(j, num_sms);
    const int* counts = reinterpret_cast<const int*>(b.part + static_cast<size_t>(blocks) * (j.experts + 1));
    return static_cast<int>(launch_after(moe_balance_join_kernel, dim3(1), dim3(1024), 0, s, static_cast<const float*>(b.part), counts,
                                         blocks, j, b));
}

int launch_moe_gate_backward(const GateJob& j, const GateGradJob& g, cudaStream_t s) {
    const bool probs = g.counts || !j.normalize;
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return by_experts(j.experts, [&](auto nv) {
            constexpr int NV = decltype(nv)::value;
            return static_cast<int>(launch_after(probs ? moe_gate_backward_kernel<T, NV, true> : moe_gate_backward_kernel<T, NV, false>,
                                                 token_grid(j.tokens, 0x7fffffff), dim3(kThreads), 0, s, j, g));
        });
    });
}

}  // namespace gns
