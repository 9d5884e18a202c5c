// The router: each token's top-k experts with their weights, the loss that keeps
// the experts' loads level, and the gradient of both with respect to the logits.
//
// A warp owns a token; lane l holds the logits of the experts l, l + 32, ... in
// registers, as order-preserving integer keys. The topk-th largest of the lanes' maxima
// is a bound that at least topk logits reach and few others do: those candidates go to
// a lane each, in expert order, and their ranks among one another are their slots. Only
// where more than 32 reach it (many equal logits) are they drawn one after the other.
//
// Bound: instructions and latency; 16384 tokens of 256 fp32 logits are 17 MB, 2.5 us of
// HBM. Those with their 8 experts take 12 us (drawn one after the other 15, by a maximum
// over every lane's values each time 20), the balance loss 13, the gradient of both 10;
// one token 2.3, 6.0 and 2.7.
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
constexpr unsigned kNoKey = 0x007fffffu, kNanKey = 0xfffffffeu;
__device__ __forceinline__ unsigned key_of(float v) {
    if (v != v) return kNanKey;
    const unsigned b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float(key == kNanKey ? 0x7fc00000u : key & 0x80000000u ? key & 0x7fffffffu : ~key);
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

// The topk largest keys one after the other: lane r gets the r-th's key and expert.
template <int NV>
__device__ __forceinline__ void draw(const unsigned (&key)[NV], int topk, int lane, unsigned& mine, int& id) {
    unsigned last = 0xffffffffu;
    int last_at = -1;
    for (int r = 0; r < topk; ++r) {
        unsigned best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool open = key[i] < last || (key[i] == last && lane + 32 * i > last_at);
            if (open && key[i] > best) best = key[i], at = lane + 32 * i;
        }
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        if (top <= kNoKey) break;  // nothing is left
        last = top;
        last_at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
        if (lane == r) mine = top, id = last_at;
    }
}

// A live row's probabilities, in place of its logits. From the row's maximum, not from
// its lse, whose rounding would be that much of every probability (4e-6 of one at 100).
template <int NV>
__device__ __forceinline__ void probabilities(float (&l)[NV]) {
    float best = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = fmaxf(best, l[i]);
    const float most = value_of(__reduce_max_sync(0xffffffffu, key_of(best)));
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        l[i] = expf(l[i] - most);
        total += l[i];
    }
    const float inv = 1.0f / warp_sum(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] *= inv;
}

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) moe_gate_kernel(GateJob j, long long* ids, float* weights, float* lse) {
    __shared__ uint2 found[kWarps][32];  // candidates: key, expert
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < j.tokens; t += static_cast<long long>(gridDim.x) * kWarps) {
        float l[NV];
        load_logits<T>(j, t, lane, l);
        unsigned key[NV], best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            key[i] = lane + 32 * i < j.experts ? key_of(l[i]) : 0;
            best = max(best, key[i]);
        }
        unsigned top = __reduce_max_sync(0xffffffffu, best), bound = top;
        const float most = top > kNoKey ? value_of(top) : 0.0f;
        for (int r = 1; r < j.topk; ++r) {
            if (best == bound) best = 0;
            bound = __reduce_max_sync(0xffffffffu, best);
        }
        bound = max(bound, kNoKey + 1);
        int count = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = key[i] >= bound;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            const int place = count + __popc(who & ((1u << lane) - 1));
            if (in && place < 32) found[warp][place] = make_uint2(key[i], lane + 32 * i);
            count += __popc(who);
        }
        __syncwarp();
        unsigned mine = 0;  // of this lane's candidate, which has slot `rank`
        int id = -1, rank = lane;
        if (count <= 32) {
            if (lane < count) {
                const uint2 c = found[warp][lane];
                mine = c.x, id = static_cast<int>(c.y);
            }
            rank = 0;
#pragma unroll 4
            for (int c = 0; c < count; ++c) rank += found[warp][c].x + (c < lane) > mine;
            if (lane >= count) rank = lane;  // the slots that are left, if count is below topk
        } else {
            draw<NV>(key, j.topk, lane, mine, id);
        }
        __syncwarp();
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += expf(l[i] - most);
        total = warp_sum(total);
        const bool chosen = id >= 0 && rank < j.topk;
        float w = chosen ? expf(value_of(mine) - most) : 0.0f;
        const float divisor = j.normalize ? warp_sum(w) : total;
        if (chosen) w = w / divisor;
        if (rank < j.topk) {
            ids[t * j.topk + rank] = chosen ? id : -1;
            weights[t * j.topk + rank] = w;
        }
        if (lane == 0) lse[t] = top > kNoKey ? most + logf(total) : -kInf;
    }
}

// ------------------------------------------------------------ the balance loss
//
// Each block sums, over its tokens, the experts' probabilities and the squares of
// lse, and counts the slots; a second kernel, one block, adds the blocks' sums in
// their order and computes the loss.

constexpr int kBalanceWarps = 16;
constexpr int kBalanceThreads = 32 * kBalanceWarps;
constexpr int kAhead = 2;  // tokens of a warp whose loads are issued together

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
    const long long step = static_cast<long long>(gridDim.x) * kBalanceWarps;
    for (long long t0 = static_cast<long long>(blockIdx.x) * kBalanceWarps + warp; t0 < j.tokens; t0 += kAhead * step) {
        float l[kAhead][NV], z[kAhead];
        long long id[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const long long t = t0 + a * step;
            const bool in = t < j.tokens;
            z[a] = in ? j.lse[t] : -kInf;
            id[a] = in && lane < j.topk ? j.ids[t * j.topk + lane] : -1;
            if (in) load_logits<T>(j, t, lane, l[a]);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (id[a] >= 0 && id[a] < j.experts) atomicAdd(&count[id[a]], 1);
            if (z[a] == -kInf) continue;
            ++rows;
            squares = fmaf(z[a], z[a], squares);
            probabilities(l[a]);
#pragma unroll
            for (int i = 0; i < NV; ++i) p[i] += l[a][i];
        }
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

// One cluster: each CTA takes every eighth strip of 32 experts, a warp every 32nd
// block's sums, and the last column, the squares and the number of rows, besides.
constexpr int kJoinCtas = 8;

__global__ void __launch_bounds__(1024) moe_balance_join_kernel(const float* part, const int* part_counts, int blocks,
                                                                GateJob j, BalanceJob b) {
    __shared__ float sum[32][33];
    __shared__ int count[32][33];
    __shared__ float terms[kJoinCtas];  // of the first CTA: the loss' sum over each CTA's experts
    __shared__ float rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = static_cast<int>(blockIdx.x), cols = j.experts + 1;
    cluster_sync();  // the first CTA has begun before any other writes to its shared memory
    grid_dependency_wait();
    grid_launch_dependents();
    float squares = 0.0f;
    if (warp == 0) {
        int n = 0;
        for (int k = lane; k < blocks; k += 32) {
            n += part_counts[static_cast<long long>(k) * cols + j.experts];
            squares += part[static_cast<long long>(k) * cols + j.experts];
        }
        n = __reduce_add_sync(0xffffffffu, n);
        squares = warp_sum(squares);
        if (lane == 0) {
            rows = static_cast<float>(max(1, n));
            if (rank == 0) b.counts[j.experts] = n;
        }
    }
    float dot = 0.0f;  // of the first warp's lanes
    for (int e0 = 32 * rank; e0 < j.experts; e0 += 32 * kJoinCtas) {
        float s = 0.0f;
        int c = 0;
        if (e0 + lane < j.experts) {
#pragma unroll 4
            for (int k = warp; k < blocks; k += 32) {
                s += part[static_cast<long long>(k) * cols + e0 + lane];
                c += part_counts[static_cast<long long>(k) * cols + e0 + lane];
            }
        }
        sum[warp][lane] = s;
        count[warp][lane] = c;
        __syncthreads();
        s = warp_sum(sum[lane][warp]);
        c = __reduce_add_sync(0xffffffffu, count[lane][warp]);
        __syncthreads();
        if (lane == 0) {
            sum[0][warp] = s;
            const int e = e0 + warp;
            if (e < j.experts) {
                b.counts[e] = c;
                b.probs[e] = s / rows;
            }
            count[0][warp] = c;
        }
        __syncthreads();
        if (warp == 0) dot = fmaf(static_cast<float>(count[0][lane]), sum[0][lane], dot);
        __syncthreads();
    }
    if (warp == 0) {
        dot = warp_sum(dot);
        if (lane == 0)
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&terms[rank]), 0)), "r"(__float_as_uint(dot)) : "memory");
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        dot = 0.0f;
        for (int k = 0; k < kJoinCtas; ++k) dot += terms[k];
        const float n = rows, level = b.balance * (static_cast<float>(j.experts) / (n * static_cast<float>(j.topk))) * (dot / n);
        // Squares beyond fp32 (|lse| > 1.8e19) matter only where they are asked for.
        *b.loss = b.z != 0.0f ? level + b.z * (squares / n) : level;
    }
}

// ------------------------------------------------------------------- backward

// PROBS: the gradient has terms in the probabilities (the loss, or weights over all experts).
template <typename T, int NV, bool PROBS>
__global__ void __launch_bounds__(kThreads) moe_gate_backward_kernel(GateJob j, GateGradJob g) {
    __shared__ float rows[kWarps][32 * NV];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* row = rows[warp];
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
        for (int i = 0; i < NV; ++i) d[i] = row[lane + 32 * i] = 0.0f;
        if (PROBS) {
            const float z = j.lse[t];
            if (z != -kInf) {
                float p[NV], level = 0.0f;
                load_logits<T>(j, t, lane, p);
                probabilities(p);
#pragma unroll
                for (int i = 0; i < NV; ++i) level = fmaf(p[i], c[i], level);
                level = warp_sum(level);
                // The weights' part and the loss' are added last: each cancels by itself.
                const float all = by_lse * z, less = j.normalize ? 0.0f : inner;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    d[i] = p[i] * (by_count * (c[i] - level) + all);
                    row[lane + 32 * i] = -p[i] * less;
                }
            }
        }
        // The chosen experts' terms, a lane each, through shared memory. A gate of one's own
        // may name an expert twice: the first of its lanes adds up, in order.
        float v = term;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)) != 0)) {
            v = 0.0f;
            for (int r = 0; r < j.topk; ++r) {
                const float o = __shfl_sync(0xffffffffu, term, r);
                if (same >> r & 1) v += o;
            }
        }
        __syncwarp();
        if (id >= 0 && __ffs(same) - 1 == lane) row[id] += v;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < j.experts) out[t * g.ldd + lane + 32 * i] = from_f32<T>(d[i] + row[lane + 32 * i]);
        __syncwarp();
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kJoinCtas);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kJoinCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, moe_balance_join_kernel, static_cast<const float*>(b.part), counts, blocks, j, b));
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
