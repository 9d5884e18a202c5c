// Block-scaled 8-bit products on tcgen05 (sm_103a): forward, data gradient and
// weight gradient of a linear layer, for one weight matrix or for the experts
// of a routed batch in one launch.
//
//   D[m][n] = sum over k blocks b of  sA(m, b) sB(n, b) sum_{k in b} A[m][k] B[n][k]
//
// with blocks of 128 along the contraction. The tensor core sums one block's
// 128 products in fp32 (kind::f8f6f4, TMEM); the epilogue warps then add
// sA sB times that partial sum to fp32 accumulators in registers. So a block
// costs one read of its 128 x 256 TMEM accumulator besides its MMAs: at full
// MMA rate a block takes about 512 cycles per SM, the TMEM reads 256 and the
// scaled adds 128 (packed pairs; 256 when both scales vary along the tile), so
// the tensor core stays the bound as long as the two overlap.
//
// One CTA (CG = 1, 128 x 256 tiles) or a pair (CG = 2, 256 x 256 tiles, paired
// MMAs; each CTA stages 128 rows of each operand, so a k block moves 32 KB per
// SM instead of 48 KB from L2) per SM (pair) walks the tiles with a static
// stride. Warp roles:
//   warp 0     TMA producer of 128-byte-wide k blocks (128-byte swizzle)
//   warp 1     TMEM owner, MMA issuer; k block i goes to accumulator buffer
//              i & 1 (256 columns each)
//   warps 4-11 epilogue: lane quarter warp & 3, column half of the tile
//              (warp - 4) >> 2, 128 accumulators per thread. The first
//              warpgroup gives registers up for them: 40 + 2 x 232 per lane of
//              the 3 x 168 the block is launched with.
// Operands whose contraction runs along the stored rows (the weights of the
// data gradient, both operands of the weight gradient) are read MN-major
// through the shared-memory descriptor; nothing is transposed in memory.
#include <algorithm>

#include "blockops.cuh"
#include "fp8.cuh"
#include "moe.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = kFp8Block;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kBand = 16;  // tile rows walked together (their A stays in L2 while the columns pass)
constexpr uint32_t kTmemCols = 2 * BN;
constexpr uint32_t A_BYTES = BM * BK;
constexpr uint32_t kBoxBytes = 128 * 128;

template <int CG>
struct Cfg {
    static constexpr int STAGES = CG == 1 ? 4 : 6;
    static constexpr uint32_t B_BYTES = BN / CG * BK;
    static constexpr int TM = BM * CG;
};

__host__ __device__ constexpr int num_bars(int stages) { return 2 * stages + 5; }

struct Groups {
    int offs[kMaxExperts + 2];  // first row of each group; offs[G + 1]: all rows
    int pre[kMaxExperts + 2];   // tile rows (weight gradient: token blocks) of the groups before
};

template <int CG>
constexpr int smem_bytes() {
    return 1024 + Cfg<CG>::STAGES * static_cast<int>(A_BYTES + Cfg<CG>::B_BYTES) + kEpiWarps * 2 * 128 * 4 +
           num_bars(Cfg<CG>::STAGES) * 8 + 16 + static_cast<int>(sizeof(Groups));
}
static_assert(smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448, "shared memory budget");

template <int CG>
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Instruction descriptor of kind::f8f6f4, fp32 accumulator.
__device__ __forceinline__ uint32_t idesc_f8(int M, int N, int fmt_a, int fmt_b, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4)                                  // D format: f32
           | (static_cast<uint32_t>(fmt_a) << 7)      // 0: e4m3, 1: e5m2
           | (static_cast<uint32_t>(fmt_b) << 10)
           | (a_mn << 15) | (b_mn << 16)
           | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// acc (two fp32) += {v0, v1} * s (two fp32), each rounded once.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t v0, uint32_t v1, uint64_t s) {
    // volatile: keeps its place between the TMEM loads (a chunk is used before
    // the next one is loaded, which the register budget counts on).
    asm volatile("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
        : "+l"(acc)
        : "r"(v0), "r"(v1), "l"(s));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

// mbar_wait with its bounded spin inline: a call in the epilogue's loop would
// have the 128 accumulators saved around it.
__device__ __forceinline__ bool mbar_wait_here(uint32_t bar, uint32_t parity, const DevStatus& st) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (call_aborted(st)) return false;
        if (globaltimer() - t0 > st.limit_ns) {
            raise_timeout(st);
            return false;
        }
    }
    return true;
}

// tcgen05.wait::ld that the uses of v depend on.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
}

struct Tile {
    int g;          // group; G: the rows past the last group (all zero)
    int m0, n0;     // origin: row within the group (weight gradient: row of D), column
    int kb0, kb1;   // k blocks
    int split;
};

// What every role needs to walk the tiles.
struct Walk {
    int G, ntn, mtn, split, wgrad, total_kb, units;
    const Groups* gr;
};

template <int CG>
__device__ __forceinline__ Tile decode(const Walk& w, int t) {
    constexpr int TM = Cfg<CG>::TM;
    Tile tl;
    tl.split = 0;
    int local, rows;
    if (w.wgrad) {
        const int per = w.mtn * w.ntn;
        tl.g = t / per;
        local = t - tl.g * per;
        rows = w.mtn;
    } else {
        if (w.split > 1) {
            tl.split = t % w.split;
            t /= w.split;
        }
        int lo = 0, hi = w.G;  // the last group whose first tile is <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (w.gr->pre[mid] * w.ntn <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        tl.g = lo;
        local = t - w.gr->pre[lo] * w.ntn;
        rows = w.gr->pre[lo + 1] - w.gr->pre[lo];
    }
    const int band = local / (kBand * w.ntn);
    const int rem = local - band * kBand * w.ntn;
    const int h = min(kBand, rows - band * kBand);
    const int nt = rem / h;
    tl.n0 = nt * BN;
    tl.m0 = (band * kBand + rem - nt * h) * TM;
    if (w.wgrad) {
        tl.kb0 = w.gr->pre[tl.g];
        tl.kb1 = w.gr->pre[tl.g + 1];
    } else if (tl.g == w.G) {
        tl.kb0 = tl.kb1 = 0;
    } else {
        tl.kb0 = static_cast<int>(static_cast<long long>(w.total_kb) * tl.split / w.split);
        tl.kb1 = static_cast<int>(static_cast<long long>(w.total_kb) * (tl.split + 1) / w.split);
    }
    return tl;
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer() - t0 > limit_ns) break;
    }
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&a)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]),
                 "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7])
                 : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float2 f) {
    if constexpr (sizeof(T) == 2) {
        const T lo = from_f32<T>(f.x), hi = from_f32<T>(f.y);
        return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&lo)) |
               (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&hi)) << 16);
    }
    return 0;
}

// The thread's 128 columns from column n0 of one row (ncol of them inside
// the matrix), straight from its registers: 32-byte stores where the row
// allows them, single elements otherwise.
template <typename T>
__device__ __forceinline__ void store_row(T* row, const uint64_t (&acc)[64], int ncol, bool direct) {
    constexpr int PER = 32 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 128; c += PER) {
        if (direct && c + PER <= ncol) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (sizeof(T) == 2) {
                    w[i] = pack_pair<T>(unpack2(acc[c / 2 + i]));
                } else {
                    const float2 f = unpack2(acc[(c + i) / 2]);
                    w[i] = __float_as_uint(i & 1 ? f.y : f.x);
                }
            }
            st_global_v8(row + c, w);
        } else {
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 f = unpack2(acc[(c + i) / 2]);
                if (c + i < ncol) row[c + i] = from_f32<T>(f.x);
                if (c + i + 1 < ncol) row[c + i + 1] = from_f32<T>(f.y);
            }
        }
    }
}

template <int CG, bool WGRAD>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmJob P) {
    constexpr int STAGES = Cfg<CG>::STAGES;
    constexpr int TM = Cfg<CG>::TM;
    constexpr int BNH = BN / CG;
    constexpr uint32_t B_BYTES = Cfg<CG>::B_BYTES;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + STAGES * A_BYTES;
    float* scales = reinterpret_cast<float*>(sB + STAGES * B_BYTES);  // [kEpiWarps][2][128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(scales + kEpiWarps * 2 * 128);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + num_bars(STAGES));
    Groups* gr = reinterpret_cast<Groups*>(tmem_slot + 4);

    const uint32_t full0 = smem_u32(bars);
    const uint32_t empty0 = smem_u32(bars + STAGES);
    const uint32_t accf0 = smem_u32(bars + 2 * STAGES);
    const uint32_t acce0 = smem_u32(bars + 2 * STAGES + 2);
    const uint32_t drain_bar = smem_u32(bars + 2 * STAGES + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const DevStatus& err = P.st;
    const uint32_t rank = CG > 1 ? cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, kEpiWarps * CG);
        }
        mbar_init(drain_bar, 1);
        fence_mbar_init();
        prefetch_tmap(&P.mapA);
        prefetch_tmap(&P.mapB);
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish<CG>();
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // The groups' first rows and the tile rows (token blocks) before each.
    const int G = P.G;
    if (P.offsets) {
        int* part = reinterpret_cast<int*>(scales);  // one sum per warp
        for (int g = threadIdx.x; g <= G; g += kThreads) gr->offs[g] = P.offsets[g];
        if (threadIdx.x == 0) gr->offs[G + 1] = P.rows;
        __syncthreads();
        const int n = G + 1;  // the rows past the last group are one more group
        const int per = (n + kThreads - 1) / kThreads;
        const int g0 = threadIdx.x * per;
        auto units = [&](int g) {
            const int c = gr->offs[g + 1] - gr->offs[g];
            return WGRAD ? (c + BK - 1) / BK : (c + TM - 1) / TM;
        };
        int mine = 0;
        for (int i = 0; i < per && g0 + i < n; ++i) mine += units(g0 + i);
        int scan = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += v;
        }
        if (lane == 31) part[warp] = scan;
        __syncthreads();
        int start = scan - mine;
        for (int w = 0; w < warp; ++w) start += part[w];
        for (int i = 0; i < per && g0 + i < n; ++i) {
            gr->pre[g0 + i] = start;
            start += units(g0 + i);
            if (g0 + i == G) gr->pre[n] = start;
        }
    } else if (threadIdx.x == 0) {
        const int u = WGRAD ? (P.rows + BK - 1) / BK : (P.rows + TM - 1) / TM;
        gr->offs[0] = 0;
        gr->offs[1] = gr->offs[2] = P.rows;
        gr->pre[0] = 0;
        gr->pre[1] = gr->pre[2] = u;
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    Walk w;
    w.G = G;
    w.ntn = (P.N + BN - 1) / BN;
    w.mtn = WGRAD ? (P.M + TM - 1) / TM : 0;
    w.split = P.split;
    w.wgrad = WGRAD;
    w.total_kb = WGRAD ? 0 : (P.K + BK - 1) / BK;
    w.gr = gr;
    const int total = WGRAD ? G * w.mtn * w.ntn : gr->pre[G + 1] * w.ntn * P.split;
    const int first = static_cast<int>(blockIdx.x) / CG, stride = static_cast<int>(gridDim.x) / CG;
    const bool a_mn = WGRAD, b_mn = WGRAD || P.b_mn;

    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            if (lane == 0) {
                uint32_t stage = 0, phase = 0;
                int issued = 0;
                bool ok = true;
                for (int t = first; ok && t < total; t += stride) {
                    const Tile tl = decode<CG>(w, t);
                    const int arow = (WGRAD ? 0 : gr->offs[tl.g]) + tl.m0 + BM * static_cast<int>(rank);
                    const int brow = tl.n0 + BNH * static_cast<int>(rank);
                    const int gb = WGRAD ? 0 : tl.g;
                    for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
                        if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = full0 + 8 * stage;
                        const uint32_t da = smem_u32(sA + stage * A_BYTES), db = smem_u32(sB + stage * B_BYTES);
                        if constexpr (CG == 1) {
                            mbar_arrive_expect_tx(fb, A_BYTES + B_BYTES);
                            if (a_mn)
                                tma_load_3d(da, &P.mapA, fb, arow, kb * BK, 0);
                            else
                                tma_load_3d(da, &P.mapA, fb, kb * BK, arow, 0);
                            if (b_mn) {
                                for (int h = 0; h < BNH / 128; ++h)
                                    tma_load_3d(db + h * kBoxBytes, &P.mapB, fb, brow + 128 * h, kb * BK, gb);
                            } else {
                                tma_load_3d(db, &P.mapB, fb, kb * BK, brow, gb);
                            }
                        } else {
                            if (rank == 0) mbar_arrive_expect_tx(fb, 2 * (A_BYTES + B_BYTES));
                            const uint32_t lead_fb = map_to_rank(fb, 0);
                            if (a_mn)
                                tma_load_3d_pair(da, &P.mapA, lead_fb, arow, kb * BK, 0);
                            else
                                tma_load_3d_pair(da, &P.mapA, lead_fb, kb * BK, arow, 0);
                            if (b_mn)
                                tma_load_3d_pair(db, &P.mapB, lead_fb, brow, kb * BK, gb);
                            else
                                tma_load_3d_pair(db, &P.mapB, lead_fb, kb * BK, brow, gb);
                        }
                        ++issued;
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                // Loads still in flight land before the CTA ends.
                if (CG == 1 || rank == 0) {
                    const int pending = issued < STAGES ? issued : STAGES;
                    for (int i = 0; i < pending; ++i) {
                        if (stage == 0) {
                            stage = STAGES;
                            phase ^= 1;
                        }
                        --stage;
                        drain_wait(full0 + 8 * stage, phase, err.limit_ns);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------- MMA issuer (pair leader)
            if (lane == 0 && rank == 0) {
                uint32_t stage = 0, phase = 0;
                int it = 0;  // k blocks issued; the accumulator buffer is it & 1
                bool ok = true;
                const uint32_t idesc = idesc_f8(TM, BN, P.fmt_a, P.fmt_b, a_mn, b_mn);
                const uint64_t a0 = a_mn ? sw128_mnmajor_desc(smem_u32(sA), kBoxBytes) : sw128_kmajor_desc(smem_u32(sA));
                const uint64_t b0 = b_mn ? sw128_mnmajor_desc(smem_u32(sB), kBoxBytes) : sw128_kmajor_desc(smem_u32(sB));
                // A 32-wide k step: 32 bytes along a K-major row, or 32 rows of an MN-major tile.
                const uint32_t a_step = a_mn ? (4096 >> 4) : (32 >> 4);
                const uint32_t b_step = b_mn ? (4096 >> 4) : (32 >> 4);
                for (int t = first; ok && t < total; t += stride) {
                    const Tile tl = decode<CG>(w, t);
                    for (int kb = tl.kb0; kb < tl.kb1; ++kb, ++it) {
                        const int buf = it & 1;
                        if (!mbar_wait(acce0 + 8 * buf, ((it >> 1) & 1) ^ 1, err) ||
                            !mbar_wait(full0 + 8 * stage, phase, err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t adesc = a0 + ((stage * A_BYTES) >> 4);
                        const uint64_t bdesc = b0 + ((stage * B_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            tc_mma_f8<CG>(tmem_base + buf * BN, adesc + a_step * kk, bdesc + b_step * kk, idesc, kk != 0);
                        if constexpr (CG == 1) {
                            tc_commit<1>(empty0 + 8 * stage);
                            tc_commit<1>(accf0 + 8 * buf);
                        } else {
                            tc_commit_pair(empty0 + 8 * stage);
                            tc_commit_pair(accf0 + 8 * buf);
                        }
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                // All MMAs issued by this thread must finish before TMEM is freed.
                tc_commit<CG>(drain_bar);
                drain_wait(drain_bar, 0, err.limit_ns);
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int q = warp & 3;           // TMEM lane quarter this warp may read
        const int ew = warp - kEpiWarp0;
        const int half = ew >> 2;         // columns 128 half .. 128 half + 127 of the tile
        float* sbuf = scales + ew * 256;  // two k blocks' column scales (weight gradient)
        const uint32_t sbuf_u32 = smem_u32(sbuf);
        const uint32_t acce_lead = CG == 2 ? map_to_rank(acce0, 0) : acce0;
        const uint32_t tmem_warp = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
        int it = 0;
        bool ok = true;
        for (int t = first; ok && t < total; t += stride) {
            const Tile tl = decode<CG>(w, t);
            const int local = tl.m0 + BM * static_cast<int>(rank) + q * 32 + lane;
            const int rows = WGRAD ? P.M : gr->offs[tl.g + 1] - gr->offs[tl.g];
            const bool live = local < rows;
            const int row = WGRAD ? local : gr->offs[tl.g] + local;
            const int col = tl.n0 + 128 * half;
            // Scales are read two k blocks ahead of their use.
            const float* pa = P.sA + row;
            const float* pb = WGRAD ? P.sB + col + 4 * lane
                                    : P.sB + tl.g * P.sB_g + static_cast<long long>(col / kFp8Block) * P.sB_n;
            const bool b_in = WGRAD ? col + 4 * lane < P.sB_k : col < P.N;
            float sa[2] = {0.0f, 0.0f};
            float sb[2] = {0.0f, 0.0f};
            float4 sv[2];
            auto fetch = [&](int kb, int slot) {
                if (kb >= tl.kb1) return;
                sa[slot] = live ? __ldg(pa + kb * P.ldsA) : 0.0f;
                if constexpr (WGRAD)
                    sv[slot] = b_in ? __ldg(reinterpret_cast<const float4*>(pb + kb * P.sB_k)) : make_float4(0, 0, 0, 0);
                else
                    sb[slot] = b_in ? __ldg(pb + kb * P.sB_k) : 0.0f;
            };
            fetch(tl.kb0, 0);
            fetch(tl.kb0 + 1, 1);
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            int slot = 0;
#pragma unroll 1
            for (int kb = tl.kb0; kb < tl.kb1; ++kb, ++it) {
                const int buf = it & 1;
                float s = WGRAD ? sa[0] : sa[0] * sb[0];
                if constexpr (WGRAD) {
                    *reinterpret_cast<float4*>(sbuf + 128 * slot + 4 * lane) = sv[0];
                    sv[0] = sv[1];
                    __syncwarp();
                }
                sa[0] = sa[1];
                sb[0] = sb[1];
                fetch(kb + 2, 1);
                const uint64_t s2 = pack2(s, s);
                if (!__all_sync(0xffffffffu, mbar_wait_here(accf0 + 8 * buf, (it >> 1) & 1, err))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem_warp + buf * BN + 32 * c, v);
                    tmem_ld_wait_for(v);
                    if (c == 3) {  // the accumulator is in registers: the next MMAs may overwrite it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (CG == 1)
                                mbar_arrive(acce0 + 8 * buf);
                            else
                                mbar_arrive_cluster(acce_lead + 8 * buf);
                        }
                    }
                    if constexpr (WGRAD) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 f = ld_shared_v4(sbuf_u32 + 4 * (128 * slot + 32 * c + 4 * i));
                            fma2(acc[16 * c + 2 * i], v[4 * i], v[4 * i + 1], mul2(s2, pack2u(f.x, f.y)));
                            fma2(acc[16 * c + 2 * i + 1], v[4 * i + 2], v[4 * i + 3], mul2(s2, pack2u(f.z, f.w)));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) fma2(acc[16 * c + i], v[2 * i], v[2 * i + 1], s2);
                    }
                }
                slot ^= 1;
            }
            if (!ok) break;
            if (!live || col >= P.N) continue;
            const int ncol = P.N - col;
            if (P.split > 1) {
                float* d = P.partial + (static_cast<long long>(tl.split) * P.rows + row) * P.N + col;
                store_row<float>(d, acc, ncol, P.N % 8 == 0);
                continue;
            }
            const long long at = (WGRAD ? tl.g * P.strideD : 0LL) + static_cast<long long>(row) * P.ldd + col;
            const int es = P.out_dtype == GNS_FP32 ? 4 : 2;
            const bool direct = ((reinterpret_cast<uintptr_t>(P.D) | static_cast<uintptr_t>(P.ldd * es) |
                                  static_cast<uintptr_t>(P.strideD * es)) & 31) == 0;
            if (P.out_dtype == GNS_BF16)
                store_row(static_cast<__nv_bfloat16*>(P.D) + at, acc, ncol, direct);
            else if (P.out_dtype == GNS_FP16)
                store_row(static_cast<__half*>(P.D) + at, acc, ncol, direct);
            else
                store_row(static_cast<float*>(P.D) + at, acc, ncol, direct);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // The leader's MMAs read the peer's shared memory and the peer's loads and
    // epilogues arrive on the leader's barriers: neither leaves before the other.
    if constexpr (CG > 1) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, kTmemCols);
    }
}

// out[r][n] = sum over the splits, in order, of partial[split][r][n].
template <typename T>
__global__ void __launch_bounds__(256) fp8_reduce_kernel(const float* partial, int split, long long elems, int N, T* out,
                                                         long long ldd) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= elems) return;
    float s = 0.0f;
#pragma unroll 8
    for (int k = 0; k < split; ++k) s += partial[k * elems + i];
    const long long r = i / N;
    out[r * ldd + (i - r * N)] = from_f32<T>(s);
}

constexpr int kMaxDevices = 64;

template <int CG, bool WGRAD>
int launch_variant(const Fp8GemmJob& job, long long max_tiles, int num_sms, cudaStream_t s) {
    // Per device: the shared-memory opt-in and the clusters that fit at once.
    static int clusters[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<CG>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    if (clusters[dev] == 0) {
        e = cudaFuncSetAttribute(fp8_gemm_kernel<CG, WGRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem_bytes<CG>());
        if (e != cudaSuccess) return e;
        int n = 0;
        cfg.gridDim = dim3(CG * (num_sms / CG > 0 ? num_sms / CG : 1));
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<CG, WGRAD>, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = num_sms / CG;
        }
        clusters[dev] = n > 0 ? n : 1;
    }
    const int fit = std::max(1, std::min(clusters[dev], num_sms / CG));
    cfg.gridDim = dim3(CG * static_cast<unsigned>(std::min<long long>(fit, max_tiles)));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<CG, WGRAD>, job);
}

}  // namespace

int fp8_gemm_tile_rows(int M, int N, int G, bool grouped, int num_sms) {
    // Pairs (256-row tiles) halve the L2 traffic of a k block's B; single CTAs
    // waste fewer rows on ragged groups and fill the machine sooner.
    const long long per = grouped ? (M + G - 1) / G : M;
    const long long tn = (N + BN - 1) / BN;
    const long long pairs = (grouped ? G : 1) * ((per + 255) / 256) * tn;
    if (per <= 384 && grouped) return 128;
    return per > 128 && 2 * pairs >= num_sms ? 256 : 128;
}

int fp8_gemm_split(int rows, int N, int K, int num_sms) {
    const long long tiles = static_cast<long long>((rows + BM - 1) / BM) * ((N + BN - 1) / BN);
    const int kb = (K + BK - 1) / BK;
    if (2 * tiles > num_sms) return 1;
    // At least four k blocks each, so that the pipeline fills.
    return static_cast<int>(std::max<long long>(1, std::min<long long>(num_sms / tiles, kb / 4)));
}

int launch_fp8_gemm(const Fp8GemmJob& job, int tile_rows, int num_sms, cudaStream_t s) {
    const long long tn = (job.N + BN - 1) / BN;
    const long long tm = job.wgrad
                             ? static_cast<long long>(job.G) * ((job.M + tile_rows - 1) / tile_rows)
                             : (job.offsets ? (job.rows + static_cast<long long>(tile_rows - 1) * (std::min(job.rows, job.G) + 1)) / tile_rows
                                            : (job.rows + tile_rows - 1) / tile_rows);
    const long long tiles = tm * tn * job.split;
    if (tiles <= 0) return cudaSuccess;
    int e;
    if (tile_rows == 256)
        e = job.wgrad ? launch_variant<2, true>(job, tiles, num_sms, s) : launch_variant<2, false>(job, tiles, num_sms, s);
    else
        e = job.wgrad ? launch_variant<1, true>(job, tiles, num_sms, s) : launch_variant<1, false>(job, tiles, num_sms, s);
    if (e != cudaSuccess || job.split <= 1) return e;
    const long long elems = static_cast<long long>(job.rows) * job.N;
    return by_dtype(job.out_dtype, [&](auto t) {
        using T = decltype(t);
        return static_cast<int>(launch_after(fp8_reduce_kernel<T>, dim3(static_cast<unsigned>((elems + 255) / 256)),
                                             dim3(256), 0, s, static_cast<const float*>(job.partial), job.split, elems,
                                             job.N, static_cast<T*>(job.D), job.ldd));
    });
}

}  // namespace gns
