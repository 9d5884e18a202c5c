// Block-scaled 8-bit products on tcgen05 (sm_103a): forward, data gradient and
// weight gradient of a linear layer, for one weight matrix or for the experts
// of a routed batch in one launch.
//
//   D[m][n] = sum over k blocks b of  sA(m, b) sB(n, b) sum_{k in b} A[m][k] B[n][k]
//
// with blocks of 128 along the contraction. The tensor core sums one block's
// 128 products in fp32 (kind::f8f6f4, TMEM); the epilogue warps then add
// sA sB times that partial sum to fp32 accumulators in registers. A block is
// 512 cycles of MMA for a 128 x 256 tile; the epilogue's share of it (TMEM
// reads 256 cycles, scaled adds 256 per scheduler) has to run beside the next
// block's MMAs, which write the other half of TMEM.
//
// One CTA per SM walks 128 x 256 tiles with a static stride. Warp roles:
//   warp 0     TMA producer of 128-byte-wide k blocks (128-byte swizzle)
//   warp 1     TMEM owner, MMA issuer; k block i goes to accumulator buffer
//              i & 1 (256 columns each)
//   warp 2     scale producer: cp.async of a k block's row and column scales
//              into a ring of shared-memory slots, several blocks ahead
//   warp 3     scheduler: decodes the CTA's tiles ahead of their use (the
//              divisions and the search for a tile's group took the other
//              roles 2200 cycles per tile) into a ring of records
//   warps 4-11 epilogue: lane quarter warp & 3, columns 128 ((warp - 4) >> 2)
//              to + 127 of the tile, 128 accumulators per thread. The first
//              warpgroup gives registers up for them: 40 + 2 x 232 per lane of
//              the 3 x 168 the block is launched with.
// Measured and left: CTA pairs (256 x 256 tiles, paired MMAs) load a third less
// from L2, but their accumulator hand-shake crosses CTAs once per block
// (8192 x 14336 x 4096 forward: 954 us against 551); sixteen epilogue warps of
// 64 columns hide no more latency than eight (598 us).
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
constexpr int kCols = 128;  // columns of an epilogue warp
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kBand = 16;  // tile rows walked together (their A stays in L2 while the columns pass)
constexpr uint32_t kTmemCols = 2 * BN;
constexpr uint32_t A_BYTES = BM * BK;
constexpr uint32_t B_BYTES = BN * BK;
constexpr uint32_t kBoxBytes = 128 * 128;
constexpr int STAGES = 3;
constexpr int kStageRow = 128;                    // bytes of a row staged for the output stores
constexpr int kStageBytes = 32 * kStageRow;        // per epilogue warp

// A scale slot holds kSlotBlocks k blocks' scales, for each the 128 row scales
// and then its two column-half scales, or 256 column scales (weight gradient).
// One barrier wait per k block costs the epilogue about 150 cycles of the 800
// it has; a slot of four shares it.
constexpr int kScaleSlots = 3;
constexpr int kSlotBlocks = 4;
template <bool WGRAD>
constexpr int kScaleFloats = WGRAD ? BM + BN : BM + 4;
template <bool WGRAD>
constexpr int kSlotFloats = kSlotBlocks * kScaleFloats<WGRAD>;

constexpr int kTileSlots = 4;
constexpr int kTileReaders = 3 + kEpiWarps;  // producer, MMA issuer, scale producer, epilogue warps

constexpr int kNumBars = 2 * STAGES + 5 + 2 * kScaleSlots + 2 * kTileSlots;

// A tile as the roles see it.
struct Tile {
    int g;         // group; G: the rows past the last group (all zero); -1: no more tiles
    int m0, n0;    // origin: row within the group (weight gradient: row of D), column
    int kb0, kb1;  // k blocks
    int split;
    int row0;      // first row of the group in A and D (0 for the weight gradient)
    int rows;      // rows of the group (weight gradient: of D)
};
static_assert(sizeof(Tile) == 32, "read as two 16-byte pieces");

struct Groups {
    int offs[kMaxExperts + 2];  // first row of each group; offs[G + 1]: all rows
    int pre[kMaxExperts + 2];   // tile rows (weight gradient: token blocks) of the groups before
};

constexpr int kSmemBytes = 1024 + STAGES * static_cast<int>(A_BYTES + B_BYTES) + kScaleSlots * kSlotFloats<true> * 4 +
                           kEpiWarps * kStageBytes + kTileSlots * static_cast<int>(sizeof(Tile)) + kNumBars * 8 + 16 + static_cast<int>(sizeof(Groups));
static_assert(kSmemBytes <= 232448, "shared memory budget");

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
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

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// tcgen05.wait::ld that the uses of v depend on.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
          "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
          "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
          "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
          "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
        :
        : "memory");
}

// BYTES from global to shared memory, zeros where `in` is false (then `safe`,
// which is not read, stands for the address).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const float* src, bool in, const float* safe) {
    const int n = in ? BYTES : 0;
    const float* p = in ? src : safe;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// What the scheduler needs to decode tiles.
struct Walk {
    int G, M, ntn, mtn, split, wgrad, total_kb;
    const Groups* gr;
};

__device__ __forceinline__ Tile decode(const Walk& w, int t) {
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
    tl.m0 = (band * kBand + rem - nt * h) * BM;
    if (w.wgrad) {
        tl.kb0 = w.gr->pre[tl.g];
        tl.kb1 = w.gr->pre[tl.g + 1];
    } else if (tl.g == w.G) {
        tl.kb0 = tl.kb1 = 0;
    } else {
        tl.kb0 = static_cast<int>(static_cast<long long>(w.total_kb) * tl.split / w.split);
        tl.kb1 = static_cast<int>(static_cast<long long>(w.total_kb) * (tl.split + 1) / w.split);
    }
    tl.row0 = w.wgrad ? 0 : w.gr->offs[tl.g];
    tl.rows = w.wgrad ? w.M : w.gr->offs[tl.g + 1] - tl.row0;
    return tl;
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer() - t0 > limit_ns) break;
    }
}

// One 32-bit word of two 16-bit results, or of one 32-bit result.
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_half2(lo, hi);
}

// The warp's 32 rows x kCols columns (a thread holds one row), clipped to
// rows x ncol, to d (row stride ldd elements of ES bytes). Rows go through
// shared memory, 128 bytes of each at a time (16-byte pieces, piece index XOR
// row mod 8), so that a store instruction writes four whole 128-byte lines
// where rows start on 16-byte boundaries, and runs of neighbouring elements
// where they do not. Straight from the registers a store would touch 32 rows:
// a 128 x 256 tile took 4000 cycles that way.
template <int ES>
__device__ __forceinline__ void store_tile(uint32_t stage, uint8_t* d, long long ldd, int rows, int ncol,
                                           const float (&acc)[kCols], bool bf16, bool aligned, int lane) {
    constexpr int PASS = kStageRow / ES;  // columns per pass
    constexpr int PIECE = 16 / ES;        // elements of a 16-byte piece
#pragma unroll
    for (int p = 0; p < kCols / PASS; ++p) {
        const int left = ncol - p * PASS;  // columns from here on
        if (left <= 0) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (ES == 2)
                    w[e] = pack_pair(acc[p * PASS + 8 * k + 2 * e], acc[p * PASS + 8 * k + 2 * e + 1], bf16);
                else
                    w[e] = __float_as_uint(acc[p * PASS + 4 * k + e]);
            }
            st_shared_v4(stage + lane * kStageRow + ((k ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        uint8_t* dp = d + static_cast<long long>(p) * kStageRow;
        if (aligned) {
            const int k = lane & 7, r0 = lane >> 3;
            uint4 piece[8];  // all reads first: each takes some 200 cycles beside the MMAs
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 4 * j + r0;
                piece[j] = ld_shared_v4(stage + r * kStageRow + ((k ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 4 * j + r0;
                const uint4 v = piece[j];
                uint8_t* a = dp + r * ldd * ES + 16 * k;
                if (r < rows) {
                    if ((k + 1) * PIECE <= left) {
                        *reinterpret_cast<uint4*>(a) = v;
                    } else {
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < PIECE; ++e) {
                            if (k * PIECE + e >= left) continue;
                            if constexpr (ES == 2)
                                reinterpret_cast<uint16_t*>(a)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
                            else
                                reinterpret_cast<uint32_t*>(a)[e] = w[e];
                        }
                    }
                }
            }
        } else {
            for (int r = 0; r < min(rows, 32); ++r) {
#pragma unroll
                for (int c = lane; c < PASS; c += 32) {
                    const uint32_t at = stage + r * kStageRow + (((c / PIECE) ^ (r & 7)) << 4) + (c % PIECE) * ES;
                    if (c < left) {
                        if constexpr (ES == 2)
                            *reinterpret_cast<uint16_t*>(dp + r * ldd * ES + c * ES) = ld_shared_u16(at);
                        else
                            *reinterpret_cast<float*>(dp + r * ldd * ES + c * ES) = ld_shared_f32(at);
                    }
                }
            }
        }
        __syncwarp();  // read before the next pass overwrites
    }
}

template <bool WGRAD>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmJob P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + STAGES * A_BYTES;
    float* scales = reinterpret_cast<float*>(sB + STAGES * B_BYTES);
    uint8_t* staging = reinterpret_cast<uint8_t*>(scales + kScaleSlots * kSlotFloats<true>);
    Tile* tiles = reinterpret_cast<Tile*>(staging + kEpiWarps * kStageBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(tiles + kTileSlots);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
    Groups* gr = reinterpret_cast<Groups*>(tmem_slot + 4);

    const uint32_t full0 = smem_u32(bars);
    const uint32_t empty0 = smem_u32(bars + STAGES);
    const uint32_t accf0 = smem_u32(bars + 2 * STAGES);
    const uint32_t acce0 = smem_u32(bars + 2 * STAGES + 2);
    const uint32_t drain_bar = smem_u32(bars + 2 * STAGES + 4);
    const uint32_t sfull0 = smem_u32(bars + 2 * STAGES + 5);
    const uint32_t sempty0 = sfull0 + 8 * kScaleSlots;
    const uint32_t tfull0 = sempty0 + 8 * kScaleSlots;
    const uint32_t tempty0 = tfull0 + 8 * kTileSlots;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const DevStatus& err = P.st;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        for (int b = 0; b < kScaleSlots; ++b) {
            mbar_init(sfull0 + 8 * b, 32);
            mbar_init(sempty0 + 8 * b, kEpiWarps);
        }
        for (int b = 0; b < kTileSlots; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, kTileReaders);
        }
        fence_mbar_init();
        prefetch_tmap(&P.mapA);
        prefetch_tmap(&P.mapB);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish<1>();
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
            return WGRAD ? (c + BK - 1) / BK : (c + BM - 1) / BM;
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
        const int u = WGRAD ? (P.rows + BK - 1) / BK : (P.rows + BM - 1) / BM;
        gr->offs[0] = 0;
        gr->offs[1] = gr->offs[2] = P.rows;
        gr->pre[0] = 0;
        gr->pre[1] = gr->pre[2] = u;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // The CTA's i-th tile, from ring slot i mod kTileSlots; false after the
    // last one or when a wait gave up. Called by a thread or by whole warps.
    const uint32_t tiles_u32 = smem_u32(tiles);
    auto take = [&](int i, Tile& tl, bool whole_warp) -> bool {
        const int slot = i % kTileSlots;
        bool got = mbar_wait_here(tfull0 + 8 * slot, (i / kTileSlots) & 1, err);
        if (whole_warp) got = __all_sync(0xffffffffu, got);
        if (!got) return false;
        const uint32_t at = tiles_u32 + slot * static_cast<uint32_t>(sizeof(Tile));
        const uint4 a = ld_shared_v4(at), b = ld_shared_v4(at + 16);
        tl = Tile{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
                  static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(tempty0 + 8 * slot);
        return tl.g >= 0;
    };
    const bool a_mn = WGRAD, b_mn = WGRAD || P.b_mn;

    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            if (lane == 0) {
                uint32_t stage = 0, phase = 0;
                int issued = 0;
                bool ok = true;
                Tile tl;
                for (int i = 0; ok && take(i, tl, false); ++i) {
                    const int arow = tl.row0 + tl.m0;
                    const int gb = WGRAD ? 0 : tl.g;
                    for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
                        if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = full0 + 8 * stage;
                        const uint32_t da = smem_u32(sA + stage * A_BYTES), db = smem_u32(sB + stage * B_BYTES);
                        mbar_arrive_expect_tx(fb, A_BYTES + B_BYTES);
                        if (a_mn)
                            tma_load_3d(da, &P.mapA, fb, arow, kb * BK, 0);
                        else
                            tma_load_3d(da, &P.mapA, fb, kb * BK, arow, 0);
                        if (b_mn) {
                            for (int h = 0; h < BN / 128; ++h)
                                tma_load_3d(db + h * kBoxBytes, &P.mapB, fb, tl.n0 + 128 * h, kb * BK, gb);
                        } else {
                            tma_load_3d(db, &P.mapB, fb, kb * BK, tl.n0, gb);
                        }
                        ++issued;
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                // Loads still in flight land before the CTA ends.
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
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------- MMA issuer
            if (lane == 0) {
                uint32_t stage = 0, phase = 0;
                int it = 0;  // k blocks issued; the accumulator buffer is it & 1
                bool ok = true;
                const uint32_t idesc = idesc_f8(BM, BN, P.fmt_a, P.fmt_b, a_mn, b_mn);
                const uint64_t a0 = a_mn ? sw128_mnmajor_desc(smem_u32(sA), kBoxBytes) : sw128_kmajor_desc(smem_u32(sA));
                const uint64_t b0 = b_mn ? sw128_mnmajor_desc(smem_u32(sB), kBoxBytes) : sw128_kmajor_desc(smem_u32(sB));
                // A 32-wide k step: 32 bytes along a K-major row, or 32 rows of an MN-major tile.
                const uint32_t a_step = a_mn ? (4096 >> 4) : (32 >> 4);
                const uint32_t b_step = b_mn ? (4096 >> 4) : (32 >> 4);
                Tile tl;
                for (int i = 0; ok && take(i, tl, false); ++i) {
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
                            tc_mma_f8(tmem_base + buf * BN, adesc + a_step * kk, bdesc + b_step * kk, idesc, kk != 0);
                        tc_commit<1>(empty0 + 8 * stage);
                        tc_commit<1>(accf0 + 8 * buf);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                // All MMAs issued by this thread must finish before TMEM is freed.
                tc_commit<1>(drain_bar);
                drain_wait(drain_bar, 0, err.limit_ns);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ----------------------------------------------- scale producer
            const uint32_t ring = smem_u32(scales);
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true;
            Tile tl;
            for (int i = 0; ok && take(i, tl, true); ++i) {
                const int local = tl.m0 + lane;
                const float* pa = P.sA + tl.row0 + local;
                const float* pb = P.sB + (WGRAD ? tl.n0 + 4 * lane
                                                : tl.g * P.sB_g + static_cast<long long>(tl.n0 / kFp8Block + lane) * P.sB_n);
                for (int kb0 = tl.kb0; kb0 < tl.kb1; kb0 += kSlotBlocks) {
                    if (!__all_sync(0xffffffffu, mbar_wait(sempty0 + 8 * slot, phase ^ 1, err))) {
                        ok = false;
                        break;
                    }
                    const int end = min(kb0 + kSlotBlocks, tl.kb1);
                    for (int kb = kb0; kb < end; ++kb) {
                        const uint32_t dst = ring + 4 * (slot * kSlotFloats<WGRAD> + (kb - kb0) * kScaleFloats<WGRAD>);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            copy_async<4>(dst + 4 * (lane + 32 * i), pa + kb * P.ldsA + 32 * i, local + 32 * i < tl.rows, P.sA);
                        if constexpr (WGRAD) {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                copy_async<16>(dst + 4 * (BM + 4 * lane + 128 * i), pb + kb * P.sB_k + 128 * i,
                                               tl.n0 + 4 * lane + 128 * i < P.sB_k, P.sB);
                        } else if (lane < 2) {
                            copy_async<4>(dst + 4 * (BM + lane), pb + kb * P.sB_k, tl.n0 + 128 * lane < P.N, P.sB);
                        }
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sfull0 + 8 * slot) : "memory");
                    if (++slot == kScaleSlots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        } else if (lane == 0) {
            // ---------------------------------------------------- scheduler
            Walk w;
            w.G = G;
            w.M = P.M;
            w.ntn = (P.N + BN - 1) / BN;
            w.mtn = WGRAD ? (P.M + BM - 1) / BM : 0;
            w.split = P.split;
            w.wgrad = WGRAD;
            w.total_kb = WGRAD ? 0 : (P.K + BK - 1) / BK;
            w.gr = gr;
            const int total = WGRAD ? G * w.mtn * w.ntn : gr->pre[G + 1] * w.ntn * P.split;
            int t = static_cast<int>(blockIdx.x);
            for (int i = 0;; ++i, t += static_cast<int>(gridDim.x)) {
                Tile tl{};
                tl.g = -1;
                if (t < total) tl = decode(w, t);
                const int slot = i % kTileSlots;
                if (!mbar_wait(tempty0 + 8 * slot, ((i / kTileSlots) & 1) ^ 1, err)) break;
                const uint32_t at = tiles_u32 + slot * static_cast<uint32_t>(sizeof(Tile));
                st_shared_v4(at, tl.g, tl.m0, tl.n0, tl.kb0);
                st_shared_v4(at + 16, tl.kb1, tl.split, tl.row0, tl.rows);
                mbar_arrive(tfull0 + 8 * slot);
                if (tl.g < 0) break;
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int q = warp & 3;           // TMEM lane quarter this warp may read
        const int ew = warp - kEpiWarp0;
        const int cq = (ew >> 2) * kCols;  // its first column within the tile
        const uint32_t ring = smem_u32(scales);
        const uint32_t tmem_warp = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + cq;
        int it = 0;    // k blocks added
        int slot = 0;  // scale slot and its phase
        uint32_t sphase = 0;
        bool ok = true;
        Tile tl;
        for (int i = 0; ok && take(i, tl, true); ++i) {
            const int col = tl.n0 + cq;
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
            // A chunk of 32 columns is loaded from TMEM while the one before it
            // is added; the next k block's barrier is polled ahead of its use
            // (a poll, like every shared-memory access, takes some 150 cycles
            // beside the MMAs' operand reads).
            bool ready = false;
            float s = 0.0f;
#pragma unroll 1
            for (int kb = tl.kb0; kb < tl.kb1; ++kb, ++it) {
                const int in_slot = (kb - tl.kb0) % kSlotBlocks;
                const uint32_t acc_tmem = tmem_warp + (it & 1) * BN;
                const uint32_t sc = ring + 4 * (slot * kSlotFloats<WGRAD> + in_slot * kScaleFloats<WGRAD>);
                if (!__all_sync(0xffffffffu, ready)) {
                    ok = (in_slot != 0 || mbar_wait_here(sfull0 + 8 * slot, sphase, err)) &&
                         mbar_wait_here(accf0 + 8 * (it & 1), (it >> 1) & 1, err);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_after();
                uint32_t v[2][32];
                tmem_ld_32x32b_x32(acc_tmem, v[0]);
                s = ld_shared_f32(sc + 4 * (q * 32 + lane));
                if (!WGRAD) s *= ld_shared_f32(sc + 4 * (BM + cq / kFp8Block));
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    const uint32_t(&x)[32] = v[c & 1];
                    tmem_ld_wait_for(v[c & 1]);
                    if (c + 1 < kCols / 32) {
                        tmem_ld_32x32b_x32(acc_tmem + 32 * (c + 1), v[(c + 1) & 1]);
                    } else {  // all in registers: the next MMAs may overwrite the accumulator
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acce0 + 8 * (it & 1));
                        ready = in_slot != kSlotBlocks - 1 && kb + 1 < tl.kb1 &&
                                mbar_test(accf0 + 8 * ((it + 1) & 1), ((it + 1) >> 1) & 1);
                    }
                    if constexpr (WGRAD) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 f = ld_shared_v4(sc + 4 * (BM + cq + 32 * c + 4 * i));
                            const uint32_t g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = 4 * i + e;
                                acc[32 * c + j] = fmaf(__uint_as_float(x[j]), s * __uint_as_float(g[e]), acc[32 * c + j]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            acc[32 * c + j] = fmaf(__uint_as_float(x[j]), s, acc[32 * c + j]);
                    }
                }
                if (in_slot == kSlotBlocks - 1 || kb + 1 == tl.kb1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sempty0 + 8 * slot);
                    if (++slot == kScaleSlots) {
                        slot = 0;
                        sphase ^= 1;
                    }
                }
            }
            if (!ok) break;
            // Rows of this warp inside the group (of D) and columns inside D.
            const int wrows = tl.rows - tl.m0 - q * 32, ncol = P.N - col;
            if (wrows <= 0 || ncol <= 0) continue;
            const int es = P.out_dtype == GNS_FP32 || P.split > 1 ? 4 : 2;
            const uint32_t stage = smem_u32(staging + ew * kStageBytes);
            const long long row0 = tl.row0 + tl.m0 + q * 32;
            uint8_t* d;
            long long ldd;
            bool aligned;
            if (P.split > 1) {
                d = reinterpret_cast<uint8_t*>(P.partial + (static_cast<long long>(tl.split) * P.rows + row0) * P.N + col);
                ldd = P.N;
                aligned = P.N % 4 == 0;
            } else {
                d = static_cast<uint8_t*>(P.D) + ((WGRAD ? tl.g * P.strideD : 0LL) + row0 * P.ldd + col) * es;
                ldd = P.ldd;
                aligned = ((reinterpret_cast<uintptr_t>(P.D) | static_cast<uintptr_t>(P.ldd * es) |
                            static_cast<uintptr_t>(P.strideD * es)) & 15) == 0;
            }
            if (es == 2)
                store_tile<2>(stage, d, ldd, wrows, ncol, acc, P.out_dtype == GNS_BF16, aligned, lane);
            else
                store_tile<4>(stage, d, ldd, wrows, ncol, acc, false, aligned, lane);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, kTmemCols);
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

template <bool WGRAD>
int launch_variant(const Fp8GemmJob& job, long long max_tiles, int num_sms, cudaStream_t s) {
    static bool configured[kMaxDevices];  // the shared-memory opt-in is per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(fp8_gemm_kernel<WGRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const unsigned grid = static_cast<unsigned>(std::min<long long>(num_sms, max_tiles));
    return launch_after(fp8_gemm_kernel<WGRAD>, dim3(grid), dim3(kThreads), kSmemBytes, s, job);
}

}  // namespace

int fp8_gemm_split(int rows, int N, int K, int num_sms) {
    const long long tiles = static_cast<long long>((rows + BM - 1) / BM) * ((N + BN - 1) / BN);
    const int kb = (K + BK - 1) / BK;
    if (2 * tiles > num_sms) return 1;
    // At least four k blocks each, so that the pipeline fills.
    return static_cast<int>(std::max<long long>(1, std::min<long long>(num_sms / tiles, kb / 4)));
}

int launch_fp8_gemm(const Fp8GemmJob& job, int num_sms, cudaStream_t s) {
    const long long tn = (job.N + BN - 1) / BN;
    long long tm;  // tile rows, an upper bound where the groups are on the device
    if (job.wgrad)
        tm = static_cast<long long>(job.G) * ((job.M + BM - 1) / BM);
    else if (job.offsets)
        tm = (job.rows + static_cast<long long>(BM - 1) * (std::min(job.rows, job.G) + 1)) / BM;
    else
        tm = (job.rows + BM - 1) / BM;
    const long long tiles = tm * tn * job.split;
    if (tiles <= 0) return cudaSuccess;
    const int e = job.wgrad ? launch_variant<true>(job, tiles, num_sms, s) : launch_variant<false>(job, tiles, num_sms, s);
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
