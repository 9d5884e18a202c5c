// Block-scaled 8-bit products on tcgen05 (sm_103a): forward, data gradient and
// weight gradient of a linear layer, for one weight matrix or for the experts
// of a routed batch in one launch.
//
//   D[m][n] = sum over k blocks b of  sA(m, b) sB(n, b) sum_{k in b} A[m][k] B[n][k]
//
// with blocks of 128 along the contraction and power-of-two scales. The tensor
// core applies the scales itself (kind::mxf8f6f4, block_scale): it takes one
// 8-bit exponent per row of A and of B and 32-wide k step, so a block of 128 is
// four steps with the same exponent, and the sum stays in TMEM in fp32. That
// accumulator truncates, an error that grows with the steps: up to about 2^-23 of
// the sum per step of 32 terms where all have one sign (3.7e-2 of a sum of 8.4
// million), 2.9e-6 of a result at 4096 terms of mixed signs. So fp32 results are
// summed in segments of kSegment blocks, each segment added to the stored result
// with one rounding (6e-7 at any length), and 16-bit results in segments of
// kFp8LongBlocks blocks (32768 terms, 1.5e-4 at most: a third of fp16's
// rounding), whose fp32 sums a tile's CTA carries on in its own part of an
// intermediate buffer. (Weight gradients over 65536 rows, two segments: N x K =
// 1024 x 4096 204 us without and 206 to 217 with it, 4096 x 4096 798 to 814 and
// 804 to 837; segments of 128 blocks cost up to twice that.)
// Applying the scales in registers instead, which any fp32 scale would need,
// reads the accumulator once per block: 1220 cycles per block beside the 512 of
// its MMAs (8192 x 14336 x 4096 forward: 470 us, with scaled MMAs 378).
//
// One CTA (CG = 1, 128 x 256 tiles) or a pair (CG = 2, 256 x 256 tiles, paired
// MMAs; each CTA stages 128 rows of each operand) per SM (pair) walks the tiles
// with a static stride. Warp roles:
//   warp 0     TMA producer of 128-byte-wide k blocks (128-byte swizzle)
//   warp 1     TMEM owner, MMA issuer (the pair's leader)
//   warp 2     scheduler: decodes the CTA's tiles ahead of their use (the
//              divisions and the search for a tile's group take some 2000
//              cycles) into a ring of records
//   warps 4-7  scale builders: a slot holds four k blocks' exponents, one
//              32-bit word per row in the order tcgen05.cp spreads over TMEM;
//              warp 4 + j writes byte j
//   warps 8-15 epilogue: lane quarter warp & 3, column half (warp - 8) >> 2
// TMEM: two accumulators of 256 columns that overlap by the 24 columns the
// scales take, so the next tile's MMAs wait for the chunk of 32 columns in the
// overlap to be read (the first thing the epilogue does) and run beside the
// rest of the epilogue.
// Operands whose contraction runs along the stored rows (the weights of the
// data gradient, both operands of the weight gradient) are read MN-major
// through the shared-memory descriptor; nothing is transposed in memory.
//
// Bound: the tensor cores for large matrices, HBM for many experts of few rows,
// the latency of one tile for small ones. 8192 x 14336 x 4096: forward 295 us
// (3.3 PFLOP/s, 0.87 of twice the measured bf16 rate), data gradient 327 (2.9),
// weight gradient 331 (2.9). 256 experts of 512 x 2048, 65536 rows: 85, 96 and
// 126 us (5.5 to 5.8 TB/s of operands and results, each once). One tile of one k
// block: 4.7 us.
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
constexpr int kBuildWarp0 = 4;
constexpr int kEpiWarp0 = 8;
constexpr int kCols = 128;  // columns of an epilogue warp
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kBand = 16;  // tile rows walked together (their A stays in L2 while the columns pass)
constexpr uint32_t A_BYTES = BM * BK;
constexpr uint32_t kBoxBytes = 128 * 128;

// TMEM columns: accumulator 0 at 0, accumulator 1 at kAcc1, two scale slots of
// 4 columns for A's 128 rows and 8 for B's 256.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCols = 12;
constexpr uint32_t kScaleTmem = kTmemCols - 2 * kScaleCols;
constexpr uint32_t kAcc1 = kScaleTmem - BN;
static_assert(BN - kAcc1 <= 32, "the overlap lies in one chunk of 32 columns of either accumulator");

// CG = 1: a CTA computes 128 x 256 tiles. CG = 2: a pair of CTAs computes 256 x
// 256 tiles with paired MMAs; each stages its 128 rows of A and 128 of B's 256.
template <int CG>
struct Cfg {
    static constexpr int STAGES = CG == 1 ? 4 : 5;
    static constexpr int STORE_ROW = fp8_store_row(CG);          // bytes of a row staged for an output store
    static constexpr uint32_t STORE_BYTES = 32 * STORE_ROW;      // an epilogue warp's buffer
    static constexpr int BNH = BN / CG;  // rows of B a CTA stages
    static constexpr uint32_t B_BYTES = BNH * BK;
    static constexpr int TM = BM * CG;
};

// A scale slot in shared memory: 512 bytes for A's 128 rows and 1024 for B's
// 256. Row r of 128 is the word at 16 (r mod 32) + 4 (r / 32); its byte j is the
// exponent of the slot's j-th k block.
constexpr int kScaleSlots = 2;
constexpr int kSlotBlocks = 4;
constexpr uint32_t kSlotBytes = 512 + 1024;
constexpr int kSegment = 16;  // k blocks of a segment of an fp32 result
static_assert(kSegment % kSlotBlocks == 0 && kFp8LongBlocks % kSlotBlocks == 0, "a scale slot lies in one segment");

constexpr int kTileSlots = 4;
constexpr int kTileReaders = 2 + kSlotBlocks + kEpiWarps;  // producer, MMA issuer, scale builder, epilogue warps

__host__ __device__ constexpr int num_bars(int stages) { return 2 * stages + 6 + 2 * kScaleSlots + 2 * kTileSlots; }

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

template <int CG>
constexpr int smem_bytes() {
    return 1024 + Cfg<CG>::STAGES * static_cast<int>(A_BYTES + Cfg<CG>::B_BYTES) + kScaleSlots * static_cast<int>(kSlotBytes) +
           kEpiWarps * static_cast<int>(Cfg<CG>::STORE_BYTES) + kTileSlots * static_cast<int>(sizeof(Tile)) + num_bars(Cfg<CG>::STAGES) * 8 + 16 +
           static_cast<int>(sizeof(Groups));
}
static_assert(smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448, "shared memory budget");

// D(tmem) (+)= A(smem) * B(smem)^T with the exponents of the rows of A and B
// at the TMEM addresses sfa and sfb (the byte idesc names).
template <int CG>
__device__ __forceinline__ void tc_mma_mx(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
}

// Instruction descriptor of kind::mxf8f6f4 with 8-bit exponents as scales; the
// byte of the scale words is added per k block (scale_id).
__device__ __forceinline__ uint32_t idesc_mx(int M, int N, int fmt_a, int fmt_b, uint32_t a_mn, uint32_t b_mn) {
    return (static_cast<uint32_t>(fmt_a) << 7)  // 0: e4m3, 1: e5m2
           | (static_cast<uint32_t>(fmt_b) << 10) | (a_mn << 15) | (b_mn << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (1u << 23)  // scale type: 8-bit exponent
           | (static_cast<uint32_t>(M >> 7) << 27);
}
__device__ __forceinline__ uint32_t scale_id(uint32_t byte) { return (byte << 4) | (byte << 29); }

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 512 bytes of scale words (32 rows of 16 bytes, contiguous) from shared memory
// to four TMEM columns of each lane quarter.
template <int CG>
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);  // start address
    d |= static_cast<uint64_t>(128 >> 4) << 32;               // stride byte offset: 8 rows of 16 bytes
    d |= static_cast<uint64_t>(1) << 46;                       // descriptor version; no swizzle
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
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

// What the scheduler needs to decode tiles.
struct Walk {
    int G, M, ntn, mtn, split, wgrad, total_kb;
    const Groups* gr;
};

template <int CG>
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
    tl.m0 = (band * kBand + rem - nt * h) * Cfg<CG>::TM;
    if (w.wgrad) {
        tl.kb0 = w.gr->pre[tl.g];
        tl.kb1 = w.gr->pre[tl.g + 1];
    } else if (tl.g == w.G) {
        tl.kb0 = tl.kb1 = 0;
    } else {
        // total_kb < 2^24 and at most 152 parts: the products fit 32 bits.
        tl.kb0 = static_cast<int>(static_cast<uint32_t>(w.total_kb) * static_cast<uint32_t>(tl.split) / static_cast<uint32_t>(w.split));
        tl.kb1 = static_cast<int>(static_cast<uint32_t>(w.total_kb) * static_cast<uint32_t>(tl.split + 1) /
                                  static_cast<uint32_t>(w.split));
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

// One 32-bit word of two 16-bit results.
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_half2(lo, hi);
    }
}

// Offset of a staged row's 16-byte piece: the 64- or 128-byte swizzle.
template <int ROW>
__device__ __forceinline__ uint32_t stage_piece(int row, int piece) {
    static_assert(ROW == 64 || ROW == 128, "a swizzle's row");
    return row * ROW + ((piece ^ (ROW == 64 ? (row >> 1) & 3 : row & 7)) << 4);
}

__device__ __forceinline__ uint32_t add_bits(uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// Stores (or, with `add`, adds, fp32) a staged block of 32 rows of 64 or 128 bytes,
// asynchronously, clipped to the map's extents.
__device__ __forceinline__ void bulk_store(const CUtensorMap* m, uint32_t src, int c0, int c1, int c2, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(m)),
                     "r"(src), "r"(c0), "r"(c1), "r"(c2)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(m)),
                     "r"(src), "r"(c0), "r"(c1), "r"(c2)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Writes a staged block (32 rows of ROW bytes, swizzled), clipped to rows x left,
// to d (row stride ldd elements of ES bytes): a store instruction covers whole
// 16-byte pieces of neighbouring rows where rows start on 16-byte boundaries, and
// runs of neighbouring elements where they do not. With `add` (fp32) the stored
// values are added to; a lane meets its own stores.
template <int ES, int ROW>
__device__ __noinline__ void store_rows(uint32_t stage, uint8_t* d, long long ldd, int rows, int left, bool aligned,
                                           bool add, int lane) {
    constexpr int PASS = ROW / ES;  // columns
    constexpr int PIECE = 16 / ES;        // elements of a 16-byte piece
    constexpr int PR = ROW / 16;    // pieces of a row
    if (aligned) {
        const int k = lane % PR, r0 = lane / PR;
        uint4 piece[PR];  // all reads first
#pragma unroll
        for (int j = 0; j < PR; ++j) {
            const int r = 32 / PR * j + r0;
            piece[j] = ld_shared_v4(stage + stage_piece<ROW>(r, k));
        }
        if (ES == 4 && add && (k + 1) * PIECE <= left) {
            uint4 old[PR];
#pragma unroll
            for (int j = 0; j < PR; ++j) {
                const int r = 32 / PR * j + r0;
                old[j] = r < rows ? *reinterpret_cast<const uint4*>(d + r * ldd * ES + 16 * k) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < PR; ++j) {
                piece[j].x = add_bits(old[j].x, piece[j].x);
                piece[j].y = add_bits(old[j].y, piece[j].y);
                piece[j].z = add_bits(old[j].z, piece[j].z);
                piece[j].w = add_bits(old[j].w, piece[j].w);
            }
        }
#pragma unroll
        for (int j = 0; j < PR; ++j) {
            const int r = 32 / PR * j + r0;
            uint8_t* a = d + r * ldd * ES + 16 * k;
            if (r >= rows) continue;
            if ((k + 1) * PIECE <= left) {
                *reinterpret_cast<uint4*>(a) = piece[j];
            } else {
                const uint32_t x[4] = {piece[j].x, piece[j].y, piece[j].z, piece[j].w};
#pragma unroll
                for (int e = 0; e < PIECE; ++e) {
                    if (k * PIECE + e >= left) continue;
                    if constexpr (ES == 2)
                        reinterpret_cast<uint16_t*>(a)[e] = static_cast<uint16_t>(x[e / 2] >> (16 * (e & 1)));
                    else
                        reinterpret_cast<uint32_t*>(a)[e] = add ? add_bits(reinterpret_cast<uint32_t*>(a)[e], x[e]) : x[e];
                }
            }
        }
    } else {
        constexpr int LANES = PASS < 32 ? PASS : 32;  // lanes on a row
        for (int r = lane / LANES; r < min(rows, 32); r += 32 / LANES) {
#pragma unroll
            for (int c = lane % LANES; c < PASS; c += LANES) {
                const uint32_t at = stage + stage_piece<ROW>(r, c / PIECE) + (c % PIECE) * ES;
                if (c < left) {
                    if constexpr (ES == 2)
                        *reinterpret_cast<uint16_t*>(d + r * ldd * ES + c * ES) = ld_shared_u16(at);
                    else {
                        float* a = reinterpret_cast<float*>(d + r * ldd * ES + c * ES);
                        const float v = ld_shared_f32(at);
                        *a = add ? *a + v : v;
                    }
                }
            }
        }
    }
    __syncwarp();  // read before the next pass overwrites
}

// Hands accumulator columns back to the MMA issuer of the pair's leader. The
// tcgen05.wait::ld before it has put their values into registers, so no memory
// operation has to be ordered and the arrive is relaxed (one with
// cluster-scope release would wait for the warp's global stores).
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// T is the type that is stored: D's, or float for the partial sums of a split.
// One kernel per type and direction rather than branches: the warps' roles run
// at the same time and share the instruction cache, which short tiles feel most
// (256 experts of 512 x 2048, 65536 rows, with three operand stages: one kernel
// for all, data gradient 137 us, weight gradient 155; one per type 119 and 138;
// one per type and direction 112 and 138). Rare paths, the plain stores and the waits' spins, are out of line for
// the same reason.
template <int CG, typename T, bool wgrad>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmJob P) {
    constexpr int STAGES = Cfg<CG>::STAGES;
    constexpr int TM = Cfg<CG>::TM;
    constexpr int BNH = Cfg<CG>::BNH;
    constexpr uint32_t B_BYTES = Cfg<CG>::B_BYTES;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + STAGES * A_BYTES;
    uint8_t* staging = sB + STAGES * B_BYTES;  // 1024-byte aligned, as the swizzle wants
    uint8_t* scales = staging + kEpiWarps * Cfg<CG>::STORE_BYTES;
    Tile* tiles = reinterpret_cast<Tile*>(scales + kScaleSlots * kSlotBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(tiles + kTileSlots);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + num_bars(STAGES));
    Groups* gr = reinterpret_cast<Groups*>(tmem_slot + 4);

    const uint32_t full0 = smem_u32(bars);
    const uint32_t empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES;   // accumulator complete
    const uint32_t acce0 = accf0 + 16;            // accumulator read
    const uint32_t overlap_bar = acce0 + 16;      // the overlap's chunk of the last accumulator read
    const uint32_t drain_bar = overlap_bar + 8;
    const uint32_t sfull0 = drain_bar + 8;
    const uint32_t sempty0 = sfull0 + 8 * kScaleSlots;
    const uint32_t tfull0 = sempty0 + 8 * kScaleSlots;
    const uint32_t tempty0 = tfull0 + 8 * kTileSlots;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const DevStatus& err = P.st;
    const int rank = CG > 1 ? static_cast<int>(cluster_ctarank()) : 0;  // 0: the pair's leader
    // k blocks summed in TMEM before the result is stored or added to (fp32) or
    // added to the sums that are carried on to the tile's last segment (16 bits).
    constexpr int ES = sizeof(T);
    constexpr int segment = ES == 4 ? kSegment : kFp8LongBlocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, kEpiWarps * CG);
        }
        mbar_init(overlap_bar, kEpiWarps / 2 * CG);
        mbar_init(drain_bar, 1);
        for (int b = 0; b < kScaleSlots; ++b) {
            mbar_init(sfull0 + 8 * b, kSlotBlocks * CG);
            mbar_init(sempty0 + 8 * b, 1);
        }
        for (int b = 0; b < kTileSlots; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, kTileReaders - (rank != 0));  // no MMA issuer on the peer
        }
        fence_mbar_init();
        prefetch_tmap(&P.mapA);
        prefetch_tmap(&P.mapB);
        if (P.bulk_store) prefetch_tmap(&P.mapD);
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
            return wgrad ? (c + BK - 1) / BK : (c + TM - 1) / TM;
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
        gr->offs[0] = 0;
        gr->offs[1] = gr->offs[2] = P.rows;
        gr->pre[0] = 0;
        gr->pre[1] = gr->pre[2] = wgrad ? (P.rows + BK - 1) / BK : (P.rows + TM - 1) / TM;
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG > 1) cluster_sync();  // the pair's barriers exist before any remote use
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // The CTA's i-th tile, from ring slot i mod kTileSlots; false after the
    // last one or when a wait gave up. Called by a thread or by whole warps.
    const uint32_t tiles_u32 = smem_u32(tiles);
    auto take = [&](int i, Tile& tl, bool whole_warp) -> bool {
        const int slot = i % kTileSlots;
        bool got = mbar_wait(tfull0 + 8 * slot, (i / kTileSlots) & 1, err);
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
    constexpr bool a_mn = wgrad;
    const bool b_mn = wgrad || P.b_mn;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int issued = 0;
            bool ok = true;
            Tile tl;
            for (int i = 0; ok && take(i, tl, false); ++i) {
                const int arow = tl.row0 + tl.m0 + BM * rank;
                const int brow = tl.n0 + BNH * rank;
                const int gb = wgrad ? 0 : tl.g;
                for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full0 + 8 * stage;
                    const uint32_t da = smem_u32(sA + stage * A_BYTES), db = smem_u32(sB + stage * B_BYTES);
                    const int ka = a_mn ? arow : kb * BK, ra = a_mn ? kb * BK : arow;
                    if constexpr (CG == 1) {
                        mbar_arrive_expect_tx(fb, A_BYTES + B_BYTES);
                        tma_load_3d(da, &P.mapA, fb, ka, ra, 0);
                        if (b_mn) {
                            for (int h = 0; h < BNH / 128; ++h)
                                tma_load_3d(db + h * kBoxBytes, &P.mapB, fb, brow + 128 * h, kb * BK, gb);
                        } else {
                            tma_load_3d(db, &P.mapB, fb, kb * BK, brow, gb);
                        }
                    } else {  // both halves complete on the leader's barrier
                        if (rank == 0) mbar_arrive_expect_tx(fb, 2 * (A_BYTES + B_BYTES));
                        const uint32_t lead_fb = map_to_rank(fb, 0);
                        tma_load_3d_pair(da, &P.mapA, lead_fb, ka, ra, 0);
                        tma_load_3d_pair(db, &P.mapB, lead_fb, b_mn ? brow : kb * BK, b_mn ? kb * BK : brow, gb);
                    }
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // Loads still in flight land before the CTA ends.
            const int pending = rank != 0 ? 0 : issued < STAGES ? issued : STAGES;
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
        // ------------------------------------------- MMA issuer (pair leader)
        if (lane == 0 && rank == 0) {
            // This thread's own instructions bound the kernel when they take
            // longer than a block's MMAs (512 cycles), so the loop runs over
            // scale slots with their four k blocks unrolled, and counts
            // instead of dividing.
            uint32_t stage = 0, phase = 0;
            int it = 0;       // segments done; the accumulator is it & 1
            uint32_t sn = 0;  // scale slots used
            bool ok = true;
            const uint32_t idesc = idesc_mx(TM, BN, P.fmt_a, P.fmt_b, a_mn, b_mn);
            const uint64_t a0 = a_mn ? sw128_mnmajor_desc(smem_u32(sA), kBoxBytes) : sw128_kmajor_desc(smem_u32(sA));
            const uint64_t b0 = b_mn ? sw128_mnmajor_desc(smem_u32(sB), kBoxBytes) : sw128_kmajor_desc(smem_u32(sB));
            // A 32-wide k step: 32 bytes along a K-major row, or 32 rows of an MN-major tile.
            const uint32_t a_step = a_mn ? (4096 >> 4) : (32 >> 4);
            const uint32_t b_step = b_mn ? (4096 >> 4) : (32 >> 4);
            auto commit = [&](uint32_t bar) {
                if constexpr (CG == 1)
                    tc_commit<1>(bar);
                else
                    tc_commit_pair(bar);
            };
            Tile tl;
            for (int i = 0; ok && take(i, tl, false); ++i) {
                int left = tl.kb1 - tl.kb0;  // k blocks
                int in_segment = 0;          // scale slots of this segment so far
                while (left > 0) {
                    const uint32_t buf = it & 1, slot = sn & 1;
                    static_assert(kScaleSlots == 2, "slot and phase come from sn's bits");
                    const uint32_t d_tmem = tmem_base + buf * kAcc1;
                    if (in_segment == 0 && (!mbar_wait(acce0 + 8 * buf, ((it >> 1) & 1) ^ 1, err) ||
                                            (it > 0 && !mbar_wait(overlap_bar, (it - 1) & 1, err)))) {
                        ok = false;
                        break;
                    }
                    // A full slot also says that the MMAs that read its TMEM
                    // columns before are done (see the builders).
                    if (!mbar_wait_cluster(sfull0 + 8 * slot, (sn >> 1) & 1, err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sf = tmem_base + kScaleTmem + slot * kScaleCols;
                    const uint32_t src = smem_u32(scales) + slot * kSlotBytes;
                    tc_copy_scales<CG>(sf, src);
                    tc_copy_scales<CG>(sf + 4, src + 512);
                    tc_copy_scales<CG>(sf + 8, src + 1024);
#pragma unroll
                    for (int j = 0; j < kSlotBlocks; ++j) {
                        if (j >= left) break;
                        if (!mbar_wait(full0 + 8 * stage, phase, err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t adesc = a0 + stage * (A_BYTES >> 4);
                        const uint64_t bdesc = b0 + stage * (B_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            tc_mma_mx<CG>(d_tmem, adesc + a_step * kk, bdesc + b_step * kk, idesc | scale_id(j), sf, sf + 4,
                                          (j | kk) != 0 || in_segment != 0);
                        commit(empty0 + 8 * stage);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    commit(sempty0 + 8 * slot);
                    ++sn;
                    left -= kSlotBlocks;
                    if (++in_segment == segment / kSlotBlocks || left <= 0) {
                        commit(accf0 + 8 * buf);
                        ++it;
                        in_segment = 0;
                    }
                }
            }
            // All MMAs issued by this thread must finish before TMEM is freed.
            tc_commit<CG>(drain_bar);
            drain_wait(drain_bar, 0, err.limit_ns);
        }
        __syncwarp();
    } else if (warp >= kBuildWarp0 && warp < kEpiWarp0) {
        // --------------------------------------------------- scale builders
        // This warp's k block of each slot; lane l holds rows l, l + 32, l +
        // 64, l + 96 of A's (and of each half of B's) 128. The exponents
        // are read before the wait for the slot, which ends when the MMAs
        // that used it are done and so frees its TMEM columns too.
        const uint32_t ring = smem_u32(scales);
        const uint32_t sfull_lead = CG == 2 ? map_to_rank(sfull0, 0) : sfull0;
        const int j = warp - kBuildWarp0;
        int groups = 0;
        bool ok = true;
        Tile tl;
        for (int i = 0; ok && take(i, tl, true); ++i) {
            const int arow = tl.m0 + BM * rank + lane;
            const uint8_t* pa = P.sA + tl.row0 + arow;
            const uint8_t* pb = P.sB + (wgrad ? tl.n0 + lane
                                            : tl.g * P.sB_g + static_cast<long long>(tl.n0 / kFp8Block) * P.sB_n);
            // Rows outside have some valid element's scale: nothing of theirs is stored.
            uint8_t va[4], vb[8];
            auto load = [&](int kb) {
                const bool in = kb < tl.kb1;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    va[r] = __ldg(in && arow + 32 * r < tl.rows ? pa + kb * P.ldsA + 32 * r : P.sA);
                if (wgrad) {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        vb[r] = __ldg(in && tl.n0 + lane + 32 * r < P.N ? pb + kb * P.sB_k + 32 * r : P.sB);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        vb[h] = __ldg(in && tl.n0 + 128 * h < P.N ? pb + kb * P.sB_k + h * P.sB_n : P.sB);
                }
            };
            load(tl.kb0 + j);
            for (int kb0 = tl.kb0; kb0 < tl.kb1; kb0 += kSlotBlocks, ++groups) {
                // This slot's exponents, then the loads for the next one.
                uint32_t ea[4], eb[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) ea[r] = va[r];
#pragma unroll
                for (int r = 0; r < 8; ++r) eb[r] = wgrad ? vb[r] : vb[r >> 2];
                load(kb0 + kSlotBlocks + j);
                const int slot = groups % kScaleSlots;
                if (!__all_sync(0xffffffffu, mbar_wait(sempty0 + 8 * slot, ((groups / kScaleSlots) & 1) ^ 1, err))) {
                    ok = false;
                    break;
                }
                const uint32_t at = ring + slot * kSlotBytes + 16 * lane + j;
#pragma unroll
                for (int r = 0; r < 4; ++r) st_shared_u8(at + 4 * r, ea[r]);
#pragma unroll
                for (int r = 0; r < 8; ++r) st_shared_u8(at + 512 + 128 * (r & ~3) + 4 * (r & 3), eb[r]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // tcgen05.cp reads through the async proxy
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1)
                        mbar_arrive(sfull0 + 8 * slot);
                    else
                        mbar_arrive_cluster(sfull_lead + 8 * slot);
                }
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // -------------------------------------------------------- scheduler
        if (lane == 0) {
            Walk w;
            w.G = G;
            w.M = P.M;
            w.ntn = (P.N + BN - 1) / BN;
            w.mtn = wgrad ? (P.M + TM - 1) / TM : 0;
            w.split = P.split;
            w.wgrad = wgrad;
            w.total_kb = wgrad ? 0 : (P.K + BK - 1) / BK;
            w.gr = gr;
            const int total = wgrad ? G * w.mtn * w.ntn : gr->pre[G + 1] * w.ntn * P.split;
            int t = static_cast<int>(blockIdx.x) / CG;
            for (int i = 0;; ++i, t += static_cast<int>(gridDim.x) / CG) {
                Tile tl{};
                tl.g = -1;
                if (t < total) tl = decode<CG>(w, t);
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
    } else if (warp >= kEpiWarp0) {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may read
        const int ew = warp - kEpiWarp0;
        const int half = ew >> 2;  // columns 128 half .. + 127 of the tile
        const uint32_t stage = smem_u32(staging + ew * Cfg<CG>::STORE_BYTES);
        const uint32_t acce_lead = CG == 2 ? map_to_rank(acce0, 0) : acce0;
        const uint32_t overlap_lead = CG == 2 ? map_to_rank(overlap_bar, 0) : overlap_bar;
        auto hand_back = [&](uint32_t bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 1)
                    mbar_arrive(bar);
                else
                    mbar_arrive_relaxed(bar);
            }
        };
        int it = 0;         // segments read; the accumulator is it & 1
        bool ok = true;
        Tile tl;
        for (int i = 0; ok && take(i, tl, true); ++i) {
            const int col = tl.n0 + kCols * half;
            const int row = tl.m0 + BM * rank + 32 * q;
            // Rows of this warp inside the group (of D) and columns inside D.
            const int rows = tl.rows - row, ncol = P.N - col;
            const bool live = rows > 0 && ncol > 0;
            const bool split = ES == 4 && P.split > 1;
            const long long row0 = static_cast<long long>(tl.row0) + row;
            const long long ldd = split ? P.N : P.ldd;
            uint8_t* d = split ? reinterpret_cast<uint8_t*>(P.partial + (static_cast<long long>(tl.split) * P.rows + row0) * P.N + col)
                               : static_cast<uint8_t*>(P.D) + ((wgrad ? tl.g * P.strideD : 0LL) + row0 * P.ldd + col) * ES;
            const bool aligned = split ? P.N % 4 == 0
                                       : ((reinterpret_cast<uintptr_t>(P.D) | static_cast<uintptr_t>(P.ldd * ES) |
                                           static_cast<uintptr_t>(P.strideD * ES)) & 15) == 0;
            int kb = tl.kb0;
            // Rows leave by bulk stores, which the map clips at D's end. Where a
            // group ends inside the 32 rows, the next one's follow, and the
            // warp stores the rows itself; so it does without 16-byte rows.
            const bool bulk = P.bulk_store && live && (rows >= 32 || wgrad || !P.offsets);
            do {  // segments; once, with zeros, for a group without rows to sum over
                const bool filled = kb < tl.kb1;
                const int buf = it & 1;
                const uint32_t acc = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * kAcc1 + kCols * half;
                if (filled) {
                    if (!__all_sync(0xffffffffu, mbar_wait(accf0 + 8 * buf, (it >> 1) & 1, err))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                // The chunk in the overlap comes first: accumulator 0's last
                // columns (the second half's warps), accumulator 1's first.
                const bool mine = half == (buf == 0);
                const bool add = ES == 4 && kb > tl.kb0;
                bool fresh = true;  // nothing of this segment has been stored
                // Chunks of 32 columns, each staged and stored in kRounds
                // pieces, or kJoin chunks in one.
                constexpr int ROW = Cfg<CG>::STORE_ROW;
                constexpr int kRounds = 32 * ES > ROW ? 32 * ES / ROW : 1, kJoin = ROW > 32 * ES ? ROW / (32 * ES) : 1;
#pragma unroll 1
                for (int n = 0; n < kCols / 32; ++n) {
                    const int p = buf == 0 ? kCols / 32 - 1 - n : n;
                    uint32_t x[32];
                    if (filled && live) {
                        tmem_ld_32x32b_x32(acc + 32 * p, x);
                        tmem_ld_wait_for(x);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = 0;
                    }
                    if (filled) {
                        if (n == 0 && mine) hand_back(overlap_lead);
                        if (n == kCols / 32 - 1) hand_back(acce_lead + 8 * buf);
                    }
                    if constexpr (ES == 2) {
                        if (live && tl.kb1 - tl.kb0 > segment) {
                            // A lane's sums are 32 words apart, a warp's neighbouring.
                            float* sums = P.carry + (static_cast<size_t>(blockIdx.x) * kEpiWarps + ew) * (32 * kCols) +
                                          1024 * p + lane;
                            if (kb > tl.kb0) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) x[j] = add_bits(__float_as_uint(sums[32 * j]), x[j]);
                            }
                            if (tl.kb1 - kb > segment) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) sums[32 * j] = __uint_as_float(x[j]);
                                continue;
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < kRounds; ++h) {
                        const int c0 = 32 * (kJoin == 2 ? p & ~1 : p) + h * (ROW / ES);
                        if (!live || c0 >= ncol) continue;
                        if (kJoin == 1 || n % 2 == 0) {
                            // The last bulk store has read the buffer. Before a
                            // segment is added, the stores it adds to are complete.
                            if (lane == 0) {
                                if (add && fresh)
                                    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                                else
                                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                            }
                            fresh = false;
                            __syncwarp();
                        }
                        constexpr int PIECES = ROW / 16 / kJoin;
#pragma unroll
                        for (int k = 0; k < PIECES; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (ES == 2)
                                    w[i] = pack_pair<T>(__uint_as_float(x[8 * k + 2 * i]), __uint_as_float(x[8 * k + 2 * i + 1]));
                                else
                                    w[i] = x[4 * PIECES * h + 4 * k + i];
                            }
                            st_shared_v4(stage + stage_piece<ROW>(lane, k + (kJoin == 2 ? PIECES * (p & 1) : 0)), w[0], w[1],
                                         w[2], w[3]);
                        }
                        if (kJoin == 2 && n % 2 == 0) continue;
                        if (bulk) {
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0)
                                bulk_store(&P.mapD, stage, col + c0, static_cast<int>(row0), split ? tl.split : wgrad ? tl.g : 0, add);
                        } else {
                            __syncwarp();
                            store_rows<ES, ROW>(stage, d + c0 * ES, ldd, rows, ncol - c0, aligned, add, lane);
                        }
                    }
                }
                it += filled;
                kb = segment < tl.kb1 - kb ? kb + segment : tl.kb1;
            } while (kb < tl.kb1);
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the stores are complete
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

// out[r][n] = sum over the splits, in order, of partial[split][r][n]; a thread
// sums V neighbouring columns of one row.
template <typename T, int V>
__global__ void __launch_bounds__(128) fp8_reduce_kernel(const float* partial, int split, int rows, int N, T* out,
                                                         long long ldd) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = (static_cast<int>(blockIdx.x) * 128 + static_cast<int>(threadIdx.x)) * V;
    if (n >= N) return;
    const long long step = static_cast<long long>(rows) * N;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        const float* p = partial + static_cast<long long>(r) * N + n;
        float s[V] = {};
#pragma unroll 8
        for (int k = 0; k < split; ++k) {
            if constexpr (V == 4) {
                const float4 f = *reinterpret_cast<const float4*>(p + k * step);
                s[0] += f.x, s[1] += f.y, s[2] += f.z, s[3] += f.w;
            } else {
                s[0] += p[k * step];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) out[r * ldd + n + i] = from_f32<T>(s[i]);
    }
}

constexpr int kMaxDevices = 64;

template <int CG, typename T, bool wgrad>
int launch_variant(const Fp8GemmJob& job, long long max_tiles, int num_sms, cudaStream_t s) {
    // Per device: the shared-memory opt-in, and the clusters that fit at once
    // (tiles go to them with a static stride).
    static int clusters[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const auto kernel = fp8_gemm_kernel<CG, T, wgrad>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<CG>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    if (clusters[dev] == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<CG>());
        if (e != cudaSuccess) return e;
        int n = 0;
        if (CG > 1) {
            cfg.attrs = attr + 1;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(static_cast<unsigned>(std::max(num_sms / CG, 1) * CG));
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) cudaGetLastError();
            cfg.attrs = attr;
        }
        clusters[dev] = n > 0 ? n : std::max(num_sms / CG, 1);
    }
    const int fit = std::max(1, std::min(clusters[dev], num_sms / CG));
    cfg.gridDim = dim3(static_cast<unsigned>(CG * std::min<long long>(fit, max_tiles)));
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, job);
}

}  // namespace

int fp8_gemm_split(int rows, int N, int K, int num_sms) {
    // Fewer tiles than SMs: the contraction is split where that pays. Measured: a
    // k block takes 0.33 us (four stages in flight at the latency of L2), the
    // second kernel 3 us, and its fp32 partial sums, written and read, 8 bytes
    // per result and split at 7.5 TB/s. (1024 x 768 x 4096, 24 tiles: 17.1 us
    // whole, 15.6 in six parts; 48 x 4096 x 14336, 16 tiles, in nine: 16.4 us.)
    const long long tiles = static_cast<long long>((rows + BM - 1) / BM) * ((N + BN - 1) / BN);
    const int kb = (K + BK - 1) / BK;
    const int most = static_cast<int>(std::min<long long>(num_sms / tiles, kb / 4));  // the pipeline fills with four
    int best = 1;
    double least = 0.33 * kb;
    for (int s = 2; s <= most; ++s) {
        const double us = 0.33 * ((kb + s - 1) / s) + 3.0 + s * (8.0 / 7.5e6) * rows * N;
        if (us < least) {
            least = us;
            best = s;
        }
    }
    return best;
}

int fp8_gemm_cg(int M, int N, bool grouped, bool forward, int out_dtype, int num_sms) {
    // A pair loads and reads from shared memory 32 KB per k block and SM where a
    // single CTA takes 48 KB, has larger output stores and a stage more; a single
    // CTA's loads come from one place and its epilogue hands back to itself.
    // Measured, pairs against singles: forward, 16-bit results, 8192 x 14336 x
    // 4096 298 and 310 us, 16384 x 8192 x 8192 683 and 689, 8192 x 4096 x 4096 95
    // and 91, 8192 x 2048 x 8192 115 and 108; data and weight gradient of the
    // first 338 and 347, 323 and 337; fp32 results of 8192 x 4096 x 14336 386 and
    // 421, its weight gradient 392 and 426.
    // Pairs need enough tiles for all of them (1021 x 712 x 4093: 15, 11, 17
    // against 13, 11, 16), and their 256 rows waste more of ragged groups (256
    // experts of 512 x 2048, 65536 rows: 94, 112, 160 against 85, 97, 126).
    const long long tiles = static_cast<long long>((M + 255) / 256) * ((N + BN - 1) / BN);
    if (grouped || tiles < num_sms / 2) return 1;
    return out_dtype == GNS_FP32 || (forward && N >= 8192) ? 2 : 1;
}

int launch_fp8_gemm(const Fp8GemmJob& job, int cg, int num_sms, cudaStream_t s) {
    const int tile = BM * cg;
    const long long tn = (job.N + BN - 1) / BN;
    long long tm;  // tile rows, an upper bound where the groups are on the device
    if (job.wgrad)
        tm = static_cast<long long>(job.G) * ((job.M + tile - 1) / tile);
    else if (job.offsets)
        tm = (job.rows + static_cast<long long>(tile - 1) * (std::min(job.rows, job.G) + 1)) / tile;
    else
        tm = (job.rows + tile - 1) / tile;
    const long long tiles = tm * tn * job.split;
    if (tiles <= 0) return cudaSuccess;
    if (!job.carry && fp8_carry_bytes(job.wgrad ? job.rows : job.K, job.out_dtype, job.split, num_sms))
        return cudaErrorInvalidValue;
    return by_dtype(job.split > 1 ? static_cast<int>(GNS_FP32) : job.out_dtype, [&](auto t) {
        using T = decltype(t);
        if (job.wgrad) {
            if constexpr (sizeof(T) == 4)
                if (cg == 2) return launch_variant<2, T, true>(job, tiles, num_sms, s);
            return launch_variant<1, T, true>(job, tiles, num_sms, s);
        }
        return cg == 2 ? launch_variant<2, T, false>(job, tiles, num_sms, s) : launch_variant<1, T, false>(job, tiles, num_sms, s);
    });
}

int launch_fp8_reduce(const Fp8GemmJob& job, cudaStream_t s) {
    const int v = job.N % 4 == 0 ? 4 : 1;
    const dim3 grid((job.N + 128 * v - 1) / (128 * v), std::min(job.rows, 65535));
    return by_dtype(job.out_dtype, [&](auto t) {
        using T = decltype(t);
        return static_cast<int>(launch_after(v == 4 ? fp8_reduce_kernel<T, 4> : fp8_reduce_kernel<T, 1>, grid, dim3(128), 0, s,
                                             static_cast<const float*>(job.partial), job.split, job.rows, job.N,
                                             static_cast<T*>(job.D), job.ldd));
    });
}

}  // namespace gns
