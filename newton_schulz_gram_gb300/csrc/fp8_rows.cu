// The block-scaled 8-bit linear layer for few rows (a decode step), in
// one launch: D[r][n] = x_r . w[g(r)][n] with x cast to 8 bits on the way.
//
// Bound: HBM, the weights once, N K bytes per group that has rows. Two blocks
// of threads per SM (one where shared memory has no room for two) cast their
// group's rows of x once and then walk strips of 16 weight rows; the sixteen
// warps split the contraction (k block b belongs to warp b mod 16). Each warp streams its own pieces of the weights, across
// strips, through a ring of cp.async slots that only its own lanes read back,
// so nothing but the sum over the warps at the end of a strip synchronizes, and
// 128 KB per SM are in flight all the time. The products run as mma.sync
// m16n8k16 with the rows of x as the 8 columns: 8-bit values are exact in fp16
// and so are their fp32 products, x is kept in shared memory as the fp16 form
// of its 8-bit values, and a lane's 16-byte loads of two weight rows convert to
// A fragments as they are, because the order of k within a block is free as
// long as x uses the same one. Tensor throughput does not matter at 8 columns;
// tcgen05 would add TMEM and descriptors to a kernel that lives for a few
// microseconds. The warps' sums are joined in a fixed order.
// One row, 14336 x 4096: 15.2 us (3.9 TB/s; 28672 x 8192 46.7, 5.0); without
// conversions and products, the loads alone, 11.9. Eight rows, whose fp16 forms
// leave room for one block of threads per SM: 20.2. The 8-bit mma.sync took
// 19.4 us for one row, a block of threads per strip without the ring 15.6, and
// more of them, of eight warps, 17.0.
#include <algorithm>

#include "blockops.cuh"
#include "fp8.cuh"
#include "fp8_convert.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStrip = 16;               // weight rows
constexpr int kSlotBytes = 4 * 32 * 16;  // a warp's k block: four 16-byte pieces per lane
// Dynamic shared memory of a block: the limit, and what lets two share an SM
// (228 KB, of which each takes 1 KB and the 18.1 KB of its static arrays).
constexpr size_t kMaxSmem = 200 * 1024;
constexpr size_t kSmemOfTwo = 94 * 1024;

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four 8-bit values of a word as two pairs of fp16.
template <bool E5M2>
__device__ __forceinline__ uint2 to_half4(uint32_t four) {
    uint2 r;
    if constexpr (E5M2)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, lo;\n\tcvt.rn.f16x2.e5m2x2 %1, hi;\n\t}"
            : "=r"(r.x), "=r"(r.y)
            : "r"(four));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(r.x), "=r"(r.y)
            : "r"(four));
    return r;
}

// Sixteen k of two weight rows (lo, hi) and of x (b, sixteen fp16).
template <bool E5M2>
__device__ __forceinline__ void product(float (&c)[4], const uint4& lo, const uint4& hi, const uint4 (&b)[2]) {
    const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
    const uint32_t x[8] = {b[0].x, b[0].y, b[0].z, b[0].w, b[1].x, b[1].y, b[1].z, b[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint2 p = to_half4<E5M2>(l[i]), q = to_half4<E5M2>(h[i]);
        mma_16816(c, p.x, q.x, p.y, q.y, x[2 * i], x[2 * i + 1]);
    }
}

// acc + part 2^(a + b - 254) for two 8-bit exponents a, b, given as (a + b) << 22:
// half of it in each of two factors, since the whole may be no fp32 number where
// the result is (a block whose scale is 2^100 may meet nothing but zeros). `nan`
// is a NaN's bits where an exponent is the one that stands for NaN.
__device__ __forceinline__ float scaled(float part, uint32_t exps, uint32_t nan, float acc) {
    const float lo = __uint_as_float((exps & 0x7F800000u) | nan);
    const float hi = __uint_as_float((exps + 0x400000u) & 0x7F800000u);
    return fmaf(part * lo, hi, acc);
}

// 16 bytes to shared memory, zeros where `in` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// The bytes of a 16-byte piece that lie inside the row (left of them).
__device__ __forceinline__ uint4 clip(uint4 v, int left) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        if (n < 4) w[i] = n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1);
    }
    return v;
}

// 8 values of a row of x from column k (K columns in all) as fp32.
template <typename T>
__device__ __forceinline__ void load_x(const T* row, int k, int K, bool vec, float (&v)[8]) {
    if (vec && k + 8 <= K) {
        Pack<T, 8> p;
        p.load(row + k);
        p.get(v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < K ? to_f32<T>(row[k + i]) : 0.0f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) fp8_rows_kernel(Fp8RowsJob j, bool vec, int slots, int chunk) {
    // [kWarps][slots] ring slots, then x in fp16: [rows + 1][K rounded up to 128, + 8], the last row zero, then its
    // scales [rows][k blocks].
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sums[2][kWarps][kStrip][kFp8FewRows + 1];
    __shared__ int found[3];  // group, its first row, its row count
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int g = 0, r0 = 0, count = j.rows;
    if (j.offsets) {
        // Row blockIdx.y stands for `chunk` rows of its group if it is the first of them.
        const int r = blockIdx.y;
        if (threadIdx.x == 0) found[0] = -1;
        __syncthreads();
        for (int i = threadIdx.x; i < j.G; i += kThreads) {
            const int beg = j.offsets[i], end = j.offsets[i + 1];
            if (beg <= r && r < end) {
                found[0] = i;
                found[1] = beg;
                found[2] = end - beg;
            }
        }
        __syncthreads();
        g = found[0];
        r0 = found[1];
        count = found[2];
        if (g < 0) {  // a row of no group: zero
            for (int n = blockIdx.x * kThreads + threadIdx.x; n < j.N; n += gridDim.x * kThreads)
                by_dtype_device(j.out_dtype, [&](auto t) {
                    using O = decltype(t);
                    static_cast<O*>(j.D)[static_cast<long long>(r) * j.ldd + n] = from_f32<O>(0.0f);
                });
            return;
        }
        if ((r - r0) % chunk != 0) return;
        count = min(count - (r - r0), chunk);
        r0 = r;
    }
    const int gq = lane >> 2, t = lane & 3;
    const uint8_t* wg = j.w + g * j.stride_w;
    const int nkb = (j.K + kFp8Block - 1) / kFp8Block;
    const uint8_t* sw = j.sw + static_cast<long long>(g) * ((j.N + kFp8Block - 1) / kFp8Block) * nkb;
    const int strips = (j.N + kStrip - 1) / kStrip;
    const int per_strip = (nkb - warp + kWarps - 1) / kWarps;  // k blocks of this warp (0 when there are fewer than warps)
    const int my_strips = (strips - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int total = my_strips * per_strip;
    const uint32_t ring = smem_u32(smem) + (warp * slots) * kSlotBytes + lane * 16;

    // The next k block of the walk into its slot; one group per call, empty
    // past the end, so that the wait below counts alike everywhere.
    int strip_at = blockIdx.x, kb_at = warp, slot_at = 0, issued = 0;
    const uint8_t* src = nullptr;   // this lane's first piece of row gq
    bool in0 = false, in1 = false;  // rows gq and gq + 8 of the strip exist
    auto enter_strip = [&]() {
        const int n = strip_at * kStrip + gq;
        in0 = n < j.N;
        in1 = n + 8 < j.N;
        src = wg + static_cast<long long>(n) * j.ldw + warp * kFp8Block + 16 * t;
        kb_at = warp;
    };
    enter_strip();
    auto issue = [&]() {
        if (issued < total) {
            const uint32_t dst = ring + slot_at * kSlotBytes;
            const int left = j.K - (kb_at * kFp8Block + 16 * t);  // columns from this lane's first piece on
            const uint8_t* row8 = src + 8 * j.ldw;
            copy16(dst, in0 && left > 0 ? src : wg, in0 && left > 0);
            copy16(dst + 512, in0 && left > 64 ? src + 64 : wg, in0 && left > 64);
            copy16(dst + 1024, in1 && left > 0 ? row8 : wg, in1 && left > 0);
            copy16(dst + 1536, in1 && left > 64 ? row8 + 64 : wg, in1 && left > 64);
            ++issued;
            kb_at += kWarps;
            src += kWarps * kFp8Block;
            if (kb_at >= nkb) {
                strip_at += gridDim.x;
                enter_strip();
            }
            if (++slot_at == slots) slot_at = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < slots; ++i) issue();

    // x to 8 bits: sixteen threads per block of 128.
    const int stride = nkb * kFp8Block + 8;
    __half* xq = reinterpret_cast<__half*>(smem + kWarps * slots * kSlotBytes);
    uint32_t* xs = reinterpret_cast<uint32_t*>(xq + (count + 1) * stride);  // exponents, as `scaled` wants them
    for (int i = threadIdx.x; i < stride / 8; i += kThreads)
        *reinterpret_cast<uint4*>(xq + count * stride + 8 * i) = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x >> 4; i < count * nkb; i += kThreads / 16) {
        const int r = i / nkb, b = i - r * nkb, l = threadIdx.x & 15;
        const int row = j.slots ? j.slots[r0 + r] / j.topk : r0 + r;
        float v[8];
        load_x(static_cast<const T*>(j.x) + row * j.ldx, b * kFp8Block + 8 * l, j.K, vec, v);
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(v[e]));
        const unsigned half = 0xFFFFu << (lane & 16);
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, m));
        const uint32_t e = scale_exponent(amax, 8);
        const float inv = exp_inverse(e);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = no_infinity(v[c]) * inv;
        const uint32_t w[2] = {cast_quad<false>(v[0], v[1], v[2], v[3]), cast_quad<false>(v[4], v[5], v[6], v[7])};
        const uint2 lo = to_half4<false>(w[0]), hi = to_half4<false>(w[1]);
        *reinterpret_cast<uint4*>(xq + r * stride + b * kFp8Block + 8 * l) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        if (l == 0) xs[r * nkb + b] = e << 22;
    }
    __syncthreads();

    const __half* xrow = xq + (gq < count ? gq : count) * stride + 16 * t;
    int slot = 0, buf = 0;
    // The weights' exponent of the walk's next k block, loaded a block ahead.
    uint32_t scale = 0;
    if (warp < nkb && static_cast<int>(blockIdx.x) < strips) scale = __ldg(sw + blockIdx.x * kStrip / kFp8Block * nkb + warp);
    for (int strip = blockIdx.x; strip < strips; strip += gridDim.x, buf ^= 1) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int b = warp; b < nkb; b += kWarps) {
            const uint32_t wexp = scale << 22, nan = scale == 255 ? 0x7FC00000u : 0u;
            {
                int next = b + kWarps, at = strip;
                if (next >= nkb) next = warp, at += gridDim.x;
                if (at < strips) scale = __ldg(sw + at * kStrip / kFp8Block * nkb + next);
            }
            // All but the slots - 1 youngest groups have landed: this block's among them.
            if (slots == 1)
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            const uint32_t at = ring + slot * kSlotBytes;
            uint4 a[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < 2; ++c) a[h][c] = ld_shared_v4(at + (2 * h + c) * 512);
            if (++slot == slots) slot = 0;
            const int k = b * kFp8Block + 16 * t;
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (k + 64 * c + 16 > j.K) {
                    a[0][c] = clip(a[0][c], j.K - k - 64 * c);
                    a[1][c] = clip(a[1][c], j.K - k - 64 * c);
                }
                const uint4* xp = reinterpret_cast<const uint4*>(xrow + b * kFp8Block + 64 * c);
                const uint4 x[2] = {xp[0], xp[1]};
                if (j.fmt_w == GNS_E5M2)
                    product<true>(part, a[0][c], a[1][c], x);
                else
                    product<false>(part, a[0][c], a[1][c], x);
            }
            issue();  // into the slot just read: a lane meets only its own pieces
            const uint32_t s0 = wexp + (2 * t < count ? xs[2 * t * nkb + b] : 0);
            const uint32_t s1 = wexp + (2 * t + 1 < count ? xs[(2 * t + 1) * nkb + b] : 0);
            acc[0] = scaled(part[0], s0, nan, acc[0]);
            acc[1] = scaled(part[1], s1, nan, acc[1]);
            acc[2] = scaled(part[2], s0, nan, acc[2]);
            acc[3] = scaled(part[3], s1, nan, acc[3]);
        }
        sums[buf][warp][gq][2 * t] = acc[0];
        sums[buf][warp][gq][2 * t + 1] = acc[1];
        sums[buf][warp][8 + gq][2 * t] = acc[2];
        sums[buf][warp][8 + gq][2 * t + 1] = acc[3];
        __syncthreads();  // one per strip: the other buffer's readers are a barrier behind
        const int r = threadIdx.x / kStrip, c = threadIdx.x % kStrip, n = strip * kStrip + c;
        if (r < count && n < j.N) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += sums[buf][k][c][r];
            by_dtype_device(j.out_dtype, [&](auto o) {
                using O = decltype(o);
                static_cast<O*>(j.D)[static_cast<long long>(r0 + r) * j.ldd + n] = from_f32<O>(v);
            });
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

static_assert(kThreads / kStrip >= kFp8FewRows, "a thread per result");

size_t rows_smem(int rows, int K, int slots) {
    const size_t nkb = (static_cast<size_t>(K) + kFp8Block - 1) / kFp8Block;
    return static_cast<size_t>(kWarps) * slots * kSlotBytes + (rows + 1) * (nkb * kFp8Block + 8) * 2 + rows * nkb * 4;
}

// Rows of one group that a block of threads takes: as many as let two blocks
// share an SM with two slots each (most groups of few rows have one or two).
int rows_of_chunk(int rows, int K) {
    int chunk = std::min(rows, kFp8FewRows);
    while (chunk > 1 && rows_smem(chunk, K, 2) > kSmemOfTwo) --chunk;
    return chunk;
}

}  // namespace

bool fp8_rows_fit(int rows, int N, int K, int groups, bool grouped, int num_sms) {
    if (!grouped) return rows <= kFp8FewRows && rows_smem(rows, K, 2) <= kMaxSmem;
    if (rows > kFp8FewRouted || rows_smem(1, K, 1) > kSmemOfTwo) return false;
    // This kernel starts at once but streams the weights of one group per row at
    // 2 to 5 TB/s (least where the warps are more than the k blocks, most where a
    // block walks over several strips); the tensor cores' kernel takes the cast
    // before it and a tile's k blocks one after another, and then streams
    // faster. Measured, us, this and that, weights from HBM: 256 experts of 512 x
    // 2048, 8 rows 5.7 and 13.4, 16 rows 10.1 and 14.3, 32 rows 15.3 and 15.2; of
    // 2048 x 512, 8 rows 8.7 and 9.7, 16 rows 11.7 and 10.2, 32 rows 17.1 and 14.0;
    // 16 of 4096 x 4096, 1 row 8.1 and 18.1, 4 rows 22.3 and 22.4; 8 of 14336 x
    // 4096, 2 rows 30.4 and 29.2, 8 rows 76.5 and 54.8. How many experts have rows
    // is on the device: the rule takes one per row.
    const int strips = (N + kStrip - 1) / kStrip, nkb = (K + kFp8Block - 1) / kFp8Block;
    const int parts = std::min(rows, groups + (rows - 1) / rows_of_chunk(rows, K));
    const double megabytes = 1e-6 * parts * N * K;
    return 3 + megabytes * (nkb < kWarps ? 0.5 : strips < 2 * num_sms ? 0.35 : 0.2) <= 8 + 0.3 * nkb;
}

int launch_fp8_rows(const Fp8RowsJob& j, int num_sms, cudaStream_t s) {
    const int strips = (j.N + kStrip - 1) / kStrip, nkb = (j.K + kFp8Block - 1) / kFp8Block;
    const int chunk = j.offsets ? rows_of_chunk(j.rows, j.K) : j.rows;
    // Two blocks per SM where two fit, whose products hide each other's waits
    // (one row of 14336 x 4096: 15.2 us, one block per SM 16.6), with two slots if
    // there is room and the walk is that long, else one. With groups, whose
    // number that have rows is on the device, enough blocks for two rounds if
    // all rows are of different groups.
    const bool two = rows_smem(chunk, j.K, 1) <= kSmemOfTwo;
    const int blocks = j.offsets ? std::min(strips, std::max(1, 4 * num_sms / j.rows)) : std::min(strips, (two ? 2 : 1) * num_sms);
    int slots = 1;
    if ((nkb + kWarps - 1) / kWarps * ((strips + blocks - 1) / blocks) > 1 &&
        rows_smem(chunk, j.K, 2) <= (two ? kSmemOfTwo : kMaxSmem))
        slots = 2;
    const size_t smem = rows_smem(chunk, j.K, slots);
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        const bool vec = (reinterpret_cast<uintptr_t>(j.x) & 15) == 0 && j.ldx * static_cast<int>(sizeof(T)) % 16 == 0;
        static bool configured[64];  // the shared-memory opt-in is per device
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
        if (e == cudaSuccess && !configured[dev]) {
            e = cudaFuncSetAttribute(fp8_rows_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(kMaxSmem));
            configured[dev] = e == cudaSuccess;
        }
        if (e != cudaSuccess) return static_cast<int>(e);
        return static_cast<int>(launch_after(fp8_rows_kernel<T>, dim3(blocks, j.offsets ? j.rows : 1), dim3(kThreads), smem,
                                             s, j, vec, slots, chunk));
    });
}

}  // namespace gns
