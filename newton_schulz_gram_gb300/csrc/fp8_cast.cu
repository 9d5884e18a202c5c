// Casts to 8-bit floating point with a power-of-two scale for each block of
// 128 values: along a row (the contraction of the forward and data-gradient
// products), along a column (that of the weight gradient), or 128 x 128 of a
// weight matrix.
//
//   s = the smallest power of two with amax / s <= 1.75 * 2^e  (448 = 1.75 * 2^8
//       for e4m3, 57344 = 1.75 * 2^15 for e5m2), at least 2^-126,
//   q = x / s rounded to nearest even; s is kept as its 8-bit exponent.
//
// The scale is a power of two so that x / s and s q are exact: the only
// rounding is the one to 8 bits, and a value's 8-bit form does not depend on
// how the scale was applied. amax is taken over the finite values; NaN and
// infinities become NaN and leave their block's other values alone.
//
// One block of threads holds a 128 x 128 tile in registers, so the row and the
// column form (and the gather of a token's row to its places) come from one
// read of x. Bound: HBM, 2 bytes read and 1 (2 for both forms) written per
// value of 16 bits: 8192 x 14336 in both forms 69 us (6.8 TB/s), weights of 256 x
// 512 x 2048 116 (6.9). Gathered rows come from L2, and there instruction issue
// bounds: 8192 tokens of 2048 to 65536 sorted rows, both forms, 87 us (3.5 TB/s).
// fp32 values go one by one: 8192 x 8192 in both forms 77 us, the row form 60, as
// weights 62 (5.2, 5.6 and 5.4 TB/s).
#include <algorithm>
#include <initializer_list>

#include "blockops.cuh"
#include "fp8.cuh"
#include "fp8_convert.cuh"
#include "ptx.cuh"

namespace gns {
namespace {

constexpr int kThreads = 256;
constexpr int kPasses = 8;   // 16 rows each; a thread owns 8 columns of one row per pass
constexpr int kWarps = kThreads / 32;

enum CastMode { kRowForm = 1, kColForm = 2, kBothForms = 3, kBlockForm = 4 };

template <bool E5M2>
__device__ __forceinline__ uint2 cast8(const float (&v)[8], const float (&inv)[8]) {
    return make_uint2(cast_quad<E5M2>(v[0] * inv[0], v[1] * inv[1], v[2] * inv[2], v[3] * inv[3]),
                      cast_quad<E5M2>(v[4] * inv[4], v[5] * inv[5], v[6] * inv[6], v[7] * inv[7]));
}

// One tile: rows r0 .. r0 + nrows - 1 of the matrix (their rows of x from
// `source` if there is one), columns c0 .. c0 + 127.
struct Tile {
    int r0, nrows, c0;
    long long qc_row;  // first row of the tile in the column form
    int sc_row;        // its row of column scales
};

// Whether column c (a multiple of 8) of an 8-bit row is written: those up to the
// next multiple of 16 are, what lies beyond in a larger row stride is the caller's.
__device__ __forceinline__ bool written(int c, int cols) { return (c & ~15) < cols; }

// Two 16-bit values at a time. max_abs has the larger magnitudes (and signs of
// no meaning); it passes over a NaN and shows an infinity, whose block then
// takes the finite maximum the slow way. scaled is a pair times a power of two
// as two floats: exact, except that a bf16 product too small to be a normal
// number may lose bits, hundreds of binades below the smallest 8-bit value.
// fp16 has no room for the inverse scales and is multiplied in fp32.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7F80u;
    static __device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    using Scale = uint32_t;  // of both values
    static __device__ __forceinline__ Scale scale(float lo, float hi) {
        return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    }
    static __device__ __forceinline__ float2 scaled(uint32_t w, Scale s) {
        uint32_t r;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(s));
        return make_float2(lo(r), hi(r));
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
};
template <>
struct Pair<__half> {
    static constexpr uint32_t kInf = 0x7C00u;
    static __device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    using Scale = float2;
    static __device__ __forceinline__ Scale scale(float lo, float hi) { return make_float2(lo, hi); }
    static __device__ __forceinline__ float2 scaled(uint32_t w, Scale s) {
        return make_float2(lo(w) * s.x, hi(w) * s.y);
    }
    static __device__ __forceinline__ float lo(uint32_t w) {
        return __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
    }
    static __device__ __forceinline__ float hi(uint32_t w) {
        return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
    }
};

__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & 0x7FFF7FFFu; }

// Maxima that are no finite value (of nothing but NaN) as zero.
template <typename T>
__device__ __forceinline__ uint32_t finite_maxima(uint32_t m) {
    return ((m & 0xFFFFu) < Pair<T>::kInf ? m & 0xFFFFu : 0u) | ((m >> 16) < Pair<T>::kInf ? m & 0xFFFF0000u : 0u);
}

// Infinities become NaN: the maximum then passes over them, and the conversion,
// which would saturate them, keeps them.
template <typename T>
__device__ __forceinline__ void nan_for_infinity(uint4& p) {
    for (uint32_t* w : {&p.x, &p.y, &p.z, &p.w}) {
        const uint32_t m = magnitudes(*w);
        *w |= ((m & 0xFFFFu) == Pair<T>::kInf ? 0x7FFFu : 0u) | ((m >> 16) == Pair<T>::kInf ? 0x7FFF0000u : 0u);
    }
}

// An infinity, or NaN alone, among the values behind these maxima.
template <typename T>
__device__ __forceinline__ bool has_infinity(uint32_t maxima) {
    return (maxima & 0xFFFFu) >= Pair<T>::kInf || (maxima >> 16) >= Pair<T>::kInf;
}

// Eight values (four words) with their inverse scales to 8 bits.
template <typename T, bool E5M2>
__device__ __forceinline__ uint2 cast_words(const uint4& p, const typename Pair<T>::Scale (&inv)[4]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = Pair<T>::scaled(w[i], inv[i]);
    return make_uint2(cast_quad<E5M2>(v[0].x, v[0].y, v[1].x, v[1].y), cast_quad<E5M2>(v[2].x, v[2].y, v[3].x, v[3].y));
}

// The tile of 16-bit values: the general tile below with the maxima taken over
// packed pairs (two rows' maxima travel through the shuffles in one word) and
// the infinities out of the way. Instruction issue bounds the casts as soon as
// HBM does not: 8192 x 14336 in both forms takes 69 us here and 208 value by
// value.
template <typename T, int MODE, bool E5M2, bool FULL>
__device__ __forceinline__ void cast_tile16(const Tile& tl, const T* x, long long ldx, const int* source,
                                            int cols, bool vec, uint8_t* q_rows, long long ld_rows, uint8_t* s_rows,
                                            long long lds_rows, uint8_t* q_cols, long long ld_cols, uint8_t* s_cols,
                                            long long lds_cols, float (&part)[kWarps][128], float (&inv_col)[128]) {
    constexpr int kTop = E5M2 ? 15 : 8;
    using P2 = Pair<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = (threadIdx.x & 15) * 8;  // this thread's columns within the tile
    const int rl = threadIdx.x >> 4;        // its row within a pass
    const int c = tl.c0 + cl;
    uint4 raw[kPasses];
    const T* base = x + (source ? c : static_cast<long long>(tl.r0 + rl) * ldx + c);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int r = 16 * p + rl;
        if (!FULL) raw[p] = make_uint4(0, 0, 0, 0);
        if (FULL || (r < tl.nrows && c < cols)) {
            const T* a = source ? base + static_cast<long long>(source[r]) * ldx : base + 16LL * p * ldx;
            if (FULL || (vec && c + 8 <= cols)) {
                raw[p] = *reinterpret_cast<const uint4*>(a);
            } else {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < cols)
                        w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(a)[i]) << (16 * (i & 1));
                raw[p] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    auto word = [&](int p, int i) {
        const uint32_t w[4] = {raw[p].x, raw[p].y, raw[p].z, raw[p].w};
        return w[i];
    };
    if (MODE & kRowForm) {
        // Row maxima, passes p and p + 4 in the halves of one word.
        uint32_t m[kPasses / 2];
        auto row_maxima = [&]() {
#pragma unroll
            for (int p = 0; p < kPasses / 2; ++p) {
                const uint32_t a = P2::max_abs(P2::max_abs(word(p, 0), word(p, 1)), P2::max_abs(word(p, 2), word(p, 3)));
                const uint32_t b = P2::max_abs(P2::max_abs(word(p + 4, 0), word(p + 4, 1)),
                                               P2::max_abs(word(p + 4, 2), word(p + 4, 3)));
                m[p] = P2::max_abs(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
#pragma unroll
                for (int p = 0; p < kPasses / 2; ++p) m[p] = P2::max_abs(m[p], __shfl_xor_sync(0xffffffffu, m[p], d));
            }
#pragma unroll
            for (int p = 0; p < kPasses / 2; ++p) m[p] = magnitudes(m[p]);
        };
        row_maxima();
        bool inf = false;
#pragma unroll
        for (int p = 0; p < kPasses / 2; ++p) inf |= has_infinity<T>(m[p]);
        if (__any_sync(0xffffffffu, inf)) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) nan_for_infinity<T>(raw[p]);
            row_maxima();
#pragma unroll
            for (int p = 0; p < kPasses / 2; ++p) m[p] = finite_maxima<T>(m[p]);
        }
        uint8_t* out = q_rows + static_cast<long long>(tl.r0 + rl) * ld_rows + c;
        uint32_t bytes[2] = {0, 0};  // the passes' exponents
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const uint32_t e = scale_exponent(p < 4 ? P2::lo(m[p & 3]) : P2::hi(m[p & 3]), kTop);
            bytes[p >> 2] |= e << (8 * (p & 3));
            if (!FULL && 16 * p >= tl.nrows) continue;  // no row of this pass is there
            const typename P2::Scale s = P2::scale(exp_inverse(e), exp_inverse(e)), inv[4] = {s, s, s, s};
            if (FULL || (16 * p + rl < tl.nrows && written(c, cols)))
                *reinterpret_cast<uint2*>(out + 16LL * p * ld_rows) =
                    cast_words<T, E5M2>(raw[p], inv);
        }
        // Lane k of a row's sixteen stores the exponent of pass k.
        const int k = threadIdx.x & 15;
        if (k < kPasses && (FULL || 16 * k + rl < tl.nrows))
            s_rows[static_cast<long long>(tl.c0 / 128) * lds_rows + tl.r0 + 16 * k + rl] =
                static_cast<uint8_t>((k & 4 ? bytes[1] : bytes[0]) >> (8 * (k & 3)));
    }
    if (MODE & (kColForm | kBlockForm)) {
        uint32_t m[4];  // maxima of columns 2 i, 2 i + 1 over this thread's rows
        auto col_maxima = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = word(0, i);
#pragma unroll
                for (int p = 1; p < kPasses; ++p) m[i] = P2::max_abs(m[i], word(p, i));
                m[i] = magnitudes(m[i]);
            }
        };
        col_maxima();
        if (__syncthreads_or(has_infinity<T>(m[0]) || has_infinity<T>(m[1]) || has_infinity<T>(m[2]) ||
                             has_infinity<T>(m[3]))) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) nan_for_infinity<T>(raw[p]);
            col_maxima();
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = finite_maxima<T>(m[i]);
        }
        typename P2::Scale iv[4];
        if (MODE & kBlockForm) {  // one maximum for the tile
            uint32_t a = P2::max_abs(P2::max_abs(m[0], m[1]), P2::max_abs(m[2], m[3]));
            a = magnitudes(P2::max_abs(a, __byte_perm(a, a, 0x1032)));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) a = magnitudes(P2::max_abs(a, __shfl_xor_sync(0xffffffffu, a, d)));
            if (lane == 0) part[warp][0] = P2::lo(a);
            __syncthreads();
            float t = part[0][0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) t = fmaxf(t, part[w][0]);
            const uint32_t e = scale_exponent(t, kTop);
            if (threadIdx.x == 0) *s_cols = static_cast<uint8_t>(e);
#pragma unroll
            for (int i = 0; i < 4; ++i) iv[i] = P2::scale(exp_inverse(e), exp_inverse(e));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = magnitudes(P2::max_abs(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16)));
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                    *reinterpret_cast<float4*>(&part[warp][cl + 2 * i]) =
                        make_float4(P2::lo(m[i]), P2::hi(m[i]), P2::lo(m[i + 1]), P2::hi(m[i + 1]));
            }
            __syncthreads();
            if (threadIdx.x < 128) {
                float t = part[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) t = fmaxf(t, part[w][threadIdx.x]);
                const uint32_t e = scale_exponent(t, kTop);
                inv_col[threadIdx.x] = exp_inverse(e);
                if (FULL || tl.c0 + static_cast<int>(threadIdx.x) < cols)
                    s_cols[static_cast<long long>(tl.sc_row) * lds_cols + tl.c0 + threadIdx.x] = static_cast<uint8_t>(e);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&inv_col[cl + i]);
                iv[i / 2] = P2::scale(f.x, f.y);
                iv[i / 2 + 1] = P2::scale(f.z, f.w);
            }
        }
        uint8_t* out = q_cols + (tl.qc_row + rl) * ld_cols + c;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            // The column form is zero to the end of its last block of 128
            // rows (the rows past nrows were loaded as zero).
            if (FULL || (written(c, cols) && (!(MODE & kBlockForm) || 16 * p + rl < tl.nrows)))
                *reinterpret_cast<uint2*>(out + 16LL * p * ld_cols) =
                    !FULL && 16 * p >= tl.nrows ? make_uint2(0, 0) : cast_words<T, E5M2>(raw[p], iv);
        }
        // part is written again only after the next tile's barrier; its readers
        // of inv_col and part are past theirs by then.
    }
}

// The tile of any type, value by value.
template <typename T, int MODE, bool E5M2>
__device__ __forceinline__ void cast_tile(const Tile& tl, const T* x, long long ldx, const int* source,
                                          int cols, bool vec, uint8_t* q_rows, long long ld_rows, uint8_t* s_rows,
                                          long long lds_rows, uint8_t* q_cols, long long ld_cols, uint8_t* s_cols,
                                          long long lds_cols, float (&part)[kWarps][128], float (&inv_col)[128]) {
    constexpr int kTop = E5M2 ? 15 : 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = (threadIdx.x & 15) * 8;  // this thread's columns within the tile
    const int rl = threadIdx.x >> 4;        // its row within a pass
    const int c = tl.c0 + cl;
    Pack<T, 8> raw[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int r = 16 * p + rl;
        raw[p].clear();
        if (r < tl.nrows && c < cols) {
            const int row = tl.r0 + r;
            const T* a = x + static_cast<long long>(source ? source[r] : row) * ldx + c;
            if (vec && c + 8 <= cols) {
                raw[p].load(a);
            } else {
                T* e = reinterpret_cast<T*>(raw[p].p);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < cols) e[i] = a[i];
            }
        }
    }
    float cmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cmax[i] = 0.0f;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        float v[8];
        raw[p].get(v);
        float rmax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = finite_abs(v[i]);
            if (MODE & kRowForm) rmax = fmaxf(rmax, a);
            if (MODE & (kColForm | kBlockForm)) cmax[i] = fmaxf(cmax[i], a);
        }
        if (MODE & kRowForm) {
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) rmax = fmaxf(rmax, __shfl_xor_sync(0xffffffffu, rmax, m));
            const uint32_t e = scale_exponent(rmax, kTop);
            const float inv = exp_inverse(e);
            const int r = 16 * p + rl;
            if (r < tl.nrows) {
                if (written(c, cols)) {
                    float w[8], iv[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        w[i] = no_infinity(v[i]);
                        iv[i] = inv;
                    }
                    *reinterpret_cast<uint2*>(q_rows + static_cast<long long>(tl.r0 + r) * ld_rows + c) =
                        cast8<E5M2>(w, iv);
                }
                if (cl == 0) s_rows[static_cast<long long>(tl.c0 / 128) * lds_rows + tl.r0 + r] = static_cast<uint8_t>(e);
            }
        }
    }
    if (MODE & (kColForm | kBlockForm)) {
        if (MODE & kBlockForm) {  // one maximum for the tile
            float m = cmax[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = fmaxf(m, cmax[i]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (lane == 0) part[warp][0] = m;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cmax[i] = fmaxf(cmax[i], __shfl_xor_sync(0xffffffffu, cmax[i], 16));
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 8; i += 4)
                    *reinterpret_cast<float4*>(&part[warp][cl + i]) =
                        make_float4(cmax[i], cmax[i + 1], cmax[i + 2], cmax[i + 3]);
            }
        }
        __syncthreads();
        if (MODE & kColForm) {
            if (threadIdx.x < 128) {
                float m = part[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) m = fmaxf(m, part[w][threadIdx.x]);
                const uint32_t e = scale_exponent(m, kTop);
                inv_col[threadIdx.x] = exp_inverse(e);
                if (tl.c0 + static_cast<int>(threadIdx.x) < cols)
                    s_cols[static_cast<long long>(tl.sc_row) * lds_cols + tl.c0 + threadIdx.x] = static_cast<uint8_t>(e);
            }
            __syncthreads();
        }
        float iv[8];
        if (MODE & kBlockForm) {
            float m = part[0][0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, part[w][0]);
            const uint32_t e = scale_exponent(m, kTop);
            if (threadIdx.x == 0) *s_cols = static_cast<uint8_t>(e);
#pragma unroll
            for (int i = 0; i < 8; ++i) iv[i] = exp_inverse(e);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&inv_col[cl + i]);
                iv[i] = f.x, iv[i + 1] = f.y, iv[i + 2] = f.z, iv[i + 3] = f.w;
            }
        }
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int r = 16 * p + rl;
            // The column form is zero to the end of its last block of 128
            // rows (the rows past nrows were loaded as zero).
            if (written(c, cols) && (!(MODE & kBlockForm) || r < tl.nrows)) {
                float v[8];
                raw[p].get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = no_infinity(v[i]);
                *reinterpret_cast<uint2*>(q_cols + (tl.qc_row + r) * ld_cols + c) = cast8<E5M2>(v, iv);
            }
        }
        __syncthreads();  // part and inv_col are free for the next tile
    }
}

template <typename T, int MODE, bool E5M2, typename... Args>
__device__ __forceinline__ void cast_tile_of(const Tile& tl, const T* x, long long ldx, const int* source, int cols,
                                             bool vec, Args&&... args) {
    if constexpr (sizeof(T) == 2) {
        if (vec && tl.nrows == kFp8Block && tl.c0 + kFp8Block <= cols)  // the common case without its edge tests
            cast_tile16<T, MODE, E5M2, true>(tl, x, ldx, source, cols, vec, args...);
        else
            cast_tile16<T, MODE, E5M2, false>(tl, x, ldx, source, cols, vec, args...);
    } else {
        cast_tile<T, MODE, E5M2>(tl, x, ldx, source, cols, vec, args...);
    }
}

// blockIdx.y: token block, after those of earlier launches (j.block0; the column
// form's pointers are this launch's); blockIdx.x: the first of the `span` column blocks.
template <typename T, int MODE, bool E5M2>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) fp8_cast_kernel(CastJob j, bool vec, int span) {
    __shared__ float part[kWarps][128];
    __shared__ __align__(16) float inv_col[128];
    __shared__ int found[3];
    __shared__ int source[kFp8Block];  // with a route, the row of x behind each row of the tile
    grid_dependency_wait();
    grid_launch_dependents();
    Tile tl;
    if (j.offsets) {
        // The group that owns this token block: thread t sums the blocks of
        // groups t * per .. t * per + per - 1.
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int per = (j.G + kThreads - 1) / kThreads;
        const int g0 = threadIdx.x * per;
        int mine = 0;
        if (threadIdx.x == 0) found[0] = -1;
        for (int i = 0; i < per && g0 + i < j.G; ++i) mine += blocks_of(j.offsets[g0 + i + 1] - j.offsets[g0 + i]);
        int scan = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += v;
        }
        if (lane == 31) part[0][warp] = __int_as_float(scan);
        __syncthreads();
        int start = scan - mine;
        for (int w = 0; w < warp; ++w) start += __float_as_int(part[0][w]);
        const int b = j.block0 + static_cast<int>(blockIdx.y);
        if (b >= start && b < start + mine) {
            for (int i = 0; i < per && g0 + i < j.G; ++i) {
                const int beg = j.offsets[g0 + i], n = j.offsets[g0 + i + 1] - beg;
                const int nb = blocks_of(n);
                if (b < start + nb) {
                    found[1] = beg + (b - start) * kFp8Block;
                    found[2] = min(n - (b - start) * kFp8Block, kFp8Block);
                    found[0] = 1;
                    break;
                }
                start += nb;
            }
        }
        __syncthreads();
        if (found[0] < 0) return;  // past the last group's blocks
        tl.r0 = found[1];
        tl.nrows = found[2];
    } else {
        tl.r0 = blockIdx.y * kFp8Block;
        tl.nrows = min(j.rows - tl.r0, kFp8Block);
    }
    if (j.slots) {  // once for all column blocks: a division per row
        if (static_cast<int>(threadIdx.x) < tl.nrows) source[threadIdx.x] = j.slots[tl.r0 + threadIdx.x] / j.topk;
        __syncthreads();
    }
    tl.qc_row = static_cast<long long>(blockIdx.y) * kFp8Block;
    tl.sc_row = blockIdx.y;
    const int nblk = (j.cols + kFp8Block - 1) / kFp8Block;
    for (int cb = blockIdx.x * span; cb < min(nblk, static_cast<int>(blockIdx.x + 1) * span); ++cb) {
        tl.c0 = cb * kFp8Block;
        cast_tile_of<T, MODE, E5M2>(tl, static_cast<const T*>(j.x), j.ldx, j.slots ? source : nullptr, j.cols, vec, j.q_rows, j.ld_rows,
                                    j.s_rows, j.lds_rows, j.q_cols, j.ld_cols, j.s_cols, j.lds_cols, part, inv_col);
    }
}

// Three blocks of threads per SM for 16-bit weights: 80 registers, of which 4 to 8
// bytes spill (four blocks spill more and took 129 us where three took 118).
template <typename T, bool E5M2>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) fp8_cast_weight_kernel(CastWeightJob j, bool vec) {
    __shared__ float part[kWarps][128];
    __shared__ __align__(16) float inv_col[128];
    grid_dependency_wait();
    grid_launch_dependents();
    const int nb = (j.rows + kFp8Block - 1) / kFp8Block, kb = (j.cols + kFp8Block - 1) / kFp8Block;
    for (int g = blockIdx.z; g < j.G; g += gridDim.z) {
        Tile tl;
        tl.r0 = blockIdx.y * kFp8Block;
        tl.nrows = min(j.rows - tl.r0, kFp8Block);
        tl.c0 = blockIdx.x * kFp8Block;
        tl.qc_row = static_cast<long long>(g) * j.rows + tl.r0;
        tl.sc_row = 0;
        uint8_t* scale = j.scale + (static_cast<long long>(g) * nb + blockIdx.y) * kb + blockIdx.x;
        cast_tile_of<T, kBlockForm, E5M2>(tl, static_cast<const T*>(j.w) + g * j.stride_w, j.ldw, nullptr, j.cols, vec,
                                          static_cast<uint8_t*>(nullptr), 0LL, static_cast<uint8_t*>(nullptr), 0LL, j.q,
                                          j.ldq, scale, 0LL, part, inv_col);
    }
}

template <typename T, bool E5M2>
int cast_typed(const CastJob& j, int num_sms, cudaStream_t s) {
    const bool vec = (reinterpret_cast<uintptr_t>(j.x) & 15) == 0 && j.ldx * static_cast<int>(sizeof(T)) % 16 == 0;
    const int nblk = (j.cols + kFp8Block - 1) / kFp8Block;
    const int tblk = fp8_cast_blocks(j);
    // With groups a block looks its token block up first, so it takes several
    // column blocks then, as long as that leaves about sixteen blocks per SM.
    int span = 1;
    if (j.offsets)
        while (span < 8 && static_cast<long long>(tblk) * ((nblk + 2 * span - 1) / (2 * span)) >= 16LL * num_sms) span *= 2;
    // Later token blocks than a launch takes: the column form begins there. (A
    // third grid dimension instead costs the kernel of both forms registers that
    // it has not: spills, 92 us instead of 88 for the gathered cast above.)
    CastJob part = j;
    if (part.q_cols) {
        part.q_cols += static_cast<long long>(j.block0) * kFp8Block * j.ld_cols;
        part.s_cols += static_cast<long long>(j.block0) * j.lds_cols;
    }
    const dim3 grid((nblk + span - 1) / span, std::min(tblk - j.block0, kFp8CastBlocks));
    auto run = [&](auto k) { return static_cast<int>(launch_after(k, grid, dim3(kThreads), 0, s, part, vec, span)); };
    if (j.q_rows && j.q_cols) return run(fp8_cast_kernel<T, kBothForms, E5M2>);
    if (j.q_rows) return run(fp8_cast_kernel<T, kRowForm, E5M2>);
    return run(fp8_cast_kernel<T, kColForm, E5M2>);
}

}  // namespace

int fp8_cast_blocks(const CastJob& j) {
    return j.offsets ? fp8_max_blocks(j.rows, j.G) : (j.rows + kFp8Block - 1) / kFp8Block;
}

int launch_fp8_cast(const CastJob& j, int num_sms, cudaStream_t s) {
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        return j.fmt == GNS_E5M2 ? cast_typed<T, true>(j, num_sms, s) : cast_typed<T, false>(j, num_sms, s);
    });
}

int launch_fp8_cast_weight(const CastWeightJob& j, cudaStream_t s) {
    return by_dtype(j.dtype, [&](auto t) {
        using T = decltype(t);
        const bool vec = (reinterpret_cast<uintptr_t>(j.w) & 15) == 0 && j.ldw * static_cast<int>(sizeof(T)) % 16 == 0 &&
                         j.stride_w * static_cast<int>(sizeof(T)) % 16 == 0;
        const dim3 grid((j.cols + kFp8Block - 1) / kFp8Block, (j.rows + kFp8Block - 1) / kFp8Block,
                        std::min(j.G, 65535));
        return static_cast<int>(j.fmt == GNS_E5M2
                                    ? launch_after(fp8_cast_weight_kernel<T, true>, grid, dim3(kThreads), 0, s, j, vec)
                                    : launch_after(fp8_cast_weight_kernel<T, false>, grid, dim3(kThreads), 0, s, j, vec));
    });
}

}  // namespace gns
