// Block-scaled 8-bit operands and their products: launchers (fp8_cast.cu,
// fp8_gemm.cu, fp8_rows.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "blockops.cuh"
#include "ptx.cuh"

namespace gns {

constexpr int kFp8Block = 128;

// Bytes of a row of the product's output that one bulk store takes (and its
// swizzle), for single CTAs and pairs. A single CTA's tile needs 48 KB per k
// block, and with 64-byte rows there is room for a fourth (data and weight
// gradient of 256 experts of 512 x 2048, 65536 rows: 103 and 129 us, 113 and 138
// with 128-byte rows and three); a pair's needs 32 KB and has five with 128.
constexpr int fp8_store_row(int cg) { return cg == 1 ? 64 : 128; }

// The cast of a rows x cols matrix; see gns_fp8_quantize. Either output may
// be null. With offsets the token blocks of the column form are those of the
// G groups of rows, and rows past offsets[G] are not written.
struct CastJob {
    const void* x;
    long long ldx;
    int dtype;
    int rows, cols;
    const int* slots;  // source row of row r is slots[r] / topk (null: r)
    int topk;
    const int* offsets;  // or null: one group of all rows
    int G;
    int fmt;
    uint8_t* q_rows;
    uint8_t* s_rows;  // scales are 8-bit exponents: b stands for 2^(b - 127)
    long long ld_rows, lds_rows;
    uint8_t* q_cols;
    uint8_t* s_cols;
    long long ld_cols, lds_cols;
    int block0;  // first token block of the launch
};

// Token blocks of the cast (with offsets, an upper bound), and those that one launch takes.
int fp8_cast_blocks(const CastJob& job);
constexpr int kFp8CastBlocks = 65535;
int launch_fp8_cast(const CastJob& job, int num_sms, cudaStream_t s);

// The cast of G matrices of rows x cols in blocks of 128 x 128.
struct CastWeightJob {
    const void* w;
    long long ldw, stride_w;
    int dtype, G, rows, cols, fmt;
    uint8_t* q;
    long long ldq;  // matrices are rows * ldq apart
    uint8_t* scale;  // [G][ceil(rows / 128)][ceil(cols / 128)]
};

int launch_fp8_cast_weight(const CastWeightJob& job, cudaStream_t s);

// Largest number of 128-row token blocks that `rows` rows in G groups need.
__host__ __device__ inline int fp8_max_blocks(long long rows, int G) {
    const long long g = rows < G ? rows : G;
    return static_cast<int>((rows + (kFp8Block - 1) * g) / kFp8Block);
}

__device__ __forceinline__ int blocks_of(int count) { return (count + kFp8Block - 1) / kFp8Block; }

// One tcgen05 product per group g of rows (fp8_gemm.cu):
//   forward / data gradient: D[r][n] over the group's rows r, contraction
//     K; A is the row form, B the group's weights, [N][K] (b_mn = 0) or its
//     stored transpose [K][N] (b_mn = 1);
//   weight gradient (wgrad = 1): D[g][m][n], contraction the group's rows; A
//     and B are column forms, [blocks * 128][M] and [blocks * 128][N].
struct Fp8GemmJob {
    CUtensorMap mapA, mapB, mapD;  // mapD: boxes of 32 rows of fp8_store_row() bytes of the output (partial when split > 1)
    int bulk_store;                // mapD holds (the output has 16-byte rows)
    int wgrad, b_mn;
    int fmt_a, fmt_b;
    int G;
    const int* offsets;  // or null: one group of all rows
    int rows;            // rows of all groups (capacity when offsets is given)
    int M, N, K;         // M: wgrad only; K: not for wgrad
    const uint8_t* sA;   // [k block or token block][row or m], row stride ldsA
    long long ldsA;
    const uint8_t* sB;   // weights: scale of (g, n block, k block) at g * sB_g + nb * sB_n + kb * sB_k
    long long sB_g, sB_n, sB_k;  // wgrad: [token block][n], row stride sB_k
    void* D;
    long long ldd, strideD;
    int out_dtype;
    float* partial;      // split > 1: fp32 [split][rows][N]
    float* carry;        // fp8_carry_bytes() bytes, or null where that is 0
    int split;           // forward / data gradient of one group only
    DevStatus st;
};

// CTAs per tile (1: 128 x 256 tiles, 2: a pair, 256 x 256) for a product with M
// rows (of all groups; the weight gradient: of each D) and N columns.
int fp8_gemm_cg(int M, int N, bool grouped, bool forward, int out_dtype, int num_sms);
// Rows of the boxes of B's tensor map.
inline int fp8_gemm_b_box(int cg, bool b_mn) { return b_mn || cg == 2 ? 128 : 256; }

int launch_fp8_gemm(const Fp8GemmJob& job, int cg, int num_sms, cudaStream_t s);
// The sum over the parts of a split contraction, after launch_fp8_gemm.
int launch_fp8_reduce(const Fp8GemmJob& job, cudaStream_t s);

// Bytes of intermediate memory for a 16-bit result whose contraction (an upper
// bound of it) is longer than the tensor core's accumulator sums alone: a tile's
// fp32 sums so far, for each CTA.
constexpr int kFp8LongBlocks = 256;  // blocks of 128 along the contraction (see fp8_gemm.cu)
inline size_t fp8_carry_bytes(long long contraction, int out_dtype, int split, int num_sms) {
    const bool carries = elem_bytes(out_dtype) == 2 && split <= 1 && contraction > kFp8LongBlocks * kFp8Block;
    return carries ? sizeof(float) * 128 * 256 * (num_sms > 1 ? num_sms : 2) : 0;  // a pair is launched whole
}

// The split of the contraction that fills the machine, 1 for none.
int fp8_gemm_split(int rows, int N, int K, int num_sms);

// The product of few rows (fp8_rows.cu): D[r][n] = x_r . w[g(r)][n], x cast on
// the way as by launch_fp8_cast.
struct Fp8RowsJob {
    const void* x;
    long long ldx;
    int dtype;
    const int* slots;
    int topk;
    const int* offsets;
    int G, rows, N, K;
    int fmt_w;
    const uint8_t* w;
    long long ldw, stride_w;
    const uint8_t* sw;  // [G][ceil(N / 128)][ceil(K / 128)]
    void* D;
    long long ldd;
    int out_dtype;
};

constexpr int kFp8FewRows = 8;     // rows of one matrix (and of a block of threads)
constexpr int kFp8FewRouted = 32;  // rows of a routed batch
// Whether launch_fp8_rows takes this product.
bool fp8_rows_fit(int rows, int N, int K, int groups, bool grouped, int num_sms);
int launch_fp8_rows(const Fp8RowsJob& job, int num_sms, cudaStream_t s);

}  // namespace gns
