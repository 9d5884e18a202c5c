// C ABI of the training-block operators: counter-based dropout, expert
// routing, block-scaled 8-bit casts and products. Argument checks, tensor maps
// and intermediate memory; the kernels are in dropout.cu, moe.cu and fp8_*.cu.
#include <algorithm>
#include <cmath>
#include <string>

#include "blockops.cuh"
#include "dropout.cuh"
#include "fp8.cuh"
#include "moe.cuh"
#include "runtime.cuh"

namespace gns {
namespace {

constexpr int64_t kMaxRows = 65535LL * kFp8Block;  // blocks of rows are a grid dimension

bool bad_dtype(int d) { return d != GNS_BF16 && d != GNS_FP16 && d != GNS_FP32; }
bool bad_format(int f) { return f != GNS_E4M3 && f != GNS_E5M2; }
bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int invalid(const char* msg) { return fail(GNS_ERR_INVALID, msg); }

// A row-major tensor of 8-bit values, `outer` rows of `inner`, G of them.
int map_u8(CUtensorMap* m, const void* p, int64_t inner, int64_t outer, int64_t G, int64_t ld, int64_t stride,
           uint32_t box_outer) {
    const auto fn = encode_fn();
    if (!fn) return fail(GNS_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(G)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld), static_cast<cuuint64_t>(stride)};
    cuuint32_t box[3] = {kFp8Block, box_outer, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(p), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(GNS_ERR_INVALID, "cuTensorMapEncodeTiled failed (" + std::to_string(static_cast<int>(r)) + "): " +
                                         std::to_string(outer) + " x " + std::to_string(inner) + ", ld " +
                                         std::to_string(ld));
    return GNS_OK;
}

// The map that whole rows of the product's output are stored through, where it
// can be described (16-byte rows).
int map_output(Fp8GemmJob& j, int cg) {
    const bool split = j.split > 1;
    const int es = split ? 4 : elem_bytes(j.out_dtype);
    void* p = split ? static_cast<void*>(j.partial) : j.D;
    const int64_t rows = j.wgrad ? j.M : j.rows, ld = split ? j.N : j.ldd;
    const int64_t G = split ? j.split : j.wgrad ? j.G : 1;
    const int64_t stride = split ? ld * rows : j.wgrad && j.G > 1 ? j.strideD : ld * rows;
    j.bulk_store = !misaligned(p, 16) && ld * es % 16 == 0 && stride * es % 16 == 0;
    if (!j.bulk_store) return GNS_OK;
    const auto fn = encode_fn();
    if (!fn) return fail(GNS_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(j.N), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(G)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * es), static_cast<cuuint64_t>(stride * es)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(fp8_store_row(cg) / es), 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(&j.mapD, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          fp8_store_row(cg) == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GNS_ERR_INVALID, "cuTensorMapEncodeTiled failed for the output");
    return GNS_OK;
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// An 8-bit operand [outer][ld] with `inner` values per row.
int check_q(const void* q, int64_t inner, int64_t ld) {
    if (!q) return invalid("null pointer");
    if (misaligned(q, 16) || ld % 16) return invalid("8-bit operands need 16-byte aligned rows");
    if (ld < up(inner, 16)) return invalid("an 8-bit operand's row stride must cover its columns rounded up to 16");
    return GNS_OK;
}

int check_route(int tokens, int topk, int num_experts) {
    if (tokens < 0 || topk < 1) return invalid("tokens >= 0 and topk >= 1 required");
    if (num_experts < 1 || num_experts > kMaxExperts) return invalid("num_experts must be in 1..GNS_MAX_EXPERTS");
    if (static_cast<int64_t>(tokens) * topk > 0x7fffffffLL - 4096) return invalid("tokens * topk must fit 31 bits");
    return GNS_OK;
}

int check_moves(int tokens, int topk, int num_experts, int cols, int dtype, const void* offsets, const void* rows) {
    RET(check_route(tokens, topk, num_experts));
    if (cols < 0) return invalid("cols >= 0 required");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (!offsets || (tokens > 0 && !rows)) return invalid("null pointer");
    return GNS_OK;
}

// Intermediate memory of such a product: the parts of a split contraction or the carried sums of a long one.
size_t product_scratch(int rows, int inner, int out, bool grouped, int out_dtype, int num_sms) {
    const int split = grouped ? 1 : fp8_gemm_split(rows, out, inner, num_sms);
    return split > 1 ? sizeof(float) * static_cast<size_t>(split) * rows * out
                     : fp8_carry_bytes(inner, out_dtype, split, num_sms);
}

// The forward and the data-gradient product: A [rows][inner_a], D [rows][n_out].
// scratch: product_scratch() bytes.
int product(const void* a, int64_t lda, const uint8_t* sa, int64_t ld_sa, int fmt_a, int rows, const void* w, int64_t ldw,
            const uint8_t* sw, int fmt_w, int groups, int N, int K, bool dgrad, const int32_t* offsets, void* D,
            int64_t ldd, int out_dtype, DeviceState* st, char* scratch, cudaStream_t s) {
    const int inner = dgrad ? N : K, out = dgrad ? K : N;
    RET(check_q(a, inner, lda));
    RET(check_q(w, K, ldw));
    if (!sa || !sw || !D) return invalid("null pointer");
    if (ld_sa < rows) return invalid("a scale's row stride must cover the rows");
    if (ldd < out) return invalid("the output's row stride must cover its columns");
    Fp8GemmJob j{};
    const int cg = fp8_gemm_cg(rows, out, offsets != nullptr, !dgrad, out_dtype, st->num_sms);
    j.split = offsets ? 1 : fp8_gemm_split(rows, out, inner, st->num_sms);
    RET(map_u8(&j.mapA, a, inner, rows, 1, lda, lda * rows, 128));
    RET(map_u8(&j.mapB, w, K, N, groups, ldw, ldw * N, fp8_gemm_b_box(cg, dgrad)));
    j.b_mn = dgrad;
    j.fmt_a = fmt_a;
    j.fmt_b = fmt_w;
    j.G = groups;
    j.offsets = offsets;
    j.rows = rows;
    j.N = out;
    j.K = inner;
    j.sA = sa;
    j.ldsA = ld_sa;
    const int64_t nb = up(N, kFp8Block) / kFp8Block, kb = up(K, kFp8Block) / kFp8Block;
    j.sB = sw;
    j.sB_g = nb * kb;
    j.sB_n = dgrad ? 1 : kb;
    j.sB_k = dgrad ? kb : 1;
    j.D = D;
    j.ldd = ldd;
    j.out_dtype = out_dtype;
    // One of the two at most, in product_scratch() bytes.
    (j.split > 1 ? j.partial : j.carry) = reinterpret_cast<float*>(scratch);
    RET(map_output(j, cg));
    j.st = new_call(*st);
    LAUNCH(kClsFp8Gemm, launch_fp8_gemm(j, cg, st->num_sms, s));
    if (j.split > 1) LAUNCH(kClsFp8Gemm, launch_fp8_reduce(j, s));
    return GNS_OK;
}

int check_product(int fmt_a, int fmt_w, int groups, int rows, int N, int K, const void* offsets, int out_dtype) {
    if (bad_format(fmt_a) || bad_format(fmt_w)) return invalid("unknown 8-bit format");
    if (bad_dtype(out_dtype)) return invalid("unknown dtype");
    if (groups < 1 || groups > kMaxExperts) return invalid("groups must be in 1..GNS_MAX_EXPERTS");
    if (groups > 1 && !offsets) return invalid("more than one group needs offsets");
    if (rows < 0 || rows > kMaxRows) return invalid("rows must be in 0..8388480");
    if (N < 1 || K < 1) return invalid("N >= 1 and K >= 1 required");
    return GNS_OK;
}

}  // namespace
}  // namespace gns

using namespace gns;

extern "C" {

int gns_dropout(const void* x, const void* residual, void* y, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr,
                int64_t ldy, int dtype, double p, uint64_t seed, uint64_t step, int64_t base_index, void* stream) {
    if (rows < 0 || cols < 0 || base_index < 0) return invalid("rows, cols and base_index must be >= 0");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (!(p >= 0.0 && p <= 1.0)) return invalid("p must be in [0, 1]");
    if (step >> 63) return invalid("step must be below 2^63");
    if (rows == 0 || cols == 0) return GNS_OK;
    if (cols > (INT64_C(1) << 40) / rows) return invalid("more than 2^40 elements");
    if (!x || !y) return invalid("null pointer");
    if (rows > 1 && (ldx < cols || ldy < cols || (residual && ldr < cols)))
        return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    DropoutJob j{};
    j.x = x;
    j.residual = residual;
    j.y = y;
    j.rows = rows;
    j.cols = cols;
    j.ldx = ldx;
    j.ldr = ldr;
    j.ldy = ldy;
    j.dtype = dtype;
    j.threshold = static_cast<uint32_t>(std::nearbyint(p * 65536.0));
    j.inv = j.threshold < 65536u ? static_cast<float>(65536.0 / (65536.0 - j.threshold)) : 0.0f;
    j.seed = seed;
    j.step = step;
    j.base = static_cast<unsigned long long>(base_index);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsDropout, launch_dropout(j, s));
    return GNS_OK;
}

int gns_moe_sort(const void* experts, int id_bytes, int tokens, int topk, int num_experts, int32_t* offsets,
                 int32_t* rows, int32_t* slots, void* stream) {
    RET(check_route(tokens, topk, num_experts));
    if (id_bytes != 4 && id_bytes != 8) return invalid("id_bytes must be 4 or 8");
    if (!offsets || (tokens > 0 && (!experts || !rows || !slots))) return invalid("null pointer");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    SortJob j{experts, id_bytes, static_cast<long long>(tokens) * topk, num_experts, offsets, rows, slots, nullptr};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch scratch;
    if (const size_t bytes = moe_sort_scratch(j.n, num_experts)) {
        RET(scratch.take(*st, bytes, s));
        j.hist = reinterpret_cast<int*>(scratch.data());
        LAUNCH(kClsMoe, launch_moe_count(j, s));
    }
    LAUNCH(kClsMoe, launch_moe_place(j, s));
    return GNS_OK;
}

int gns_moe_gather(const void* x, int64_t ldx, int tokens, int topk, int num_experts, int cols, int dtype,
                   const int32_t* offsets, const int32_t* rows, void* y, int64_t ldy, void* stream) {
    RET(check_moves(tokens, topk, num_experts, cols, dtype, offsets, rows));
    if (tokens == 0 || cols == 0) return GNS_OK;
    if (!x || !y) return invalid("null pointer");
    if (ldx < cols || ldy < cols) return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsMoe, launch_moe_gather(RouteJob{tokens, topk, num_experts, cols, offsets, rows, dtype}, x, ldx, y, ldy, s));
    return GNS_OK;
}

int gns_moe_combine(const void* y, int64_t ldy, const float* weights, int tokens, int topk, int num_experts, int cols,
                    int dtype, const int32_t* offsets, const int32_t* rows, void* out, int64_t ldo, void* stream) {
    RET(check_moves(tokens, topk, num_experts, cols, dtype, offsets, rows));
    if (tokens == 0 || cols == 0) return GNS_OK;
    if (!y || !out) return invalid("null pointer");
    if (ldy < cols || ldo < cols) return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsMoe, launch_moe_combine(RouteJob{tokens, topk, num_experts, cols, offsets, rows, dtype}, y, ldy, weights,
                                       out, ldo, s));
    return GNS_OK;
}

int gns_moe_combine_backward(const void* dout, int64_t lddo, const void* y, int64_t ldy, const float* weights,
                             int tokens, int topk, int num_experts, int cols, int dtype, const int32_t* offsets,
                             const int32_t* rows, void* dy, int64_t lddy, float* dweights, void* stream) {
    RET(check_moves(tokens, topk, num_experts, cols, dtype, offsets, rows));
    if (tokens == 0) return GNS_OK;
    if (!weights || (dweights && !y && cols > 0)) return invalid("null pointer");
    if (cols > 0 && (!dout || !dy)) return invalid("null pointer");
    if (lddo < cols || lddy < cols || (dweights && ldy < cols)) return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsMoe, launch_moe_combine_backward(RouteJob{tokens, topk, num_experts, cols, offsets, rows, dtype}, dout,
                                                lddo, y, ldy, weights, dy, lddy, dweights, s));
    return GNS_OK;
}

int gns_fp8_quantize(const void* x, int64_t ldx, int dtype, int rows, int cols, const int32_t* slots, int topk,
                     const int32_t* offsets, int groups, int format, void* q_rows, int64_t ld_rows, uint8_t* scale_rows,
                     int64_t ld_scale_rows, void* q_cols, int64_t ld_cols, uint8_t* scale_cols, int64_t ld_scale_cols,
                     void* stream) {
    if (rows < 0 || rows > kMaxRows || cols < 1) return invalid("rows must be in 0..8388480 and cols >= 1");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (bad_format(format)) return invalid("unknown 8-bit format");
    if (slots && topk < 1) return invalid("topk >= 1 required");
    if (offsets && (groups < 1 || groups > kMaxExperts)) return invalid("groups must be in 1..GNS_MAX_EXPERTS");
    if (rows == 0) return GNS_OK;
    if (!q_rows && !q_cols) return invalid("null pointer");
    if (q_rows) {
        RET(check_q(q_rows, cols, ld_rows));
        if (!scale_rows) return invalid("null pointer");
        if (ld_scale_rows < rows) return invalid("a scale's row stride must cover the rows");
    }
    if (q_cols) {
        RET(check_q(q_cols, cols, ld_cols));
        if (!scale_cols) return invalid("null pointer");
        if (ld_scale_cols < cols) return invalid("a scale's row stride must cover the columns");
    }
    if (!x) return invalid("null pointer");
    if (ldx < cols) return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    CastJob j{};
    j.x = x;
    j.ldx = ldx;
    j.dtype = dtype;
    j.rows = rows;
    j.cols = cols;
    j.slots = slots;
    j.topk = slots ? topk : 1;
    // Groups matter to the column form's blocks alone.
    j.offsets = q_cols ? offsets : nullptr;
    j.G = j.offsets ? groups : 1;
    j.fmt = format;
    j.q_rows = static_cast<uint8_t*>(q_rows);
    j.s_rows = scale_rows;
    j.ld_rows = ld_rows;
    j.lds_rows = ld_scale_rows;
    j.q_cols = static_cast<uint8_t*>(q_cols);
    j.s_cols = scale_cols;
    j.ld_cols = ld_cols;
    j.lds_cols = ld_scale_cols;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Without groups there are at most 65535 token blocks, the limit of a launch;
    // groups may add one each.
    const int blocks = fp8_cast_blocks(j);
    for (; j.block0 < blocks; j.block0 += kFp8CastBlocks) LAUNCH(kClsFp8Cast, launch_fp8_cast(j, st->num_sms, s));
    return GNS_OK;
}

int gns_fp8_quantize_weight(const void* w, int64_t ldw, int64_t stride_w, int dtype, int groups, int N, int K,
                            int format, void* q, int64_t ldq, uint8_t* scale, void* stream) {
    if (groups < 0 || N < 1 || N > kMaxRows || K < 1) return invalid("groups >= 0, N in 1..8388480 and K >= 1 required");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (bad_format(format)) return invalid("unknown 8-bit format");
    if (groups == 0) return GNS_OK;
    RET(check_q(q, K, ldq));
    if (!w || !scale) return invalid("null pointer");
    if (ldw < K) return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    CastWeightJob j{w, ldw, stride_w, dtype, groups, N, K, format, static_cast<uint8_t*>(q), ldq, scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsFp8Cast, launch_fp8_cast_weight(j, s));
    return GNS_OK;
}

int gns_fp8_matmul(const void* a, int64_t lda, const uint8_t* scale_a, int64_t ld_scale_a, int format_a, int rows,
                   const void* w, int64_t ldw, const uint8_t* scale_w, int format_w, int groups, int N, int K,
                   const int32_t* offsets, void* y, int64_t ldy, int out_dtype, void* stream) {
    RET(check_product(format_a, format_w, groups, rows, N, K, offsets, out_dtype));
    if (rows == 0) return GNS_OK;
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch scratch;
    if (const size_t bytes = product_scratch(rows, K, N, offsets != nullptr, out_dtype, st->num_sms))
        RET(scratch.take(*st, bytes, s));
    return product(a, lda, scale_a, ld_scale_a, format_a, rows, w, ldw, scale_w, format_w, groups, N, K, false, offsets,
                   y, ldy, out_dtype, st, scratch.data(), s);
}

int gns_fp8_matmul_dgrad(const void* dy, int64_t lddy, const uint8_t* scale_dy, int64_t ld_scale_dy, int format_dy,
                         int rows, const void* w, int64_t ldw, const uint8_t* scale_w, int format_w, int groups, int N,
                         int K, const int32_t* offsets, void* dx, int64_t lddx, int out_dtype, void* stream) {
    RET(check_product(format_dy, format_w, groups, rows, N, K, offsets, out_dtype));
    if (rows == 0) return GNS_OK;
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch scratch;
    if (const size_t bytes = product_scratch(rows, N, K, offsets != nullptr, out_dtype, st->num_sms))
        RET(scratch.take(*st, bytes, s));
    return product(dy, lddy, scale_dy, ld_scale_dy, format_dy, rows, w, ldw, scale_w, format_w, groups, N, K, true,
                   offsets, dx, lddx, out_dtype, st, scratch.data(), s);
}

int gns_fp8_matmul_wgrad(const void* dy, int64_t lddy, const uint8_t* scale_dy, int64_t ld_scale_dy, int format_dy,
                         const void* x, int64_t ldx, const uint8_t* scale_x, int64_t ld_scale_x, int format_x, int rows,
                         int groups, int N, int K, const int32_t* offsets, void* dw, int64_t lddw, int64_t stride_dw,
                         int out_dtype, void* stream) {
    RET(check_product(format_dy, format_x, groups, rows, N, K, offsets, out_dtype));
    if (!dw) return invalid("null pointer");
    if (lddw < K || stride_dw < 0) return invalid("a row stride must cover the columns");
    if (rows > 0) {
        RET(check_q(dy, N, lddy));
        RET(check_q(x, K, ldx));
        if (!scale_dy || !scale_x) return invalid("null pointer");
        if (ld_scale_dy < N || ld_scale_x < K) return invalid("a scale's row stride must cover the columns");
    }
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t es = static_cast<size_t>(elem_bytes(out_dtype));
    if (rows == 0) {  // no tokens: the gradient is zero
        for (int g = 0; g < groups; ++g)
            CK(cudaMemset2DAsync(static_cast<char*>(dw) + es * g * stride_dw, es * lddw, 0, es * K, N, s));
        return GNS_OK;
    }
    Fp8GemmJob j{};
    const int64_t qrows = offsets ? static_cast<int64_t>(fp8_max_blocks(rows, groups)) * kFp8Block : up(rows, kFp8Block);
    const int cg = fp8_gemm_cg(N, K, groups > 1, false, out_dtype, st->num_sms);
    RET(map_u8(&j.mapA, dy, N, qrows, 1, lddy, lddy * qrows, 128));
    RET(map_u8(&j.mapB, x, K, qrows, 1, ldx, ldx * qrows, 128));
    j.wgrad = 1;
    j.b_mn = 1;
    j.fmt_a = format_dy;
    j.fmt_b = format_x;
    j.G = groups;
    j.offsets = offsets;
    j.rows = rows;
    j.M = N;
    j.N = K;
    j.sA = scale_dy;
    j.ldsA = ld_scale_dy;
    j.sB = scale_x;
    j.sB_k = ld_scale_x;
    j.D = dw;
    j.ldd = lddw;
    j.strideD = stride_dw;
    j.out_dtype = out_dtype;
    j.split = 1;
    Scratch carry;
    if (const size_t bytes = fp8_carry_bytes(rows, out_dtype, 1, st->num_sms)) {
        RET(carry.take(*st, bytes, s));
        j.carry = reinterpret_cast<float*>(carry.data());
    }
    RET(map_output(j, cg));
    j.st = new_call(*st);
    LAUNCH(kClsFp8Gemm, launch_fp8_gemm(j, cg, st->num_sms, s));
    return GNS_OK;
}

int gns_fp8_linear(const void* x, int64_t ldx, int dtype, int rows, const int32_t* slots, int topk,
                   const int32_t* offsets, const void* w, int64_t ldw, const uint8_t* scale_w, int format_w, int groups,
                   int N, int K, void* y, int64_t ldy, int out_dtype, void* stream) {
    RET(check_product(GNS_E4M3, format_w, groups, rows, N, K, offsets, out_dtype));
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (slots && topk < 1) return invalid("topk >= 1 required");
    if (rows == 0) return GNS_OK;
    if (!x || !y || !scale_w) return invalid("null pointer");
    if (ldx < K || ldy < N) return invalid("a row stride must cover the columns");
    RET(check_q(w, K, ldw));
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (fp8_rows_fit(rows, N, K, groups, offsets != nullptr, st->num_sms)) {
        Fp8RowsJob j{x,       ldx, dtype, slots, slots ? topk : 1, offsets, groups, rows, N, K, format_w,
                     static_cast<const uint8_t*>(w), ldw, ldw * N, scale_w, y, ldy, out_dtype};
        LAUNCH(kClsFp8Gemm, launch_fp8_rows(j, st->num_sms, s));
        return GNS_OK;
    }
    // Every SM reads the cast rows at the same time, and from less than 128 KB
    // that is slower: few rows lie apart (9 to 31 rows by 14336 x 4096: 16.0 to
    // 16.6 us instead of 19.8 to 20.4 with the weights in L2, 20.0 to 20.7 instead
    // of 21.0 to 21.3 with weights from HBM).
    const int64_t ldq = std::max(up(K, 16), up((256 << 10) / rows, 128));
    const size_t q_bytes = static_cast<size_t>(up(ldq * rows, 256));
    const size_t s_bytes = static_cast<size_t>(up(up(K, kFp8Block) / kFp8Block * rows, 256));
    Scratch scratch;
    RET(scratch.take(*st, q_bytes + s_bytes + product_scratch(rows, K, N, offsets != nullptr, out_dtype, st->num_sms), s));
    uint8_t* scale = reinterpret_cast<uint8_t*>(scratch.data() + q_bytes);
    RET(gns_fp8_quantize(x, ldx, dtype, rows, K, slots, topk, nullptr, 1, GNS_E4M3, scratch.data(), ldq, scale, rows,
                         nullptr, 0, nullptr, 0, stream));
    return product(scratch.data(), ldq, scale, rows, GNS_E4M3, rows, w, ldw, scale_w, format_w, groups, N, K, false,
                   offsets, y, ldy, out_dtype, st, scratch.data() + q_bytes + s_bytes, s);
}

}  // extern "C"
