// C ABI of the layer operators around an expert block: layer norm. Argument checks
// and intermediate memory; the kernels are in layer_norm*.cu.
#include <cmath>

#include "blockops.cuh"
#include "layer_norm.cuh"
#include "runtime.cuh"

namespace gns {
namespace {

bool bad_dtype(int d) { return d != GNS_BF16 && d != GNS_FP16 && d != GNS_FP32; }

int invalid(const char* msg) { return fail(GNS_ERR_INVALID, msg); }

constexpr int kMaxNormCols = 1 << 24;  // as far as fp32 counts

int check_norm(int64_t rows, int cols, int dtype, int weight_dtype) {
    if (rows < 0 || rows > 0x7fffffffLL) return invalid("rows must be in 0..2^31 - 1");
    if (cols < 0 || cols > kMaxNormCols) return invalid("cols must be in 0..2^24");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (weight_dtype != dtype && weight_dtype != GNS_FP32) return invalid("weight and bias must be fp32 or of x's type");
    return GNS_OK;
}

}  // namespace
}  // namespace gns

using namespace gns;

extern "C" {

int gns_layer_norm(const void* x, int64_t ldx, int64_t rows, int cols, int dtype, const void* weight, const void* bias,
                   int weight_dtype, double eps, int rms, void* y, int64_t ldy, float* stats, void* stream) {
    RET(check_norm(rows, cols, dtype, weight_dtype));
    if (!(eps >= 0.0 && std::isfinite(static_cast<float>(eps)))) return invalid("eps must be a finite fp32 value of at least 0");
    if (rows == 0 || cols == 0) return GNS_OK;
    if (!x || !y || !stats) return invalid("null pointer");
    if (ldx < cols || ldy < cols) return invalid("a row stride must cover the columns");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    NormJob j{};
    j.x = x;
    j.ldx = ldx;
    j.rows = rows;
    j.cols = cols;
    j.dtype = dtype;
    j.weight = weight;
    j.bias = bias;
    j.wf32 = weight_dtype == GNS_FP32;
    j.rms = rms != 0;
    j.eps = static_cast<float>(eps);
    j.y = y;
    j.ldy = ldy;
    j.stats = stats;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsLayerNorm, launch_layer_norm(j, st->num_sms, s));
    return GNS_OK;
}

int gns_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* stats, int64_t rows,
                            int cols, int dtype, const void* weight, int weight_dtype, int rms, const void* residual,
                            int64_t ldr, void* dx, int64_t lddx, void* dweight, void* dbias, void* stream) {
    RET(check_norm(rows, cols, dtype, weight_dtype));
    if (cols == 0) return GNS_OK;
    if (rows > 0 && (!dy || !x || !stats || !dx)) return invalid("null pointer");
    if (rows > 0 && (lddy < cols || ldx < cols || lddx < cols || (residual && ldr < cols)))
        return invalid("a row stride must cover the columns");
    if (rows == 0 && !dweight && !dbias) return GNS_OK;
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // no rows: the sums over them are zero
        const size_t bytes = static_cast<size_t>(cols) * elem_bytes(weight_dtype);
        if (dweight) CK(cudaMemsetAsync(dweight, 0, bytes, s));
        if (dbias) CK(cudaMemsetAsync(dbias, 0, bytes, s));
        return GNS_OK;
    }
    NormJob j{};
    j.x = x;
    j.ldx = ldx;
    j.rows = rows;
    j.cols = cols;
    j.dtype = dtype;
    j.weight = weight;
    j.wf32 = weight_dtype == GNS_FP32;
    j.rms = rms != 0;
    j.stats = const_cast<float*>(stats);
    j.dy = dy;
    j.lddy = lddy;
    j.residual = residual;
    j.ldr = ldr;
    j.dx = dx;
    j.lddx = lddx;
    j.dweight = dweight;
    j.dbias = dbias;
    Scratch scratch;
    if (const size_t bytes = norm_backward_scratch(j, st->num_sms)) {
        RET(scratch.take(*st, bytes, s));
        j.part = reinterpret_cast<float*>(scratch.data());
    }
    LAUNCH(kClsLayerNorm, launch_layer_norm_backward(j, st->num_sms, s));
    if (!j.part) return GNS_OK;
    if (layer_norm_columns_apart(j)) LAUNCH(kClsLayerNorm, launch_layer_norm_columns(j, st->num_sms, s));
    LAUNCH(kClsLayerNorm, launch_layer_norm_join(j, st->num_sms, s));
    return GNS_OK;
}

}  // extern "C"
