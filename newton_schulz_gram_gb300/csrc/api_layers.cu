// C ABI of the layer operators around an expert block: layer norm, the
// router's gates with the balance loss, and the embedding. Argument checks and
// intermediate memory; the kernels are in layer_norm*.cu, moe_gate.cu and embedding.cu.
#include <cmath>

#include "blockops.cuh"
#include "embedding.cuh"
#include "layer_norm.cuh"
#include "moe_gate.cuh"
#include "runtime.cuh"

namespace gns {
namespace {

bool bad_dtype(int d) { return d != GNS_BF16 && d != GNS_FP16 && d != GNS_FP32; }

int invalid(const char* msg) { return fail(GNS_ERR_INVALID, msg); }

constexpr int kMaxNormCols = 1 << 24;  // as far as fp32 counts

int check_norm(int64_t rows, int cols, int dtype, int weight_dtype) {
    if (rows < 0 || rows > 0x7fffffffLL) return invalid("rows must be in 0..2^31 - 1");
    if (cols < 1 || cols > kMaxNormCols) return invalid("cols must be in 1..2^24");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (weight_dtype != dtype && weight_dtype != GNS_FP32) return invalid("weight and bias must be fp32 or of x's type");
    return GNS_OK;
}

// Whether [rows][ld] rows of cols elements at a and b share memory.
bool overlap(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int cols, int es) {
    const auto end = [&](const void* p, int64_t ld) { return static_cast<const char*>(p) + ((rows - 1) * ld + cols) * es; };
    return a < end(b, ldb) && b < end(a, lda);
}

int check_gate(const void* logits, int64_t ld, int tokens, int experts, int topk, int dtype) {
    if (tokens < 0) return invalid("tokens >= 0 required");
    if (experts < 1 || experts > kMaxExperts) return invalid("num_experts must be in 1..GNS_MAX_EXPERTS");
    if (topk < 1 || topk > kMaxTopk || topk > experts) return invalid("topk must be in 1..num_experts and at most GNS_MAX_TOPK");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (static_cast<int64_t>(tokens) * topk > 0x7fffffffLL - 4096) return invalid("tokens * topk must fit 31 bits");
    if (tokens > 0 && !logits) return invalid("null pointer");
    if (ld < experts) return invalid("a row stride must cover the experts");
    return GNS_OK;
}

constexpr int kMaxVocab = 1 << 30;

int check_embedding(const void* ids, int id_bytes, int64_t tokens, int64_t vocab, int64_t cols, int dtype, double scale) {
    if (tokens < 0 || tokens > 0x7fffffffLL - 4096) return invalid("tokens must fit 31 bits");
    if (vocab < 1 || vocab > kMaxVocab) return invalid("vocab must be in 1..2^30");
    if (cols < 0 || cols > (1 << 24)) return invalid("cols must be in 0..2^24");
    if (id_bytes != 4 && id_bytes != 8) return invalid("id_bytes must be 4 or 8");
    if (bad_dtype(dtype)) return invalid("unknown dtype");
    if (!std::isfinite(static_cast<float>(scale))) return invalid("scale must be a finite fp32 value");
    if (tokens > 0 && cols > 0 && !ids) return invalid("null pointer");
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
    if (rows == 0) return GNS_OK;
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
    j.again = !overlap(x, ldx, y, ldy, rows, cols, elem_bytes(dtype));
    j.stats = stats;
    j.st = new_call(*st);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsLayerNorm, launch_layer_norm(j, st->num_sms, s));
    return GNS_OK;
}

int gns_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* stats, int64_t rows,
                            int cols, int dtype, const void* weight, int weight_dtype, int rms, const void* residual,
                            int64_t ldr, void* dx, int64_t lddx, void* dweight, void* dbias, void* stream) {
    RET(check_norm(rows, cols, dtype, weight_dtype));
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
    j.st = new_call(*st);
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

int gns_moe_gate(const void* logits, int64_t ld, int tokens, int num_experts, int topk, int dtype, int normalize,
                 int64_t* ids, float* weights, float* lse, void* stream) {
    RET(check_gate(logits, ld, tokens, num_experts, topk, dtype));
    if (tokens == 0) return GNS_OK;
    if (!ids || !weights || !lse) return invalid("null pointer");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    GateJob j{logits, ld, tokens, num_experts, topk, dtype, normalize != 0, reinterpret_cast<const long long*>(ids), weights, lse};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsMoe, launch_moe_gate(j, s));
    return GNS_OK;
}

int gns_moe_balance(const void* logits, int64_t ld, int tokens, int num_experts, int topk, int dtype, const int64_t* ids,
                    const float* lse, double balance, double z, float* loss, int32_t* counts, float* probs, void* stream) {
    RET(check_gate(logits, ld, tokens, num_experts, topk, dtype));
    if (tokens > 0 && (!ids || !lse)) return invalid("null pointer");
    if (!loss || !counts || !probs) return invalid("null pointer");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    GateJob j{logits, ld, tokens, num_experts, topk, dtype, 0, reinterpret_cast<const long long*>(ids), nullptr, lse};
    BalanceJob b{static_cast<float>(balance), static_cast<float>(z), loss, counts, probs, nullptr};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch scratch;
    RET(scratch.take(*st, moe_balance_scratch(j, st->num_sms), s));
    b.part = reinterpret_cast<float*>(scratch.data());
    LAUNCH(kClsMoe, launch_moe_balance(j, b, st->num_sms, s));
    LAUNCH(kClsMoe, launch_moe_balance_join(j, b, st->num_sms, s));
    return GNS_OK;
}

int gns_moe_gate_backward(const float* dweights, const void* logits, int64_t ld, int tokens, int num_experts, int topk,
                          int dtype, int normalize, const int64_t* ids, const float* weights, const float* lse,
                          const int32_t* counts, double balance, double z, const float* dloss, void* dlogits, int64_t ldd,
                          void* stream) {
    RET(check_gate(logits, ld, tokens, num_experts, topk, dtype));
    if (ldd < num_experts) return invalid("a row stride must cover the experts");
    if (tokens == 0) return GNS_OK;
    if (!dweights || !ids || !weights || !lse || !dlogits) return invalid("null pointer");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    GateJob j{logits, ld, tokens, num_experts, topk, dtype, normalize != 0, reinterpret_cast<const long long*>(ids), weights, lse};
    GateGradJob g{dweights, counts, static_cast<float>(balance), static_cast<float>(z), dloss, dlogits, ldd};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsMoe, launch_moe_gate_backward(j, g, s));
    return GNS_OK;
}

int gns_embedding(const void* ids, int id_bytes, int64_t tokens, const void* table, int64_t ldt, int64_t vocab, int64_t cols,
                  int dtype, double scale, void* y, int64_t ldy, void* stream) {
    RET(check_embedding(ids, id_bytes, tokens, vocab, cols, dtype, scale));
    if (ldt < cols || ldy < cols) return invalid("a row stride must cover the columns");
    if (tokens == 0 || cols == 0) return GNS_OK;
    if (!table || !y) return invalid("null pointer");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    EmbeddingJob j{};
    j.ids = ids;
    j.id_bytes = id_bytes;
    j.tokens = static_cast<int>(tokens);
    j.vocab = static_cast<int>(vocab);
    j.cols = static_cast<int>(cols);
    j.scale = static_cast<float>(scale);
    j.table = table;
    j.ldt = ldt;
    j.y = y;
    j.ldy = ldy;
    j.dtype = dtype;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LAUNCH(kClsEmbedding, launch_embedding(j, s));
    return GNS_OK;
}

int gns_embedding_backward(const void* dy, int64_t lddy, const void* ids, int id_bytes, int64_t tokens, int64_t vocab,
                           int64_t cols, int dtype, double scale, void* dtable, int64_t lddt, int out_dtype, void* stream) {
    RET(check_embedding(ids, id_bytes, tokens, vocab, cols, dtype, scale));
    if (bad_dtype(out_dtype)) return invalid("unknown dtype");
    if (lddt < cols || (tokens > 0 && lddy < cols)) return invalid("a row stride must cover the columns");
    if (cols == 0) return GNS_OK;
    if (!dtable || (tokens > 0 && !dy)) return invalid("null pointer");
    DeviceState* st = nullptr;
    RET(get_state(&st));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {  // no tokens: the gradient is zero
        const size_t es = static_cast<size_t>(elem_bytes(out_dtype));
        CK(cudaMemset2DAsync(dtable, es * lddt, 0, es * cols, vocab, s));
        return GNS_OK;
    }
    EmbeddingJob j{};
    j.ids = ids;
    j.id_bytes = id_bytes;
    j.tokens = static_cast<int>(tokens);
    j.vocab = static_cast<int>(vocab);
    j.cols = static_cast<int>(cols);
    j.scale = static_cast<float>(scale);
    j.dy = dy;
    j.lddy = lddy;
    j.dtable = dtable;
    j.lddt = lddt;
    j.dtype = dtype;
    j.out_dtype = out_dtype;
    Scratch scratch;
    RET(scratch.take(*st, embedding_plan(j, nullptr).bytes, s));
    const EmbeddingPlan p = embedding_plan(j, scratch.data());
    CK(cudaMemsetAsync(p.ready, 0, p.cleared, s));
    for (int pass = 0; pass < p.passes; ++pass) {
        if (p.counts) LAUNCH(kClsEmbedding, launch_embedding_count(j, p, pass, s));
        LAUNCH(kClsEmbedding, launch_embedding_place(j, p, pass, s));
    }
    LAUNCH(kClsEmbedding, launch_embedding_runs(j, p, s));
    if (p.chunks > 1) LAUNCH(kClsEmbedding, launch_embedding_joins(j, p, s));
    return GNS_OK;
}

}  // extern "C"
