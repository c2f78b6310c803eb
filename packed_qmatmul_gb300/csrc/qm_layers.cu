// qm_layers.cu -- C entry points around a layer's products: the checks of an
// epilogue (qm_apply_fused, qm_apply_experts_fused), the choice of experts and
// the sum over a token's experts. Each refusal names the part.
#include <cuda_runtime.h>

#include <cmath>
#include <limits>
#include <string>

#include "qm.h"
#include "qm_internal.h"

namespace qm {

static bool meets(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const char* p = static_cast<const char*>(a);
    const char* q = static_cast<const char*>(b);
    return a_bytes > 0 && b_bytes > 0 && p < q + b_bytes && q < p + a_bytes;
}

// Bytes from the first to the last of `rows` rows of `n` 16-bit elements, or -1.
static int64_t span16(int64_t rows, int64_t stride, int64_t n) {
    int64_t v = 0;
    if (rows < 1 || n < 1) return 0;
    if (!mul_ok(rows - 1, stride, &v) || v > (std::numeric_limits<int64_t>::max() >> 2) - n) return -1;
    return (v + n) * 2;
}

// A residual of `rows` rows of n elements: any even address, whole rows apart or one for all.
static qm_status check_residual(const void* residual, int64_t stride, int64_t rows, int64_t n) {
    if (!residual) return QM_OK;
    if (stride < 0) return fail(QM_EINVAL, "residual: negative stride");
    if (reinterpret_cast<uintptr_t>(residual) & 1u) return fail(QM_EINVAL, "residual: misaligned");
    if (span16(rows, stride, n) < 0) return fail(QM_EINVAL, "residual: shape too large");
    return QM_OK;
}

static qm_status residual_meets(const void* residual, int64_t stride, int64_t rows, int64_t n, const void* out,
                                const std::string& name) {
    if (!residual || !meets(residual, span16(rows, stride, n), out, rows * n * 2)) return QM_OK;
    if (residual == out && (rows <= 1 || stride == n)) return QM_OK;  // each result is read where it is written
    return fail(QM_EINVAL, "residual: overlaps " + name);
}

qm_status validate_epilogue(const qm_epilogue* ep, const WDesc& w, int64_t M, Epi* e) {
    if (ep->act < QM_ACT_NONE || ep->act > QM_ACT_GELU_TANH) return fail(QM_EINVAL, "epilogue: unknown act");
    if (ep->gated != 0 && ep->gated != 1) return fail(QM_EINVAL, "epilogue: gated must be 0 or 1");
    if (ep->act == QM_ACT_SILU && !std::isfinite(ep->alpha)) return fail(QM_EINVAL, "epilogue: alpha must be finite");
    if (!(ep->limit >= 0.0f)) return fail(QM_EINVAL, "epilogue: limit must not be negative");
    if (!std::isfinite(ep->up_offset)) return fail(QM_EINVAL, "epilogue: up_offset must be finite");
    if (!ep->gated && (ep->limit != 0.0f || ep->up_offset != 0.0f))
        return fail(QM_EINVAL, "epilogue: limit and up_offset are a gate's");
    if (ep->gated && w.n % 2 != 0) return fail(QM_EINVAL, "w: a gate pairs rows, and n is odd");
    e->yn = ep->gated ? w.n / 2 : w.n;
    if (ep->bias) {
        if (ep->bias_dtype != QM_F32 && ep->bias_dtype != QM_BF16 && ep->bias_dtype != QM_F16)
            return fail(QM_EINVAL, "bias: dtype must be QM_F32, QM_BF16 or QM_F16");
        if (!aligned16(ep->bias)) return fail(QM_EINVAL, "bias: base address must be 16-byte aligned");
    }
    if (ep->residual && w.ndim != 2) return fail(QM_EINVAL, "residual: not with experts; experts_combine adds one");
    const qm_status s = check_residual(ep->residual, ep->residual_stride, M, e->yn);
    if (s != QM_OK) return s;
    e->bias = ep->bias;
    e->residual = static_cast<const uint16_t*>(ep->residual);
    e->residual_stride = ep->residual_stride;
    e->bias_dtype = ep->bias_dtype;
    e->act = ep->act;
    e->gated = ep->gated;
    e->alpha = ep->alpha == 0.0f ? 1.0f : ep->alpha;
    e->limit = ep->limit == 0.0f ? std::numeric_limits<float>::infinity() : ep->limit;
    e->up_offset = ep->up_offset;
    e->on = e->bias || e->residual || e->act != QM_ACT_NONE || e->gated;
    return QM_OK;
}

qm_status check_epilogue_overlap(const Epi& e, const WDesc& w, int64_t M, const void* y) {
    if (e.bias && meets(e.bias, w.rows * (e.bias_dtype == QM_F32 ? 4 : 2), y, M * e.yn * 2))
        return fail(QM_EINVAL, "bias: overlaps y");
    return residual_meets(e.residual, e.residual_stride, M, e.yn, y, "y");
}

}  // namespace qm

using namespace qm;

extern "C" {

qm_status qm_experts_select(const qm_router* r, const void* logits, int32_t logits_dtype, int64_t logits_stride,
                            int64_t T, int32_t* ids, float* weights, qm_stream_t stream) {
    set_error("");
    if (!r) return fail(QM_EINVAL, "router: NULL");
    if (r->experts < 1 || r->experts > QM_MAX_EXPERTS)
        return fail(QM_EINVAL, "router: experts must be 1 .. " + std::to_string(QM_MAX_EXPERTS));
    if (r->topk < 1 || r->topk > QM_MAX_TOPK || r->topk > r->experts)
        return fail(QM_EINVAL, "router: topk must be 1 .. " + std::to_string(QM_MAX_TOPK) + " and at most experts");
    if (r->score != QM_SCORE_SOFTMAX && r->score != QM_SCORE_SIGMOID)
        return fail(QM_EINVAL, "router: score must be QM_SCORE_SOFTMAX or QM_SCORE_SIGMOID");
    if (r->groups < 1 || r->groups > QM_MAX_GROUPS || r->experts % r->groups != 0)
        return fail(QM_EINVAL, "router: groups must be 1 .. " + std::to_string(QM_MAX_GROUPS) + " and divide experts");
    if (r->topk_groups < 1 || r->topk_groups > r->groups) return fail(QM_EINVAL, "router: topk_groups must be 1 .. groups");
    if (r->group_score != QM_GROUP_MAX && r->group_score != QM_GROUP_TOP2)
        return fail(QM_EINVAL, "router: group_score must be QM_GROUP_MAX or QM_GROUP_TOP2");
    if (r->groups > 1 && r->group_score == QM_GROUP_TOP2 && r->experts / r->groups < 2)
        return fail(QM_EINVAL, "router: QM_GROUP_TOP2 needs two experts to a group");
    if (r->renormalize != 0 && r->renormalize != 1) return fail(QM_EINVAL, "router: renormalize must be 0 or 1");
    if (!std::isfinite(r->scale)) return fail(QM_EINVAL, "router: scale must be finite");
    if (reinterpret_cast<uintptr_t>(r->bias) & 3u) return fail(QM_EINVAL, "bias: misaligned");
    if (logits_dtype != QM_F32 && logits_dtype != QM_BF16 && logits_dtype != QM_F16)
        return fail(QM_EINVAL, "logits: dtype must be QM_F32, QM_BF16 or QM_F16");
    if (T < 0 || T > std::numeric_limits<int32_t>::max()) return fail(QM_EINVAL, "logits: T must be 0 .. 2^31-1");
    if (logits_stride < 0) return fail(QM_EINVAL, "logits: negative stride");
    if (T == 0) return QM_OK;
    if (!logits) return fail(QM_EINVAL, "logits: NULL");
    if (reinterpret_cast<uintptr_t>(logits) & (logits_dtype == QM_F32 ? 3u : 1u)) return fail(QM_EINVAL, "logits: misaligned");
    const int64_t span = span16(T, logits_stride, r->experts);
    if (span < 0) return fail(QM_EINVAL, "logits: shape too large");
    if (!ids) return fail(QM_EINVAL, "ids: NULL");
    if (!weights) return fail(QM_EINVAL, "weights: NULL");
    if (reinterpret_cast<uintptr_t>(ids) & 3u) return fail(QM_EINVAL, "ids: misaligned");
    if (reinterpret_cast<uintptr_t>(weights) & 3u) return fail(QM_EINVAL, "weights: misaligned");
    const int64_t out = T * r->topk * 4, in = span * (logits_dtype == QM_F32 ? 2 : 1);
    if (meets(ids, out, weights, out)) return fail(QM_EINVAL, "ids: overlaps weights");
    if (meets(ids, out, logits, in) || meets(weights, out, logits, in)) return fail(QM_EINVAL, "logits: overlaps an output");
    if (meets(ids, out, r->bias, r->bias ? r->experts * 4 : 0) || meets(weights, out, r->bias, r->bias ? r->experts * 4 : 0))
        return fail(QM_EINVAL, "bias: overlaps an output");
    return check_launch(launch_experts_select(*r, logits, logits_dtype, logits_stride, T, ids, weights,
                                              reinterpret_cast<cudaStream_t>(stream)),
                        "select launch");
}

qm_status qm_experts_combine(const void* y, const float* weights, int64_t T, int64_t topk, int64_t n, int32_t dtype,
                             const void* residual, int64_t residual_stride, void* out, qm_stream_t stream) {
    set_error("");
    if (dtype != QM_BF16) return fail(QM_ENOTSUP, "y: experts_combine takes bfloat16 rows");
    if (T < 0 || topk < 0 || n < 0) return fail(QM_EINVAL, "y: negative shape");
    int64_t rows = 0, all = 0;
    if (!mul_ok(T, topk, &rows) || !mul_ok(rows, n, &all) || all > (std::numeric_limits<int64_t>::max() >> 2))
        return fail(QM_EINVAL, "y: shape too large");
    if (!mul_ok(T, n, &all) || all > (std::numeric_limits<int64_t>::max() >> 2)) return fail(QM_EINVAL, "out: shape too large");
    if (topk > std::numeric_limits<int32_t>::max() - 8) return fail(QM_EINVAL, "y: topk too large");
    const qm_status s = check_residual(residual, residual_stride, T, n);
    if (s != QM_OK) return s;
    if (T == 0 || n == 0) return QM_OK;
    if (!out) return fail(QM_EINVAL, "out: NULL");
    if (!aligned16(out)) return fail(QM_EINVAL, "out: base address must be 16-byte aligned");
    if (topk > 0) {
        if (!y) return fail(QM_EINVAL, "y: NULL");
        if (!aligned16(y)) return fail(QM_EINVAL, "y: base address must be 16-byte aligned");
        if (!weights) return fail(QM_EINVAL, "weights: NULL");
        if (reinterpret_cast<uintptr_t>(weights) & 3u) return fail(QM_EINVAL, "weights: misaligned");
        if (meets(y, rows * n * 2, out, T * n * 2)) return fail(QM_EINVAL, "out: overlaps y");
        if (meets(weights, rows * 4, out, T * n * 2)) return fail(QM_EINVAL, "out: overlaps weights");
    }
    const qm_status o = residual_meets(residual, residual_stride, T, n, out, "out");
    if (o != QM_OK) return o;
    return check_launch(launch_experts_combine(y, weights, T, topk, n, residual, residual_stride, out,
                                               reinterpret_cast<cudaStream_t>(stream)),
                        "combine launch");
}

}  // extern "C"
