// qm_cache.cu -- C entry points of the operators around a paged key/value
// cache: host-side validation (each refusal names the part) and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <limits>
#include <string>

#include "qm.h"
#include "qm_internal.h"

namespace qm {

static const int64_t kMaxI32 = std::numeric_limits<int32_t>::max();

static const int64_t kMaxPieces = int64_t(0xFFFFFFFE) * 16;  // in bytes

static bool float16ish(int32_t dt) { return dt == QM_BF16 || dt == QM_F16; }

static qm_status check_heads(const qm_heads* x, const std::string& name, int64_t tokens) {
    const bool live = tokens > 0;
    if (!x) return fail(QM_EINVAL, name + ": NULL");
    if (x->heads < 1) return fail(QM_EINVAL, name + ": needs at least one head");
    if (!float16ish(x->dtype)) return fail(QM_EINVAL, name + ": dtype must be QM_BF16 or QM_F16");
    if (x->token_stride < 0 || x->head_stride < 0) return fail(QM_EINVAL, name + ": negative stride");
    if ((tokens > 1 && x->token_stride % 8 != 0) || (x->heads > 1 && x->head_stride % 8 != 0))  // an axis of one has none
        return fail(QM_EINVAL, name + ": strides must be multiples of 8 elements");
    if (live && !x->data) return fail(QM_EINVAL, name + ": NULL");
    if (live && !aligned16(x->data)) return fail(QM_EINVAL, name + ": base address must be 16-byte aligned");
    return QM_OK;
}

// Rows that are written: two of them must not meet.
static qm_status check_written(const qm_heads& x, const std::string& name, int64_t tokens, int dim) {
    if ((x.heads > 1 && x.head_stride < dim) || (tokens > 1 && x.token_stride < dim))
        return fail(QM_EINVAL, name + ": strides make rows overlap");
    return QM_OK;
}

static qm_status check_rope(const qm_rope* rope, int dim) {
    if (!rope) return QM_OK;
    if (rope->style != QM_ROPE_HALF && rope->style != QM_ROPE_PAIRS)
        return fail(QM_EINVAL, "rope: style must be QM_ROPE_HALF or QM_ROPE_PAIRS");
    if (rope->dim < 8 || rope->dim % 8 != 0 || rope->dim > dim)
        return fail(QM_EINVAL, "rope: dim must be a multiple of 8, from 8 to the head's dim");
    if (rope->rows < 0) return fail(QM_EINVAL, "rope: negative rows");
    if (rope->rows > 0 && !rope->table) return fail(QM_EINVAL, "rope: table is NULL");
    if (!aligned16(rope->table)) return fail(QM_EINVAL, "rope: table must be 16-byte aligned");
    return QM_OK;
}

static qm_status check_eps(float eps) {
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(QM_EINVAL, "eps: must be finite and not negative");
    return QM_OK;
}

static qm_status check_cache(const qm_cache* c) {
    if (!c) return fail(QM_EINVAL, "cache: NULL");
    if (!float16ish(c->dtype) && c->dtype != QM_I8)
        return fail(QM_EINVAL, "cache: dtype must be QM_BF16, QM_F16 or QM_I8");
    const bool i8 = c->dtype == QM_I8;
    const int step = i8 ? 16 : 8;
    if (c->dim < step || c->dim % step != 0)
        return fail(QM_EINVAL, "cache: dim must be a multiple of " + std::to_string(step));
    if (c->dim > 128) return fail(QM_ENOTSUP, "cache: dim is at most 128");
    if (c->heads < 1) return fail(QM_EINVAL, "cache: needs at least one head");
    if (c->page_size < 1) return fail(QM_EINVAL, "cache: page_size must be at least 1");
    if (c->pages < 0 || c->pages > kMaxI32) return fail(QM_EINVAL, "cache: pages must be 0 .. 2^31-1");
    if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < 0)
        return fail(QM_EINVAL, "cache: negative stride");
    if ((c->pages > 1 && c->page_stride % step != 0) || (c->heads > 1 && c->head_stride % step != 0) ||
        (c->page_size > 1 && c->token_stride % step != 0))
        return fail(QM_EINVAL, "cache: strides must be multiples of " + std::to_string(step) + " elements");
    if ((c->pages > 1 && c->page_stride < c->dim) || (c->heads > 1 && c->head_stride < c->dim) ||
        (c->page_size > 1 && c->token_stride < c->dim))
        return fail(QM_EINVAL, "cache: strides make rows overlap");
    if (c->pages > 0) {
        if (!c->k) return fail(QM_EINVAL, "k: cache has no keys (NULL)");
        if (!c->v) return fail(QM_EINVAL, "v: cache has no values (NULL)");
        if (!aligned16(c->k)) return fail(QM_EINVAL, "k: base address must be 16-byte aligned");
        if (!aligned16(c->v)) return fail(QM_EINVAL, "v: base address must be 16-byte aligned");
    }
    // the kernels count a part's 16-byte pieces in 32 bits
    int64_t pg = 0, hd = 0, tk = 0;
    if (c->pages > 0 && (!mul_ok(c->pages - 1, c->page_stride, &pg) || !mul_ok(c->heads - 1, c->head_stride, &hd) ||
                         !mul_ok(c->page_size - 1, c->token_stride, &tk) || pg > kMaxPieces || hd > kMaxPieces || tk > kMaxPieces ||
                         pg + hd + tk + c->dim > kMaxPieces / (i8 ? 1 : 2)))
        return fail(QM_ENOTSUP, "cache: k and v may span at most 64 GB each");
    if (i8) {
        if (c->scale_page_stride < 0 || c->scale_head_stride < 0 || c->scale_token_stride < 0)
            return fail(QM_EINVAL, "k_scales: negative stride");
        if (c->pages > 0) {
            if (!c->k_scales) return fail(QM_EINVAL, "k_scales: NULL");
            if (!c->v_scales) return fail(QM_EINVAL, "v_scales: NULL");
            if (reinterpret_cast<uintptr_t>(c->k_scales) & 3u) return fail(QM_EINVAL, "k_scales: misaligned");
            if (reinterpret_cast<uintptr_t>(c->v_scales) & 3u) return fail(QM_EINVAL, "v_scales: misaligned");
        }
    } else {
        if (c->k_scales) return fail(QM_EINVAL, "k_scales: only a QM_I8 cache has scales; pass NULL");
        if (c->v_scales) return fail(QM_EINVAL, "v_scales: only a QM_I8 cache has scales; pass NULL");
    }
    return QM_OK;
}

static qm_status check_batch(const qm_batch* b) {
    if (!b) return fail(QM_EINVAL, "batch: NULL");
    if (b->seqs < 0) return fail(QM_EINVAL, "batch: negative seqs");
    if (b->tokens < 0 || b->tokens > kMaxI32) return fail(QM_EINVAL, "batch: tokens must be 0 .. 2^31-1");
    if (b->max_new < 0) return fail(QM_EINVAL, "batch: negative max_new");
    if (b->table_width < 0 || b->table_stride < 0) return fail(QM_EINVAL, "page_table: negative shape");
    if (b->tokens == 0 || b->seqs == 0) return QM_OK;
    if (!b->q_offsets && b->tokens % b->seqs != 0)
        return fail(QM_EINVAL, "q_offsets: NULL needs tokens to be a multiple of seqs");
    if (!b->lens) return fail(QM_EINVAL, "lens: NULL");
    if (b->table_width > 0 && !b->page_table) return fail(QM_EINVAL, "page_table: NULL");
    const void* arrays[3] = {b->lens, b->page_table, b->q_offsets};
    const char* names[3] = {"lens", "page_table", "q_offsets"};
    for (int i = 0; i < 3; ++i)
        if (reinterpret_cast<uintptr_t>(arrays[i]) & 3u) return fail(QM_EINVAL, std::string(names[i]) + ": misaligned");
    return QM_OK;
}

}  // namespace qm

using namespace qm;

extern "C" {

qm_status qm_head_norm_rope(const qm_heads* xs, const qm_heads* outs, const void* const* weights, int32_t count,
                            int64_t tokens, int32_t dim, float eps, const qm_rope* rope, const void* positions,
                            int32_t pos_type, qm_stream_t stream) {
    set_error("");
    if (count < 1 || count > QM_MAX_HEAD_SETS) return fail(QM_EINVAL, "count: must be 1 .. QM_MAX_HEAD_SETS");
    if (!xs) return fail(QM_EINVAL, "x: NULL");
    if (!outs) return fail(QM_EINVAL, "out: NULL");
    if (tokens < 0 || tokens > kMaxI32) return fail(QM_EINVAL, "x: tokens must be 0 .. 2^31-1");
    if (dim < 8 || dim % 8 != 0) return fail(QM_EINVAL, "x: dim must be a multiple of 8");
    if (dim > 256) return fail(QM_ENOTSUP, "x: dim is at most 256");
    qm_status s = check_eps(eps);
    if (s != QM_OK) return s;
    s = check_rope(rope, dim);
    if (s != QM_OK) return s;
    for (int i = 0; i < count; ++i) {
        const std::string at = "[" + std::to_string(i) + "]";
        if ((s = check_heads(&xs[i], "x" + at, tokens)) != QM_OK) return s;
        if ((s = check_heads(&outs[i], "out" + at, tokens)) != QM_OK) return s;
        if ((s = check_written(outs[i], "out" + at, tokens, dim)) != QM_OK) return s;
        if (xs[i].dtype != xs[0].dtype) return fail(QM_EINVAL, "x" + at + ": dtype differs from x[0]");
        if (outs[i].dtype != xs[i].dtype) return fail(QM_EINVAL, "out" + at + ": dtype differs from x" + at);
        if (outs[i].heads != xs[i].heads) return fail(QM_EINVAL, "out" + at + ": heads differ from x" + at);
        if (outs[i].data == xs[i].data && tokens > 0 &&
            (outs[i].token_stride != xs[i].token_stride || outs[i].head_stride != xs[i].head_stride))
            return fail(QM_EINVAL, "out" + at + ": shares x" + at + "'s address with other strides");
        if (weights && weights[i] && !aligned16(weights[i]))
            return fail(QM_EINVAL, "weights" + at + ": must be 16-byte aligned");
    }
    if (tokens == 0) return QM_OK;
    if (rope) {
        if (pos_type != QM_I32 && pos_type != QM_I64)
            return fail(QM_EINVAL, "positions: pos_type must be QM_I32 or QM_I64");
        if (!positions) return fail(QM_EINVAL, "positions: NULL");
        if (reinterpret_cast<uintptr_t>(positions) & (pos_type == QM_I64 ? 7u : 3u))
            return fail(QM_EINVAL, "positions: misaligned");
    }
    return check_launch(launch_head_norm_rope(xs, outs, weights, count, tokens, dim, eps, rope, positions,
                                              pos_type == QM_I64, reinterpret_cast<cudaStream_t>(stream)),
                        "head_norm_rope launch");
}

qm_status qm_cache_append(const qm_cache* cache, const qm_batch* batch, const qm_heads* k, const qm_heads* v,
                          const void* k_weight, float eps, const qm_rope* rope, qm_stream_t stream) {
    set_error("");
    qm_status s = check_cache(cache);
    if (s != QM_OK) return s;
    if ((s = check_batch(batch)) != QM_OK) return s;
    if ((s = check_eps(eps)) != QM_OK) return s;
    if ((s = check_rope(rope, cache->dim)) != QM_OK) return s;
    const bool live = batch->tokens > 0 && batch->seqs > 0;
    if ((s = check_heads(k, "k", live ? batch->tokens : 0)) != QM_OK) return s;
    if ((s = check_heads(v, "v", live ? batch->tokens : 0)) != QM_OK) return s;
    if (k->heads != cache->heads) return fail(QM_EINVAL, "k: heads differ from the cache's");
    if (v->heads != cache->heads) return fail(QM_EINVAL, "v: heads differ from the cache's");
    if (v->dtype != k->dtype) return fail(QM_EINVAL, "v: dtype differs from k's");
    if (cache->dtype != QM_I8 && k->dtype != cache->dtype) return fail(QM_EINVAL, "k: dtype differs from the cache's");
    if (!aligned16(k_weight)) return fail(QM_EINVAL, "k_weight: must be 16-byte aligned");
    if (!live || cache->pages == 0 || batch->table_width == 0) return QM_OK;
    return check_launch(launch_cache_append(*cache, *batch, *k, *v, k_weight, eps, rope,
                                            reinterpret_cast<cudaStream_t>(stream)),
                        "cache_append launch");
}

size_t qm_cache_attend_workspace(const qm_cache* cache, const qm_batch* batch, int32_t q_heads) {
    set_error("");
    if (check_cache(cache) != QM_OK || check_batch(batch) != QM_OK || q_heads < 1 || q_heads % cache->heads != 0 ||
        batch->tokens == 0 || batch->seqs == 0)
        return 0;
    return attend_workspace_bytes(*cache, *batch, q_heads);
}

qm_status qm_cache_attend(const qm_cache* cache, const qm_batch* batch, const qm_heads* q, const qm_heads* out,
                          float* lse, float scale, int64_t window, void* workspace, size_t workspace_bytes,
                          qm_stream_t stream) {
    set_error("");
    qm_status s = check_cache(cache);
    if (s != QM_OK) return s;
    if ((s = check_batch(batch)) != QM_OK) return s;
    const bool live = batch->tokens > 0 && batch->seqs > 0;
    if ((s = check_heads(q, "q", live ? batch->tokens : 0)) != QM_OK) return s;
    if ((s = check_heads(out, "out", live ? batch->tokens : 0)) != QM_OK) return s;
    if (q->heads % cache->heads != 0) return fail(QM_EINVAL, "q: heads must be a multiple of the cache's");
    if (q->heads / cache->heads > 32768) return fail(QM_ENOTSUP, "q: at most 32768 query heads to a key head");
    if (cache->dtype != QM_I8 && q->dtype != cache->dtype) return fail(QM_EINVAL, "q: dtype differs from the cache's");
    if (out->heads != q->heads) return fail(QM_EINVAL, "out: heads differ from q's");
    if (out->dtype != q->dtype) return fail(QM_EINVAL, "out: dtype differs from q's");
    if ((s = check_written(*out, "out", batch->tokens, cache->dim)) != QM_OK) return s;
    if (live && out->data == q->data) return fail(QM_EINVAL, "out: shares q's address");
    int64_t rows = 0;
    if (!mul_ok(batch->tokens, q->heads, &rows) || rows > kMaxI32)
        return fail(QM_EINVAL, "q: more than 2^31-1 rows of heads");
    if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(QM_EINVAL, "lse: misaligned");
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(QM_EINVAL, "scale: must be finite and above 0");
    if (window < 0) return fail(QM_EINVAL, "window: negative");
    if (!live) return QM_OK;
    const size_t need = attend_workspace_bytes(*cache, *batch, q->heads);
    if (!workspace || workspace_bytes < need)
        return fail(QM_EINVAL, "workspace: needs " + std::to_string(need) + " bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 31u) return fail(QM_EINVAL, "workspace: must be 32-byte aligned");
    return check_launch(launch_cache_attend(*cache, *batch, *q, *out, lse, scale, window, workspace,
                                            reinterpret_cast<cudaStream_t>(stream)),
                        "cache_attend launch");
}

}  // extern "C"
