// C ABI of the rotary positions, the paged key/value cache and attention over
// it: argument validation and dispatch.  Every check runs on the host before
// anything is enqueued.
#include "kv_checks.h"

using namespace q4::check;

namespace {

// What a norm of heads asks for beside the rotation; null where there is none.
struct Norm {
    const void* gain[2];
    int type;
    float eps;
};

q4_status check_norm(const char* fn, const Norm& n) {
    if (!(n.eps >= 0.0f) || !std::isfinite(n.eps)) return fail(Q4_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    if (!n.gain[0] && !n.gain[1]) return Q4_OK;
    const int b = type_bytes(n.type);
    if (!b) return fail(Q4_ERR_INVALID_ARG, "%s: the gains have an unknown type %d", fn, n.type);
    if (!aligned(n.gain[0], b) || !aligned(n.gain[1], b)) return fail(Q4_ERR_MISALIGNED, "%s: the gains must be aligned to their elements", fn);
    return Q4_OK;
}

Span gain_span(const Norm* n, int which, int dim) {
    return n && n->gain[which] ? span(n->gain[which], (uint64_t)dim * type_bytes(n->type)) : Span{0, 0};
}

q4_status launch_heads(const q4::RopeArgs& a, const Norm* norm, int in_type, int out_type, int layout, void* stream, const char* what) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (!norm) return hip_status(q4::launch_rope(a, in_type, out_type, layout, s), what);
    q4::NormRopeArgs n = {};
    n.rope = a;
    for (int i = 0; i < 2; ++i) n.gain[i] = static_cast<const char*>(norm->gain[i]);
    n.gain_type = norm->type;
    n.eps = norm->eps;
    return hip_status(q4::launch_norm_rope(n, in_type, out_type, layout, s), what);
}

q4_status rope(const char* fn, const char* what, const q4_heads* x, const q4_heads* out, const Norm* norm, const int32_t* positions,
               const double* inv_freq, int64_t tokens, int heads, int head_dim, int rot_dim, int layout, float mscale, void* stream) {
    q4_status st = check_sizes(fn, tokens, heads, head_dim);
    if (st) return st;
    st = check_rotation(fn, inv_freq, rot_dim, head_dim, layout, mscale);
    if (st) return st;
    if (!norm && rot_dim < 2) return fail(Q4_ERR_INVALID_ARG, "%s: rot_dim must be at least 2", fn);
    if (norm && (st = check_norm(fn, *norm))) return st;
    st = check_heads(fn, "x", x, tokens, heads, head_dim, false);
    if (st) return st;
    st = check_heads(fn, "out", out, tokens, heads, head_dim, true);
    if (st) return st;
    if (rot_dim && !positions) return fail(Q4_ERR_INVALID_ARG, "%s: null positions", fn);
    if (!aligned(positions, 4)) return fail(Q4_ERR_MISALIGNED, "%s: positions must be 4-byte aligned", fn);
    const Rows ro = rows_of(*out, tokens, heads, head_dim);
    if (!same(*x, *out) && overlap(ro, rows_of(*x, tokens, heads, head_dim)))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps x without being x", fn);
    if (overlap(ro.all, span(positions, positions ? 4 * (uint64_t)tokens : 0)) || overlap(ro.all, span(inv_freq, 4 * (uint64_t)rot_dim)))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps positions or inv_freq", fn);
    if (overlap(ro.all, gain_span(norm, 0, head_dim))) return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps the gain", fn);
    q4::RopeArgs a = {};
    a.in[0] = heads_arg(*x, tokens, heads);
    a.out = heads_arg(*out, tokens, heads);
    a.heads[0] = heads;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.tokens = tokens;
    a.head_dim = head_dim;
    a.rot_dim = rot_dim;
    a.mscale = mscale;
    return launch_heads(a, norm, x->type, out->type, layout, stream, what);
}

q4_status append(const char* fn, const char* what, const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* k, const q4_heads* v,
                 const q4_heads* q, const q4_heads* q_out, int q_heads, int64_t tokens, const Norm* norm, const int32_t* positions,
                 const double* inv_freq, int rot_dim, int layout, float mscale, void* stream) {
    q4_status st = check_cache(fn, cache);
    if (st) return st;
    st = check_batch(fn, batch, cache);
    if (st) return st;
    const int dim = cache->head_dim;
    st = check_sizes(fn, tokens, q ? q_heads : 1, dim);
    if (st) return st;
    st = check_rotation(fn, inv_freq, rot_dim, dim, layout, mscale);
    if (st) return st;
    if (norm && (st = check_norm(fn, *norm))) return st;
    st = check_heads(fn, "k", k, tokens, cache->kv_heads, dim, false);
    if (st) return st;
    st = check_heads(fn, "v", v, tokens, cache->kv_heads, dim, false);
    if (st) return st;
    Axis ak[3], av[3];
    const int nk = cache_axes(cache, false, ak), nv = cache_axes(cache, true, av);
    if (!axes_nest(ak, nk, dim) || !axes_nest(av, nv, dim))
        return fail(Q4_ERR_INVALID_ARG, "%s: the heads of the cache overlap each other", fn);
    if (blocks_meet(ak, nk, av, nv, dim, (int64_t)((intptr_t)cache->v - (intptr_t)cache->k) / 2))
        return fail(Q4_ERR_INVALID_ARG, "%s: the cache's keys and values are the same memory, or parts of them", fn);
    if (k->type != v->type || (q && q->type != k->type)) return fail(Q4_ERR_INVALID_ARG, "%s: q, k and v must have one type", fn);
    if (!q != !q_out) return fail(Q4_ERR_INVALID_ARG, "%s: q and q_out go together", fn);
    if (!aligned(positions, 4)) return fail(Q4_ERR_MISALIGNED, "%s: positions must be 4-byte aligned", fn);
    const Rows rk = rows_of(*k, tokens, cache->kv_heads, dim), rv = rows_of(*v, tokens, cache->kv_heads, dim);
    const Span ck = cache_span(cache, false), cv = cache_span(cache, true);
    const Span read[4] = {span(positions, positions ? 4 * (uint64_t)tokens : 0), span(inv_freq, rot_dim ? 4 * (uint64_t)rot_dim : 0),
                          gain_span(norm, 0, dim), gain_span(norm, 1, dim)};
    if (q) {
        st = check_heads(fn, "q", q, tokens, q_heads, dim, false);
        if (st) return st;
        st = check_heads(fn, "q_out", q_out, tokens, q_heads, dim, true);
        if (st) return st;
        if (q_out->type != cache->type) return fail(Q4_ERR_INVALID_ARG, "%s: q_out must have the cache's type", fn);
        const Rows rq = rows_of(*q, tokens, q_heads, dim), ro = rows_of(*q_out, tokens, q_heads, dim);
        if ((!same(*q, *q_out) && overlap(ro, rq)) || overlap(ro, rk) || overlap(ro, rv) || overlap(ro.all, read[0]) ||
            overlap(ro.all, read[1]) || overlap(ro.all, read[2]) || overlap(ro.all, read[3]) || overlaps_batch(ro.all, batch) || overlap(ro.all, ck) || overlap(ro.all, cv))
            return fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps another tensor (or q without being q)", fn);
        if (overlap(rq.all, ck) || overlap(rq.all, cv)) return fail(Q4_ERR_INVALID_ARG, "%s: q overlaps the cache", fn);
    }
    for (const Span& c : {ck, cv})
        if (overlap(c, rk.all) || overlap(c, rv.all) || overlap(c, read[0]) || overlap(c, read[1]) || overlap(c, read[2]) ||
            overlap(c, read[3]) || overlaps_batch(c, batch))
            return fail(Q4_ERR_INVALID_ARG, "%s: the cache overlaps an input", fn);
    q4::RopeArgs a = {};
    if (q) {
        a.in[0] = heads_arg(*q, tokens, q_heads);
        a.out = heads_arg(*q_out, tokens, q_heads);
        a.heads[0] = q_heads;
    }
    a.in[1] = heads_arg(*k, tokens, cache->kv_heads);
    a.in[2] = heads_arg(*v, tokens, cache->kv_heads);
    a.heads[1] = a.heads[2] = cache->kv_heads;
    a.paged = 1;
    a.cache = cache_arg(*cache);
    a.batch = batch_arg(*batch);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.tokens = tokens;
    a.head_dim = dim;
    a.rot_dim = rot_dim;
    a.mscale = mscale;
    return launch_heads(a, norm, k->type, cache->type, layout, stream, what);
}

// Attention of new tokens over the cache, causal or, with a mask, over trees of them.
q4_status attention(const char* fn, const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* q, const q4_heads* out,
                    const uint64_t* mask, int mask_words, float* lse, int q_heads, int64_t tokens, float scale, int64_t window,
                    void* workspace, size_t workspace_bytes, void* stream) {
    q4_status st = check_attention(fn, cache, batch, q_heads, tokens, window);
    if (st) return st;
    const int dim = cache->head_dim;
    st = check_heads(fn, "q", q, tokens, q_heads, dim, false);
    if (st) return st;
    st = check_heads(fn, "out", out, tokens, q_heads, dim, true);
    if (st) return st;
    if (q->type != cache->type || out->type != cache->type) return fail(Q4_ERR_INVALID_ARG, "%s: q and out must have the cache's type", fn);
    const q4::HeadsArg qa = heads_arg(*q, tokens, q_heads), oa = heads_arg(*out, tokens, q_heads);
    if (!aligned(qa.data, 16) || !aligned(oa.data, 16) || (qa.token_stride | qa.head_stride | oa.token_stride | oa.head_stride) % 8)
        return fail(Q4_ERR_MISALIGNED, "%s: q and out must be 16-byte aligned with strides that are multiples of 8", fn);
    if (!aligned(lse, 4)) return fail(Q4_ERR_MISALIGNED, "%s: lse must be 4-byte aligned", fn);
    if (!(scale > 0.0f) || !std::isfinite(scale) || !std::isfinite(scale * 1.4426950408889634f))
        return fail(Q4_ERR_INVALID_ARG, "%s: scale must be finite and > 0", fn);
    const q4::CacheArg c = cache_arg(*cache);
    const q4::BatchArg b = batch_arg(*batch);
    const q4::AttnShape shape = q4::attn_shape(c, b, q_heads, tokens, window_arg(window), batch->max_query, batch->max_context, mask != nullptr);
    if (shape.bytes) {
        if (!workspace || workspace_bytes < shape.bytes) return fail(Q4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, shape.bytes);
        if (!aligned(workspace, 16)) return fail(Q4_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    }
    const Rows rq = rows_of(*q, tokens, q_heads, dim), ro = rows_of(*out, tokens, q_heads, dim);
    const Span written[3] = {ro.all, span(lse, lse ? 4 * (uint64_t)tokens * q_heads : 0), span(workspace, shape.bytes)};
    const Span read[3] = {rq.all, cache_span(cache, false), cache_span(cache, true)};
    for (int i = 0; i < 3; ++i) {
        if (written[i].lo == written[i].hi) continue;
        if (overlap(written[i], span(mask, mask ? 8 * (uint64_t)tokens * mask_words : 0)))
            return fail(Q4_ERR_INVALID_ARG, "%s: an output or the workspace overlaps the mask", fn);
        for (int j = 0; j < 3; ++j)
            if (i == 0 && j == 0 ? overlap(ro, rq) : overlap(written[i], read[j]))
                return fail(Q4_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", fn);
        if (overlaps_batch(written[i], batch)) return fail(Q4_ERR_INVALID_ARG, "%s: an output or the workspace overlaps the batch", fn);
        for (int j = i + 1; j < 3; ++j)
            if (written[j].lo != written[j].hi && overlap(written[i], written[j]))
                return fail(Q4_ERR_INVALID_ARG, "%s: outputs and workspace must not overlap", fn);
    }
    q4::TreeArgs a = {};
    a.q = qa;
    a.out = oa;
    a.lse = lse;
    a.cache = c;
    a.batch = b;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.window = window_arg(window);
    a.workspace = workspace;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (!mask) return hip_status(q4::launch_attention(a, shape, cache->type, s), "q4_attention_paged launch");
    a.mask = mask;
    a.mask_words = mask_words;
    return hip_status(q4::launch_attention_tree(a, shape, cache->type, s), "q4_attention_tree launch");
}

}  // namespace

extern "C" {

q4_status q4_rope(const q4_heads* x, const q4_heads* out, const int32_t* positions, const double* inv_freq,
                  int64_t tokens, int heads, int head_dim, int rot_dim, int layout, float mscale, void* stream) {
    return rope("q4_rope", "q4_rope launch", x, out, nullptr, positions, inv_freq, tokens, heads, head_dim, rot_dim, layout, mscale, stream);
}

q4_status q4_norm_rope(const q4_heads* x, const q4_heads* out, const void* gain, int gain_type, float eps, const int32_t* positions,
                       const double* inv_freq, int64_t tokens, int heads, int head_dim, int rot_dim, int layout, float mscale,
                       void* stream) {
    const Norm norm = {{gain, nullptr}, gain_type, eps};
    return rope("q4_norm_rope", "q4_norm_rope launch", x, out, &norm, positions, inv_freq, tokens, heads, head_dim, rot_dim, layout, mscale,
                stream);
}

q4_status q4_kv_append(const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* k, const q4_heads* v,
                       const q4_heads* q, const q4_heads* q_out, int q_heads, int64_t tokens, const int32_t* positions,
                       const double* inv_freq, int rot_dim, int layout, float mscale, void* stream) {
    return append("q4_kv_append", "q4_kv_append launch", cache, batch, k, v, q, q_out, q_heads, tokens, nullptr, positions, inv_freq, rot_dim,
                  layout, mscale, stream);
}

q4_status q4_kv_append_norm(const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* k, const q4_heads* v,
                            const q4_heads* q, const q4_heads* q_out, int q_heads, int64_t tokens, const void* q_gain,
                            const void* k_gain, int gain_type, float eps, const int32_t* positions, const double* inv_freq,
                            int rot_dim, int layout, float mscale, void* stream) {
    const Norm norm = {{q_gain, k_gain}, gain_type, eps};
    return append("q4_kv_append_norm", "q4_kv_append_norm launch", cache, batch, k, v, q, q_out, q_heads, tokens, &norm, positions, inv_freq,
                  rot_dim, layout, mscale, stream);
}

size_t q4_attention_paged_workspace_bytes(const q4_kv_cache* cache, const q4_kv_batch* batch, int q_heads, int64_t tokens,
                                          int64_t window) {
    if (check_attention("q4_attention_paged_workspace_bytes", cache, batch, q_heads, tokens, window)) return 0;
    ok();
    return q4::attn_shape(cache_arg(*cache), batch_arg(*batch), q_heads, tokens, window_arg(window), batch->max_query, batch->max_context).bytes;
}

size_t q4_attention_tree_workspace_bytes(const q4_kv_cache* cache, const q4_kv_batch* batch, int q_heads, int64_t tokens,
                                         int64_t window) {
    if (check_attention("q4_attention_tree_workspace_bytes", cache, batch, q_heads, tokens, window)) return 0;
    ok();
    return q4::attn_shape(cache_arg(*cache), batch_arg(*batch), q_heads, tokens, window_arg(window), batch->max_query, batch->max_context, true).bytes;
}

size_t q4_attention_workspace_most(const q4_kv_cache* cache, int q_heads, int64_t tokens) {
    const char* fn = "q4_attention_workspace_most";
    if (check_cache(fn, cache) || check_attention_sizes(fn, cache, q_heads, tokens)) return 0;
    ok();
    return q4::attn_most_bytes(cache->head_dim, tokens * (q_heads / cache->kv_heads));
}

q4_status q4_attention_paged(const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* q, const q4_heads* out,
                             float* lse, int q_heads, int64_t tokens, float scale, int64_t window, void* workspace,
                             size_t workspace_bytes, void* stream) {
    return attention("q4_attention_paged", cache, batch, q, out, nullptr, 0, lse, q_heads, tokens, scale, window, workspace, workspace_bytes,
                     stream);
}

q4_status q4_attention_tree(const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* q, const q4_heads* out,
                            const uint64_t* mask, int mask_words, float* lse, int q_heads, int64_t tokens, float scale,
                            int64_t window, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "q4_attention_tree";
    if (!mask) return fail(Q4_ERR_INVALID_ARG, "%s: null mask", fn);
    if (!aligned(mask, 8)) return fail(Q4_ERR_MISALIGNED, "%s: mask must be 8-byte aligned", fn);
    if (mask_words < 1 || mask_words > 16) return fail(Q4_ERR_INVALID_ARG, "%s: mask_words = %d outside [1, 16]", fn, mask_words);
    return attention(fn, cache, batch, q, out, mask, mask_words, lse, q_heads, tokens, scale, window, workspace, workspace_bytes, stream);
}

}  // extern "C"
