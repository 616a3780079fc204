// C ABI of the rotary positions, the paged key/value cache and attention over
// it: argument validation and dispatch.  Every check runs on the host before
// anything is enqueued.
#include "kv_launch.h"
#include "q4_status.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace {

__attribute__((format(printf, 2, 3))) q4_status fail(q4_status code, const char* fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return q4::set_status(code, text);
}

q4_status ok() { return q4::set_status(Q4_OK, ""); }

q4_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(Q4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int type_bytes(int type) { return type == Q4_TYPE_F32 ? 4 : type == Q4_TYPE_F16 || type == Q4_TYPE_BF16 ? 2 : 0; }

// Limits that keep every row, position and unit index inside 32 bits, and every
// byte offset inside int64: strides alone do not, their products with the counts
// are bounded by kMaxReach.
constexpr int64_t kMaxTokens = int64_t(1) << 27;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxReach = int64_t(1) << 60;  // elements, of at most 4 bytes
constexpr int kMaxHeads = 4096;
constexpr int kMaxHeadDim = 1024;
constexpr int kMaxPage = 65536;

// Elements from the first to behind the last of `count` blocks of `block` elements
// that are `stride` apart (kMaxReach where there are more).
int64_t reach(int64_t block, int64_t count, int64_t stride) {
    int64_t r;
    if (__builtin_mul_overflow(count - 1, stride, &r) || __builtin_add_overflow(block, r, &r)) return kMaxReach;
    return std::min(r, kMaxReach);
}

struct Span {
    uintptr_t lo, hi;  // [lo, hi) bytes
};
bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }
Span span(const void* p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + bytes};
}

// A strided block of heads as bytes: `len` bytes of each token from `lo` on,
// tokens `step` bytes apart.
struct Rows {
    Span all;
    uint64_t len, step;
};
Rows rows_of(const q4_heads& x, int64_t tokens, int heads, int dim) {
    const uint64_t b = type_bytes(x.type);
    Rows r;
    r.len = ((uint64_t)(heads - 1) * x.head_stride + dim) * b;
    r.step = (uint64_t)x.token_stride * b;
    r.all = span(x.data, (uint64_t)(tokens - 1) * r.step + r.len);
    return r;
}
// Parts of the same packed rows (equal steps, disjoint within a step) do not
// overlap although their spans do.
bool overlap(const Rows& a, const Rows& b) {
    if (!overlap(a.all, b.all)) return false;
    if (a.step != b.step || a.len > a.step || b.len > b.step) return true;
    const uint64_t at = b.all.lo >= a.all.lo ? (b.all.lo - a.all.lo) % a.step : (a.step - (a.all.lo - b.all.lo) % a.step) % a.step;
    return !(at >= a.len && at + b.len <= a.step);
}

bool same(const q4_heads& a, const q4_heads& b) {
    return a.data == b.data && a.type == b.type && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

q4_status check_heads(const char* fn, const char* name, const q4_heads* x, int64_t tokens, int heads, int dim, bool output) {
    if (!x || !x->data) return fail(Q4_ERR_INVALID_ARG, "%s: null %s", fn, name);
    const int b = type_bytes(x->type);
    if (!b) return fail(Q4_ERR_INVALID_ARG, "%s: %s has an unknown type %d", fn, name, x->type);
    if (!aligned(x->data, b)) return fail(Q4_ERR_MISALIGNED, "%s: %s must be aligned to its elements", fn, name);
    if (x->token_stride < 0 || x->token_stride > kMaxStride || x->head_stride < 0 || x->head_stride > kMaxStride)
        return fail(Q4_ERR_INVALID_ARG, "%s: a stride of %s is negative or too large", fn, name);
    if (reach(reach(dim, heads, x->head_stride), tokens, x->token_stride) >= kMaxReach)
        return fail(Q4_ERR_INVALID_ARG, "%s: the strides of %s reach too far", fn, name);
    if (output) {
        const int64_t ts = x->token_stride, hs = x->head_stride;
        const bool by_token = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= (heads - 1) * hs + dim);
        const bool by_head = (tokens == 1 || ts >= dim) && (heads == 1 || hs >= (tokens - 1) * ts + dim);
        if (!by_token && !by_head) return fail(Q4_ERR_INVALID_ARG, "%s: the heads of %s overlap each other", fn, name);
    }
    return Q4_OK;
}

q4_status check_sizes(const char* fn, int64_t tokens, int heads, int dim) {
    if (tokens < 1 || tokens > kMaxTokens) return fail(Q4_ERR_INVALID_ARG, "%s: tokens = %lld outside [1, %lld]", fn, (long long)tokens, (long long)kMaxTokens);
    if (heads < 1 || heads > kMaxHeads) return fail(Q4_ERR_INVALID_ARG, "%s: heads = %d outside [1, %d]", fn, heads, kMaxHeads);
    if (dim < 1 || dim > kMaxHeadDim) return fail(Q4_ERR_INVALID_ARG, "%s: head_dim = %d outside [1, %d]", fn, dim, kMaxHeadDim);
    return Q4_OK;
}

q4_status check_rotation(const char* fn, const double* inv_freq, int rot_dim, int head_dim, int layout, float mscale) {
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2) return fail(Q4_ERR_INVALID_ARG, "%s: rot_dim = %d must be even and in [0, head_dim = %d]", fn, rot_dim, head_dim);
    if (layout != Q4_ROPE_HALF && layout != Q4_ROPE_INTERLEAVED) return fail(Q4_ERR_INVALID_ARG, "%s: unknown layout %d", fn, layout);
    if (rot_dim && !inv_freq) return fail(Q4_ERR_INVALID_ARG, "%s: null inv_freq", fn);
    if (!aligned(inv_freq, 8)) return fail(Q4_ERR_MISALIGNED, "%s: inv_freq must be 8-byte aligned", fn);
    if (!std::isfinite(mscale)) return fail(Q4_ERR_INVALID_ARG, "%s: mscale must be finite", fn);
    return Q4_OK;
}

q4_status check_cache(const char* fn, const q4_kv_cache* c) {
    if (!c || !c->k || !c->v) return fail(Q4_ERR_INVALID_ARG, "%s: null cache", fn);
    if (c->type != Q4_TYPE_F16 && c->type != Q4_TYPE_BF16) return fail(Q4_ERR_INVALID_ARG, "%s: the cache must hold binary16 or bfloat16", fn);
    if (!aligned(c->k, 2) || !aligned(c->v, 2)) return fail(Q4_ERR_MISALIGNED, "%s: the cache must be aligned to its elements", fn);
    if (c->pages < 1 || c->pages > 0x7fffffff) return fail(Q4_ERR_INVALID_ARG, "%s: pages = %lld outside [1, 2^31)", fn, (long long)c->pages);
    if (c->page_size < 8 || c->page_size > kMaxPage || c->page_size % 8) return fail(Q4_ERR_INVALID_ARG, "%s: page_size = %d must be a multiple of 8 in [8, %d]", fn, c->page_size, kMaxPage);
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads) return fail(Q4_ERR_INVALID_ARG, "%s: kv_heads = %d outside [1, %d]", fn, c->kv_heads, kMaxHeads);
    if (c->head_dim < 1 || c->head_dim > kMaxHeadDim) return fail(Q4_ERR_INVALID_ARG, "%s: head_dim = %d outside [1, %d]", fn, c->head_dim, kMaxHeadDim);
    const int64_t s[6] = {c->k_page_stride, c->k_head_stride, c->k_slot_stride, c->v_page_stride, c->v_head_stride, c->v_slot_stride};
    for (int i = 0; i < 6; ++i) {
        if (s[i] < 0 || s[i] > kMaxStride) return fail(Q4_ERR_INVALID_ARG, "%s: a stride of the cache is negative or too large", fn);
        const int64_t count = i % 3 == 0 ? c->pages : i % 3 == 1 ? c->kv_heads : c->page_size;
        if (count > 1 && s[i] < c->head_dim) return fail(Q4_ERR_INVALID_ARG, "%s: the heads of the cache overlap each other", fn);
    }
    for (int i = 0; i < 6; i += 3)
        if (reach(reach(reach(c->head_dim, c->page_size, s[i + 2]), c->kv_heads, s[i + 1]), c->pages, s[i]) >= kMaxReach)
            return fail(Q4_ERR_INVALID_ARG, "%s: the strides of the cache reach too far", fn);
    return Q4_OK;
}

// The axes of keys or values that have more than one entry, the largest stride first.
struct Axis {
    int64_t stride, count;
};
int cache_axes(const q4_kv_cache* c, bool values, Axis (&axis)[3]) {
    const Axis all[3] = {{values ? c->v_page_stride : c->k_page_stride, c->pages},
                         {values ? c->v_head_stride : c->k_head_stride, c->kv_heads},
                         {values ? c->v_slot_stride : c->k_slot_stride, c->page_size}};
    int n = 0;
    for (const Axis& a : all)
        if (a.count > 1) axis[n++] = a;
    std::sort(axis, axis + n, [](const Axis& a, const Axis& b) { return a.stride > b.stride; });
    return n;
}

// Each stride steps over all that the smaller ones reach: no two elements of a
// cache that is written are the same memory.
bool axes_nest(const Axis* axis, int n, int64_t dim) {
    for (int i = n - 1; i >= 0; --i) {
        if (axis[i].stride < dim) return false;
        dim = reach(dim, axis[i].count, axis[i].stride);
    }
    return true;
}

// Whether an element of the values, `delta` elements behind the keys, may be one of
// the keys (nested axes, largest first).  With equal strides the outermost can
// bring a block of the one near a block of the other in two ways only, rounding
// delta / stride down and up; where the layouts differ the spans decide.
bool blocks_meet(const Axis* k, int nk, const Axis* v, int nv, int64_t dim, int64_t delta) {
    int64_t rk = dim, rv = dim;
    for (int i = 0; i < nk; ++i) rk = reach(rk, k[i].count, k[i].stride);
    for (int i = 0; i < nv; ++i) rv = reach(rv, v[i].count, v[i].stride);
    if (delta >= rk || -delta >= rv) return false;
    if (!nk || !nv || k->stride != v->stride || k->count != v->count) return true;
    const int64_t down = delta / k->stride - (delta % k->stride < 0);
    for (int64_t i = down; i <= down + 1; ++i)
        if (i > -k->count && i < k->count && blocks_meet(k + 1, nk - 1, v + 1, nv - 1, dim, delta - i * k->stride)) return true;
    return false;
}

Span cache_span(const q4_kv_cache* c, bool values) {
    const int64_t p = values ? c->v_page_stride : c->k_page_stride, h = values ? c->v_head_stride : c->k_head_stride,
                  s = values ? c->v_slot_stride : c->k_slot_stride;
    return span(values ? c->v : c->k, 2 * (uint64_t)((c->pages - 1) * p + (c->kv_heads - 1) * h + (c->page_size - 1) * s + c->head_dim));
}

q4_status check_batch(const char* fn, const q4_kv_batch* b, const q4_kv_cache* c) {
    if (!b || !b->block_table || !b->query_start || !b->context_len) return fail(Q4_ERR_INVALID_ARG, "%s: null batch, block table or lengths", fn);
    if (!aligned(b->block_table, 4) || !aligned(b->query_start, 4) || !aligned(b->context_len, 4))
        return fail(Q4_ERR_MISALIGNED, "%s: block table and lengths must be 4-byte aligned", fn);
    if (b->seqs < 1 || b->seqs > (1 << 24)) return fail(Q4_ERR_INVALID_ARG, "%s: seqs = %d outside [1, 2^24]", fn, b->seqs);
    if (b->table_pages < 1 || (int64_t)b->table_pages * c->page_size > (int64_t(1) << 30))
        return fail(Q4_ERR_INVALID_ARG, "%s: a block table of %d pages: it must hold 1 page and at most 2^30 tokens", fn, b->table_pages);
    if (b->table_stride < 0 || b->table_stride > kMaxStride || (b->seqs > 1 && b->table_stride < b->table_pages))
        return fail(Q4_ERR_INVALID_ARG, "%s: the block table's stride is smaller than a row", fn);
    if (reach(b->table_pages, b->seqs, b->table_stride) >= kMaxReach)
        return fail(Q4_ERR_INVALID_ARG, "%s: the block table's stride reaches too far", fn);
    if (b->max_query < 0 || b->max_context < 0) return fail(Q4_ERR_INVALID_ARG, "%s: max_query and max_context must not be negative", fn);
    return Q4_OK;
}

// Block table, starts and lengths: what no output may overlap.
bool overlaps_batch(Span x, const q4_kv_batch* b) {
    return overlap(x, span(b->block_table, 4 * (uint64_t)((b->seqs - 1) * b->table_stride + b->table_pages))) ||
           overlap(x, span(b->query_start, 4 * (uint64_t)(b->seqs + 1))) || overlap(x, span(b->context_len, 4 * (uint64_t)b->seqs));
}

// (strides of a single token or head are never used: as 0 they do not decide about alignment)
q4::HeadsArg heads_arg(const q4_heads& x, int64_t tokens, int heads) {
    return q4::HeadsArg{static_cast<char*>(x.data), tokens > 1 ? x.token_stride : 0, heads > 1 ? x.head_stride : 0};
}

q4::CacheArg cache_arg(const q4_kv_cache& c) {
    q4::CacheArg r;
    r.k = static_cast<char*>(c.k);
    r.v = static_cast<char*>(c.v);
    r.k_page = c.pages > 1 ? c.k_page_stride : 0;
    r.v_page = c.pages > 1 ? c.v_page_stride : 0;
    r.k_head = c.kv_heads > 1 ? c.k_head_stride : 0;
    r.v_head = c.kv_heads > 1 ? c.v_head_stride : 0;
    r.k_slot = c.k_slot_stride;
    r.v_slot = c.v_slot_stride;
    r.pages = (uint32_t)c.pages;
    r.page_size = q4::FastDiv((uint32_t)c.page_size);
    r.kv_heads = c.kv_heads;
    r.head_dim = c.head_dim;
    return r;
}

int window_arg(int64_t window) { return (int)std::min<int64_t>(window, int64_t(1) << 30); }  // a table holds no more

q4::BatchArg batch_arg(const q4_kv_batch& b) {
    return q4::BatchArg{b.block_table, b.table_stride, b.table_pages, b.seqs, b.query_start, b.context_len};
}

q4_status check_attention(const char* fn, const q4_kv_cache* cache, const q4_kv_batch* batch, int q_heads, int64_t tokens,
                          int64_t window) {
    q4_status st = check_cache(fn, cache);
    if (st) return st;
    st = check_batch(fn, batch, cache);
    if (st) return st;
    st = check_sizes(fn, tokens, q_heads, cache->head_dim);
    if (st) return st;
    if (!q4::attn_head_dim_ok(cache->head_dim)) return fail(Q4_ERR_INVALID_ARG, "%s: head_dim = %d must be 64, 96, 128 or 256", fn, cache->head_dim);
    if (q_heads % cache->kv_heads) return fail(Q4_ERR_INVALID_ARG, "%s: q_heads = %d must be a multiple of kv_heads = %d", fn, q_heads, cache->kv_heads);
    if (tokens * q_heads > (int64_t(1) << 30)) return fail(Q4_ERR_INVALID_ARG, "%s: more than 2^30 query rows", fn);
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16)) return fail(Q4_ERR_MISALIGNED, "%s: the cache must be 16-byte aligned", fn);
    const q4::CacheArg c = cache_arg(*cache);
    if ((c.k_page | c.k_head | c.k_slot | c.v_page | c.v_head | c.v_slot) % 8)
        return fail(Q4_ERR_MISALIGNED, "%s: the cache's strides must be multiples of 8", fn);
    if (cache->k_slot_stride > (1 << 26) || cache->v_slot_stride > (1 << 26))
        return fail(Q4_ERR_INVALID_ARG, "%s: the slots of the cache must not be more than 2^26 elements apart", fn);
    if (window < 0) return fail(Q4_ERR_INVALID_ARG, "%s: window must not be negative", fn);
    return Q4_OK;
}

}  // namespace

extern "C" {

q4_status q4_rope(const q4_heads* x, const q4_heads* out, const int32_t* positions, const double* inv_freq,
                  int64_t tokens, int heads, int head_dim, int rot_dim, int layout, float mscale, void* stream) {
    const char* fn = "q4_rope";
    q4_status st = check_sizes(fn, tokens, heads, head_dim);
    if (st) return st;
    st = check_rotation(fn, inv_freq, rot_dim, head_dim, layout, mscale);
    if (st) return st;
    if (rot_dim < 2) return fail(Q4_ERR_INVALID_ARG, "%s: rot_dim must be at least 2", fn);
    st = check_heads(fn, "x", x, tokens, heads, head_dim, false);
    if (st) return st;
    st = check_heads(fn, "out", out, tokens, heads, head_dim, true);
    if (st) return st;
    if (!positions) return fail(Q4_ERR_INVALID_ARG, "%s: null positions", fn);
    if (!aligned(positions, 4)) return fail(Q4_ERR_MISALIGNED, "%s: positions must be 4-byte aligned", fn);
    const Rows ro = rows_of(*out, tokens, heads, head_dim);
    if (!same(*x, *out) && overlap(ro, rows_of(*x, tokens, heads, head_dim)))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps x without being x", fn);
    if (overlap(ro.all, span(positions, 4 * (uint64_t)tokens)) || overlap(ro.all, span(inv_freq, 4 * (uint64_t)rot_dim)))
        return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps positions or inv_freq", fn);
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
    return hip_status(q4::launch_rope(a, x->type, out->type, layout, static_cast<hipStream_t>(stream)), "q4_rope launch");
}

q4_status q4_kv_append(const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* k, const q4_heads* v,
                       const q4_heads* q, const q4_heads* q_out, int q_heads, int64_t tokens, const int32_t* positions,
                       const double* inv_freq, int rot_dim, int layout, float mscale, void* stream) {
    const char* fn = "q4_kv_append";
    q4_status st = check_cache(fn, cache);
    if (st) return st;
    st = check_batch(fn, batch, cache);
    if (st) return st;
    const int dim = cache->head_dim;
    st = check_sizes(fn, tokens, q ? q_heads : 1, dim);
    if (st) return st;
    st = check_rotation(fn, inv_freq, rot_dim, dim, layout, mscale);
    if (st) return st;
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
    Span read[2] = {span(positions, positions ? 4 * (uint64_t)tokens : 0), span(inv_freq, rot_dim ? 4 * (uint64_t)rot_dim : 0)};
    if (q) {
        st = check_heads(fn, "q", q, tokens, q_heads, dim, false);
        if (st) return st;
        st = check_heads(fn, "q_out", q_out, tokens, q_heads, dim, true);
        if (st) return st;
        if (q_out->type != cache->type) return fail(Q4_ERR_INVALID_ARG, "%s: q_out must have the cache's type", fn);
        const Rows rq = rows_of(*q, tokens, q_heads, dim), ro = rows_of(*q_out, tokens, q_heads, dim);
        if ((!same(*q, *q_out) && overlap(ro, rq)) || overlap(ro, rk) || overlap(ro, rv) || overlap(ro.all, read[0]) ||
            overlap(ro.all, read[1]) || overlaps_batch(ro.all, batch) || overlap(ro.all, ck) || overlap(ro.all, cv))
            return fail(Q4_ERR_INVALID_ARG, "%s: q_out overlaps another tensor (or q without being q)", fn);
        if (overlap(rq.all, ck) || overlap(rq.all, cv)) return fail(Q4_ERR_INVALID_ARG, "%s: q overlaps the cache", fn);
    }
    for (const Span& c : {ck, cv})
        if (overlap(c, rk.all) || overlap(c, rv.all) || overlap(c, read[0]) || overlap(c, read[1]) || overlaps_batch(c, batch))
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
    return hip_status(q4::launch_rope(a, k->type, cache->type, layout, static_cast<hipStream_t>(stream)), "q4_kv_append launch");
}

size_t q4_attention_paged_workspace_bytes(const q4_kv_cache* cache, const q4_kv_batch* batch, int q_heads, int64_t tokens,
                                          int64_t window) {
    if (check_attention("q4_attention_paged_workspace_bytes", cache, batch, q_heads, tokens, window)) return 0;
    ok();
    return q4::attn_shape(cache_arg(*cache), batch_arg(*batch), q_heads, tokens, window_arg(window), batch->max_query, batch->max_context).bytes;
}

q4_status q4_attention_paged(const q4_kv_cache* cache, const q4_kv_batch* batch, const q4_heads* q, const q4_heads* out,
                             float* lse, int q_heads, int64_t tokens, float scale, int64_t window, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const char* fn = "q4_attention_paged";
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
    const q4::AttnShape shape = q4::attn_shape(c, b, q_heads, tokens, window_arg(window), batch->max_query, batch->max_context);
    if (shape.bytes) {
        if (!workspace || workspace_bytes < shape.bytes) return fail(Q4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, shape.bytes);
        if (!aligned(workspace, 16)) return fail(Q4_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    }
    const Rows rq = rows_of(*q, tokens, q_heads, dim), ro = rows_of(*out, tokens, q_heads, dim);
    const Span written[3] = {ro.all, span(lse, lse ? 4 * (uint64_t)tokens * q_heads : 0), span(workspace, shape.bytes)};
    const Span read[3] = {rq.all, cache_span(cache, false), cache_span(cache, true)};
    for (int i = 0; i < 3; ++i) {
        if (written[i].lo == written[i].hi) continue;
        for (int j = 0; j < 3; ++j)
            if (i == 0 && j == 0 ? overlap(ro, rq) : overlap(written[i], read[j]))
                return fail(Q4_ERR_INVALID_ARG, "%s: an output or the workspace overlaps an input", fn);
        if (overlaps_batch(written[i], batch)) return fail(Q4_ERR_INVALID_ARG, "%s: an output or the workspace overlaps the batch", fn);
        for (int j = i + 1; j < 3; ++j)
            if (written[j].lo != written[j].hi && overlap(written[i], written[j]))
                return fail(Q4_ERR_INVALID_ARG, "%s: outputs and workspace must not overlap", fn);
    }
    q4::AttnArgs a = {};
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
    return hip_status(q4::launch_attention(a, shape, cache->type, static_cast<hipStream_t>(stream)), "q4_attention_paged launch");
}

}  // extern "C"
