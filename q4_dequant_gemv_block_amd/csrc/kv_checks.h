// Checks of arguments shared by the entry points of the paged cache's operators (host).
// Every check runs before anything is enqueued.
#pragma once

#include "kv_launch.h"
#include "q4_status.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace q4 {
namespace check {

__attribute__((format(printf, 2, 3))) inline q4_status fail(q4_status code, const char* fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return q4::set_status(code, text);
}

inline q4_status ok() { return q4::set_status(Q4_OK, ""); }

inline q4_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(Q4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int type_bytes(int type) { return type == Q4_TYPE_F32 ? 4 : type == Q4_TYPE_F16 || type == Q4_TYPE_BF16 ? 2 : 0; }

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
inline int64_t reach(int64_t block, int64_t count, int64_t stride) {
    int64_t r;
    if (__builtin_mul_overflow(count - 1, stride, &r) || __builtin_add_overflow(block, r, &r)) return kMaxReach;
    return std::min(r, kMaxReach);
}

struct Span {
    uintptr_t lo, hi;  // [lo, hi) bytes
};
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }
inline Span span(const void* p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + bytes};
}

// A strided block of heads as bytes: `len` bytes of each token from `lo` on,
// tokens `step` bytes apart.
struct Rows {
    Span all;
    uint64_t len, step;
};
inline Rows rows_of(const q4_heads& x, int64_t tokens, int heads, int dim) {
    const uint64_t b = type_bytes(x.type);
    Rows r;
    r.len = ((uint64_t)(heads - 1) * x.head_stride + dim) * b;
    r.step = (uint64_t)x.token_stride * b;
    r.all = span(x.data, (uint64_t)(tokens - 1) * r.step + r.len);
    return r;
}
// Parts of the same packed rows (equal steps, disjoint within a step) do not
// overlap although their spans do.
inline bool overlap(const Rows& a, const Rows& b) {
    if (!overlap(a.all, b.all)) return false;
    if (a.step != b.step || a.len > a.step || b.len > b.step) return true;
    const uint64_t at = b.all.lo >= a.all.lo ? (b.all.lo - a.all.lo) % a.step : (a.step - (a.all.lo - b.all.lo) % a.step) % a.step;
    return !(at >= a.len && at + b.len <= a.step);
}

inline bool same(const q4_heads& a, const q4_heads& b) {
    return a.data == b.data && a.type == b.type && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

inline q4_status check_heads(const char* fn, const char* name, const q4_heads* x, int64_t tokens, int heads, int dim, bool output) {
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

inline q4_status check_sizes(const char* fn, int64_t tokens, int heads, int dim) {
    if (tokens < 1 || tokens > kMaxTokens) return fail(Q4_ERR_INVALID_ARG, "%s: tokens = %lld outside [1, %lld]", fn, (long long)tokens, (long long)kMaxTokens);
    if (heads < 1 || heads > kMaxHeads) return fail(Q4_ERR_INVALID_ARG, "%s: heads = %d outside [1, %d]", fn, heads, kMaxHeads);
    if (dim < 1 || dim > kMaxHeadDim) return fail(Q4_ERR_INVALID_ARG, "%s: head_dim = %d outside [1, %d]", fn, dim, kMaxHeadDim);
    return Q4_OK;
}

inline q4_status check_rotation(const char* fn, const double* inv_freq, int rot_dim, int head_dim, int layout, float mscale) {
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2) return fail(Q4_ERR_INVALID_ARG, "%s: rot_dim = %d must be even and in [0, head_dim = %d]", fn, rot_dim, head_dim);
    if (layout != Q4_ROPE_HALF && layout != Q4_ROPE_INTERLEAVED) return fail(Q4_ERR_INVALID_ARG, "%s: unknown layout %d", fn, layout);
    if (rot_dim && !inv_freq) return fail(Q4_ERR_INVALID_ARG, "%s: null inv_freq", fn);
    if (!aligned(inv_freq, 8)) return fail(Q4_ERR_MISALIGNED, "%s: inv_freq must be 8-byte aligned", fn);
    if (!std::isfinite(mscale)) return fail(Q4_ERR_INVALID_ARG, "%s: mscale must be finite", fn);
    return Q4_OK;
}

inline q4_status check_cache(const char* fn, const q4_kv_cache* c) {
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
inline int cache_axes(const q4_kv_cache* c, bool values, Axis (&axis)[3]) {
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
inline bool axes_nest(const Axis* axis, int n, int64_t dim) {
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
inline bool blocks_meet(const Axis* k, int nk, const Axis* v, int nv, int64_t dim, int64_t delta) {
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

inline Span cache_span(const q4_kv_cache* c, bool values) {
    const int64_t p = values ? c->v_page_stride : c->k_page_stride, h = values ? c->v_head_stride : c->k_head_stride,
                  s = values ? c->v_slot_stride : c->k_slot_stride;
    return span(values ? c->v : c->k, 2 * (uint64_t)((c->pages - 1) * p + (c->kv_heads - 1) * h + (c->page_size - 1) * s + c->head_dim));
}

inline q4_status check_batch(const char* fn, const q4_kv_batch* b, const q4_kv_cache* c) {
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
inline bool overlaps_batch(Span x, const q4_kv_batch* b) {
    return overlap(x, span(b->block_table, 4 * (uint64_t)((b->seqs - 1) * b->table_stride + b->table_pages))) ||
           overlap(x, span(b->query_start, 4 * (uint64_t)(b->seqs + 1))) || overlap(x, span(b->context_len, 4 * (uint64_t)b->seqs));
}

// (strides of a single token or head are never used: as 0 they do not decide about alignment)
inline q4::HeadsArg heads_arg(const q4_heads& x, int64_t tokens, int heads) {
    return q4::HeadsArg{static_cast<char*>(x.data), tokens > 1 ? x.token_stride : 0, heads > 1 ? x.head_stride : 0};
}

inline q4::CacheArg cache_arg(const q4_kv_cache& c) {
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

inline int window_arg(int64_t window) { return (int)std::min<int64_t>(window, int64_t(1) << 30); }  // a table holds no more

inline q4::BatchArg batch_arg(const q4_kv_batch& b) {
    return q4::BatchArg{b.block_table, b.table_stride, b.table_pages, b.seqs, b.query_start, b.context_len};
}

// Heads and tokens of attention over a cache that is checked.
inline q4_status check_attention_sizes(const char* fn, const q4_kv_cache* cache, int q_heads, int64_t tokens) {
    const q4_status st = check_sizes(fn, tokens, q_heads, cache->head_dim);
    if (st) return st;
    if (!q4::attn_head_dim_ok(cache->head_dim)) return fail(Q4_ERR_INVALID_ARG, "%s: head_dim = %d must be 64, 96, 128 or 256", fn, cache->head_dim);
    if (q_heads % cache->kv_heads) return fail(Q4_ERR_INVALID_ARG, "%s: q_heads = %d must be a multiple of kv_heads = %d", fn, q_heads, cache->kv_heads);
    if (tokens * q_heads > (int64_t(1) << 30)) return fail(Q4_ERR_INVALID_ARG, "%s: more than 2^30 query rows", fn);
    return Q4_OK;
}

inline q4_status check_attention(const char* fn, const q4_kv_cache* cache, const q4_kv_batch* batch, int q_heads, int64_t tokens,
                          int64_t window) {
    q4_status st = check_cache(fn, cache);
    if (st) return st;
    st = check_batch(fn, batch, cache);
    if (st) return st;
    st = check_attention_sizes(fn, cache, q_heads, tokens);
    if (st) return st;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16)) return fail(Q4_ERR_MISALIGNED, "%s: the cache must be 16-byte aligned", fn);
    const q4::CacheArg c = cache_arg(*cache);
    if ((c.k_page | c.k_head | c.k_slot | c.v_page | c.v_head | c.v_slot) % 8)
        return fail(Q4_ERR_MISALIGNED, "%s: the cache's strides must be multiples of 8", fn);
    if (cache->k_slot_stride > (1 << 26) || cache->v_slot_stride > (1 << 26))
        return fail(Q4_ERR_INVALID_ARG, "%s: the slots of the cache must not be more than 2^26 elements apart", fn);
    if (window < 0) return fail(Q4_ERR_INVALID_ARG, "%s: window must not be negative", fn);
    return Q4_OK;
}

}  // namespace check
}  // namespace q4
