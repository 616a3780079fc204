// C ABI of a decode step with drafted trees beside the cache's own operators: block
// tables from lengths, rules on logits, the path taken and the move of its slots.
// Every check runs on the host before anything is enqueued.
#include "kv_checks.h"
#include "step_launch.h"

#include <algorithm>
#include <initializer_list>

using namespace q4::check;

namespace {

struct Named {
    const char* name;
    Span at;
    int align;
    bool optional;
};

Span ints(const void* p, int64_t n) { return span(p, p ? 4 * (uint64_t)n : 0); }
Span rows(const void* p, int64_t n, int64_t stride, int64_t width, int bytes) {
    return span(p, p ? (uint64_t)reach(width, n, stride) * bytes : 0);
}

q4_status check_tensors(const char* fn, std::initializer_list<Named> all) {
    for (const Named& x : all) {
        if (!x.at.lo && !x.optional) return fail(Q4_ERR_INVALID_ARG, "%s: null %s", fn, x.name);
        if (x.at.lo & (x.align - 1)) return fail(Q4_ERR_MISALIGNED, "%s: %s must be %d-byte aligned", fn, x.name, x.align);
        if (x.at.hi - x.at.lo >= uint64_t(1) << 61) return fail(Q4_ERR_INVALID_ARG, "%s: the stride of %s reaches too far", fn, x.name);
    }
    return Q4_OK;
}
// No tensor that is written overlaps another one.
q4_status check_apart(const char* fn, std::initializer_list<Named> written, std::initializer_list<Named> read) {
    for (const Named* w = written.begin(); w != written.end(); ++w) {
        for (const Named* o = w + 1; o != written.end(); ++o)
            if (overlap(w->at, o->at)) return fail(Q4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, w->name, o->name);
        for (const Named& r : read)
            if (overlap(w->at, r.at)) return fail(Q4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, w->name, r.name);
    }
    return Q4_OK;
}

constexpr int kMaxWords = 16;
constexpr int64_t kMaxRows = int64_t(1) << 24;

q4_status accept(const char* fn, const char* what, const int32_t* query_start, const int32_t* context_len, int seqs, const int32_t* choice,
                 const int32_t* draft, const int32_t* parents, const int64_t* slots, int64_t tokens, int32_t* accepted, int32_t* next,
                 int32_t* path, int32_t* lens, int32_t* history, int64_t history_stride, int history_tokens, void* stream) {
    if (seqs < 1 || seqs > kMaxRows) return fail(Q4_ERR_INVALID_ARG, "%s: seqs = %d outside [1, 2^24]", fn, seqs);
    if (tokens < 1 || tokens > kMaxTokens) return fail(Q4_ERR_INVALID_ARG, "%s: tokens = %lld outside [1, %lld]", fn, (long long)tokens, (long long)kMaxTokens);
    if (history && (history_tokens < 1 || history_stride < 0 || history_stride > kMaxStride || (seqs > 1 && history_stride < history_tokens)))
        return fail(Q4_ERR_INVALID_ARG, "%s: history_tokens = %d must be at least 1 and history_stride no smaller", fn, history_tokens);
    const Named start = {"query_start", ints(query_start, (int64_t)seqs + 1), 4, false}, context = {"context_len", ints(context_len, seqs), 4, false};
    const Named c = {"choice", ints(choice, tokens), 4, false}, d = {"draft", ints(draft, tokens), 4, false}, p = {"parents", ints(parents, tokens), 4, true};
    const Named sl = {"slots", span(slots, slots ? 8 * (uint64_t)tokens : 0), 8, true};
    const Named acc = {"accepted", ints(accepted, seqs), 4, false}, nx = {"next", ints(next, seqs), 4, false};
    const Named pa = {"path", ints(path, tokens), 4, false}, le = {"lens", ints(lens, seqs), 4, false};
    const Named hi = {"history", rows(history, seqs, history_stride, history_tokens, 4), 4, true};
    q4_status st = check_tensors(fn, {start, context, c, d, p, sl, acc, nx, pa, le, hi});
    if (!st) st = check_apart(fn, {acc, nx, pa, le, hi}, {start, context, c, d, p, sl});
    if (st) return st;
    const q4::AcceptArgs a = {query_start, context_len, choice, draft, parents, slots, accepted, next, path, lens,
                              history, seqs > 1 ? history_stride : 0, history_tokens, seqs, tokens};
    return hip_status(q4::launch_accept(a, static_cast<hipStream_t>(stream)), what);
}

}  // namespace

extern "C" {

q4_status q4_kv_assign(const q4_kv_step* x, void* stream) {
    const char* fn = "q4_kv_assign";
    if (!x) return fail(Q4_ERR_INVALID_ARG, "%s: null step", fn);
    if (x->seqs < 1 || x->seqs > 65536) return fail(Q4_ERR_INVALID_ARG, "%s: seqs = %d outside [1, 65536]", fn, x->seqs);
    if (x->tokens < 1 || x->tokens > kMaxTokens) return fail(Q4_ERR_INVALID_ARG, "%s: tokens = %lld outside [1, %lld]", fn, (long long)x->tokens, (long long)kMaxTokens);
    if (x->page_size < 8 || x->page_size > kMaxPage || x->page_size % 8) return fail(Q4_ERR_INVALID_ARG, "%s: page_size = %d must be a multiple of 8 in [8, %d]", fn, x->page_size, kMaxPage);
    if (x->table_pages < 1 || (int64_t)x->table_pages * x->page_size > (int64_t(1) << 30))
        return fail(Q4_ERR_INVALID_ARG, "%s: a block table of %d pages: it must hold 1 page and at most 2^30 tokens", fn, x->table_pages);
    for (const int64_t s : {x->table_in_stride, x->table_stride})
        if (s < 0 || s > kMaxStride || (x->seqs > 1 && s < x->table_pages))
            return fail(Q4_ERR_INVALID_ARG, "%s: a block table's stride is smaller than a row or too large", fn);
    if (x->free_capacity < 0 || x->free_capacity > 0x7fffffff) return fail(Q4_ERR_INVALID_ARG, "%s: free_capacity outside [0, 2^31)", fn);
    if (x->mask ? x->mask_words < 1 || x->mask_words > kMaxWords : x->mask_words != 0)
        return fail(Q4_ERR_INVALID_ARG, "%s: mask_words = %d must be in [1, %d] with a mask and 0 without", fn, x->mask_words, kMaxWords);
    const Named in = {"table_in", rows(x->table_in, x->seqs, x->table_in_stride, x->table_pages, 4), 4, false};
    const Named out = {"table", rows(x->table, x->seqs, x->table_stride, x->table_pages, 4), 4, false};
    const bool in_place = x->table == x->table_in && (x->seqs == 1 || x->table_stride == x->table_in_stride);
    const Named held_in = {"held_in", ints(x->held_in, x->seqs), 4, false}, past = {"past_len", ints(x->past_len, x->seqs), 4, false};
    const Named fresh = {"new_len", ints(x->new_len, x->seqs), 4, false}, pages = {"free_pages", ints(x->free_pages, x->free_capacity), 4, !x->free_capacity};
    const Named count = {"free_count", ints(x->free_count, 1), 4, false}, parents = {"parents", ints(x->parents, x->tokens), 4, true};
    const Named held = {"held", ints(x->held, x->seqs), 4, false}, start = {"query_start", ints(x->query_start, x->seqs + 1), 4, false};
    const Named context = {"context_len", ints(x->context_len, x->seqs), 4, false}, missing = {"missing", ints(x->missing, x->seqs), 4, false};
    const Named left = {"free_left", ints(x->free_left, 1), 4, false}, positions = {"positions", ints(x->positions, x->tokens), 4, false};
    const Named slots = {"slots", span(x->slots, 8 * (uint64_t)x->tokens), 8, false};
    const Named mask = {"mask", span(x->mask, x->mask ? 8 * (uint64_t)x->tokens * x->mask_words : 0), 8, true};
    q4_status st = check_tensors(fn, {in, out, held_in, past, fresh, pages, count, parents, held, start, context, missing, left, positions});
    if (st) return st;
    if (!x->slots) return fail(Q4_ERR_INVALID_ARG, "%s: null slots", fn);
    st = check_tensors(fn, {slots, mask});
    if (st) return st;
    if (!in_place && overlap(out.at, in.at)) return fail(Q4_ERR_INVALID_ARG, "%s: table overlaps table_in without being it", fn);
    st = check_apart(fn, {out, held, start, context, missing, left, positions, slots, mask}, {held_in, past, fresh, pages, count, parents});
    if (st) return st;
    st = check_apart(fn, {held, start, context, missing, left, positions, slots, mask}, {in});
    if (st) return st;
    q4::AssignArgs a = {};
    a.table_in = x->table_in;
    a.table_in_stride = x->seqs > 1 ? x->table_in_stride : 0;
    a.held_in = x->held_in;
    a.past = x->past_len;
    a.fresh = x->new_len;
    a.free_pages = x->free_pages;
    a.free_count = x->free_count;
    a.parents = x->parents;
    a.table = x->table;
    a.table_stride = x->seqs > 1 ? x->table_stride : 0;
    a.held = x->held;
    a.query_start = x->query_start;
    a.context_len = x->context_len;
    a.missing = x->missing;
    a.free_left = x->free_left;
    a.positions = x->positions;
    a.slots = x->slots;
    a.mask = x->mask;
    a.mask_words = x->mask_words;
    a.seqs = x->seqs;
    a.table_pages = x->table_pages;
    a.page = q4::FastDiv((uint32_t)x->page_size);
    a.free_capacity = x->free_capacity;
    a.tokens = x->tokens;
    return hip_status(q4::launch_assign(a, static_cast<hipStream_t>(stream)), "q4_kv_assign launch");
}

// No fewer for more rows or entries, so that what was made for the largest call serves all:
// slices shorter than the longest are taken where a call has no more than kLogitFew of
// them, the longest ones' number grows with both sizes.
size_t q4_logits_argmax_workspace_bytes(int64_t n, int64_t vocab) {
    if (n < 1 || n > kMaxRows || vocab < 1 || vocab > kMaxRows) return 0;
    auto slices = [&](int64_t slice) { return (vocab + slice - 1) / slice; };
    if (slices(q4::kLogitShort) == 1) return 0;
    const int64_t few = std::min<int64_t>(n * slices(q4::kLogitShort), q4::kLogitFew);
    const int64_t many = slices(q4::kLogitLong) > 1 ? n * slices(q4::kLogitLong) : 0;
    return (size_t)std::max(few, many) * q4::kLogitKeys * 8;
}

q4_status q4_logits_argmax(const void* logits, int type, int64_t row_stride, int64_t n, int64_t vocab, const q4_logit_rules* r,
                           float* out, int64_t out_stride, int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "q4_logits_argmax";
    if (n < 1 || n > kMaxRows) return fail(Q4_ERR_INVALID_ARG, "%s: rows = %lld outside [1, 2^24]", fn, (long long)n);
    if (vocab < 1 || vocab > kMaxRows) return fail(Q4_ERR_INVALID_ARG, "%s: vocab = %lld outside [1, 2^24]", fn, (long long)vocab);
    const int b = type_bytes(type);
    if (!b) return fail(Q4_ERR_INVALID_ARG, "%s: unknown type %d", fn, type);
    for (const int64_t s : {row_stride, out ? out_stride : row_stride})
        if (s < 0 || s > kMaxStride) return fail(Q4_ERR_INVALID_ARG, "%s: a stride is negative or too large", fn);
    if (out && n > 1 && out_stride < vocab) return fail(Q4_ERR_INVALID_ARG, "%s: the rows of out overlap each other", fn);
    const Named in = {"logits", rows(logits, n, row_stride, vocab, b), b, false};
    const Named res = {"out", rows(out, n, out_stride, vocab, 4), 4, true}, tok = {"tokens", ints(tokens, n), 4, false};
    const int64_t slice = q4::logit_slice(n, vocab), slices = (vocab + slice - 1) / slice;
    const size_t need = slices > 1 ? (size_t)n * slices * q4::kLogitKeys * 8 : 0;
    const Named ws = {"workspace", span(workspace, workspace ? need : 0), 8, true};
    q4_status st = check_tensors(fn, {in, res, tok});
    if (st) return st;
    if (need) {
        if (!workspace || workspace_bytes < need) return fail(Q4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", fn, need);
        st = check_tensors(fn, {ws});
        if (st) return st;
    }
    const bool in_place = out && (const void*)out == logits && type == Q4_TYPE_F32 && (n == 1 || out_stride == row_stride);
    if (!in_place && overlap(res.at, in.at)) return fail(Q4_ERR_INVALID_ARG, "%s: out overlaps logits without being it", fn);
    st = check_apart(fn, {res, tok, ws}, {});
    if (!st) st = check_apart(fn, {tok, ws}, {in});
    if (st) return st;
    q4::LogitArgs a = {};
    if (r) {
        if (r->seqs < 1 || r->seqs > kMaxRows) return fail(Q4_ERR_INVALID_ARG, "%s: seqs = %d outside [1, 2^24]", fn, r->seqs);
        if (!r->query_start && n > r->seqs) return fail(Q4_ERR_INVALID_ARG, "%s: %lld rows of %d sequences without query_start", fn, (long long)n, r->seqs);
        if (!r->history != !r->history_len) return fail(Q4_ERR_INVALID_ARG, "%s: history and history_len go together", fn);
        if (r->history && (r->history_tokens < 1 || r->history_tokens > (1 << 29) || r->history_stride < 0 || r->history_stride > kMaxStride ||
                           (r->seqs > 1 && r->history_stride < r->history_tokens)))
            return fail(Q4_ERR_INVALID_ARG, "%s: history_tokens = %d must be in [1, 2^29] and history_stride no smaller", fn, r->history_tokens);
        if (r->prompt_len && !r->history) return fail(Q4_ERR_INVALID_ARG, "%s: prompt_len without history", fn);
        if (r->mask && !r->draft) return fail(Q4_ERR_INVALID_ARG, "%s: a mask without draft", fn);
        if (r->mask ? r->mask_words < 1 || r->mask_words > kMaxWords : r->mask_words != 0)
            return fail(Q4_ERR_INVALID_ARG, "%s: mask_words = %d must be in [1, %d] with a mask and 0 without", fn, r->mask_words, kMaxWords);
        if (r->biases < 0 || r->biases > (1 << 29)) return fail(Q4_ERR_INVALID_ARG, "%s: biases outside [0, 2^29]", fn);
        if (r->bias_start ? r->biases && (!r->bias_tokens || !r->bias_values) : r->bias_tokens || r->bias_values || r->biases)
            return fail(Q4_ERR_INVALID_ARG, "%s: bias_start, bias_tokens and bias_values go together", fn);
        const int64_t words = (vocab + 31) / 32;
        if (r->allowed && (r->allowed_rows < 1 || r->allowed_rows > kMaxRows || r->allowed_stride < 0 || r->allowed_stride > kMaxStride))
            return fail(Q4_ERR_INVALID_ARG, "%s: allowed_rows = %lld must be in [1, 2^24] and allowed_stride not negative", fn, (long long)r->allowed_rows);
        if (r->allowed_row && !r->allowed) return fail(Q4_ERR_INVALID_ARG, "%s: allowed_row without allowed", fn);
        const Named read[] = {{"query_start", ints(r->query_start, (int64_t)r->seqs + 1), 4, true},
                              {"history", rows(r->history, r->seqs, r->history_stride, r->history_tokens, 4), 4, true},
                              {"history_len", ints(r->history_len, r->seqs), 4, true}, {"prompt_len", ints(r->prompt_len, r->seqs), 4, true},
                              {"draft", ints(r->draft, n), 4, true}, {"mask", span(r->mask, r->mask ? 8 * (uint64_t)n * r->mask_words : 0), 8, true},
                              {"repetition", ints(r->repetition, r->seqs), 4, true}, {"presence", ints(r->presence, r->seqs), 4, true},
                              {"frequency", ints(r->frequency, r->seqs), 4, true}, {"bias_start", ints(r->bias_start, (int64_t)r->seqs + 1), 4, true},
                              {"bias_tokens", ints(r->bias_tokens, r->biases), 4, true}, {"bias_values", ints(r->bias_values, r->biases), 4, true},
                              {"allowed", rows(r->allowed, r->allowed_rows, r->allowed_stride, words, 4), 4, true},
                              {"allowed_row", ints(r->allowed_row, n), 4, true}};
        for (const Named& x : read) {
            st = check_tensors(fn, {x});
            if (!st) st = check_apart(fn, {res}, {x});
            if (!st) st = check_apart(fn, {tok}, {x});
            if (!st) st = check_apart(fn, {ws}, {x});
            if (st) return st;
        }
        a.seqs = r->seqs;
        a.query_start = r->query_start;
        a.history = r->history;
        a.history_stride = r->seqs > 1 ? r->history_stride : 0;
        a.history_tokens = r->history_tokens;
        a.history_len = r->history_len;
        a.prompt_len = r->prompt_len;
        a.draft = r->draft;
        a.mask = r->mask;
        a.mask_words = r->mask_words;
        a.repetition = r->repetition;
        a.presence = r->presence;
        a.frequency = r->frequency;
        a.bias_start = r->biases ? r->bias_start : nullptr;
        a.bias_tokens = r->bias_tokens;
        a.bias_values = r->bias_values;
        a.biases = r->biases;
        a.allowed = r->allowed;
        a.allowed_stride = r->allowed_rows > 1 ? r->allowed_stride : 0;
        a.allowed_rows = r->allowed_rows;
        a.allowed_row = r->allowed_row;
    }
    a.logits = static_cast<const char*>(logits);
    a.row_stride = n > 1 ? row_stride : 0;
    a.rows = n;
    a.vocab = vocab;
    a.out = out;
    a.out_stride = n > 1 ? out_stride : 0;
    a.tokens = tokens;
    a.keys = static_cast<uint64_t*>(workspace);
    return hip_status(q4::launch_logits(a, type, static_cast<hipStream_t>(stream)), "q4_logits_argmax launch");
}

q4_status q4_tree_accept(const int32_t* query_start, const int32_t* context_len, int seqs, const int32_t* choice, const int32_t* draft,
                         const int32_t* parents, int64_t tokens, int32_t* accepted, int32_t* next, int32_t* path, int32_t* lens,
                         int32_t* history, int64_t history_stride, int history_tokens, void* stream) {
    return accept("q4_tree_accept", "q4_tree_accept launch", query_start, context_len, seqs, choice, draft, parents, nullptr, tokens, accepted,
                  next, path, lens, history, history_stride, history_tokens, stream);
}

q4_status q4_tree_accept_stored(const int32_t* query_start, const int32_t* context_len, int seqs, const int32_t* choice,
                                const int32_t* draft, const int32_t* parents, const int64_t* slots, int64_t tokens, int32_t* accepted,
                                int32_t* next, int32_t* path, int32_t* lens, int32_t* history, int64_t history_stride,
                                int history_tokens, void* stream) {
    return accept("q4_tree_accept_stored", "q4_tree_accept_stored launch", query_start, context_len, seqs, choice, draft, parents, slots,
                  tokens, accepted, next, path, lens, history, history_stride, history_tokens, stream);
}

q4_status q4_kv_move(const q4_kv_cache* caches, int layers, const q4_kv_batch* batch, const int32_t* path, const int32_t* accepted,
                     int64_t tokens, void* stream) {
    const char* fn = "q4_kv_move";
    constexpr int kMostLayers = 512;
    if (layers < 1 || layers > kMostLayers) return fail(Q4_ERR_INVALID_ARG, "%s: layers = %d outside [1, %d]", fn, layers, kMostLayers);
    q4_status st = check_cache(fn, caches);
    if (st) return st;
    st = check_batch(fn, batch, caches);
    if (st) return st;
    if (tokens < 1 || tokens > kMaxTokens) return fail(Q4_ERR_INVALID_ARG, "%s: tokens = %lld outside [1, %lld]", fn, (long long)tokens, (long long)kMaxTokens);
    const Named p = {"path", ints(path, tokens), 4, false}, acc = {"accepted", ints(accepted, batch->seqs), 4, false};
    Axis ak[3], av[3];
    const int nk = cache_axes(caches, false, ak), nv = cache_axes(caches, true, av);
    if (!axes_nest(ak, nk, caches->head_dim) || !axes_nest(av, nv, caches->head_dim))
        return fail(Q4_ERR_INVALID_ARG, "%s: the heads of the cache overlap each other", fn);
    const q4::CacheArg size = cache_arg(*caches);
    bool wide = caches->head_dim % 8 == 0 && (size.k_page | size.k_head | size.k_slot | size.v_page | size.v_head | size.v_slot) % 8 == 0;
    struct Block {
        Span at;
        const void* data;
        bool values;
        int64_t rest;  // where in a period of the outermost axis it starts
    };
    Block blocks[2 * kMostLayers];
    int count = 0;
    for (int i = 0; i < layers; ++i) {
        const q4_kv_cache& c = caches[i];
        if (!c.k || !c.v) return fail(Q4_ERR_INVALID_ARG, "%s: null cache", fn);
        if (!aligned(c.k, 2) || !aligned(c.v, 2)) return fail(Q4_ERR_MISALIGNED, "%s: the cache must be aligned to its elements", fn);
        const q4::CacheArg x = cache_arg(c);
        if (c.pages != caches->pages || c.page_size != caches->page_size || c.kv_heads != caches->kv_heads || c.head_dim != caches->head_dim ||
            c.type != caches->type || x.k_page != size.k_page || x.k_head != size.k_head || x.k_slot != size.k_slot || x.v_page != size.v_page ||
            x.v_head != size.v_head || x.v_slot != size.v_slot)
            return fail(Q4_ERR_INVALID_ARG, "%s: the caches of all layers must have the same sizes, strides and type", fn);
        wide = wide && aligned(c.k, 16) && aligned(c.v, 16);
        for (const bool values : {false, true}) {
            const Span at = cache_span(&c, values);
            if (overlap(at, p.at) || overlap(at, acc.at) || overlaps_batch(at, batch))
                return fail(Q4_ERR_INVALID_ARG, "%s: the cache overlaps an input", fn);
            blocks[count++] = Block{at, values ? c.v : c.k, values, 0};
        }
    }
    // Blocks whose spans overlap may still lie beside each other (layers or sides of one
    // tensor).  Those with the same outermost axis only meet if what is inside it does,
    // one period or another apart: then neighbours in the period are compared, not all
    // pairs (1024 blocks side by side in one tensor 12 ms with all pairs, 0.03 with neighbours).
    auto meet = [&](const Block& x, const Block& y) {
        return overlap(x.at, y.at) && blocks_meet(x.values ? av : ak, x.values ? nv : nk, y.values ? av : ak, y.values ? nv : nk,
                                                  caches->head_dim, (int64_t)((intptr_t)y.data - (intptr_t)x.data) / 2);
    };
    std::sort(blocks, blocks + count, [](const Block& x, const Block& y) { return x.at.lo < y.at.lo; });
    bool apart = true;
    for (int i = 1; i < count && apart; ++i) apart = blocks[i].at.lo >= blocks[i - 1].at.hi;
    bool met = false;
    if (!apart && nk && nv && ak->stride == av->stride && ak->count == av->count) {
        int64_t inner = 0;
        for (const bool values : {false, true}) {
            int64_t r = caches->head_dim;
            for (int i = 1; i < (values ? nv : nk); ++i) r = reach(r, (values ? av : ak)[i].count, (values ? av : ak)[i].stride);
            inner = std::max(inner, r);
        }
        for (int i = 0; i < count; ++i) blocks[i].rest = (int64_t)((uint64_t)(uintptr_t)blocks[i].data / 2 % (uint64_t)ak->stride);
        std::sort(blocks, blocks + count, [](const Block& x, const Block& y) { return x.rest < y.rest; });
        for (int i = 0; i < count && !met; ++i)
            for (int k = 1; k < count && !met; ++k) {
                const int j = i + k < count ? i + k : i + k - count;
                if (blocks[j].rest - blocks[i].rest + (j < i ? ak->stride : 0) >= inner) break;
                met = meet(blocks[i], blocks[j]);
            }
    } else if (!apart) {
        for (int i = 0; i < count && !met; ++i)
            for (int j = i + 1; j < count && blocks[j].at.lo < blocks[i].at.hi && !met; ++j) met = meet(blocks[i], blocks[j]);
    }
    if (met) return fail(Q4_ERR_INVALID_ARG, "%s: keys and values of two layers are the same memory, or parts of them", fn);
    st = check_tensors(fn, {p, acc});
    if (st) return st;
    q4::MoveArgs a = {};
    a.cache = size;
    a.path = path;
    a.accepted = accepted;
    a.tokens = tokens;
    for (int at = 0; at < layers; at += q4::kMoveLayers) {
        a.batch = batch_arg(*batch);
        a.accepted = accepted;
        a.layers = std::min(layers - at, q4::kMoveLayers);
        for (int i = 0; i < a.layers; ++i) {
            a.at[2 * i] = static_cast<char*>(caches[at + i].k);
            a.at[2 * i + 1] = static_cast<char*>(caches[at + i].v);
        }
        const hipError_t e = q4::launch_move(a, wide, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_status(e, "q4_kv_move launch");
    }
    return ok();
}

}  // extern "C"
