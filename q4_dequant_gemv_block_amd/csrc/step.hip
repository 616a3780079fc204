// A decode step's tables from its lengths, the path taken through a drafted tree,
// and the cache's slots closed up behind it (gfx950).  Whole numbers and copies:
// bound by latency, so each is one launch whose workgroups need nothing from each
// other.  Measured (an empty launch is 3.8 us): tables of 8 sequences of a token 3.8 us,
// of 256 trees of up to 64 tokens over 16384 5.9; the path through a tree of 16 2.5, 48
// through trees of up to 48 6.0; their slots in 36 layers' caches 6.5.
#include "kv_device.h"
#include "step_launch.h"

#include <algorithm>

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxNodes = 1024;  // of a tree with masks: 16 words

// Sequence b's lengths, in range whatever the tensors hold.
struct Lengths {
    int past, fresh, held, lack;  // lack: pages it needs and does not hold
};
__device__ __forceinline__ Lengths lengths_of(const AssignArgs& a, int b) {
    constexpr int most = 1 << 30;
    Lengths x;
    x.past = min(max(a.past[b], 0), most);
    x.fresh = min(max(a.fresh[b], 0), most);
    x.held = min(max(a.held_in[b], 0), a.table_pages);
    // (up to 2^31 tokens: rounded up without passing it)
    const uint32_t tokens = (uint32_t)min(x.past + (int64_t)x.fresh, (int64_t)0x7fffffff);
    const uint32_t full = a.page.div(tokens);
    const int need = (int)min(full + (full * a.page.d < tokens), (uint32_t)a.table_pages);
    x.lack = max(need - x.held, 0);
    return x;
}

// Sums over the workgroup (in turn: sh is free again behind it).
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* sh) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, o), hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o);
        v += (int64_t)(((uint64_t)hi << 32) | lo);
    }
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    int64_t r = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) r += sh[w];
    __syncthreads();
    return r;
}

// Workgroup (g, y) takes the sequences [g per, (g + 1) per) and every gridDim.y-th
// batch of their columns and tokens.  What stands before them, new tokens and pages,
// it sums from the lengths itself: 12 bytes a sequence from the L2 cost less than a
// launch that hands sums on.
__global__ void __launch_bounds__(kThreads) k_assign(const AssignArgs a) {
    __shared__ int64_t sums[kThreads / 64];
    __shared__ int32_t parent[kMaxNodes];
    const int first = blockIdx.x * a.per, last = min(first + a.per, a.seqs);
    const int64_t free_count = min(max((int64_t)*a.free_count, (int64_t)0), a.free_capacity);
    int64_t start = 0, upto = 0;  // new tokens, lacking pages of the sequences before
    for (int b = threadIdx.x; b < first; b += kThreads) {
        const Lengths x = lengths_of(a, b);
        start += x.fresh;
        upto += x.lack;
    }
    if (first) {
        start = block_sum(start, sums);
        upto = block_sum(upto, sums);
    }
    const int from = blockIdx.y * kThreads + threadIdx.x, step = gridDim.y * kThreads;
    for (int b = first; b < last; ++b) {
        const Lengths x = lengths_of(a, b);
        const int64_t before = upto;
        upto += x.lack;
        const bool served = x.lack == 0 || upto <= free_count;
        const int taken = served ? x.lack : 0;
        const int32_t* row_in = a.table_in + b * a.table_in_stride;
        // the page behind column c: one taken, none for a column that lacks one (whatever
        // stands there: it may be another sequence's by now), or the row's
        auto entry = [&](int c) {
            if (c < x.held || c >= x.held + x.lack) return row_in[c];
            return served ? a.free_pages[free_count - 1 - before - (c - x.held)] : -1;
        };
        if (from == 0) {
            constexpr int64_t most = 0x7fffffff;
            a.query_start[b] = (int32_t)min(start, most);
            a.context_len[b] = (int32_t)min(x.past + (int64_t)x.fresh, most);
            a.held[b] = x.held + taken;
            a.missing[b] = x.lack - taken;
            if (b == a.seqs - 1) a.query_start[a.seqs] = (int32_t)min(start + x.fresh, most);
            // of the last sequence, or of the first whose pages do not fit: one of all
            if (before <= free_count && upto > free_count)
                *a.free_left = (int32_t)(free_count - before);
            else if (b == a.seqs - 1 && upto <= free_count)
                *a.free_left = (int32_t)(free_count - upto);
        }
        // (a table in its own place keeps the other columns)
        const bool in_place = a.table_in == a.table;
        int32_t* row = a.table + b * a.table_stride;
        for (int c = (in_place ? x.held : 0) + from; c < (in_place ? x.held + x.lack : a.table_pages); c += step) row[c] = entry(c);
        if (start < a.tokens) {
            const int n = (int)min((int64_t)x.fresh, a.tokens - start);
            for (int i = from; i < n; i += step) {
                const uint32_t place = (uint32_t)(x.past + i);  // below 2^31
                const uint32_t c = a.page.div(place);
                const int page = c < (uint32_t)a.table_pages ? entry((int)c) : -1;
                a.slots[start + i] = page >= 0 ? (int64_t)page * a.page.d + (place - c * a.page.d) : -1;
                if (!a.parents) a.positions[start + i] = (int32_t)place;
            }
            if (a.parents || a.mask) {
                // Nodes that masks have bits for; a parent that is not before its child is none.
                const int words = max(a.mask_words, 1), nodes = min(n, a.mask ? 64 * words : kMaxNodes);
                if (a.parents) {
                    for (int i = threadIdx.x; i < nodes; i += kThreads) parent[i] = a.parents[start + i];
                    __syncthreads();
                }
                for (int64_t u = from; u < (int64_t)n * words; u += step) {
                    const int i = (int)(u / words), w = (int)(u - (int64_t)i * words);
                    uint64_t bits = 0;
                    int depth = 0;
                    if (!a.parents) {
                        const int bit = i - 64 * w;  // bits 0 .. i
                        bits = bit < 0 ? 0 : bit >= 63 ? ~uint64_t(0) : (uint64_t(2) << bit) - 1;
                    } else if (i < nodes) {
                        for (int j = i;;) {
                            if (j >> 6 == w) bits |= uint64_t(1) << (j & 63);
                            const int p = parent[j];
                            if (p < 0 || p >= j) break;
                            j = p;
                            ++depth;
                        }
                    }
                    if (a.mask) a.mask[(start + i) * words + w] = bits;
                    if (a.parents && w == 0) a.positions[start + i] = x.past + depth;
                }
                if (a.parents) __syncthreads();  // read before the next sequence's
            }
        }
        start += x.fresh;
    }
}

// A wave walks through one sequence's tree from its first new token: the child that
// was drafted as what the trunk chose is the next, found with a ballot over the
// nodes, 64 a register.  Nodes without a slot are nobody's children: their keys and
// values were not stored, so neither they nor what was chosen behind them may count.
constexpr int kHold = 4;  // registers of nodes; longer trees are read again for every step

__global__ void __launch_bounds__(kThreads) k_accept(const AcceptArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t b = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (b >= a.seqs) return;
    const int first = a.query_start[b], last = a.query_start[b + 1], context = a.context_len[b];
    const int n = first < 0 || last > a.tokens || last < first ? 0 : last - first;
    const int past = context - max(last - first, 0);
    const int32_t *choice = a.choice + first, *draft = a.draft + first, *parents = a.parents ? a.parents + first : nullptr;
    const int64_t* slots = a.slots ? a.slots + first : nullptr;
    int cur = 0, count = 0;
    int mine[kHold], token[kHold];  // nodes of the path at 64 k + lane, and their tokens
    int p[kHold], d[kHold], c[kHold];
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int i = 64 * k + lane;
        mine[k] = -1;
        token[k] = 0;
        p[k] = -1;
        d[k] = c[k] = 0;
        if (i < n) {
            p[k] = parents ? parents[i] : i - 1;
            d[k] = draft[i];
            c[k] = choice[i];
            if (slots && slots[i] < 0) p[k] = -1;
        }
    }
    auto write = [&](int j, int node, int tok) {
        a.path[first + j] = node;
        if (a.history && node >= 0 && past + j >= 0 && past + j < a.history_tokens) a.history[b * a.history_stride + past + j] = tok;
    };
    const bool held = n <= 64 * kHold;
    int chosen = -1;
    if (n) {
        int tok = held ? __builtin_amdgcn_readlane(d[0], 0) : draft[0];
        const bool stored = !slots || slots[0] >= 0;
        if (!stored) chosen = tok;  // the step again, from the same token
        while (stored) {
            // node `cur` is the path's next
            if (held) {
#pragma unroll
                for (int k = 0; k < kHold; ++k)
                    if (count == 64 * k + lane) {
                        mine[k] = cur;
                        token[k] = tok;
                    }
            } else if (lane == 0) {
                write(count, cur, tok);
            }
            ++count;
            int next = -1;
            if (held) {
                int v = 0;
#pragma unroll
                for (int k = 0; k < kHold; ++k)
                    if (cur >> 6 == k) v = __builtin_amdgcn_readlane(c[k], cur & 63);
                chosen = v;
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
                    const int i = 64 * k + lane;
                    const uint64_t is = __ballot(i > cur && i < n && p[k] == cur && d[k] == chosen && chosen >= 0);
                    if (is && next < 0) next = 64 * k + (int)__builtin_ctzll(is);
                }
            } else {
                chosen = choice[cur];
                for (int at = (cur + 1) & ~63; at < n && next < 0; at += 64) {
                    const int i = at + lane;
                    const bool in = i > cur && i < n && (!slots || slots[i] >= 0);
                    const int parent = in ? (parents ? parents[i] : i - 1) : -1;
                    const uint64_t is = __ballot(in && parent == cur && draft[in ? i : cur] == chosen && chosen >= 0);
                    if (is) next = at + (int)__builtin_ctzll(is);
                    if (!parents) break;
                }
            }
            if (next < 0) break;
            cur = next;
            tok = chosen;
        }
    }
    if (held) {
#pragma unroll
        for (int k = 0; k < kHold; ++k)
            if (64 * k + lane < n) write(64 * k + lane, mine[k], token[k]);
    } else {
        for (int j = count + lane; j < n; j += 64) a.path[first + j] = -1;
    }
    if (lane == 0) {
        a.accepted[b] = count;
        a.next[b] = chosen;
        a.lens[b] = past + count;
    }
}

// The keys and values of a path's nodes from their slots to the path's: a thread has
// one piece of a head in one layer and takes it through all of its sequence's path.
// A node lies at or behind its place on the path, so no slot is written before it is
// read, whatever is requested ahead.
template <typename P>
__global__ void __launch_bounds__(kThreads) k_move(const MoveArgs a, uint32_t groups, uint32_t total) {
    constexpr int kSteps = 64, kAhead = 8;
    __shared__ int64_t places[2][2][kSteps];  // keys and values: from, to
    __shared__ int moves;
    const int lane = threadIdx.x & 63;
    for (uint32_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int b = (int)(u / groups);
        const int first = a.batch.query_start[b], last = a.batch.query_start[b + 1];
        const int n = first < 0 || last > a.tokens || last < first ? 0 : last - first;
        const int past = a.batch.context_len[b] - n, m = min(a.accepted[b], n);
        // this thread's piece
        const uint32_t piece = (u - (uint32_t)b * groups) * kThreads + threadIdx.x;
        const bool any = piece < a.units.d;
        const uint32_t head_of = a.chunks.div(any ? piece : 0), chunk = (any ? piece : 0) - head_of * a.chunks.d;
        const uint32_t side = a.heads.div(head_of);  // 2 layer + values
        const int64_t head = head_of - side * a.heads.d;
        char* base = a.at[side] + head * (side & 1 ? a.cache.v_head : a.cache.k_head) * 2 + chunk * sizeof(P);
        for (int j0 = 0; j0 < m; j0 += kSteps) {
            if (threadIdx.x < 64) {
                const int j = j0 + lane, node = j < m ? a.path[first + j] : -1;
                int pf = -1, pt = -1;
                if (node > j && node < n) {
                    const int32_t* table = a.batch.table + b * a.batch.table_stride;
                    pf = page_of(a.cache, a.batch, table, past + node);
                    pt = page_of(a.cache, a.batch, table, past + j);
                }
                const bool moved = pf >= 0 && pt >= 0;
                const uint64_t all = __ballot(moved);
                if (moved) {
                    const int at = __popcll(all & ((uint64_t(1) << lane) - 1));
                    const int64_t sf = (past + node) - (int64_t)a.cache.page_size.div((uint32_t)(past + node)) * a.cache.page_size.d;
                    const int64_t st = (past + j) - (int64_t)a.cache.page_size.div((uint32_t)(past + j)) * a.cache.page_size.d;
                    places[0][0][at] = (pf * a.cache.k_page + sf * a.cache.k_slot) * 2;
                    places[0][1][at] = (pt * a.cache.k_page + st * a.cache.k_slot) * 2;
                    places[1][0][at] = (pf * a.cache.v_page + sf * a.cache.v_slot) * 2;
                    places[1][1][at] = (pt * a.cache.v_page + st * a.cache.v_slot) * 2;
                }
                if (lane == 0) moves = __popcll(all);
            }
            __syncthreads();
            const int count = moves;
            if (any) {
                for (int k = 0; k < count; k += kAhead) {
                    P x[kAhead];
#pragma unroll
                    for (int e = 0; e < kAhead; ++e)
                        if (k + e < count) x[e] = *reinterpret_cast<const P*>(base + places[side & 1][0][k + e]);
#pragma unroll
                    for (int e = 0; e < kAhead; ++e)
                        if (k + e < count) *reinterpret_cast<P*>(base + places[side & 1][1][k + e]) = x[e];
                }
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_assign(AssignArgs a, hipStream_t s) {
    // A workgroup a sequence up to 512 (each sums what is before its own).
    a.per = (a.seqs + 511) / 512;
    const int groups = (a.seqs + a.per - 1) / a.per;
    const int64_t units = a.tokens / groups * (a.mask ? a.mask_words : 1) + a.table_pages;
    const int y = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(1024 / groups + 1, 64), units / 1024));
    hipLaunchKernelGGL(k_assign, dim3(groups, y), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_accept(const AcceptArgs& a, hipStream_t s) {
    const int per = kThreads / 64;
    hipLaunchKernelGGL(k_accept, dim3((a.seqs + per - 1) / per), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_move(MoveArgs& a, bool wide, hipStream_t s) {
    const uint32_t chunks = wide ? a.cache.head_dim / 8 : a.cache.head_dim;
    a.chunks = FastDiv(chunks);
    a.heads = FastDiv((uint32_t)a.cache.kv_heads);
    a.units = FastDiv(2u * a.layers * a.cache.kv_heads * chunks);  // at most 128 * 4096 * 1024
    const uint32_t groups = (a.units.d + kThreads - 1) / kThreads;
    // (sequences a launch, so that workgroups are counted in 31 bits)
    const int most = (int)std::max<int64_t>(1, std::min<int64_t>(a.batch.seqs, (int64_t(1) << 30) / groups));
    const BatchArg all = a.batch;
    const int32_t* accepted = a.accepted;
    for (int b = 0; b < all.seqs; b += most) {
        const int seqs = std::min(most, all.seqs - b);
        a.batch.table = all.table + b * all.table_stride;
        a.batch.query_start = all.query_start + b;
        a.batch.context_len = all.context_len + b;
        a.batch.seqs = seqs;
        a.accepted = accepted + b;
        const uint32_t total = groups * (uint32_t)seqs;
        const unsigned grid = std::min<uint32_t>(total, 1 << 22);
        if (wide)
            hipLaunchKernelGGL((k_move<u4>), dim3(grid), dim3(kThreads), 0, s, a, groups, total);
        else
            hipLaunchKernelGGL((k_move<uint16_t>), dim3(grid), dim3(kThreads), 0, s, a, groups, total);
    }
    return hipGetLastError();
}

}  // namespace q4
