// Host side of the packed-batch entry points: a layer's tokens of sequences
// of different lengths appended, attended with and dropped again.  Checks,
// the host mirror and the launches, as in hikv_host.cu.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <new>
#include <utility>
#include <vector>

#include "hikv_cache.cuh"
#include "hikv_packed.cuh"

using namespace hikv;

namespace {

// What is wrong with packed rows, or null.  `distinct`: rows that must not
// overlap one another -- written ones, and the queries of the attention, which
// one tensor map describes (no stride of it may be zero).
const char* rows_fault(const hikv_cache* c, const hikv_rows* r, int64_t total, int heads, bool distinct) {
    const int64_t e = c->esz;
    if (!r->data) return "null data";
    if ((uintptr_t)r->data & 15) return "data not 16-byte aligned";
    if (r->token_stride < 0 || r->head_stride < 0) return "a negative stride";
    if (r->token_stride > (INT64_MAX >> 32) || r->head_stride > (INT64_MAX >> 32)) return "a stride too large";
    if (r->token_stride * e % 16 || r->head_stride * e % 16) return "a stride that is no multiple of 16 bytes";
    if (distinct) {
        const int64_t d = c->d, ts = r->token_stride, hs = r->head_stride;
        const bool heads_inside = (heads == 1 || hs >= d) && (total <= 1 || ts >= (heads - 1) * hs + d);
        const bool tokens_inside = (total <= 1 || ts >= d) && (heads == 1 || hs >= (total - 1) * ts + d);
        if (!heads_inside && !tokens_inside) return "rows that overlap one another";
    }
    return nullptr;
}

// Whether rows that are written may share memory with rows that are read: not
// if their extents are apart, nor if they are slices of one buffer (equal
// strides) that keep to their own part of the longer stride.
bool rows_meet(const hikv_cache* c, const hikv_rows* w, int wh, const hikv_rows* r, int rh, int64_t total) {
    auto extent = [&](const hikv_rows* x, int h) { return (total - 1) * x->token_stride + (h - 1) * x->head_stride + c->d; };
    const int64_t at = ((int64_t)(uintptr_t)r->data - (int64_t)(uintptr_t)w->data) / c->esz;   // r's start from w's
    if (at >= extent(w, wh) || -at >= extent(r, rh)) return false;
    if (w->token_stride != r->token_stride || w->head_stride != r->head_stride) return true;
    const bool by_token = w->token_stride >= w->head_stride;
    const int64_t period = by_token ? w->token_stride : w->head_stride;
    if (period == 0) return true;
    auto part = [&](int h) { return (by_token ? (h - 1) * w->head_stride : (total - 1) * w->token_stride) + c->d; };
    const int64_t off = (at % period + period) % period;
    return off < part(wh) || period - off < part(rh);
}

RowsArg rows_arg(const hikv_cache* c, const hikv_rows* r) {
    return {(uint8_t*)r->data, r->token_stride * c->esz, r->head_stride * c->esz};
}

// Packed token counts of a call: their sum, or -1 when one is negative or
// the sum passes 32 bits.
int64_t packed_total(const hikv_cache* c, const int32_t* ntok) {
    int64_t total = 0;
    for (int b = 0; b < c->B; ++b) {
        if (ntok[b] < 0) return -1;
        total += ntok[b];
    }
    return total <= INT32_MAX ? total : -1;
}

// The shape of the work items of the bf16 and of the fp32 kernel: query rows,
// keys per step, what an item costs beside its steps and the join's launch,
// in steps (about 1.5 us of the first kernel, 3 of the second), and the bytes
// of partial results that are written and read in the time of a step.
struct ItemShape {
    int rows, keys;
    double item_steps, join_steps, step_bytes;
};
constexpr ItemShape kTcShape{kTcRows, kTcKeys, 2.0, 3.0, 7.5e6};
constexpr ItemShape kF32Shape{kF32Rows, kF32Keys, 1.5, 1.5, 15e6};

// What the queries of a call see (hikv_packed.cuh), and the KV heads by window.
struct Sees {
    int kind = CausalMask::kind;
    WindowMask window{};
    TreeMask tree{};
    std::vector<std::pair<int32_t, int>> heads;   // window length, KV heads
};

// A sequence of a call: its batch row, first packed row, queries, and the
// longest and the mean length of its heads, and whether all are as long.
struct AttendSeq {
    int32_t brow, start, nq, n, mean;
    bool equal;
};

// Keys of the work items of row tile t of a sequence, for heads of one window
int64_t item_keys(const hikv_cache* c, const ItemShape& k, const Sees& sees, const AttendSeq& s, int64_t t, int32_t window) {
    if (sees.kind == TreeMask::kind) return s.n;
    const int64_t seen = s.n - s.nq + std::min<int64_t>(s.nq, (t + 1) * k.rows / c->G);
    if (sees.kind == CausalMask::kind) return seen;
    const int64_t align = sees.window.align, gap = (sees.window.sink + align - 1) / align * align;
    const int64_t start = std::max<int64_t>(s.n - s.nq + t * k.rows / c->G - window + 1, 0) / align * align;
    return seen - std::max<int64_t>(start - gap, 0);
}
// the most keys of a work item of a sequence, for heads of one window and for all
int64_t most_keys(const hikv_cache* c, const ItemShape& k, const Sees& sees, const AttendSeq& s, int32_t window) {
    if (sees.kind != WindowMask::kind) return s.n;
    const int64_t tiles = ((int64_t)s.nq * c->G + k.rows - 1) / k.rows;
    int64_t most = 0;   // the last tiles span most keys; the last but one may have more rows
    for (int64_t t = std::max<int64_t>(0, tiles - 2); t < tiles; ++t) most = std::max(most, item_keys(c, k, sees, s, t, window));
    return std::min<int64_t>(most + sees.window.align, s.n);   // (windows of inner tiles may start lower in a box)
}
int64_t most_keys(const hikv_cache* c, const ItemShape& k, const Sees& sees, const AttendSeq& s) {
    int64_t most = 0;
    for (const auto& h : sees.heads) most = std::max(most, most_keys(c, k, sees, s, h.first));
    return most;
}

// Keys per split, a multiple of the keys of a step (INT32_MAX: no split).
// The candidates cut the longest sequence into 1 .. 64 parts; partial results
// must fit the work buffer.  Splitting pays where few rows see many keys:
// five drafted tokens over eight 8K-32K caches take 311 us in one part, 163 in
// two, 119 in three and 145 in five; two times 512 tokens over 16K 173 us in
// one, 195 in two and 202 in three (the 34 and 51 MB of partial results cost
// more than even work gains).
int32_t attend_chunk(const hikv_cache* c, const ItemShape& k, const Sees& sees, const AttendSeq* sq, int nseq,
                     int64_t total) {
    static constexpr int kParts[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32, 40, 48, 56, 64};
    const int64_t slots = c->sm_count;
    int64_t base_items = 0, most = 0;
    for (int i = 0; i < nseq; ++i) base_items += (((int64_t)sq[i].nq * c->G + k.rows - 1) / k.rows) * c->Hkv;
    if (base_items >= 4 * slots) return INT32_MAX;
    for (int i = 0; i < nseq; ++i) most = std::max(most, most_keys(c, k, sees, sq[i]));
    const int64_t maxsteps = (most + k.keys - 1) / k.keys;
    double best = 0;
    int32_t best_chunk = INT32_MAX;
    int64_t last = 0;
    for (const int parts : kParts) {
        const int64_t ct = (maxsteps + parts - 1) / parts;   // steps per split
        if (ct == last || (parts > 1 && ct < 2)) continue;
        last = ct;
        const int64_t splits = (maxsteps + ct - 1) / ct;
        const int64_t partial = splits * total * c->Hq * (c->d + 2);
        if (splits > 1 && partial > c->attend_room) break;
        int64_t items = 0;
        double steps = 0, longest = 0;
        for (int i = 0; i < nseq; ++i) {
            const int64_t tiles = ((int64_t)sq[i].nq * c->G + k.rows - 1) / k.rows;
            const double share = (double)sq[i].mean / sq[i].n;
            for (int64_t t = 0; t < tiles; ++t)
                for (const auto& h : sees.heads) {
                    const int64_t st = (item_keys(c, k, sees, sq[i], t, h.first) + k.keys - 1) / k.keys;
                    items += (st + ct - 1) / ct * h.second;
                    steps += share * st * h.second;
                    longest = std::max(longest, (double)std::min(st, ct));
                }
        }
        double cost = std::max((steps + items * k.item_steps) / slots, longest + k.item_steps);
        if (items > slots) cost += 0.5 * longest;
        if (splits > 1) cost += k.join_steps + 8.0 * partial / k.step_bytes;
        if (parts == 1 || cost < best) {
            best = cost;
            best_chunk = splits > 1 ? (int32_t)(ct * k.keys) : INT32_MAX;
        }
    }
    return best_chunk;
}

// When the last of the items given out one by one, longest first, is done: `items`
// of (steps, count) in descending order.
double rounds(const std::vector<std::pair<double, int64_t>>& items, int64_t slots) {
    std::vector<std::pair<double, int64_t>> busy{{0.0, slots}};   // until when, slots; ascending
    for (auto [len, n] : items)
        while (n > 0) {
            auto [at, have] = busy.front();
            const int64_t m = std::min(n, have);
            if (m == have) busy.erase(busy.begin());
            else busy.front().second -= m;
            const auto to = std::lower_bound(busy.begin(), busy.end(), at + len, [](const auto& x, double y) { return x.first < y; });
            if (to != busy.end() && to->first == at + len) to->second += m;
            else busy.insert(to, {at + len, m});
            n -= m;
        }
    return busy.back().first;
}

// Windows and trees with a few more work items than SMs: the sequences that fill
// whole rounds stay whole, the others' keys are split to fill the last one.  64
// single tokens in windows of 2044 (512 items of 17 steps, 32/8 heads): 99.5 us, all
// whole 104.  With 256 rows an item partial results cost what it gains (60 tree nodes of
// twelve sequences, 192 items, 64/8 heads: 53 us whole, 60 split).
// (A model of cost alone: heads count as long as the sequence's longest, an item of
// one row tile as one of two.)
// Returns how many of the first sequences stay whole, *chunk keys per split of
// the others; all of them and INT32_MAX where that does not pay.
int attend_tail(const hikv_cache* c, const ItemShape& k, const Sees& sees, const AttendSeq* sq, int nseq, int32_t* chunk) {
    const int64_t slots = c->sm_count;
    *chunk = INT32_MAX;
    std::vector<std::pair<double, int64_t>> all;   // (steps, items) of every sequence and window
    std::vector<int> of;                           // its sequence
    int64_t items = 0, most = 0;
    int whole = 0;
    for (int i = 0; i < nseq; ++i) {
        const int64_t tiles = ((int64_t)sq[i].nq * c->G + k.rows - 1) / k.rows;
        items += tiles * c->Hkv;
        for (const auto& h : sees.heads) {
            const int64_t keys = most_keys(c, k, sees, sq[i], h.first);
            all.push_back({(double)((keys + k.keys - 1) / k.keys), tiles * h.second});
            of.push_back(i);
            most = std::max(most, keys);
        }
    }
    if (items <= slots || items >= 4 * slots) return nseq;
    int64_t full = 0;
    for (; whole < nseq; ++whole) {
        const int64_t n = (((int64_t)sq[whole].nq * c->G + k.rows - 1) / k.rows) * c->Hkv;
        if (full + n > items / slots * slots) break;
        full += n;
    }
    const int64_t maxsteps = (most + k.keys - 1) / k.keys;
    auto cost = [&](int first, int64_t ct) {   // sequences from `first` on split into parts of ct steps
        std::vector<std::pair<double, int64_t>> parts;
        for (size_t x = 0; x < all.size(); ++x) {
            const auto [st, n] = all[x];
            if (of[x] < first || st <= ct) parts.push_back({st + k.item_steps, n});
            else {
                const int64_t p = (int64_t)st / ct;
                parts.push_back({ct + k.item_steps, p * n});
                if (st - p * ct > 0) parts.push_back({st - p * ct + k.item_steps, n});
            }
        }
        std::sort(parts.begin(), parts.end(), [](const auto& x, const auto& y) { return x.first > y.first; });
        size_t n = 0;   // those of a length as one
        for (const auto& p : parts)
            if (n > 0 && parts[n - 1].first == p.first) parts[n - 1].second += p.second;
            else parts[n++] = p;
        parts.resize(n);
        return rounds(parts, slots);
    };
    double best = cost(nseq, maxsteps);
    int best_whole = nseq;
    int64_t tokens = 0;
    for (int i = whole; i < nseq; ++i) tokens += sq[i].nq;
    for (const int parts : {2, 3, 4}) {
        const int64_t ct = (maxsteps + parts - 1) / parts, splits = (maxsteps + ct - 1) / ct;
        const int64_t partial = splits * tokens * c->Hq * (c->d + 2);
        if (ct < 2 || partial > c->attend_room) break;
        const double x = cost(whole, ct) + k.join_steps + 8.0 * partial / k.step_bytes;
        if (x < best) {
            best = x;
            best_whole = whole;
            *chunk = (int32_t)(ct * k.keys);
        }
    }
    return best_whole;
}

cudaError_t launch_kernels(const hikv_cache* c, const Sees& sees, const AttendArgs& a, const CUtensorMap& qmap, cudaStream_t s) {
    const bool bf16 = c->dtype == HIKV_BF16;
    if (sees.kind == WindowMask::kind)
        return bf16 ? launch_attend_tc_window(a, sees.window, qmap, c->tmap_page, c->d, s)
                    : launch_attend_f32_window(a, sees.window, c->d, s);
    if (sees.kind == TreeMask::kind)
        return bf16 ? launch_attend_tc_tree(a, sees.tree, qmap, c->tmap_page, c->d, s)
                    : launch_attend_f32_tree(a, sees.tree, c->d, s);
    return bf16 ? launch_attend_tc(a, qmap, c->tmap_page, c->d, s) : launch_attend_f32(a, c->d, s);
}
cudaError_t launch_join(const hikv_cache* c, const Sees& sees, const AttendArgs& a, cudaStream_t s) {
    if (sees.kind == WindowMask::kind) return launch_attend_join_window(a, sees.window, c->dtype, c->d, s);
    if (sees.kind == TreeMask::kind) return launch_attend_join_tree(a, sees.tree, c->dtype, c->d, s);
    return launch_attend_join(a, c->dtype, c->d, s);
}

// The launches of the packed attention calls, their arguments checked.
hikv_status attend_launch(hikv_cache* c, int u0, const int32_t* nq, int64_t total, const hikv_rows* q,
                          const hikv_rows* out, Sees& sees, hikv_stream_t stream, const char* who) {
    DeviceGuard guard(c->device);
    if (guard.status != cudaSuccess) return cuda_fail(guard.status, who, "device");
    pdl_forget(c);
    const bool bf16 = c->dtype == HIKV_BF16;
    sees.window.align = bf16 ? std::min(c->P, 128) : 1;   // rows of a box of the tensor map of the pages
    if (sees.kind != WindowMask::kind) sees.heads.assign(1, {kAllSlots, c->Hkv});
    CUtensorMap qmap;
    if (bf16) {
        // q as [tokens][heads][d], boxes of 128 query rows x 128 bytes
        cuuint64_t dims[3] = {(cuuint64_t)c->d, (cuuint64_t)c->Hq, (cuuint64_t)total};
        cuuint64_t strides[2] = {(cuuint64_t)(c->Hq > 1 ? q->head_stride : c->d) * 2,
                                 (cuuint64_t)(total > 1 ? q->token_stride : c->d) * 2};
        cuuint32_t box[3] = {64u, (cuuint32_t)c->G, (cuuint32_t)(128 / c->G)};
        cuuint32_t estr[3] = {1u, 1u, 1u};
        const CUresult r = tensor_map_encoder()(
            &qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q->data, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(HIKV_ERR_INVALID_ARG, "%s: no tensor map of q (%d)", who, (int)r);
    }
    AttendArgs a{};
    a.v = c->v;
    a.u0 = u0;
    while ((1 << a.gshift) < c->G) ++a.gshift;
    a.hkv_shift = 0;
    while ((1 << a.hkv_shift) < c->Hkv) ++a.hkv_shift;
    if ((1 << a.hkv_shift) != c->Hkv) a.hkv_shift = -1;
    a.q = rows_arg(c, q);
    a.out = rows_arg(c, out);
    a.qscale = c->scale * 1.4426950408889634f;
    a.part_rows = total * c->Hq;
    // the sequences with queries, longest first: the work items start with the heaviest
    std::vector<AttendSeq> seqs;
    for (int b = 0, row = 0; b < c->B; row += nq[b++])
        if (nq[b] > 0) {
            const int32_t* len = c->len.data() + u0 + b * c->Hkv;
            int64_t sum = 0;
            bool equal = true;
            for (int g = 0; g < c->Hkv; ++g) {
                sum += len[g];
                equal &= len[g] == len[0];
            }
            seqs.push_back({b, row, nq[b], *std::max_element(len, len + c->Hkv), (int32_t)(sum / c->Hkv), equal});
        }
    std::stable_sort(seqs.begin(), seqs.end(), [](const AttendSeq& x, const AttendSeq& y) { return x.n > y.n; });
    const ItemShape& shape = bf16 ? kTcShape : kF32Shape;
    for (size_t s0 = 0; s0 < seqs.size(); s0 += kAttSeqs) {
        a.nseq = (int32_t)std::min<size_t>(kAttSeqs, seqs.size() - s0);
        const AttendSeq* sq = seqs.data() + s0;
        a.chunk = attend_chunk(c, shape, sees, sq, a.nseq, total);
        int whole = 0;   // of the first sequences, those that stay whole
        if (sees.kind != CausalMask::kind && a.chunk == INT32_MAX)
            whole = attend_tail(c, shape, sees, sq, a.nseq, &a.chunk);
        a.once = std::all_of(sq, sq + a.nseq, [&](const AttendSeq& s) { return (int64_t)s.nq * c->G <= shape.rows; });
        int64_t items = 0, split_tokens = 0, splits_max = 0;
        for (int i = 0; i < a.nseq; ++i) {
            const int64_t tiles = ((int64_t)sq[i].nq * c->G + shape.rows - 1) / shape.rows;
            const int64_t splits = i < whole ? 1 : (most_keys(c, shape, sees, sq[i]) + a.chunk - 1) / a.chunk;
            a.brow[i] = sq[i].brow;
            a.start[i] = sq[i].start;
            a.nq[i] = sq[i].nq;
            a.len[i] = sq[i].equal ? sq[i].n : -1;
            a.parts[i] = (int32_t)splits;
            a.item0[i] = (int32_t)items;
            a.comb0[i] = (int32_t)split_tokens;
            items += tiles * splits * c->Hkv;
            split_tokens += splits > 1 ? sq[i].nq : 0;
            splits_max = std::max(splits_max, splits);
        }
        if (items > INT32_MAX) return fail(HIKV_ERR_UNSUPPORTED, "%s: too many queries in one call", who);
        a.item0[a.nseq] = a.items = (int32_t)items;
        a.comb0[a.nseq] = (int32_t)split_tokens;
        a.splits = (int32_t)splits_max;
        if (sees.kind != CausalMask::kind) a.part_rows = split_tokens * c->Hq;
        a.part = c->d_logits;
        a.part_ml = c->d_logits + splits_max * a.part_rows * c->d;
        cudaError_t e = launch_kernels(c, sees, a, qmap, (cudaStream_t)stream);
        c->launches += 1;
        if (e == cudaSuccess && split_tokens > 0) {
            e = launch_join(c, sees, a, (cudaStream_t)stream);
            c->launches += 1;
        }
        if (e != cudaSuccess) return cuda_fail(e, who, "launch");
    }
    return HIKV_OK;
}

// The checks that the packed attention calls share; *total = 0: nothing to do
hikv_status attend_check(const hikv_cache* c, int32_t layer, const int32_t* nq, const hikv_rows* q, const hikv_rows* out,
                         int64_t* total, const char* who) {
    *total = 0;
    if (!range_ok(c, layer, 1)) return fail(HIKV_ERR_INVALID_ARG, "%s: bad cache or layer", who);
    if (!nq || !q || !out) return fail(HIKV_ERR_INVALID_ARG, "%s: null nq, q or out", who);
    const int64_t n = packed_total(c, nq);
    if (n < 0) return fail(HIKV_ERR_INVALID_ARG, "%s: a query count is negative or their sum too large", who);
    if (n == 0) return HIKV_OK;
    if (n * c->Hq > INT32_MAX / 2) return fail(HIKV_ERR_UNSUPPORTED, "%s: too many queries in one call", who);
    const char* bad = nullptr;
    if ((bad = rows_fault(c, q, n, c->Hq, true))) return fail(HIKV_ERR_INVALID_ARG, "%s: q has %s", who, bad);
    if ((bad = rows_fault(c, out, n, c->Hq, true))) return fail(HIKV_ERR_INVALID_ARG, "%s: out has %s", who, bad);
    if (rows_meet(c, out, c->Hq, q, c->Hq, n)) return fail(HIKV_ERR_INVALID_ARG, "%s: out overlaps q", who);
    const int u0 = layer * c->per_layer;
    for (int i = 0; i < c->per_layer; ++i)
        if (nq[i / c->Hkv] > c->tail[u0 + i])
            return fail(HIKV_ERR_STATE, "%s: %d queries of unit %d, which holds its newest %d in order", who,
                        nq[i / c->Hkv], u0 + i, c->tail[u0 + i]);
    *total = n;
    return HIKV_OK;
}

// attend_launch for a C caller
hikv_status attend_call(hikv_cache* c, int32_t layer, const int32_t* nq, int64_t total, const hikv_rows* q,
                        const hikv_rows* out, Sees& sees, hikv_stream_t stream, const char* who) {
    try {
        return attend_launch(c, layer * c->per_layer, nq, total, q, out, sees, stream, who);
    } catch (const std::bad_alloc&) {
        return fail(HIKV_ERR_OUT_OF_MEMORY, "%s: host memory", who);
    }
}

}  // namespace

extern "C" {

namespace {
// hikv_append_packed, and (tree) hikv_append_tree
hikv_status append_rows(hikv_cache* c, int32_t layer, const int32_t* ntok, bool tree, const int32_t* depth, const hikv_rows* k,
                        const hikv_rows* vv, const hikv_rows* q, const hikv_rows* q_out, const hikv_rope* rope,
                        hikv_stream_t stream, const char* who) {
    if (!range_ok(c, layer, 1)) return fail(HIKV_ERR_INVALID_ARG, "%s: bad cache or layer", who);
    if (!ntok || !k || !vv) return fail(HIKV_ERR_INVALID_ARG, "%s: null ntok, k or v", who);
    const int64_t total = packed_total(c, ntok);
    if (total < 0) return fail(HIKV_ERR_INVALID_ARG, "%s: a token count is negative or their sum too large", who);
    if (total == 0) return HIKV_OK;
    if ((q != nullptr) != (q_out != nullptr))
        return fail(HIKV_ERR_INVALID_ARG, "%s: q and q_out go together", who);
    if (q && !rope) return fail(HIKV_ERR_INVALID_ARG, "%s: q without a rope", who);
    if (tree && (!depth || ((uintptr_t)depth & 3) || !rope))
        return fail(HIKV_ERR_INVALID_ARG, "%s: null or misaligned depth, or no rope", who);
    const char* bad = nullptr;
    if ((bad = rows_fault(c, k, total, c->Hkv, false))) return fail(HIKV_ERR_INVALID_ARG, "%s: k has %s", who, bad);
    if ((bad = rows_fault(c, vv, total, c->Hkv, false))) return fail(HIKV_ERR_INVALID_ARG, "%s: v has %s", who, bad);
    if (q) {
        if ((bad = rows_fault(c, q, total, c->Hq, false))) return fail(HIKV_ERR_INVALID_ARG, "%s: q has %s", who, bad);
        if ((bad = rows_fault(c, q_out, total, c->Hq, true)))
            return fail(HIKV_ERR_INVALID_ARG, "%s: q_out has %s", who, bad);
        if (q->data == q_out->data && (q->token_stride != q_out->token_stride || q->head_stride != q_out->head_stride))
            return fail(HIKV_ERR_INVALID_ARG, "%s: q_out in the place of q needs its strides", who);
        if ((q->data != q_out->data && rows_meet(c, q_out, c->Hq, q, c->Hq, total)) ||
            rows_meet(c, q_out, c->Hq, k, c->Hkv, total) || rows_meet(c, q_out, c->Hq, vv, c->Hkv, total))
            return fail(HIKV_ERR_INVALID_ARG, "%s: q_out overlaps q, k or v", who);
    }
    if (rope) {
        if (!rope->cos || !rope->sin || (((uintptr_t)rope->cos | (uintptr_t)rope->sin) & 15))
            return fail(HIKV_ERR_INVALID_ARG, "%s: null or misaligned rope tables", who);
        if (rope->interleaved != 0 && rope->interleaved != 1)
            return fail(HIKV_ERR_INVALID_ARG, "%s: interleaved %d not in {0, 1}", who, rope->interleaved);
        if (rope->rot_dim < 16 || rope->rot_dim > c->d || rope->rot_dim % 16)
            return fail(HIKV_ERR_UNSUPPORTED, "%s: rot_dim %d is no multiple of 16 up to head_dim %d", who,
                        rope->rot_dim, c->d);
    }
    const int u0 = layer * c->per_layer, Hkv = c->Hkv;
    int64_t new_pages = 0;
    for (int b = 0; b < c->B; ++b) {
        const int m = ntok[b];
        if (m == 0) continue;
        const int ub = u0 + b * Hkv;
        const int32_t *len = c->len.data() + ub, *mapped = c->mapped.data() + ub, *next_pos = c->next_pos.data() + ub;
        for (int g = 0; g < Hkv; ++g) {
            if ((int64_t)len[g] + m > c->cap)
                return fail(HIKV_ERR_CAPACITY, "%s: unit %d would hold %lld > max_tokens %d", who, ub + g,
                            (long long)len[g] + m, c->cap);
            if (next_pos[g] != next_pos[0])
                return fail(HIKV_ERR_STATE, "%s: units %d and %d are at different positions", who, ub + g, ub);
            new_pages += std::max(0, ((len[g] + m - 1) >> c->page_shift) + 1 - mapped[g]);
        }
        const int64_t end = (int64_t)next_pos[0] + m;
        if (end > INT32_MAX) return fail(HIKV_ERR_CAPACITY, "%s: positions of batch row %d overflow int32", who, b);
        if (rope && end > rope->positions)
            return fail(HIKV_ERR_INVALID_ARG, "%s: batch row %d reaches position %lld, the rope has %d", who, b,
                        (long long)end - 1, rope->positions);
    }
    if (c->pages_in_use + new_pages > c->pool_pages)
        return fail(HIKV_ERR_CAPACITY, "%s: page pool exhausted (%lld in use + %lld > %lld)", who,
                    (long long)c->pages_in_use, (long long)new_pages, (long long)c->pool_pages);
    DeviceGuard guard(c->device);
    if (guard.status != cudaSuccess) return cuda_fail(guard.status, who, "device");
    pdl_forget(c);
    PackedAppendArgs a{};
    a.v = c->v;
    a.u0 = u0;
    a.k = rows_arg(c, k);
    a.vv = rows_arg(c, vv);
    if (q) {
        a.q = rows_arg(c, q);
        a.qo = rows_arg(c, q_out);
    }
    if (rope) {
        a.cos = rope->cos;
        a.sin = rope->sin;
        a.rot = rope->rot_dim;
        a.interleaved = rope->interleaved;
        a.depth = depth;
    }
    int32_t row = 0;
    for (int b0 = 0; b0 < c->B; b0 += kSeqMax) {
        const int n = std::min(kSeqMax, c->B - b0);
        a.seqs.n = n;
        a.seqs.row0 = b0;
        for (int i = 0; i < n; ++i) {
            a.seqs.start[i] = row;
            row += ntok[b0 + i];
        }
        a.seqs.start[n] = row;
        if (row == a.seqs.start[0]) continue;
        // one launch where the host knows every slot: equal heads, no page to take
        bool known = true;
        for (int i = 0; i < n; ++i) {
            const int ub = u0 + (b0 + i) * Hkv, m = ntok[b0 + i];
            const int32_t *len = c->len.data() + ub, *mapped = c->mapped.data() + ub;
            a.pos0[i] = c->next_pos[ub];
            a.base[i] = len[0];
            if (m == 0) continue;
            for (int g = 0; g < Hkv; ++g) known &= len[g] == len[0] && ((len[g] + m - 1) >> c->page_shift) < mapped[g];
        }
        a.reserved = known ? nullptr : c->d_append_base;
        cudaError_t e = launch_append_packed(a, c->dtype, c->sm_count, (cudaStream_t)stream);
        c->launches += known ? 1 : 2;
        if (e != cudaSuccess) return cuda_fail(e, who, "launch");
        for (int i = 0; i < n; ++i) {
            const int m = ntok[b0 + i], ub = u0 + (b0 + i) * Hkv;
            if (m == 0) continue;
            for (int u = ub; u < ub + Hkv; ++u) {
                c->len[u] += m;
                c->next_pos[u] += m;
                c->tail[u] += m;
                c->fresh[u] = 0;
                const int pages = ((c->len[u] - 1) >> c->page_shift) + 1;
                if (pages > c->mapped[u]) {
                    c->pages_in_use += pages - c->mapped[u];
                    c->mapped[u] = pages;
                }
            }
        }
    }
    return HIKV_OK;
}

}  // namespace

hikv_status hikv_append_packed(hikv_cache* c, int32_t layer, const int32_t* ntok, const hikv_rows* k,
                               const hikv_rows* vv, const hikv_rows* q, const hikv_rows* q_out,
                               const hikv_rope* rope, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_append_packed");
    return append_rows(c, layer, ntok, false, nullptr, k, vv, q, q_out, rope, stream, "append_packed");
}

hikv_status hikv_append_tree(hikv_cache* c, int32_t layer, const int32_t* ntok, const int32_t* depth,
                             const hikv_rows* k, const hikv_rows* vv, const hikv_rows* q, const hikv_rows* q_out,
                             const hikv_rope* rope, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_append_tree");
    return append_rows(c, layer, ntok, true, depth, k, vv, q, q_out, rope, stream, "append_tree");
}

hikv_status hikv_attend_packed(hikv_cache* c, int32_t layer, const int32_t* nq, const hikv_rows* q,
                               const hikv_rows* out, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_attend_packed");
    int64_t total;
    const hikv_status st = attend_check(c, layer, nq, q, out, &total, "attend_packed");
    if (st != HIKV_OK || total == 0) return st;
    Sees sees;
    return attend_call(c, layer, nq, total, q, out, sees, stream, "attend_packed");
}

hikv_status hikv_attend_window(hikv_cache* c, int32_t layer, const int32_t* nq, const int32_t* window, int32_t sink,
                               const hikv_rows* q, const hikv_rows* out, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_attend_window");
    int64_t total;
    const hikv_status st = attend_check(c, layer, nq, q, out, &total, "attend_window");
    if (st != HIKV_OK) return st;
    if (!window || sink < 0) return fail(HIKV_ERR_INVALID_ARG, "attend_window: null window or negative sink");
    for (int g = 0; g < c->Hkv; ++g)
        if (window[g] < 0) return fail(HIKV_ERR_INVALID_ARG, "attend_window: window[%d]=%d is negative", g, window[g]);
    if (c->Hkv > kAttHeads)
        return fail(HIKV_ERR_UNSUPPORTED, "attend_window: %d KV heads, more than %d", c->Hkv, kAttHeads);
    if (total == 0) return HIKV_OK;
    const int u0 = layer * c->per_layer;
    int longest = 0;
    for (int i = 0; i < c->per_layer; ++i) {
        const int u = u0 + i, n = nq[i / c->Hkv], w = window[i % c->Hkv];
        if (n == 0) continue;
        longest = std::max(longest, c->len[u]);
        // a cut moves survivors: the window has to lie in what was appended since, the first tokens where they stay
        if (w > 0 && c->tail[u] < c->len[u] && (c->tail[u] < (int64_t)n + w - 1 || sink > c->S))
            return fail(HIKV_ERR_STATE,
                        "attend_window: unit %d was cut and holds its newest %d in order, %d queries with a window of %d "
                        "need %lld, and at most %d first tokens", u, c->tail[u], n, w, (long long)n + w - 1, c->S);
    }
    Sees sees;
    sees.window.sink = std::min(sink, c->cap);
    bool hides = false;
    try {
        for (int g = 0; g < c->Hkv; ++g) {
            // (a window that reaches the first tokens hides nothing)
            const int32_t w = window[g] == 0 || (int64_t)window[g] + sink >= longest ? kAllSlots : window[g];
            sees.window.window[g] = w;
            hides |= w != kAllSlots;
            auto h = std::find_if(sees.heads.begin(), sees.heads.end(), [&](const auto& x) { return x.first == w; });
            if (h != sees.heads.end()) ++h->second;
            else sees.heads.push_back({w, 1});
        }
    } catch (const std::bad_alloc&) {
        return fail(HIKV_ERR_OUT_OF_MEMORY, "attend_window: host memory");
    }
    sees.kind = hides ? WindowMask::kind : CausalMask::kind;
    std::sort(sees.heads.begin(), sees.heads.end(), [](const auto& x, const auto& y) { return x.first > y.first; });
    WindowMask& m = sees.window;
    int at = 0;
    for (const auto& h : sees.heads) {
        m.first[m.classes++] = (uint8_t)at;
        for (int g = 0; g < c->Hkv; ++g)
            if (m.window[g] == h.first) m.order[at++] = (uint8_t)g;
    }
    m.first[m.classes] = (uint8_t)at;
    return attend_call(c, layer, nq, total, q, out, sees, stream, "attend_window");
}

hikv_status hikv_attend_tree(hikv_cache* c, int32_t layer, const int32_t* nq, const uint32_t* mask, int32_t words,
                             const hikv_rows* q, const hikv_rows* out, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_attend_tree");
    for (int b = 0; c && nq && b < c->B; ++b)
        if (nq[b] > 32 * (int64_t)words)
            return fail(HIKV_ERR_INVALID_ARG, "attend_tree: %d words a row for the %d nodes of batch row %d", words, nq[b], b);
    int64_t total;
    const hikv_status st = attend_check(c, layer, nq, q, out, &total, "attend_tree");
    if (st != HIKV_OK || total == 0) return st;
    if (!mask || ((uintptr_t)mask & 3)) return fail(HIKV_ERR_INVALID_ARG, "attend_tree: null or misaligned mask");
    Sees sees;
    sees.kind = TreeMask::kind;
    sees.tree = {mask, words};
    return attend_call(c, layer, nq, total, q, out, sees, stream, "attend_tree");
}

hikv_status hikv_drop(hikv_cache* c, int32_t layer0, int32_t nl, const int32_t* ndrop, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_drop");
    if (!range_ok(c, layer0, nl)) return fail(HIKV_ERR_INVALID_ARG, "drop: bad cache or layer range");
    const int u0 = layer0 * c->per_layer;
    auto count = [&](int b) { return ndrop ? ndrop[b] : -1; };
    bool any = false;
    for (int b = 0; b < c->B; ++b) {
        if (count(b) < -1) return fail(HIKV_ERR_INVALID_ARG, "drop: %d tokens of batch row %d", count(b), b);
        any |= count(b) != 0;
    }
    if (!any) return HIKV_OK;
    const int rows = nl * c->B;   // (layer, batch row) pairs
    for (int r = 0; r < rows; ++r) {
        const int n = count(r % c->B), ub = u0 + r * c->Hkv;
        for (int u = ub; u < ub + c->Hkv; ++u)
            if (n > c->tail[u])
                return fail(HIKV_ERR_STATE, "drop: %d tokens of unit %d, which holds its newest %d in order", n, u,
                            c->tail[u]);
    }
    DeviceGuard guard(c->device);
    if (guard.status != cudaSuccess) return cuda_fail(guard.status, "drop: device");
    pdl_forget(c);
    DropArgs a{};
    a.v = c->v;
    a.layer0 = layer0;
    a.nlayers = nl;
    for (int b0 = 0; b0 < c->B; b0 += kDropMax) {
        a.row0 = b0;
        a.n = std::min(kDropMax, c->B - b0);
        for (int i = 0; i < a.n; ++i) a.count[i] = count(b0 + i);
        cudaError_t e = launch_drop(a, (cudaStream_t)stream);
        c->launches += 1;
        if (e != cudaSuccess) return cuda_fail(e, "drop: launch");
    }
    for (int r = 0; r < rows; ++r) {
        const int n = count(r % c->B), ub = u0 + r * c->Hkv;
        if (n == 0) continue;
        for (int u = ub; u < ub + c->Hkv; ++u) {
            const int left = n < 0 ? 0 : c->len[u] - n;
            c->next_pos[u] = n < 0 ? 0 : c->next_pos[u] - n;
            c->tail[u] = n < 0 ? 0 : c->tail[u] - n;
            c->len[u] = left;
            c->fresh[u] = 0;
            if (!c->v.home_pages) {
                const int mapped = std::min(c->mapped[u], ceil_div(left, c->P));
                c->pages_in_use -= c->mapped[u] - mapped;
                c->mapped[u] = mapped;
            }
        }
    }
    return HIKV_OK;
}

hikv_status hikv_device_view(const hikv_cache* c, hikv_view* out) {
    set_last_error("");
    if (!c || !out) return fail(HIKV_ERR_INVALID_ARG, "device_view: null cache or output");
    *out = hikv_view{};
    out->pool = c->v.pool;
    out->page_bytes = c->v.page_bytes;
    out->pool_pages = c->pool_pages;
    out->page_table = c->v.page_table;
    out->max_pages = c->max_pages;
    out->units = c->units;
    out->importance = c->v.imp;
    out->positions = c->v.pos;
    out->lengths = c->v.len;
    return HIKV_OK;
}

}  // extern "C"
