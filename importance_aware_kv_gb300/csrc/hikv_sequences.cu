// Host side of the entry points that treat a batch row as a sequence: trees of
// drafted tokens and the accepted path of each, copies of rows.  Checks, the
// host mirror and the launches, as in hikv_host.cu.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <new>
#include <vector>

#include "hikv_cache.cuh"
#include "hikv_packed.cuh"

using namespace hikv;

namespace {

// Host mirror of shorten_unit.
void shorten(hikv_cache* c, int u, int left, int next_pos) {
    c->len[u] = left;
    c->next_pos[u] = next_pos;
    c->fresh[u] = 0;
    if (c->v.home_pages) return;
    const int mapped = std::min(c->mapped[u], ceil_div(left, c->P));
    c->pages_in_use -= c->mapped[u] - mapped;
    c->mapped[u] = mapped;
}

hikv_status fork_launch(hikv_cache* c, int32_t layer0, int32_t nl, const int32_t* src, const int32_t* same,
                        hikv_stream_t stream) {
    // copies by source, then row
    std::vector<int32_t> rows;
    for (int b = 0; b < c->B; ++b)
        if (src[b] >= 0 && src[b] != b) rows.push_back(b);
    std::stable_sort(rows.begin(), rows.end(), [&](int32_t x, int32_t y) { return src[x] < src[y]; });
    DeviceGuard guard(c->device);
    if (guard.status != cudaSuccess) return cuda_fail(guard.status, "fork: device");
    pdl_forget(c);
    ForkArgs a{};
    a.v = c->v;
    a.layer0 = layer0;
    a.nlayers = nl;
    auto part = [&](size_t i0) {   // copies [i0, i0 + kForkRows)
        a.copies = (int32_t)std::min<size_t>(kForkRows, rows.size() - i0);
        a.groups = 0;
        int longest = 0, rest = 0;   // slots of a source, and those that not every copy shares
        for (int i = 0; i < a.copies; ++i) {
            const int b = rows[i0 + i], s = src[b];
            if (i == 0 || s != a.src[a.groups - 1]) {
                a.src[a.groups] = s;
                a.from[a.groups] = INT32_MAX;
                a.first[a.groups++] = i;
            }
            a.dst[i] = b;
            a.same[i] = same ? same[b] : 0;
            a.from[a.groups - 1] = std::min(a.from[a.groups - 1], a.same[i] / kForkSlots * kForkSlots);
        }
        a.first[a.groups] = a.copies;
        for (int x = 0; x < a.groups; ++x)
            for (int l = layer0; l < layer0 + nl; ++l)
                for (int g = 0; g < c->Hkv; ++g) {
                    const int n = c->len[(l * c->B + a.src[x]) * c->Hkv + g];
                    longest = std::max(longest, n);
                    rest = std::max(rest, n - a.from[x]);
                }
        a.meta = std::max(1, ceil_div(longest, kForkMeta));
        a.chunks = ceil_div(std::max(0, rest), kForkSlots);
    };
    // every page that goes back does so before the first is taken
    for (size_t i0 = 0; i0 < rows.size() && (!c->v.home_pages || c->v.debug); i0 += kForkRows) {
        part(i0);
        const cudaError_t e = launch_fork_release(a, (cudaStream_t)stream);
        c->launches += 1;
        if (e != cudaSuccess) return cuda_fail(e, "fork: launch");
    }
    for (size_t i0 = 0; i0 < rows.size(); i0 += kForkRows) {
        part(i0);
        cudaError_t e = cudaSuccess;
        if (!c->v.home_pages) {
            e = launch_fork_reserve(a, (cudaStream_t)stream);
            c->launches += 1;
        }
        if (e == cudaSuccess) {
            e = launch_fork(a, (cudaStream_t)stream);
            c->launches += 1;
        }
        if (e != cudaSuccess) return cuda_fail(e, "fork: launch");
        for (int i = 0; i < a.copies; ++i)
            for (int l = layer0; l < layer0 + nl; ++l)
                for (int g = 0; g < c->Hkv; ++g) {
                    const int u = (l * c->B + a.dst[i]) * c->Hkv + g, s = (l * c->B + src[a.dst[i]]) * c->Hkv + g;
                    if (c->len[u] > c->len[s]) shorten(c, u, c->len[s], 0);
                    c->len[u] = c->len[s];
                    c->next_pos[u] = c->next_pos[s];
                    c->tail[u] = c->tail[s];
                    c->fresh[u] = 0;
                    const int pages = ceil_div(c->len[u], c->P);
                    if (pages > c->mapped[u]) {
                        c->pages_in_use += pages - c->mapped[u];
                        c->mapped[u] = pages;
                    }
                }
    }
    return HIKV_OK;
}

}  // namespace

extern "C" {

hikv_status hikv_tree_masks(hikv_cache* c, const int32_t* ntok, const int32_t* parent, uint32_t* mask, int32_t words,
                            int32_t* depth, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_tree_masks");
    if (!c || !ntok) return fail(HIKV_ERR_INVALID_ARG, "tree_masks: null cache or ntok");
    int64_t total = 0;
    for (int b = 0; b < c->B; ++b) {
        if (ntok[b] < 0 || words < 1 || ntok[b] > 32 * (int64_t)words)
            return fail(HIKV_ERR_INVALID_ARG, "tree_masks: %d words a row for the %d nodes of batch row %d", words, ntok[b], b);
        total += ntok[b];
    }
    if (total > INT32_MAX) return fail(HIKV_ERR_INVALID_ARG, "tree_masks: too many nodes");
    if (total == 0) return HIKV_OK;
    if (!parent || !mask || !depth || (((uintptr_t)parent | (uintptr_t)mask | (uintptr_t)depth) & 3))
        return fail(HIKV_ERR_INVALID_ARG, "tree_masks: null or misaligned parent, mask or depth");
    DeviceGuard guard(c->device);
    if (guard.status != cudaSuccess) return cuda_fail(guard.status, "tree_masks: device");
    pdl_forget(c);
    TreeArgs a{};
    a.parent = parent;
    a.mask = mask;
    a.words = words;
    a.depth = depth;
    a.err = c->v.err;
    int32_t row = 0;
    for (int b0 = 0; b0 < c->B; b0 += kSeqMax) {
        a.seqs.n = std::min(kSeqMax, c->B - b0);
        a.seqs.row0 = b0;
        for (int i = 0; i < a.seqs.n; ++i) {
            a.seqs.start[i] = row;
            row += ntok[b0 + i];
        }
        a.seqs.start[a.seqs.n] = row;
        if (row == a.seqs.start[0]) continue;
        const cudaError_t e = launch_tree_masks(a, (cudaStream_t)stream);
        c->launches += 1;
        if (e != cudaSuccess) return cuda_fail(e, "tree_masks: launch");
    }
    return HIKV_OK;
}

hikv_status hikv_accept(hikv_cache* c, int32_t layer0, int32_t nl, const int32_t* ntree, const int32_t* naccept,
                        const int32_t* index, hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_accept");
    if (!range_ok(c, layer0, nl)) return fail(HIKV_ERR_INVALID_ARG, "accept: bad cache or layer range");
    if (!ntree || !naccept) return fail(HIKV_ERR_INVALID_ARG, "accept: null ntree or naccept");
    int64_t at = 0;
    bool any = false;
    for (int b = 0; b < c->B; ++b) {
        if (ntree[b] < 0 || naccept[b] < 0 || naccept[b] > ntree[b])
            return fail(HIKV_ERR_INVALID_ARG, "accept: %d of the newest %d tokens of batch row %d", naccept[b], ntree[b], b);
        if (naccept[b] > 0 && !index) return fail(HIKV_ERR_INVALID_ARG, "accept: null index");
        for (int j = 0; j < naccept[b]; ++j) {
            const int32_t x = index[at + j];
            if (x < (j ? index[at + j - 1] + 1 : 0) || x >= ntree[b])
                return fail(HIKV_ERR_INVALID_ARG, "accept: index %d of batch row %d is not ascending in [0, %d)", x, b, ntree[b]);
        }
        at += naccept[b];
        any |= ntree[b] > 0;
    }
    const int rows = nl * c->B, u0 = layer0 * c->per_layer;
    for (int r = 0; r < rows; ++r) {
        const int n = ntree[r % c->B], ub = u0 + r * c->Hkv;
        for (int u = ub; u < ub + c->Hkv; ++u)
            if (n > c->tail[u])
                return fail(HIKV_ERR_STATE, "accept: the newest %d tokens of unit %d, which holds its newest %d in order", n, u,
                            c->tail[u]);
    }
    if (!any) return HIKV_OK;
    DeviceGuard guard(c->device);
    if (guard.status != cudaSuccess) return cuda_fail(guard.status, "accept: device");
    pdl_forget(c);
    AcceptArgs a;   // (its lists are filled as far as they are used)
    a.n = a.start[0] = 0;
    a.v = c->v;
    a.layer0 = layer0;
    a.nlayers = nl;
    auto flush = [&] {
        if (a.n == 0) return cudaSuccess;
        const cudaError_t e = launch_accept(a, (cudaStream_t)stream);
        c->launches += 1;
        a.n = 0;
        return e;
    };
    at = 0;
    cudaError_t e = cudaSuccess;
    for (int b = 0; b < c->B && e == cudaSuccess; ++b) {
        if (ntree[b] == 0) continue;
        // a row's list in parts that fit, the next part in the next launch
        int done = 0;
        do {
            if (a.n == kAcceptRows || (a.n > 0 && a.start[a.n] == kAcceptIndex)) e = flush();
            const int room = kAcceptIndex - a.start[a.n], cnt = std::min(room, naccept[b] - done);
            a.brow[a.n] = b;
            a.tree[a.n] = ntree[b];
            a.rank[a.n] = done;
            std::copy(index + at + done, index + at + done + cnt, a.index + a.start[a.n]);
            done += cnt;
            a.last[a.n] = done == naccept[b] ? done : -1;
            a.start[a.n + 1] = a.start[a.n] + cnt;
            ++a.n;
            if (done < naccept[b] && e == cudaSuccess) e = flush();
        } while (done < naccept[b] && e == cudaSuccess);
        at += naccept[b];
    }
    if (e == cudaSuccess) e = flush();
    if (e != cudaSuccess) return cuda_fail(e, "accept: launch");
    for (int r = 0; r < rows; ++r) {
        const int b = r % c->B, gone = ntree[b] - naccept[b], ub = u0 + r * c->Hkv;
        if (ntree[b] == 0) continue;
        for (int u = ub; u < ub + c->Hkv; ++u) {
            c->tail[u] -= gone;
            shorten(c, u, c->len[u] - gone, c->next_pos[u] - gone);
        }
    }
    return HIKV_OK;
}

hikv_status hikv_fork(hikv_cache* c, int32_t layer0, int32_t nl, const int32_t* src, const int32_t* same,
                      hikv_stream_t stream) {
    set_last_error("");
    NvtxRange nvtx("hikv_fork");
    if (!range_ok(c, layer0, nl)) return fail(HIKV_ERR_INVALID_ARG, "fork: bad cache or layer range");
    if (!src) return fail(HIKV_ERR_INVALID_ARG, "fork: null src");
    bool any = false;
    int64_t pages = 0, longest = 0;
    for (int b = 0; b < c->B; ++b) {
        const int s = src[b];
        if (s < -1 || s >= c->B) return fail(HIKV_ERR_INVALID_ARG, "fork: batch row %d of row %d", b, s);
        if (s < 0 || s == b) continue;
        if (src[s] >= 0 && src[s] != s)
            return fail(HIKV_ERR_INVALID_ARG, "fork: batch row %d is to be a copy of row %d, itself a copy of row %d", b, s, src[s]);
        any = true;
        for (int l = layer0; l < layer0 + nl; ++l)
            for (int g = 0; g < c->Hkv; ++g) {
                const int u = (l * c->B + b) * c->Hkv + g, from = (l * c->B + s) * c->Hkv + g;
                if (same && (same[b] < 0 || same[b] > std::min(c->len[u], c->len[from])))
                    return fail(HIKV_ERR_INVALID_ARG, "fork: %d tokens of batch row %d are not to be copied, unit %d holds %d and unit %d %d",
                                same[b], b, u, c->len[u], from, c->len[from]);
                const int need = ceil_div(c->len[from], c->P);
                longest = std::max<int64_t>(longest, c->len[from]);
                if (c->v.home_pages) continue;
                pages += c->len[u] > c->len[from] ? std::min(c->mapped[u], need) - c->mapped[u]
                                                  : std::max(c->mapped[u], need) - c->mapped[u];
            }
    }
    if (!any) return HIKV_OK;
    if ((longest / kForkSlots + longest / kForkMeta + 2) * std::min(kForkRows, c->B) * nl * c->Hkv > INT32_MAX)
        return fail(HIKV_ERR_UNSUPPORTED, "fork: too much for one launch; fewer layers or rows a call");
    if (c->pages_in_use + pages > c->pool_pages)
        return fail(HIKV_ERR_CAPACITY, "fork: page pool exhausted (%lld in use + %lld > %lld)", (long long)c->pages_in_use,
                    (long long)pages, (long long)c->pool_pages);
    try {
        return fork_launch(c, layer0, nl, src, same, stream);
    } catch (const std::bad_alloc&) {
        return fail(HIKV_ERR_OUT_OF_MEMORY, "fork: host memory");
    }
}

}  // extern "C"
