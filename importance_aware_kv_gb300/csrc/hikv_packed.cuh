// Definitions of the packed-batch kernels (hikv_append_packed,
// hikv_attend_packed, hikv_drop) beside the shared ones.
#pragma once

#include "hikv_internal.cuh"

namespace hikv {

enum : uint32_t { kWaitAttend = 9 };   // the next kWait* code: packed attention
// the next DEVERR_* bit: a wait of packed attention gave up (its launches start
// nothing more until the error is read: each work item would wait as long)
enum : uint32_t { DEVERR_ATTEND = 16u };
// A wait of these kernels, bounded as mbar_wait_bounded.  Where one gives up, it
// notes that in the CTA's word `where` (zero at first), which one thread records at
// the end: recording at each wait made the kernels 1 to 3 % slower.
__device__ __forceinline__ bool attend_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* where, uint32_t index,
                                            uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait_hint(bar, parity, 1000u)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 24); ++i) {
        if (mbar_try_wait_hint(bar, parity, 1000u)) return true;
        if ((i & 63u) == 63u && global_ns() - t0 > limit_ns) break;
    }
    *where = index;
    return false;
}
__device__ __forceinline__ void attend_record(uint32_t* err, uint32_t where, uint64_t limit_ns = kWaitLimitNs) {
    if (where == 0) return;
    atomicOr(err, DEVERR_ATTEND);
    record_timeout(err, kWaitAttend, where, limit_ns);
}
__device__ __forceinline__ bool attend_gave_up(const View& v) {
    return (*reinterpret_cast<const volatile uint32_t*>(v.err) & DEVERR_ATTEND) != 0;
}

// Address of the K (or V) row of slot s of unit u through unit_page (no table
// read with home pages); nullptr if the page is bad.
__device__ __forceinline__ uint8_t* slot_row(const View& v, int32_t u, int32_t s, bool is_v) {
    const int32_t pg = unit_page(v, u, s);
    if (pg < 0 || pg >= v.pool_pages) {
        atomicOr(v.err, DEVERR_PAGE);
        return nullptr;
    }
    const int32_t r = s & (v.page_tokens - 1);
    return v.pool + (int64_t)pg * v.page_bytes + ((is_v ? (int64_t)v.page_tokens : 0) + r) * v.row_bytes;
}

// Per unit: reserve ntok slots and map the pages they need.  Writes the
// first slot to base[u - u0] (-1 when the pool ran dry, which the host's
// capacity check makes impossible).
__device__ inline void reserve_unit(const View& v, int32_t u, int32_t ntok, int32_t* base_out) {
    int32_t n = v.len[u];
    int32_t need = ceil_div(n + ntok, v.page_tokens);
    int32_t m = v.mapped[u];
    if (n + ntok > v.cap || need > v.max_pages) {
        atomicOr(v.err, DEVERR_STATE);
        *base_out = -1;
        return;
    }
    if (need > m) {
        int32_t cnt = need - m;
        int32_t old = atomicSub(v.free_top, cnt);
        if (old - cnt < 0) {
            atomicAdd(v.free_top, cnt);
            atomicOr(v.err, DEVERR_POOL);
            *base_out = -1;
            return;
        }
        for (int32_t i = 0; i < cnt; ++i)
            v.page_table[(int64_t)u * v.max_pages + m + i] = v.free_stack[old - cnt + i];
        v.mapped[u] = need;
    }
    *base_out = n;
    v.len[u] = n + ntok;
    v.next_pos[u] += ntok;
}

// Leave unit u its first `left` tokens, the next one to be at next_pos; with a
// shared pool the whole pages past them go back.  One thread a unit; nothing may
// take pages in the same launch.
__device__ inline void shorten_unit(const View& v, int32_t u, int32_t left, int32_t next_pos) {
    v.len[u] = left;
    v.next_pos[u] = next_pos;
    v.victim[u] = -1;
    const int32_t keep = ceil_div(left, v.page_tokens), m = v.mapped[u];
    if (v.home_pages || m <= keep) return;
    const int32_t cnt = m - keep;
    const int32_t old = atomicAdd(v.free_top, cnt);
    if (old + cnt > v.pool_pages) atomicOr(v.err, DEVERR_POOL);
    for (int32_t i = 0; i < cnt; ++i) {
        const int64_t e = (int64_t)u * v.max_pages + keep + i;
        if (old + i < v.pool_pages) v.free_stack[old + i] = v.page_table[e];
        v.page_table[e] = -1;
    }
    v.mapped[u] = keep;
}

// 3-D tiled TMA load of box {x, y, z} of `tmap` into shared memory.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tmap, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// tma_load_2d with a policy for the lines that it brings into L2
__device__ __forceinline__ void tma_load_2d_hint(void* dst, const CUtensorMap* tmap, int32_t x, int32_t y, uint64_t* bar,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
        "%3}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// packed fp32 pair addition
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long*>(&d))
        : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)));
    return d;
}

// Launch `kernel` so that it may start before the previous grid in the stream
// has ended (programmatic dependent launch): every thread must call
// griddep_wait() before it touches anything another kernel reads or writes.
template <typename... P, typename... A>
inline cudaError_t launch_overlapped(void (*kernel)(P...), int32_t grid, int32_t threads, size_t smem, cudaStream_t s,
                                     const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A packed batch of one layer in kernel parameters: up to kSeqMax sequences,
// batch rows row0 .. row0 + n, sequence i's tokens at packed rows
// [start[i], start[i + 1]).  Parameters are copied with the launch, so calls
// need no device copy of the lengths and may be captured into a graph; longer
// batches take one launch per kSeqMax sequences.
constexpr int kSeqMax = 256;
struct PackedSeqs {
    int32_t n, row0;
    int32_t start[kSeqMax + 1];
};
// rows (t, h) of packed tensors, strides in bytes
struct RowsArg {
    uint8_t* p;
    int64_t ts, hs;
    __device__ __forceinline__ uint8_t* row(int64_t t, int32_t h) const { return p + t * ts + (int64_t)h * hs; }
};
struct PackedAppendArgs {
    View v;
    PackedSeqs seqs;
    int32_t u0;             // unit of (the layer, batch row 0, KV head 0)
    RowsArg k, vv, q, qo;   // q.p null: no queries
    const float* cos;       // null: no rotation
    const float* sin;
    int32_t rot, interleaved;
    int32_t slices;         // warps a token (set by the launch)
    int32_t pos0[kSeqMax];  // position of each sequence's first token
    int32_t base[kSeqMax];  // its slot, where the sequence's heads all hold as many tokens, else ...
    int32_t* reserved;      // ... scratch [units]: reserve slots and pages in a launch of their own (null: base)
    const int32_t* depth;   // turn by the first token's position + depth[row], not by the token's own (null)
};
cudaError_t launch_append_packed(PackedAppendArgs& a, int dtype, int sm_count, cudaStream_t s);

// Causal attention of packed queries over the cache (hikv_attend_packed).
// Query row r of a (sequence, KV head) is token r / G, head r % G of its
// group: the G heads that read one KV head share its tiles.  A work item is
// (sequence, tile of query rows, split of the keys, KV head), numbered
// sequence by sequence (longest first) and in a sequence from its last tile,
// which sees most, to its first.  As the packed batch above, the sequences
// come in kernel parameters.
constexpr int kAttSeqs = 128;
struct AttendArgs {
    View v;
    int32_t u0;             // unit of (the layer, batch row 0, KV head 0)
    int32_t gshift;         // log2(G)
    RowsArg q, out;
    float qscale;           // scale * log2(e)
    int32_t chunk;          // keys per split (a multiple of the kernel's key tile)
    float* part;            // partial results of split items: [splits][part_rows][d] outputs, ...
    float* part_ml;         // ... [splits][part_rows][2] references and sums
    int64_t part_rows;      // rows (t, h) of the packed batch; windows and trees: of its split sequences
    int32_t splits;         // the most parts a sequence's keys are split into
    int32_t hkv_shift;      // log2 of the KV heads, -1: no power of two
    int32_t once;           // every key is read by one work item
    int32_t nseq, items;
    int32_t brow[kAttSeqs];        // batch row
    int32_t start[kAttSeqs];       // first packed row
    int32_t nq[kAttSeqs];          // queries
    int32_t len[kAttSeqs];         // tokens its units hold, -1: not all the same (read v.len)
    int32_t parts[kAttSeqs];       // parts its keys are split into
    int32_t item0[kAttSeqs + 1];   // first work item
    int32_t comb0[kAttSeqs + 1];   // tokens of the sequences before it whose items are split
};
// the sequence that holds element x of a prefix table
__device__ __forceinline__ int32_t prefix_find(const int32_t* first, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}
// windows and trees: from a packed row of sequence i to its place among the split sequences' tokens
__device__ __forceinline__ int32_t part_token(const AttendArgs& a, int32_t i) { return a.comb0[i] - a.start[i]; }
// tokens of unit u, of sequence i of the call
__device__ __forceinline__ int32_t unit_len(const AttendArgs& a, int32_t i, int32_t u) {
    return a.len[i] >= 0 ? a.len[i] : a.v.len[u];
}
// What the queries of a call see (beside the slots up to the newest one).
//
// Causal: each query everything up to its own slot.
struct CausalMask {
    static constexpr int kind = 0;
};
// A window for every KV head: the newest window[g] slots up to the query's own,
// and the first `sink`.  The keys of a work item are then numbered without the
// slots between: number s is slot s below `gap` and slot s + shift from there
// on, where gap is `sink` and gap + shift the first row's window start, both
// rounded away from each other to multiples of `align` (the rows of a TMA box, 1
// where rows are loaded one by one).  In these numbers a row's window is as
// long as in slots, and no row sees a number from `sink` up to `gap`.
constexpr int kAttHeads = 128;
struct WindowMask {
    static constexpr int kind = 1;
    int32_t sink, align;
    int32_t window[kAttHeads];   // all slots: kAllSlots
    int32_t classes;             // heads of equal windows, the longest first: heads order[first[c]] .. of class c
    uint8_t first[kAttHeads + 1], order[kAttHeads];
};
constexpr int32_t kAllSlots = 0x3FFFFFFF;
// Trees: all slots in front of the sequence's new ones, and the new ones whose
// bits are set in the row's words (bit j of word j / 32: new slot j).
struct TreeMask {
    static constexpr int kind = 2;
    const uint32_t* bits;        // [packed rows][words]
    int32_t words;
};
// The head and the place among a head's items (of which there are `per`) of a
// sequence's work item: heads in turn, but for windows of several lengths those of
// the longest first, so that the longest items do not start last.
template <class M>
__device__ __forceinline__ void item_head(const AttendArgs& a, const M& m, int32_t item, int32_t per, int32_t& g, int32_t& x) {
    if constexpr (M::kind == 1) {
        int32_t c = 0;
        while (c + 1 < m.classes && m.first[c + 1] * per <= item) ++c;
        const int32_t heads = m.first[c + 1] - m.first[c], r = item - m.first[c] * per;
        x = r / heads;
        g = m.order[m.first[c] + r - x * heads];
    } else {
        x = a.hkv_shift >= 0 ? item >> a.hkv_shift : item / a.v.hkv;
        g = item - x * a.v.hkv;
    }
}
// the numbering of keys for rows from one that sees slots up to lim on
template <class M>
__device__ __forceinline__ void key_gap(const M& m, int32_t g, int32_t lim, int32_t& gap, int32_t& shift) {
    gap = shift = 0;
    if constexpr (M::kind == 1) {
        const int32_t start = max(lim - m.window[g] + 1, 0) & -m.align;
        gap = (m.sink + m.align - 1) & -m.align;
        shift = max(start - gap, 0);
    }
}
template <class M>
__device__ __forceinline__ int32_t key_slot(int32_t s, int32_t gap, int32_t shift) {
    return M::kind != 1 || s < gap ? s : s + shift;
}
// bits j < n of a word
__device__ __forceinline__ uint32_t bits_below(int32_t n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
// What one row sees: word k of its visible keys from key number s0 on.
template <class M>
struct RowSight;
template <>
struct RowSight<CausalMask> {   // (the kernels compare with the row's last slot instead)
    __device__ __forceinline__ RowSight(const CausalMask&, int32_t, int32_t, int32_t, int32_t, int32_t) {}
};
template <>
struct RowSight<WindowMask> {
    int32_t lim, from, sink;   // keys [from, lim], and below sink
    __device__ __forceinline__ RowSight(const WindowMask& m, int32_t g, int32_t, int32_t, int32_t, int32_t row_lim)
        : lim(row_lim), from(row_lim - m.window[g] + 1), sink(m.sink) {}
    __device__ __forceinline__ uint32_t word(int32_t s0) const {
        return bits_below(lim + 1 - s0) & (~bits_below(from - s0) | bits_below(sink - s0));
    }
};
template <>
struct RowSight<TreeMask> {
    const uint32_t* bits;
    int32_t seen0, nq;
    __device__ __forceinline__ RowSight(const TreeMask& m, int32_t, int32_t packed_row, int32_t before, int32_t n, int32_t)
        : bits(m.bits + (int64_t)packed_row * m.words), seen0(before), nq(n) {}
    // word i of the row, with ones before the tree's first slot and zeros past its last
    __device__ __forceinline__ uint32_t at(int32_t i) const {
        if (i < 0) return 0xFFFFFFFFu;
        return 32 * i < nq ? bits[i] & bits_below(nq - 32 * i) : 0u;
    }
    __device__ __forceinline__ uint32_t word(int32_t s0) const {
        const int32_t b = s0 - seen0, i = b >> 5;   // (rounds down)
        const uint32_t lo = at(i);
        return b & 31 ? __funnelshift_r(lo, at(i + 1), b & 31) : lo;
    }
    // (rare) Whether the row sees nothing.  A sum of weights of zero does not say so:
    // the logits of what it sees can all be -inf.
    __device__ __forceinline__ bool blind() const {
        if (seen0 > 0) return false;
        for (int32_t i = 0; 32 * i < nq; ++i)
            if (at(i)) return false;
        return true;
    }
};

cudaError_t launch_attend_tc(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kvmap, int d,
                             cudaStream_t s);
cudaError_t launch_attend_tc_window(const AttendArgs& a, const WindowMask& m, const CUtensorMap& qmap,
                                    const CUtensorMap& kvmap, int d, cudaStream_t s);
cudaError_t launch_attend_tc_tree(const AttendArgs& a, const TreeMask& m, const CUtensorMap& qmap,
                                  const CUtensorMap& kvmap, int d, cudaStream_t s);
constexpr int kTcRows = 256, kTcKeys = 128;    // query rows of a work item of the bf16 kernel, keys per tile
cudaError_t launch_attend_f32(const AttendArgs& a, int d, cudaStream_t s);
cudaError_t launch_attend_f32_window(const AttendArgs& a, const WindowMask& m, int d, cudaStream_t s);
cudaError_t launch_attend_f32_tree(const AttendArgs& a, const TreeMask& m, int d, cudaStream_t s);
constexpr int kF32Rows = 128, kF32Keys = 64;   // of the fp32 kernel
cudaError_t launch_attend_join(const AttendArgs& a, int dtype, int d, cudaStream_t s);
cudaError_t launch_attend_join_window(const AttendArgs& a, const WindowMask& m, int dtype, int d, cudaStream_t s);
cudaError_t launch_attend_join_tree(const AttendArgs& a, const TreeMask& m, int dtype, int d, cudaStream_t s);
cudaError_t launch_selftest_attend(const View& v, uint64_t limit_ns, cudaStream_t s);

// Trees of drafted tokens (hikv_tree_masks): parents to ancestors' bits and depths.
struct TreeArgs {
    PackedSeqs seqs;
    const int32_t* parent;
    uint32_t* mask;
    int32_t* depth;
    int32_t words;
    uint32_t* err;
};
cudaError_t launch_tree_masks(const TreeArgs& a, cudaStream_t s);

// hikv_accept: parts of the batch rows' lists of kept tokens, at most one part of a row in a launch
constexpr int kAcceptRows = 256, kAcceptIndex = 1024;
struct AcceptArgs {
    View v;
    int32_t layer0, nlayers, n;
    int32_t brow[kAcceptRows];
    int32_t tree[kAcceptRows];           // newest tokens that the row's list is of
    int32_t rank[kAcceptRows];           // place of this part's first token in the list
    int32_t last[kAcceptRows];           // tokens the row keeps in all where this is its last part, else -1
    int32_t start[kAcceptRows + 1];      // the part in index
    int32_t index[kAcceptIndex];
};
cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t s);

// hikv_fork: copies of batch rows, grouped by the row they are of
constexpr int kForkRows = 512;                        // copies of a launch
constexpr int kForkSlots = 32, kForkMeta = 1024;      // slots of a CTA: K and V, scores and positions
struct ForkArgs {
    View v;
    int32_t layer0, nlayers;
    int32_t groups, copies;
    int32_t meta, chunks;                // parts of the longest source, of kForkMeta and of kForkSlots slots ...
    int32_t from[kForkRows];             // ... [groups] from the first slot that a copy lacks on (whole parts)
    int32_t src[kForkRows];              // [groups]
    int32_t first[kForkRows + 1];        // [groups + 1] its copies
    int32_t dst[kForkRows], same[kForkRows];
};
cudaError_t launch_fork_release(const ForkArgs& a, cudaStream_t s);   // shared pools, debug mode
cudaError_t launch_fork_reserve(const ForkArgs& a, cudaStream_t s);   // shared pools
cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s);

constexpr int kDropMax = 512;
struct DropArgs {
    View v;
    int32_t layer0, nlayers, row0, n;   // batch rows row0 .. row0 + n of every layer of the range
    int32_t count[kDropMax];            // tokens to drop, -1: all
};
cudaError_t launch_drop(const DropArgs& a, cudaStream_t s);

}  // namespace hikv
