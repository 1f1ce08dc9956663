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

// 3-D tiled TMA load of box {x, y, z} of `tmap` into shared memory.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tmap, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
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
    int64_t part_rows;      // rows (t, h) of the packed batch
    int32_t splits;         // the most parts a sequence's keys are split into
    int32_t hkv_shift;      // log2 of the KV heads, -1: no power of two
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
// tokens of unit u, of sequence i of the call
__device__ __forceinline__ int32_t unit_len(const AttendArgs& a, int32_t i, int32_t u) {
    return a.len[i] >= 0 ? a.len[i] : a.v.len[u];
}
cudaError_t launch_attend_tc(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kvmap, int d,
                             cudaStream_t s);
constexpr int kTcRows = 256, kTcKeys = 128;    // query rows of a work item of the bf16 kernel, keys per tile
cudaError_t launch_attend_f32(const AttendArgs& a, int d, cudaStream_t s);
constexpr int kF32Rows = 128, kF32Keys = 64;   // of the fp32 kernel
cudaError_t launch_attend_join(const AttendArgs& a, int dtype, int d, cudaStream_t s);
cudaError_t launch_selftest_attend(const View& v, uint64_t limit_ns, cudaStream_t s);

constexpr int kDropMax = 512;
struct DropArgs {
    View v;
    int32_t layer0, nlayers, row0, n;   // batch rows row0 .. row0 + n of every layer of the range
    int32_t count[kDropMax];            // tokens to drop, -1: all
};
cudaError_t launch_drop(const DropArgs& a, cudaStream_t s);

}  // namespace hikv
