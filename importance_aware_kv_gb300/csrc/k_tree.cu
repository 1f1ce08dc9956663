// Trees of drafted tokens: what each node sees, and the accepted path moved to
// the place of the tree.
//
// The nodes of a tree enter the cache in the caller's order, parents before
// children, in the unit's next slots.  Node i's mask has the bits of the nodes
// on its path to the root, its own among them; its depth is the path's length
// less one.  Both are bound by latency: a thread a node follows its path through
// the parents (a few dependent loads of one L2 line), from its own bit down, so
// that each word of the mask is complete when the path leaves it and is written
// once.
//
// Acceptance is a copy within every unit: list entry j's slot base + index[j]
// moves to base + j.  The list ascends, so index[j] >= j and a destination is
// never a later entry's source: a warp a unit, whose lanes each own 16-byte
// columns of the K and V rows, can load several entries ahead of their stores
// without a barrier.  Bound by latency as well: four of 32 nodes in 512 units take
// 5 to 6 us, the masks of those 2,048 nodes 3.4.
#include "hikv_packed.cuh"

namespace hikv {
namespace {

__global__ void __launch_bounds__(128) k_tree_masks(const __grid_constant__ TreeArgs a) {
    const int32_t t = a.seqs.start[0] + blockIdx.x * 128 + threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    if (t >= a.seqs.start[a.seqs.n]) return;
    const int32_t first = a.seqs.start[prefix_find(a.seqs.start, a.seqs.n, t)];
    uint32_t* row = a.mask + (int64_t)t * a.words;
    int32_t at = t - first, depth = -1;
    for (int32_t w = a.words - 1; w >= 0; --w) {
        uint32_t bits = 0;
        while (at >= 32 * w) {   // (at < 32 (w + 1): a parent is an earlier node)
            bits |= 1u << (at & 31);
            ++depth;
            const int32_t up = a.parent[first + at];
            if (up < -1 || up >= at) {
                atomicOr(a.err, DEVERR_STATE);
                at = -1;
            } else {
                at = up;
            }
        }
        row[w] = bits;
    }
    a.depth[t] = depth;
}

// warp per (layer, part of a row's list, KV head)
constexpr int kAhead = 4;   // entries in flight
__global__ void __launch_bounds__(128) k_accept(const __grid_constant__ AcceptArgs a) {
    const View& v = a.v;
    const int32_t w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    if (w >= a.nlayers * a.n * v.hkv) return;
    const int32_t g = w % v.hkv, i = w / v.hkv % a.n, layer = a.layer0 + w / v.hkv / a.n;
    const int32_t u = (layer * v.batch + a.brow[i]) * v.hkv + g;
    const int32_t n = v.len[u], base = n - a.tree[i];
    if (base < 0 || n > v.cap) {
        if (lane == 0) atomicOr(v.err, DEVERR_STATE);
        return;
    }
    const int32_t* index = a.index + a.start[i];
    const int32_t cnt = a.start[i + 1] - a.start[i], rank = a.rank[i];
    const int32_t vec = v.row_bytes / 16;   // 16-byte columns of a row: 8, 16 or 32
    // lane c owns columns c, c + 32 of the K row followed by the V row
    for (int32_t j0 = 0; j0 < cnt; j0 += kAhead) {
        for (int32_t c = lane; c < 2 * vec; c += 32) {
            const bool is_v = c >= vec;
            const int32_t col = is_v ? c - vec : c;
            uint4 x[kAhead];
            uint4* to[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                to[k] = nullptr;
                if (j0 + k >= cnt || index[j0 + k] == rank + j0 + k) continue;   // in its place already
                const uint8_t* src = slot_row(v, u, base + index[j0 + k], is_v);
                uint8_t* dst = slot_row(v, u, base + rank + j0 + k, is_v);
                if (!src || !dst) continue;
                x[k] = reinterpret_cast<const uint4*>(src)[col];
                to[k] = reinterpret_cast<uint4*>(dst) + col;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (to[k]) *to[k] = x[k];
        }
    }
    // scores move with their tokens; positions are the slots' own (a row's newest tokens count up)
    float* imp = v.imp + (int64_t)u * v.cap + base;
    for (int32_t j0 = 0; j0 < cnt; j0 += 32) {
        const int32_t j = j0 + lane;
        const float x = j < cnt ? imp[index[j]] : 0.f;
        __syncwarp();   // a destination of these is no later source, but may be one of theirs
        if (j < cnt) imp[rank + j] = x;
        __syncwarp();
    }
    if (a.last[i] < 0) return;
    const int32_t left = base + a.last[i];
    if (v.debug) {
        __syncwarp();
        for (int32_t s = left; s < n; ++s) poison_slot(v, u, s, lane, 32);
        __syncwarp();
    }
    if (lane == 0) shorten_unit(v, u, left, v.next_pos[u] - (n - left));
}

}  // namespace

cudaError_t launch_tree_masks(const TreeArgs& a, cudaStream_t s) {
    const int32_t total = a.seqs.start[a.seqs.n] - a.seqs.start[0];
    return launch_overlapped(k_tree_masks, ceil_div(total, 128), 128, 0, s, a);
}

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t s) {
    const int64_t warps = (int64_t)a.nlayers * a.n * a.v.hkv;   // at most the units of a cache
    return launch_overlapped(k_accept, (int32_t)((warps + 3) / 4), 128, 0, s, a);
}

}  // namespace hikv
