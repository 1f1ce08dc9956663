// Copies of whole sequences of the cache: rows of the batch become what other
// rows are.
//
// A copy, bound by bytes: a source's K and V rows are read once for all its
// copies and written once to each.  A CTA takes 32 slots of one unit of a
// source, every lane 16 bytes of several rows at once, and skips what a copy
// shares with its source already.  An 8K prompt of two layers to seven more rows
// (545 MB): 82 us, 0.98 of the copy rate; with 64 slots a CTA in two batches 91.
// Beams that share all but their newest 64 to 130 tokens: 7.3 us with the call (12.8
// where every CTA of 64 slots copied scores too, most of them nothing else).
#include <algorithm>

#include "hikv_packed.cuh"

namespace hikv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int32_t unit_of(const View& v, int32_t layer, int32_t row, int32_t g) {
    return (layer * v.batch + row) * v.hkv + g;
}
__device__ __forceinline__ int32_t group_of(const ForkArgs& a, int32_t c) { return prefix_find(a.first, a.groups, c); }

// Warp per unit of a copy, shared pools (and debug mode): give back the pages
// past what the source holds, poison what goes.
__global__ void __launch_bounds__(128) k_fork_release(const __grid_constant__ ForkArgs a) {
    const View& v = a.v;
    const int32_t w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    if (w >= a.nlayers * a.copies * v.hkv) return;
    const int32_t g = w % v.hkv, c = w / v.hkv % a.copies, layer = a.layer0 + w / v.hkv / a.copies;
    const int32_t u = unit_of(v, layer, a.dst[c], g), n = v.len[unit_of(v, layer, a.src[group_of(a, c)], g)];
    const int32_t old = v.len[u];
    if (old <= n) return;
    if (v.debug) {
        for (int32_t s = n; s < old; ++s) poison_slot(v, u, s, lane, 32);
        __syncwarp();
    }
    if (lane == 0) shorten_unit(v, u, n, v.next_pos[u]);
}

// Thread per unit of a copy, shared pools: take the pages that are missing.
__global__ void k_fork_reserve(const __grid_constant__ ForkArgs a) {
    const View& v = a.v;
    const int32_t w = blockIdx.x * blockDim.x + threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    if (w >= a.nlayers * a.copies * v.hkv) return;
    const int32_t g = w % v.hkv, c = w / v.hkv % a.copies, layer = a.layer0 + w / v.hkv / a.copies;
    const int32_t u = unit_of(v, layer, a.dst[c], g), n = v.len[unit_of(v, layer, a.src[group_of(a, c)], g)];
    int32_t first;
    if (n > v.len[u]) reserve_unit(v, u, n - v.len[u], &first);
}

// CTA per (source, layer, KV head, part): first the parts of the scores and
// positions, then those of K and V
template <int VEC>
__global__ void __launch_bounds__(kThreads) k_fork(const __grid_constant__ ForkArgs a) {
    constexpr int BATCH = kForkSlots * 2 * VEC / kThreads;   // 16-byte columns of a lane, all in flight at once
    const View& v = a.v;
    const int32_t parts = a.meta + a.chunks;
    const int32_t part = blockIdx.x % parts, x = blockIdx.x / parts;
    const int32_t g = x % v.hkv, y = x / v.hkv, layer = a.layer0 + y % a.nlayers, grp = y / a.nlayers;
    const int32_t us = unit_of(v, layer, a.src[grp], g), c0 = a.first[grp], c1 = a.first[grp + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int32_t n = v.len[us];
    if (n > v.cap) {
        if (threadIdx.x == 0) atomicOr(v.err, DEVERR_STATE);
        return;
    }
    if (part < a.meta) {
        if (part == 0 && threadIdx.x == 0) {
            const int32_t next_pos = v.next_pos[us];
            for (int32_t c = c0; c < c1; ++c) {
                const int32_t u = unit_of(v, layer, a.dst[c], g);
                v.len[u] = n;
                v.next_pos[u] = next_pos;
                v.victim[u] = -1;
            }
        }
        const int32_t s0 = part * kForkMeta + threadIdx.x;
        float imp[kForkMeta / kThreads];
        int32_t pos[kForkMeta / kThreads];
#pragma unroll
        for (int k = 0; k < kForkMeta / kThreads; ++k) {
            const int32_t s = s0 + k * kThreads;
            if (s < n) {
                imp[k] = v.imp[(int64_t)us * v.cap + s];
                pos[k] = v.pos[(int64_t)us * v.cap + s];
            }
        }
        for (int32_t c = c0; c < c1; ++c) {
            const int64_t at = (int64_t)unit_of(v, layer, a.dst[c], g) * v.cap;
#pragma unroll
            for (int k = 0; k < kForkMeta / kThreads; ++k) {
                const int32_t s = s0 + k * kThreads;
                if (s < n) {
                    v.imp[at + s] = imp[k];
                    v.pos[at + s] = pos[k];
                }
            }
        }
        return;
    }
    const int32_t s0 = a.from[grp] + (part - a.meta) * kForkSlots;
    if (s0 >= n) return;
    // columns of the K rows, then of the V rows
    uint4 d[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
        const int32_t i = threadIdx.x + k * kThreads, s = s0 + i / VEC % kForkSlots;
        const uint8_t* p = s < n ? slot_row(v, us, s, i >= kForkSlots * VEC) : nullptr;
        if (p) d[k] = reinterpret_cast<const uint4*>(p)[i % VEC];
    }
    for (int32_t c = c0; c < c1; ++c) {
        const int32_t u = unit_of(v, layer, a.dst[c], g), same = a.same[c];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int32_t i = threadIdx.x + k * kThreads, s = s0 + i / VEC % kForkSlots;
            uint8_t* p = s < n && s >= same ? slot_row(v, u, s, i >= kForkSlots * VEC) : nullptr;
            if (p) reinterpret_cast<uint4*>(p)[i % VEC] = d[k];
        }
    }
}

}  // namespace

cudaError_t launch_fork_release(const ForkArgs& a, cudaStream_t s) {
    const int64_t units = (int64_t)a.nlayers * a.copies * a.v.hkv;
    return launch_overlapped(k_fork_release, (int32_t)((units + 3) / 4), 128, 0, s, a);
}

cudaError_t launch_fork_reserve(const ForkArgs& a, cudaStream_t s) {
    const int64_t units = (int64_t)a.nlayers * a.copies * a.v.hkv;
    return launch_overlapped(k_fork_reserve, (int32_t)((units + 127) / 128), 128, 0, s, a);
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s) {
    const int32_t grid = (int32_t)((int64_t)a.groups * a.nlayers * a.v.hkv * (a.meta + a.chunks));
    switch (a.v.row_bytes) {
        case 128: return launch_overlapped(k_fork<8>, grid, kThreads, 0, s, a);
        case 256: return launch_overlapped(k_fork<16>, grid, kThreads, 0, s, a);
        default: return launch_overlapped(k_fork<32>, grid, kThreads, 0, s, a);
    }
}

}  // namespace hikv
