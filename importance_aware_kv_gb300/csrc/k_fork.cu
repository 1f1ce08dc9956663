// Copies of whole sequences of the cache: rows of the batch become what other
// rows are.
//
// A copy, bound by bytes: a source's K and V rows are read once for all its
// copies and written once to each.  A CTA takes 64 slots of one unit of a
// source, every lane 16 bytes of several rows at once, and skips what a copy
// shares with its source already.
#include <algorithm>

#include "hikv_packed.cuh"

namespace hikv {
namespace {

constexpr int kThreads = 256;

// the unit of copy c (or of its source) and the tokens that the source holds
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

__global__ void __launch_bounds__(kThreads) k_fork(const __grid_constant__ ForkArgs a) {
    constexpr int BATCH = 4;
    const View& v = a.v;
    const int32_t per = a.chunks * v.hkv * a.nlayers;
    const int32_t grp = blockIdx.x / per, rem = blockIdx.x % per;
    const int32_t chunk = rem % a.chunks, g = rem / a.chunks % v.hkv, layer = a.layer0 + rem / a.chunks / v.hkv;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t us = unit_of(v, layer, a.src[grp], g), n = v.len[us], next_pos = v.next_pos[us];
    const int32_t c0 = a.first[grp], c1 = a.first[grp + 1];
    if (n > v.cap) {
        if (threadIdx.x == 0) atomicOr(v.err, DEVERR_STATE);
        return;
    }
    if (chunk == 0 && threadIdx.x == 0) {
        for (int32_t c = c0; c < c1; ++c) {
            const int32_t u = unit_of(v, layer, a.dst[c], g);
            v.len[u] = n;
            v.next_pos[u] = next_pos;
            v.victim[u] = -1;
        }
    }
    const int32_t s0 = chunk * kForkSlots, s1 = min(s0 + kForkSlots, n);
    for (int32_t s = s0 + threadIdx.x; s < s1; s += kThreads) {
        const float x = v.imp[(int64_t)us * v.cap + s];
        const int32_t p = v.pos[(int64_t)us * v.cap + s];
        for (int32_t c = c0; c < c1; ++c) {
            const int64_t m = (int64_t)unit_of(v, layer, a.dst[c], g) * v.cap + s;
            v.imp[m] = x;
            v.pos[m] = p;
        }
    }
    int32_t lo = n;
    for (int32_t c = c0; c < c1; ++c) lo = min(lo, a.same[c]);
    lo = max(lo, s0);
    if (lo >= s1) return;
    const int32_t vec = v.row_bytes / 16, vshift = __ffs(vec) - 1;   // 16-byte columns of a row (8, 16 or 32)
    const int32_t total = (s1 - lo) * 2 * vec;   // K rows, then V rows
    for (int32_t i0 = threadIdx.x; i0 < total; i0 += BATCH * kThreads) {
        uint4 x[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int32_t i = i0 + k * kThreads;
            const bool is_v = i >= total / 2;
            const int32_t e = is_v ? i - total / 2 : i;
            const uint8_t* p = i < total ? slot_row(v, us, lo + (e >> vshift), is_v) : nullptr;
            if (p) x[k] = reinterpret_cast<const uint4*>(p)[e & (vec - 1)];
        }
        for (int32_t c = c0; c < c1; ++c) {
            const int32_t u = unit_of(v, layer, a.dst[c], g), same = a.same[c];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int32_t i = i0 + k * kThreads;
                const bool is_v = i >= total / 2;
                const int32_t e = is_v ? i - total / 2 : i, s = lo + (e >> vshift);
                uint8_t* p = i < total && s >= same ? slot_row(v, u, s, is_v) : nullptr;
                if (p) reinterpret_cast<uint4*>(p)[e & (vec - 1)] = x[k];
            }
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
    const int64_t grid = (int64_t)a.groups * a.nlayers * a.v.hkv * a.chunks;
    return launch_overlapped(k_fork, (int32_t)grid, kThreads, 0, s, a);
}

}  // namespace hikv
