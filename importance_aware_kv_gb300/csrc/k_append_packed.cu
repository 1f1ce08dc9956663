// Append a packed batch of sequences to one layer, rotating k (and q) by
// position on the way, and drop the newest tokens again.
//
// The rotary embedding turns each pair (a, b) of a row by its position's
// angle: a' = a c - b s, b' = b c + a s, with c, s from the caller's fp32
// tables; the products and their difference are fp32 and the result is
// rounded once to the cache dtype.
//
// A copy with a little arithmetic, bound by bytes: every row is read and
// written once, 16 bytes an access.  A lane owns two 16-byte chunks of a row
// that hold whole pairs -- chunk i and its partner half a rotation on, or
// two neighbours where pairs are interleaved or nothing turns -- and the
// same two of every row of its token, so that it loads its cosines and sines
// once.  A warp takes a token's rows 32 / (chunk pairs a row) at a time, up to
// kBatch of them in flight; a token's rows are dealt to more warps
// when there are few tokens (a decode step: latency).
#include <algorithm>

#include "../../include/hikv.h"
#include "hikv_packed.cuh"

namespace hikv {
namespace {

// thread per (sequence, KV head): reserve the slots and map their pages
__global__ void k_reserve_packed(const __grid_constant__ PackedAppendArgs a) {
    const int32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    if (i >= a.seqs.n * a.v.hkv) return;
    const int32_t b = i / a.v.hkv;
    const int32_t ntok = a.seqs.start[b + 1] - a.seqs.start[b];
    if (ntok == 0) return;
    const int32_t u = a.u0 + (a.seqs.row0 + b) * a.v.hkv + i % a.v.hkv;
    int32_t first;
    reserve_unit(a.v, u, ntok, &first);
    a.reserved[u] = first;
}

constexpr int kWarps = 8;
constexpr int kBatch = 2;   // rows a lane has in flight; with 32 warps an SM (64 registers) 208 us for 4 x 8192
                            // tokens of 64/8 heads, four rows and 16 warps 225 us, four and 32 warps 236 us

template <typename T, int VE>
__device__ __forceinline__ void unpack(const uint4& x, float* f);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16, 8>(const uint4& x, float* f) {
    Widen<__nv_bfloat16, 8>::run(x, f);
}
template <>
__device__ __forceinline__ void unpack<float, 4>(const uint4& x, float* f) {
    Widen<float, 4>::run(x, f);
}
template <typename T, int VE>
__device__ __forceinline__ uint4 pack(const float* f);
template <>
__device__ __forceinline__ uint4 pack<__nv_bfloat16, 8>(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
template <>
__device__ __forceinline__ uint4 pack<float, 4>(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// turn the pairs of two chunks: (x[e], y[e]), or (x[2e], x[2e + 1]) and on into y
template <typename T, int VE, bool INTER>
__device__ __forceinline__ void turn(uint4& cx, uint4& cy, const float* c, const float* s) {
    float f[2 * VE];
    unpack<T, VE>(cx, f);
    unpack<T, VE>(cy, f + VE);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        float& x = f[INTER ? 2 * e : e];
        float& y = f[INTER ? 2 * e + 1 : e + VE];
        const float x0 = x;
        x = x0 * c[e] - y * s[e];
        y = y * c[e] + x0 * s[e];
    }
    cx = pack<T, VE>(f);
    cy = pack<T, VE>(f + VE);
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(32 * kWarps, 4) k_append_packed(const __grid_constant__ PackedAppendArgs a) {
    constexpr int VE = 16 / (int)sizeof(T);      // elements of a chunk
    constexpr int PAIRS = D / (2 * VE);          // chunk pairs of a row
    constexpr int ROWS = 32 / PAIRS;             // rows a warp covers at once
    const View& v = a.v;
    const int lane = threadIdx.x & 31;
    const int32_t gw = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int32_t tok = gw / a.slices, slice = gw - tok * a.slices;
    const int32_t t = a.seqs.start[0] + tok;
    griddep_launch_dependents();
    const int32_t b = prefix_find(a.seqs.start, a.seqs.n, t);
    const int32_t u0 = a.u0 + (a.seqs.row0 + b) * v.hkv;
    const int32_t i = t - a.seqs.start[b], ntok = a.seqs.start[b + 1] - a.seqs.start[b];
    const int32_t p = a.pos0[b] + i;
    const int pair = lane % PAIRS, turned = a.rot / (2 * VE);
    const bool rotates = pair < turned;
    // byte offsets of the lane's chunks where the row turns, and where it does not
    const int32_t x1 = rotates ? (INTER ? 32 * pair : 16 * pair) : 32 * pair;
    const int32_t y1 = rotates ? (INTER ? x1 + 16 : x1 + 16 * turned) : x1 + 16;
    const int32_t x0 = 32 * pair, y0 = x0 + 16;
    float c[VE], s[VE];
    // (so far all of it was launch parameters)
    griddep_wait();   // the rows' producer, and whoever still reads the pages
    if (t >= a.seqs.start[a.seqs.n]) return;
    int32_t at = p;   // the position to turn by
    if (a.depth) {
        const int32_t x = a.depth[t];
        at = a.pos0[b] + min(max(x, 0), ntok - 1);   // (the host has checked that the tables reach ntok)
        if (at != a.pos0[b] + x && lane == 0) atomicOr(v.err, DEVERR_STATE);
    }
    if (rotates) {
        const float* cp = a.cos + (int64_t)at * (a.rot / 2) + VE * pair;
        const float* sp = a.sin + (int64_t)at * (a.rot / 2) + VE * pair;
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            *reinterpret_cast<float4*>(c + e) = __ldg(reinterpret_cast<const float4*>(cp + e));
            *reinterpret_cast<float4*>(s + e) = __ldg(reinterpret_cast<const float4*>(sp + e));
        }
    }
    const int32_t hq = a.q.p ? v.hq : 0, rows = hq + 2 * v.hkv;
    for (int32_t r0 = slice * ROWS + lane / PAIRS; r0 < rows; r0 += kBatch * ROWS * a.slices) {
        uint4 cx[kBatch], cy[kBatch];
        uint8_t* dst[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t r = r0 + k * ROWS * a.slices;
            dst[k] = nullptr;
            if (r >= rows) continue;
            const uint8_t* src;
            const bool is_v = r >= hq + v.hkv;
            if (r < hq) {
                src = a.q.row(t, r);
                dst[k] = a.qo.row(t, r);
            } else {
                const int32_t g = is_v ? r - hq - v.hkv : r - hq;
                src = is_v ? a.vv.row(t, g) : a.k.row(t, g);
                const int32_t first = a.reserved ? a.reserved[u0 + g] : a.base[b];
                if (first < 0) continue;
                dst[k] = slot_row(v, u0 + g, first + i, is_v);
                if (!dst[k]) continue;
            }
            cx[k] = *reinterpret_cast<const uint4*>(src + (is_v ? x0 : x1));
            cy[k] = *reinterpret_cast<const uint4*>(src + (is_v ? y0 : y1));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!dst[k]) continue;
            const bool is_v = r0 + k * ROWS * a.slices >= hq + v.hkv;
            if (rotates && !is_v) turn<T, VE, INTER>(cx[k], cy[k], c, s);
            *reinterpret_cast<uint4*>(dst[k] + (is_v ? x0 : x1)) = cx[k];
            *reinterpret_cast<uint4*>(dst[k] + (is_v ? y0 : y1)) = cy[k];
        }
    }
    if (slice != 0) return;
    for (int32_t g = lane; g < v.hkv; g += 32) {
        const int32_t first = a.reserved ? a.reserved[u0 + g] : a.base[b];
        if (first < 0) continue;
        const int64_t m = (int64_t)(u0 + g) * v.cap + first + i;
        v.imp[m] = 0.0f;
        v.pos[m] = p;
        if (!a.reserved && i == ntok - 1) {   // nobody reads these before the next launch
            v.len[u0 + g] = first + ntok;
            v.next_pos[u0 + g] = p + 1;
        }
    }
}

// Warp per unit: shorten it; with a shared pool give the pages past the
// remaining tokens back; in debug mode poison what is dropped.
__global__ void __launch_bounds__(128) k_drop(const __grid_constant__ DropArgs a) {
    const View& v = a.v;
    const int32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const int32_t per_layer = a.n * v.hkv;
    griddep_launch_dependents();
    griddep_wait();
    if (w >= a.nlayers * per_layer) return;
    const int32_t b = w % per_layer / v.hkv;
    const int32_t u = ((a.layer0 + w / per_layer) * v.batch + a.row0 + b) * v.hkv + w % v.hkv;
    const int32_t n = v.len[u], c = a.count[b];
    if (c == 0) return;
    if (c > n) {
        if (lane == 0) atomicOr(v.err, DEVERR_STATE);
        return;
    }
    const int32_t left = c < 0 ? 0 : n - c;
    if (v.debug) {
        for (int32_t s = left; s < n; ++s) poison_slot(v, u, s, lane, 32);
        __syncwarp();
    }
    if (lane != 0) return;
    shorten_unit(v, u, left, c < 0 ? 0 : v.next_pos[u] - c);
}

}  // namespace

namespace {
template <typename T, int D>
cudaError_t launch_rows(const PackedAppendArgs& a, int32_t grid, cudaStream_t s) {
    return a.interleaved ? launch_overlapped(k_append_packed<T, D, true>, grid, 32 * kWarps, 0, s, a)
                         : launch_overlapped(k_append_packed<T, D, false>, grid, 32 * kWarps, 0, s, a);
}
}  // namespace

cudaError_t launch_append_packed(PackedAppendArgs& a, int dtype, int sm_count, cudaStream_t s) {
    const int32_t total = a.seqs.start[a.seqs.n] - a.seqs.start[0];
    if (a.reserved) {
        const cudaError_t e = launch_overlapped(k_reserve_packed, ceil_div(a.seqs.n * a.v.hkv, 128), 128, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    // warps a token: enough to give every SM sixteen, at most one per warpful of rows
    const int rows = (a.q.p ? a.v.hq : 0) + 2 * a.v.hkv, at_once = 32 * 32 / a.v.row_bytes;
    a.slices = std::max(1, std::min(ceil_div(rows, at_once), ceil_div(16 * sm_count, total)));
    const int32_t grid = (int32_t)(((int64_t)total * a.slices + kWarps - 1) / kWarps);
    if (dtype == HIKV_BF16)
        return a.v.d == 128 ? launch_rows<__nv_bfloat16, 128>(a, grid, s) : launch_rows<__nv_bfloat16, 64>(a, grid, s);
    return a.v.d == 128 ? launch_rows<float, 128>(a, grid, s) : launch_rows<float, 64>(a, grid, s);
}

cudaError_t launch_drop(const DropArgs& a, cudaStream_t s) {
    const int32_t warps = a.nlayers * a.n * a.v.hkv;
    return launch_overlapped(k_drop, ceil_div(warps, 4), 128, 0, s, a);
}

}  // namespace hikv
