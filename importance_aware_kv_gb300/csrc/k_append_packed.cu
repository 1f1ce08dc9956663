// Append a packed batch of sequences to one layer, rotating k (and q) by
// position on the way, and drop the newest tokens again.
//
// The rotary embedding turns each pair (a, b) of a row by its position's
// angle: a' = a c - b s, b' = b c + a s, with c, s from the caller's fp32
// tables; the products and their difference are fp32 and the result is
// rounded once to the cache dtype.
#include "../../include/hikv.h"
#include "hikv_internal.cuh"

namespace hikv {
namespace {

// thread per (sequence, KV head): reserve the slots and map their pages
__global__ void k_reserve_packed(const __grid_constant__ PackedAppendArgs a) {
    const int32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.seqs.n * a.v.hkv) return;
    const int32_t b = i / a.v.hkv;
    const int32_t ntok = a.seqs.start[b + 1] - a.seqs.start[b];
    if (ntok == 0) return;
    const int32_t u = a.u0 + (a.seqs.row0 + b) * a.v.hkv + i % a.v.hkv;
    int32_t first;
    reserve_unit(a.v, u, ntok, &first);
    a.base[u] = first;
}

// CTA per packed token: its q, k and v rows, element pair by element pair
template <typename T>
__global__ void __launch_bounds__(128) k_append_packed(const __grid_constant__ PackedAppendArgs a) {
    const View& v = a.v;
    const int32_t t = a.seqs.start[0] + blockIdx.x;
    const int32_t b = prefix_find(a.seqs.start, a.seqs.n, t);
    const int32_t u0 = a.u0 + (a.seqs.row0 + b) * v.hkv;
    const int32_t i = t - a.seqs.start[b], ntok = a.seqs.start[b + 1] - a.seqs.start[b];
    const int32_t half = a.rot / 2, pairs = v.d / 2;
    const int32_t hq = a.q.p ? v.hq : 0;
    const int32_t p = v.next_pos[u0] - ntok + i;   // one position count per sequence
    const float* cs = a.cos + (int64_t)p * half;
    const float* sn = a.sin + (int64_t)p * half;
    for (int32_t w = threadIdx.x; w < (hq + 2 * v.hkv) * pairs; w += blockDim.x) {
        const int32_t h = w / pairs, j = w % pairs;
        const bool is_q = h < hq, is_k = !is_q && h < hq + v.hkv;
        const int32_t g = is_q ? 0 : (is_k ? h - hq : h - hq - v.hkv);
        const T* src = reinterpret_cast<const T*>(is_q ? a.q.row(t, h) : (is_k ? a.k.row(t, g) : a.vv.row(t, g)));
        T* dst;
        if (is_q) {
            dst = reinterpret_cast<T*>(a.qo.row(t, h));
        } else {
            const int32_t first = a.base[u0 + g];
            if (first < 0) continue;
            dst = reinterpret_cast<T*>(row_ptr(v, u0 + g, first + i, !is_k));
            if (!dst) continue;
        }
        const bool turn = (is_q || is_k) && j < half;
        const int32_t x = turn ? (a.interleaved ? 2 * j : j) : 2 * j;
        const int32_t y = turn ? (a.interleaved ? 2 * j + 1 : j + half) : 2 * j + 1;
        if (!turn) {
            dst[x] = src[x];
            dst[y] = src[y];
            continue;
        }
        const float ax = Elem<T>::to_f(src[x]), ay = Elem<T>::to_f(src[y]), c = cs[j], s = sn[j];
        dst[x] = Elem<T>::from_f(ax * c - ay * s);
        dst[y] = Elem<T>::from_f(ay * c + ax * s);
    }
    for (int32_t g = threadIdx.x; g < v.hkv; g += blockDim.x) {
        const int32_t first = a.base[u0 + g];
        if (first < 0) continue;
        const int64_t m = (int64_t)(u0 + g) * v.cap + first + i;
        v.imp[m] = 0.0f;
        v.pos[m] = p;
    }
}

// Warp per unit: shorten it; with a shared pool give the pages past the
// remaining tokens back; in debug mode poison what is dropped.
__global__ void __launch_bounds__(128) k_drop(const __grid_constant__ DropArgs a) {
    const View& v = a.v;
    const int32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const int32_t per_layer = a.n * v.hkv;
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
    v.len[u] = left;
    v.next_pos[u] = c < 0 ? 0 : v.next_pos[u] - c;
    v.victim[u] = -1;
    const int32_t keep = ceil_div(left, v.page_tokens), m = v.mapped[u];
    if (!v.home_pages && m > keep) {
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
}

}  // namespace

cudaError_t launch_append_packed(const PackedAppendArgs& a, int dtype, cudaStream_t s) {
    const int32_t total = a.seqs.start[a.seqs.n] - a.seqs.start[0];
    k_reserve_packed<<<ceil_div(a.seqs.n * a.v.hkv, 128), 128, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (dtype == HIKV_BF16) k_append_packed<__nv_bfloat16><<<total, 128, 0, s>>>(a);
    else k_append_packed<float><<<total, 128, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_drop(const DropArgs& a, cudaStream_t s) {
    const int32_t warps = a.nlayers * a.n * a.v.hkv;
    k_drop<<<ceil_div(warps, 4), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hikv
