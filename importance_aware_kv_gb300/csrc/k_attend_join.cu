// The join of attention results whose keys were split over work items.
#include "../../include/hikv.h"
#include "hikv_packed.cuh"

namespace hikv {
namespace {

// Warp per query row (t, h) of the sequences that were split, a lane per
// split first: with m_s the parts' references, m the largest and f_s = 2^(m_s - m),
//   o = sum_s f_s O_s / sum_s f_s l_s.
// Bound by the latency of its three dependent reads (length, references, parts).
template <typename T, int D, class M>
__global__ void __launch_bounds__(128) k_attend_join(const __grid_constant__ AttendArgs a, const __grid_constant__ M mask) {
    constexpr int E = D / 32;   // elements of a lane
    const View& v = a.v;
    const int32_t x = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const bool gave_up = attend_gave_up(v);   // parts are missing: write nothing
    const int32_t tok = x / v.hq, h = x % v.hq;
    if (tok >= a.comb0[a.nseq]) return;
    const int32_t i = prefix_find(a.comb0, a.nseq, tok);
    const int32_t j = tok - a.comb0[i];
    const int32_t n = unit_len(a, i, a.u0 + a.brow[i] * v.hkv + (h >> a.gshift));
    int32_t lim = n - a.nq[i] + j;   // the row sees no slot past lim
    if (lim < 0 || n > v.cap) return;
    if constexpr (M::kind == 1) {    // in the key numbers of its work item
        constexpr int rows = sizeof(T) == 2 ? kTcRows : kF32Rows;
        const int32_t row = (j << a.gshift) + (h & ((1 << a.gshift) - 1)), r0 = row / rows * rows;
        int32_t gap, shift;
        key_gap(mask, h >> a.gshift, n - a.nq[i] + (r0 >> a.gshift), gap, shift);
        lim -= shift;
    }
    if (M::kind == 2) lim = n - 1;
    const int32_t ns = min(lim / a.chunk + 1, a.splits);
    const int64_t row = (int64_t)(M::kind == 0 ? a.start[i] + j : tok) * v.hq + h;
    float m = -INFINITY;
    for (int32_t s = lane; s < ns; s += 32) m = fmaxf(m, a.part_ml[(s * a.part_rows + row) * 2]);
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[E] = {};
    for (int32_t s0 = 0; s0 < ns; s0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (s0 + lane < ns) ml = *reinterpret_cast<const float2*>(a.part_ml + ((s0 + lane) * a.part_rows + row) * 2);
        const float f = exp2f(ml.x - base);
        l = fmaf(f, ml.y, l);
        const int32_t cnt = min(32, ns - s0);
#pragma unroll 4
        for (int32_t s = 0; s < cnt; ++s) {
            const float fs = __shfl_sync(0xffffffffu, f, s);
            const float* p = a.part + ((s0 + s) * a.part_rows + row) * D + lane * E;
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = fmaf(fs, p[k], o[k]);
        }
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (gave_up) return;
    if constexpr (M::kind == 2) {
        if (l == 0.f && RowSight<M>(mask, h >> a.gshift, a.start[i] + j, n - a.nq[i], a.nq[i], lim).blind()) l = 1.f;   // (o is zero)
    }
    T* dst = reinterpret_cast<T*>(a.out.row(a.start[i] + j, h)) + lane * E;
#pragma unroll
    for (int k = 0; k < E; ++k) dst[k] = Elem<T>::from_f(o[k] / l);
}

template <class M>
cudaError_t launch(const AttendArgs& a, const M& m, int dtype, int d, cudaStream_t s) {
    const int32_t grid = (int32_t)(((int64_t)a.comb0[a.nseq] * a.v.hq + 3) / 4);
    using B = __nv_bfloat16;
    if (dtype == HIKV_BF16)
        return d == 128 ? launch_overlapped(k_attend_join<B, 128, M>, grid, 128, 0, s, a, m)
                        : launch_overlapped(k_attend_join<B, 64, M>, grid, 128, 0, s, a, m);
    return d == 128 ? launch_overlapped(k_attend_join<float, 128, M>, grid, 128, 0, s, a, m)
                    : launch_overlapped(k_attend_join<float, 64, M>, grid, 128, 0, s, a, m);
}

// one CTA whose wait on a barrier that nothing arrives on gives up after limit_ns
__global__ void k_selftest_attend(View v, uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t where;
    if (threadIdx.x == 0) {
        where = 0;
        mbar_init(&bar, 1);
        fence_mbar_init();
        attend_wait(&bar, 0u, &where, 1u, limit_ns);
        attend_record(v.err, where, limit_ns);
    }
}

}  // namespace

cudaError_t launch_selftest_attend(const View& v, uint64_t limit_ns, cudaStream_t s) {
    k_selftest_attend<<<1, 32, 0, s>>>(v, limit_ns);
    return cudaGetLastError();
}

cudaError_t launch_attend_join(const AttendArgs& a, int dtype, int d, cudaStream_t s) {
    return launch(a, CausalMask{}, dtype, d, s);
}
cudaError_t launch_attend_join_window(const AttendArgs& a, const WindowMask& m, int dtype, int d, cudaStream_t s) {
    return launch(a, m, dtype, d, s);
}
cudaError_t launch_attend_join_tree(const AttendArgs& a, const TreeMask& m, int dtype, int d, cudaStream_t s) {
    return launch(a, m, dtype, d, s);
}

}  // namespace hikv
