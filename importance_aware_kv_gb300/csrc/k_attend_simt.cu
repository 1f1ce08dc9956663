// Causal attention of packed queries over the paged cache on the CUDA cores (fp32).
//
// One pass over the keys with a running maximum and sum per query row
// (online softmax): with m the largest logit so far and l = sum 2^(t - m),
// a new tile with maximum m' scales l and the accumulated output by
// 2^(m - m').  Logits are in the log2 domain (scale * log2 e folded in).
//
// A CTA of 16 x 16 threads takes 64 query rows -- row = token * G + head of
// the group, so the G heads that share a KV head share its tiles -- against
// tiles of 64 keys staged in shared memory; a thread forms 4 x 4 logits and
// 4 x D/16 outputs with packed pairs of fp32 multiply-adds, all sums in
// fp32.  Calls too small to give every SM two such CTAs take 32 rows, 2 x 4
// logits a thread (prompts of 256, 100, 511 and 1 tokens with 4/2 heads, d =
// 64: 50 -> 43 us; five drafted tokens over eight 16K caches with 32/8 heads,
// d = 128: 827 -> 634 us).  Bound by the latency between shared-memory reads
// and the fp32 pipes they feed (4096 tokens with 32/8 heads, d = 128: 2.95 ms,
// 46.6 TFLOP/s); two CTAs share an SM, for which P lies over K at d = 128.
// K and V come by asynchronous copies, at d = 64 a tile ahead.  With few rows
// the keys are split over CTAs (chunk) and the parts joined.
#include "hikv_packed.cuh"

namespace hikv {
namespace {

constexpr int kBN = kSimtKeys, kThreads = 256;

template <int D, int BM>
struct Simt {
    static constexpr int LD = D + 4;        // row strides that spread the banks of 16-byte reads
    static constexpr int LP = kBN + 4;
    static constexpr int BUFS = D == 64 ? 2 : 1;   // tiles of K and V: the next one loads under this one's work
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + BM * LD;
    static constexpr int OFF_V = OFF_K + BUFS * kBN * LD;
    // P lies over K (which is read before P is written) where K has one buffer
    static constexpr int OFF_P = BUFS == 1 ? OFF_K : OFF_V + BUFS * kBN * D;
    static constexpr int FLOATS = OFF_V + BUFS * kBN * D + (BUFS == 1 ? 0 : BM * LP);
    static_assert(LD >= LP && BM <= kBN, "P fits over K");
};

// 16 bytes global -> shared without a register, or zeros
__device__ __forceinline__ void copy16(float* dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {   // all but the N newest groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float2 lo(const float4& x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi(const float4& x) { return make_float2(x.z, x.w); }

template <int D, int BM>
__global__ void __launch_bounds__(kThreads, 2) k_attend_simt(const __grid_constant__ AttendArgs a) {
    using C = Simt<D, BM>;
    constexpr int R = BM / 16;   // rows of a thread
    constexpr int NV = D / 64;   // 16-byte column groups of a thread
    extern __shared__ float sm[];
    float* Qs = sm + C::OFF_Q;
    float* Ks = sm + C::OFF_K;
    float* Vs = sm + C::OFF_V;
    float* Ps = sm + C::OFF_P;
    const View& v = a.v;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t i0 = prefix_find(a.item0, a.nseq, blockIdx.x);
    const int32_t nq = a.nq[i0], first = a.start[i0];
    const int32_t rows = nq << a.gshift, tiles = ceil_div(rows, BM);
    const int32_t splits = (a.item0[i0 + 1] - a.item0[i0]) / (tiles * v.hkv);
    const int32_t rem = blockIdx.x - a.item0[i0], g = rem % v.hkv, split = rem / v.hkv % splits;
    const int32_t r0 = (tiles - 1 - rem / v.hkv / splits) * BM;   // the last rows, which see most, first
    const int32_t u = a.u0 + a.brow[i0] * v.hkv + g;
    const int32_t n = unit_len(a, i0, u);
    if (n < nq || n > v.cap) {
        if (tid == 0) atomicOr(v.err, DEVERR_STATE);
        return;
    }
    const int32_t G = 1 << a.gshift;
    const int32_t seen0 = n - nq;   // slots before the first query's own
    const int32_t first_lim = seen0 + (r0 >> a.gshift);                            // slots [0, lim] are seen by the
    const int32_t last_lim = seen0 + ((min(r0 + BM, rows) - 1) >> a.gshift);      // first and the last row
    const int32_t lo_slot = splits > 1 ? split * a.chunk : 0;
    const int32_t end = splits > 1 ? min(last_lim + 1, lo_slot + a.chunk) : last_lim + 1;
    if (lo_slot >= end) return;

    for (int i = tid; i < BM * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows) {
            const int32_t t = first + ((r0 + r) >> a.gshift), h = (g << a.gshift) + ((r0 + r) & (G - 1));
            x = *reinterpret_cast<const float4*>(a.q.row(t, h) + 4 * c);
        }
        *reinterpret_cast<float4*>(Qs + r * C::LD + c) = x;
    }
    int32_t lim[R];   // this thread's rows see slots [0, lim]
    float m[R], l[R];
    float2 o[R][2 * NV];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int32_t r = r0 + ty + 16 * i;
        lim[i] = r < rows ? seen0 + (r >> a.gshift) : -1;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * NV; ++j) o[i][j] = make_float2(0.f, 0.f);
    }

    // queue the keys, then the values of the tile at s0; rows past `end` are zero
    auto queue = [&](int32_t s0, int buf) {
        constexpr int PER = kBN * (D / 4) / kThreads;   // 16-byte pieces of a thread, in as many rows
        const int c = tid % (D / 4) * 4, r0t = tid / (D / 4);
        const int64_t to_v = (int64_t)v.page_tokens * v.row_bytes;
        const uint8_t* row[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = r0t + i * (kBN / PER);
            float* x = Ks + buf * kBN * C::LD + r * C::LD + c;
            row[i] = s0 + r < end ? slot_row(v, u, s0 + r, false) : nullptr;
            if (row[i]) copy16(x, row[i] + 4 * c);
            else *reinterpret_cast<float4*>(x) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        copy_commit();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float* x = Vs + buf * kBN * D + (r0t + i * (kBN / PER)) * D + c;
            if (row[i]) copy16(x, row[i] + to_v + 4 * c);
            else *reinterpret_cast<float4*>(x) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        copy_commit();
    };
    if (C::BUFS == 2) queue(lo_slot, 0);
    int buf = 0;
    for (int32_t s0 = lo_slot; s0 < end; s0 += kBN, buf ^= C::BUFS - 1) {
        __syncthreads();   // the tile before is done with
        if (C::BUFS == 2) {
            if (s0 + kBN < end) {
                queue(s0 + kBN, buf ^ 1);
                copy_wait<3>();
            } else {
                copy_wait<1>();
            }
        } else {
            queue(s0, 0);
            copy_wait<1>();
        }
        const float* Kt = Ks + buf * kBN * C::LD;
        const float* Vt = Vs + buf * kBN * D;
        __syncthreads();
        float2 s2[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int c = 0; c < D; c += 4) {
            float4 q[R], k[4];
#pragma unroll
            for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * C::LD + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(Kt + (tx + 16 * j) * C::LD + c);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s2[i][j] = ffma2(hi(q[i]), hi(k[j]), ffma2(lo(q[i]), lo(k[j]), s2[i][j]));
        }
        // the values are there; and K is read: P may lie over it
        if (C::BUFS == 2 && s0 + kBN < end) copy_wait<2>();
        else copy_wait<0>();
        __syncthreads();
        const bool edge = s0 + kBN - 1 > first_lim || s0 + kBN > end;   // some row does not see the whole tile
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float mx = m[i], s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = (s2[i][j].x + s2[i][j].y) * a.qscale;
                if (edge && (s0 + tx + 16 * j > lim[i] || s0 + tx + 16 * j >= end)) s[j] = -INFINITY;
                mx = fmaxf(mx, s[j]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float base = mx == -INFINITY ? 0.f : mx;   // nothing but -inf so far
            const float f = exp2f(m[i] - base);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[j] - base);
                sum += p;
                Ps[(ty + 16 * i) * C::LP + tx + 16 * j] = p;
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int j = 0; j < 2 * NV; ++j) {
                o[i][j].x *= f;
                o[i][j].y *= f;
            }
        }
        __syncwarp();   // a row's probabilities are written and read by the same half warp
        if (!edge) {
#pragma unroll 4
            for (int k = 0; k < kBN; k += 4) {
                float4 p[R];
#pragma unroll
                for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * C::LP + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    float4 x[NV];
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        x[j] = *reinterpret_cast<const float4*>(Vt + (k + kk) * D + tx * 4 + 64 * j);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float y = kk == 0 ? p[i].x : (kk == 1 ? p[i].y : (kk == 2 ? p[i].z : p[i].w));
                        const float2 y2 = make_float2(y, y);
#pragma unroll
                        for (int j = 0; j < NV; ++j) {
                            o[i][2 * j] = ffma2(y2, lo(x[j]), o[i][2 * j]);
                            o[i][2 * j + 1] = ffma2(y2, hi(x[j]), o[i][2 * j + 1]);
                        }
                    }
                }
            }
        } else {
            // a row skips the values it does not see: 0 x inf is not 0
            const int32_t kn = min(kBN, end - s0);
            for (int k = 0; k < kn; ++k) {
                float4 x[NV];
#pragma unroll
                for (int j = 0; j < NV; ++j) x[j] = *reinterpret_cast<const float4*>(Vt + k * D + tx * 4 + 64 * j);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (s0 + k > lim[i]) continue;
                    const float y = Ps[(ty + 16 * i) * C::LP + k];
                    const float2 y2 = make_float2(y, y);
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        o[i][2 * j] = ffma2(y2, lo(x[j]), o[i][2 * j]);
                        o[i][2 * j + 1] = ffma2(y2, hi(x[j]), o[i][2 * j + 1]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int32_t r = r0 + ty + 16 * i;
        if (r >= rows) continue;
        const int32_t t = first + (r >> a.gshift), h = (g << a.gshift) + (r & (G - 1));
        const int64_t pr = (int64_t)split * a.part_rows + (int64_t)t * v.hq + h;
        const float f = splits > 1 ? 1.f : 1.0f / l[i];
        float* dst = splits > 1 ? a.part + pr * D : reinterpret_cast<float*>(a.out.row(t, h));
#pragma unroll
        for (int j = 0; j < NV; ++j)
            *reinterpret_cast<float4*>(dst + tx * 4 + 64 * j) =
                make_float4(o[i][2 * j].x * f, o[i][2 * j].y * f, o[i][2 * j + 1].x * f, o[i][2 * j + 1].y * f);
        if (splits > 1 && tx == 0) *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m[i], l[i]);
    }
}

template <int D, int BM>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
    const size_t smem = Simt<D, BM>::FLOATS * sizeof(float);
    const cudaError_t e = func_smem_optin((const void*)k_attend_simt<D, BM>, smem);
    if (e != cudaSuccess) return e;
    return launch_overlapped(k_attend_simt<D, BM>, a.items, kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_attend_simt(const AttendArgs& a, int d, int rows, cudaStream_t s) {
    if (rows == kSimtRows) return d == 128 ? launch<128, kSimtRows>(a, s) : launch<64, kSimtRows>(a, s);
    return d == 128 ? launch<128, kSimtFewRows>(a, s) : launch<64, kSimtFewRows>(a, s);
}

}  // namespace hikv
