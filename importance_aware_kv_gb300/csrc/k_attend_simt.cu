// Causal attention of packed queries over the paged cache on the CUDA cores (fp32).
//
// One pass over the keys with a running maximum and sum per query row
// (online softmax): with m the largest logit so far and l = sum 2^(t - m),
// a new tile with maximum m' scales l and the accumulated output by
// 2^(m - m').  Logits are in the log2 domain (scale * log2 e folded in).
//
// A CTA of 16 x 16 threads takes 64 query rows -- row = token * G + head of
// the group, so the G heads that share a KV head share its tiles -- against
// tiles of 64 keys staged in shared memory as fp32; a thread forms 4 x 4
// logits and 4 x D/16 outputs, all sums in fp32.
#include "hikv_internal.cuh"

namespace hikv {
namespace {

constexpr int kBM = kSimtRows, kBN = 64, kThreads = 256;

template <int D>
struct Simt {
    static constexpr int LD = D + 4;        // row strides that spread the banks of 16-byte reads
    static constexpr int LP = kBN + 4;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + kBM * LD;
    static constexpr int OFF_V = OFF_K + kBN * LD;
    static constexpr int OFF_P = OFF_V + kBN * D;
    static constexpr int FLOATS = OFF_P + kBM * LP;
};

template <int D>
__global__ void __launch_bounds__(kThreads) k_attend_simt(const __grid_constant__ AttendArgs a) {
    using C = Simt<D>;
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
    const int32_t g = (blockIdx.x - a.item0[i0]) % v.hkv;
    const int32_t tile = (a.item0[i0 + 1] - 1 - (int32_t)blockIdx.x) / v.hkv;   // the last one first
    const int32_t u = a.u0 + a.brow[i0] * v.hkv + g;
    const int32_t n = v.len[u];
    if (n < nq || n > v.cap) {
        if (tid == 0) atomicOr(v.err, DEVERR_STATE);
        return;
    }
    const int32_t G = 1 << a.gshift;
    const int64_t rows = (int64_t)nq << a.gshift;
    const int64_t r0 = (int64_t)tile * kBM;
    const int32_t seen0 = n - nq;   // slots before the first query's own

    for (int i = tid; i < kBM * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows) {
            const int32_t t = first + (int32_t)((r0 + r) >> a.gshift), h = (g << a.gshift) + (int32_t)((r0 + r) & (G - 1));
            x = *reinterpret_cast<const float4*>(a.q.row(t, h) + 4 * c);
        }
        *reinterpret_cast<float4*>(Qs + r * C::LD + c) = x;
    }
    // the slots each of this thread's rows sees: [0, lim]
    int32_t lim[4];
    float m[4], l[4];
    float4 o[4][D / 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + ty + 16 * i;
        lim[i] = r < rows ? seen0 + (int32_t)(r >> a.gshift) : -1;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int64_t rlast = r0 + kBM < rows ? r0 + kBM - 1 : rows - 1;
    const int32_t first_lim = seen0 + (int32_t)(r0 >> a.gshift), last_lim = seen0 + (int32_t)(rlast >> a.gshift);

    for (int32_t s0 = 0; s0 <= last_lim; s0 += kBN) {
        __syncthreads();
        for (int i = tid; i < kBN * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (s0 + r <= last_lim) {
                const uint8_t* kp = row_ptr(v, u, s0 + r, false);
                const uint8_t* vp = row_ptr(v, u, s0 + r, true);
                if (kp) x = *reinterpret_cast<const float4*>(kp + 4 * c);
                if (vp) y = *reinterpret_cast<const float4*>(vp + 4 * c);
            }
            *reinterpret_cast<float4*>(Ks + r * C::LD + c) = x;
            *reinterpret_cast<float4*>(Vs + r * D + c) = y;
        }
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 q[4], k[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * C::LD + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * C::LD + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[i][j] = fmaf(q[i].w, k[j].w, fmaf(q[i].z, k[j].z, fmaf(q[i].y, k[j].y, fmaf(q[i].x, k[j].x, s[i][j]))));
        }
        const bool edge = s0 + kBN - 1 > first_lim;   // some row does not see the whole tile
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= a.qscale;
                if (edge && s0 + tx + 16 * j > lim[i]) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float base = mx == -INFINITY ? 0.f : mx;   // nothing but -inf so far
            const float f = exp2f(m[i] - base);
            m[i] = mx;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                Ps[(ty + 16 * i) * C::LP + tx + 16 * j] = p;
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                o[i][j].x *= f;
                o[i][j].y *= f;
                o[i][j].z *= f;
                o[i][j].w *= f;
            }
        }
        __syncwarp();   // a row's probabilities are written and read by the same half warp
        for (int k = 0; k < kBN; ++k) {
            float4 x[D / 64];
#pragma unroll
            for (int j = 0; j < D / 64; ++j) x[j] = *reinterpret_cast<const float4*>(Vs + k * D + tx * 4 + 64 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // at the edge a row skips the values it does not see: 0 x inf is not 0
                if (edge && s0 + k > lim[i]) continue;
                const float p = Ps[(ty + 16 * i) * C::LP + k];
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    o[i][j].x = fmaf(p, x[j].x, o[i][j].x);
                    o[i][j].y = fmaf(p, x[j].y, o[i][j].y);
                    o[i][j].z = fmaf(p, x[j].z, o[i][j].z);
                    o[i][j].w = fmaf(p, x[j].w, o[i][j].w);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + ty + 16 * i;
        if (r >= rows) continue;
        const int32_t t = first + (int32_t)(r >> a.gshift), h = (g << a.gshift) + (int32_t)(r & (G - 1));
        float* dst = reinterpret_cast<float*>(a.out.row(t, h));
        const float inv = 1.0f / l[i];
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            *reinterpret_cast<float4*>(dst + tx * 4 + 64 * j) =
                make_float4(o[i][j].x * inv, o[i][j].y * inv, o[i][j].z * inv, o[i][j].w * inv);
    }
}

template <int D>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
    const void* f = (const void*)k_attend_simt<D>;
    const size_t smem = Simt<D>::FLOATS * sizeof(float);
    cudaError_t e = func_smem_optin(f, smem);
    if (e != cudaSuccess) return e;
    return launch_overlapped(k_attend_simt<D>, a.items, kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_attend_simt(const AttendArgs& a, int d, cudaStream_t s) {
    return d == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace hikv
