// Causal attention of packed queries over the paged cache, fp32, on the
// tensor cores.
//
// Every fp32 operand x enters as three bf16 parts, x = h + m + l: h is x
// rounded to bf16, m what is left rounded, l what is left of that (3 x 8
// significant bits).  A product of two operands is the six products of parts
// above 2^-24 of it, the smallest first so that the fp32 accumulator rounds
// at full size in the last pass only:
//   x y = m m' + h l' + l h' + h m' + m h' + h h'  (+ m l' + l m' + l l', dropped).
// Each key tile's P V forms from zero in tensor memory and is added to the
// row's sums in registers, so that long sums round as fp32 additions do.
//
// A work item is 128 query rows (row = token * G + head) of one KV head, its
// keys in tiles of 64:
//   warps 0-3   softmax, one thread a row: the parts of its query into tensor
//               memory, S of a tile from there, the parts of P back, the row's
//               output sums in registers
//   warps 4-11  read K (4-7) and V (8-11) from global memory and write their parts to
//               shared memory, swizzled as the products want them, two tiles each
//   warp 12     one thread issues the products; S of the next tile forms under the
//               softmax of this one, whose S is in registers by then
// Queries in tensor memory leave shared memory to two tiles of keys and values.
// What bounds it: the six products.  A 128 x 64 x 16 product takes 73 cycles, as
// long as one of 128 columns would (its rows' operand, 4 KB, comes at 64 bytes a
// cycle), so a 128 x 64 tile's S takes 3,500 cycles and its P V 1,536 of the
// 5,800 a step; 128 keys a tile would need 544 columns of tensor memory.
// 4096 tokens with 32/8 heads, d = 128: 690 us, 199 TFLOP/s of fp32 work (the same
// on the CUDA cores, 4 x 4 tiles in registers: 2,947 us, 46.7).
//
// Non-finite V elements do not go through the products (0 x inf): they are
// noted with their slots and added to the rows that see them.  A non-finite
// element of k (or q) makes the logits of its key (or row) NaN.
//
// The same kernel serves sliding windows with visible first tokens and trees of
// drafted tokens, as the bf16 kernel does (k_attend_tc.cuh).
#pragma once

#include "hikv_tcgen05.cuh"

namespace hikv {
namespace {

constexpr int kThreads = 512, kConvert = 256;
constexpr int kRows = kF32Rows, kKeys = kF32Keys;
// 128 x 224 + 384 x 96 registers = the 512 x 128 at launch
constexpr int kRegsSoftmax = 224, kRegsOther = 96;
// How far the maximum may pass the one that a row's exponents refer to before the
// reference moves, in powers of two, and the factor that keeps the weights at one
// or below till then, so that sums of finite values do not overflow on the way;
// the largest weight is above 2^-16.  (4096 tokens took 688 us with 16, 710 with
// 8, 743 with 0 in one build: more rows move.  Values below 2^-94 may lose low bits.)
constexpr float kAhead = 16.f, kWeight = 1.f / 65536.f;

template <int D>
struct F3 {
    static constexpr int HALVES = D / 64;
    static constexpr int KBLOCK = kKeys * 128;            // 64 columns of a part
    static constexpr int KPART = HALVES * KBLOCK, TILE = 3 * KPART;
    static constexpr int OFF_K = 0;                       // two tiles
    static constexpr int OFF_V = 2 * TILE;
    // barriers: k_full[2], k_empty[2], v_full[2], v_empty[2], q_full, s_full, s_read, p_full, o_full, drained
    static constexpr int OFF_BAR = 4 * TILE;
    static constexpr int OFF_MISC = OFF_BAR + 14 * 8;     // tensor memory address, non-finite values noted
    static constexpr int OFF_WHERE = OFF_MISC + 8;        // where a wait gave up
    static constexpr int OFF_EDGE = OFF_MISC + 12;        // non-finite values that not every row sees
    static constexpr int OFF_OVER = OFF_MISC + 16;        // [3][D] first slots of +inf, -inf, NaN
    static constexpr int BYTES = OFF_OVER + 3 * D * 4 + 1024;
};
// columns of tensor memory: three parts of Q, S, three parts of P, O
constexpr int kTmQ = 0, kTmS = 192, kTmP = 256, kTmO = 352;

// magnitudes that round to a bf16 infinity (the finite ones from 0x7F7F8000 on too), and NaN
__device__ __forceinline__ bool rounds_to_inf(float x) { return (__float_as_uint(x) & 0x7FFFFFFFu) >= 0x7F7F8000u; }
__device__ __forceinline__ bool non_finite(float x) { return (__float_as_uint(x) & 0x7FFFFFFFu) >= 0x7F800000u; }

// Two fp32 values as three packed bf16 pairs; each remainder is exact in fp32.
// CUT: the first part cut off instead of rounded, for values that would round to
// infinity (the parts still hold 24 bits between them; NaN stays NaN in each).
template <bool CUT = false>
__device__ __forceinline__ void three_parts(float2 x, uint32_t& h, uint32_t& m, uint32_t& l) {
    const float2 minus = make_float2(-1.f, -1.f);
    h = CUT ? __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632) : pack_bf16x2(x.x, x.y);
    const float2 r = ffma2(make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u)), minus, x);
    m = pack_bf16x2(r.x, r.y);
    const float2 q = ffma2(make_float2(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), minus, r);
    l = pack_bf16x2(q.x, q.y);
}
// Eight consecutive elements as three parts, 16 bytes each, at `at` + part *
// stride; where one rounds to infinity or is NaN, mend() changes it first
template <typename F>
__device__ __forceinline__ void put_parts(uint8_t* at, int stride, float* x, F mend) {
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) three_parts(make_float2(x[2 * i], x[2 * i + 1]), h[i], m[i], l[i]);
    const uint32_t top = __vmaxu2(__vmaxu2(h[0] & 0x7FFF7FFFu, h[1] & 0x7FFF7FFFu),
                                  __vmaxu2(h[2] & 0x7FFF7FFFu, h[3] & 0x7FFF7FFFu));
    if ((top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u) {
        mend(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) three_parts<true>(make_float2(x[2 * i], x[2 * i + 1]), h[i], m[i], l[i]);
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(at + stride) = make_uint4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<uint4*>(at + 2 * stride) = make_uint4(l[0], l[1], l[2], l[3]);
}
// (NaN splits into NaN three times: its products are NaN, and nothing else)
__device__ __forceinline__ void mark_nan(float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (non_finite(x[i])) x[i] = __int_as_float(0x7FC00000);
}

template <int D, class M>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend_f32(const __grid_constant__ AttendArgs a, const __grid_constant__ M mask) {
    using C = F3<D>;
    extern __shared__ __align__(128) uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
    uint64_t* k_empty = k_full + 2;
    uint64_t* v_full = k_empty + 2;
    uint64_t* v_empty = v_full + 2;
    uint64_t* q_full = v_empty + 2;
    uint64_t* s_full = q_full + 1;
    uint64_t* s_read = s_full + 1;
    uint64_t* p_full = s_read + 1;
    uint64_t* o_full = p_full + 1;
    uint64_t* drained = o_full + 1;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_MISC);
    volatile uint32_t* where = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_WHERE);
    volatile uint32_t* edge_bad = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_EDGE);
    int32_t* over = reinterpret_cast<int32_t*>(sm + C::OFF_OVER);
    const View& v = a.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], kConvert / 64);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], kConvert / 64);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(q_full, 4);
        mbar_init(s_full, 1);
        mbar_init(s_read, 4);
        mbar_init(p_full, 4);
        mbar_init(o_full, 1);
        mbar_init(drained, 1);
        misc[1] = 0;
        *edge_bad = 0;
        *where = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 3 * D; i += kThreads) over[i] = 0x7FFFFFFF;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(sm + C::OFF_MISC))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();

    // the work item: rows [r0, r0 + kRows) of (sequence i, KV head g), keys [lo, end)
    const int32_t i = prefix_find(a.item0, a.nseq, blockIdx.x);
    const int32_t nq = a.nq[i], first = a.start[i], rows = nq << a.gshift, tiles = ceil_div(rows, kRows);
    const int32_t splits = a.parts[i];
    int32_t g, x;
    item_head(a, mask, blockIdx.x - a.item0[i], tiles * splits, g, x);
    const int32_t split = x % splits;
    const int32_t r0 = (tiles - 1 - x / splits) * kRows;   // the last rows, which see most, first
    const int32_t u = a.u0 + a.brow[i] * v.hkv + g;
    const int32_t n = unit_len(a, i, u);
    int32_t gap, shift;             // slot of key number s: s < gap ? s : s + shift (below, "slot" means number)
    key_gap(mask, g, n - nq + (r0 >> a.gshift), gap, shift);
    const int32_t seen0 = n - nq - shift;   // slots before the first query's own
    const int32_t last_row = seen0 + ((min(r0 + kRows, rows) - 1) >> a.gshift);
    const int32_t last_lim = M::kind == 2 ? n - 1 : last_row;   // what the last row sees
    // whether every row sees all of slots [s, s + n) (masks other than the causal one)
    auto all_see = [&](int32_t s, int32_t n) {
        if constexpr (M::kind == 1)
            return s + n - 1 <= seen0 + (r0 >> a.gshift) && (s > last_row - mask.window[g] || s + n - 1 < mask.sink);
        return s + n <= seen0;
    };
    const int32_t lo = splits > 1 ? split * a.chunk : 0;
    const int32_t end = splits > 1 ? min(last_lim + 1, lo + a.chunk) : last_lim + 1;
    const bool sane = n >= nq && n <= v.cap;
    if (!sane && threadIdx.x == 0) atomicOr(v.err, DEVERR_STATE);
    const bool bad = !sane || attend_gave_up(v);
    const int32_t nt = bad || end <= lo ? 0 : (end - lo + kKeys - 1) / kKeys;

    tc_fence_before();
    // (every thread has read the error word the same way: a late time-out of another item changes nothing here)
    const bool run = __syncthreads_and(nt > 0);
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp < 4) {
        // ---------------- softmax ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const uint32_t base_lane = (uint32_t)(32 * warp) << 16;
        const uint32_t tp = tmem + base_lane + kTmP, to = tmem + base_lane + kTmO;
        const int32_t row = r0 + 32 * warp + lane;
        const int32_t lim = seen0 + (min(row, rows - 1) >> a.gshift);                     // sees slots [0, lim]
        const int32_t lim_w = seen0 + (min(r0 + 32 * warp, rows - 1) >> a.gshift);        // the warp's first row
        const float c = a.qscale;
        bool ok = run;
        {
            // this row's query in parts, 16 elements (8 columns of each part) at a time
            const int32_t tok = first + (row >> a.gshift), h = (g << a.gshift) + (row & ((1 << a.gshift) - 1));
            const float4* src = reinterpret_cast<const float4*>(a.q.row(tok, h));
#pragma unroll 2
            for (int j = 0; j < D / 16; ++j) {
                float x[16] = {};
                if (row < rows) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) *reinterpret_cast<float4*>(x + 4 * k) = src[4 * j + k];
                    mark_nan(x);
                    mark_nan(x + 8);
                }
                bool big = false;
#pragma unroll
                for (int k = 0; k < 16; ++k) big |= rounds_to_inf(x[k]);
                uint32_t hi[8], mi[8], lw[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) three_parts(make_float2(x[2 * k], x[2 * k + 1]), hi[k], mi[k], lw[k]);
                if (big) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) three_parts<true>(make_float2(x[2 * k], x[2 * k + 1]), hi[k], mi[k], lw[k]);
                }
                const uint32_t tq = tmem + base_lane + kTmQ + 8 * j;
                tmem_st8(tq, hi);
                tmem_st8(tq + D / 2, mi);
                tmem_st8(tq + D, lw);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        float m = -INFINITY, l = 0.f;   // m: the maximum at the reference's last move
        float2 acc[D / 2];
#pragma unroll
        for (int j = 0; j < D / 2; ++j) acc[j] = make_float2(0.f, 0.f);
        // add the tile's P V
        auto add = [&](uint32_t parity) {
            ok = warp_wait(o_full, parity, where, 0x800);
            if (!ok) return;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < D; j += 16) {
                uint32_t o[16];
                tmem_ld16(o, to + j);
                tmem_wait_ld();
                held16(o);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    acc[j / 2 + k] = fadd2(acc[j / 2 + k], make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])));
            }
        };
        for (int32_t t = 0; ok && t < nt; ++t) {
            ok = warp_wait(s_full, t & 1, where, 0x801);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[64];
            tmem_ld32(s, tmem + base_lane + kTmS);
            tmem_ld32(s + 32, tmem + base_lane + kTmS + 32);
            tmem_wait_ld();
            held(s);
            held(s + 32);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_read);   // the next tile's S may form
            const int32_t s0 = lo + t * kKeys;
            if constexpr (M::kind == 0) {
                if (s0 + kKeys - 1 > lim_w || s0 + kKeys > end) {
                    const int32_t left = min(lim, end - 1) - s0;   // columns [0, left] are seen
#pragma unroll
                    for (int j = 0; j < 64; ++j) s[j] = j <= left ? s[j] : 0xFF800000u;
                }
            } else if (!all_see(s0, kKeys) || s0 + kKeys > end) {
                const RowSight<M> sight(mask, g, first + (min(row, rows - 1) >> a.gshift), seen0, nq, lim);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t sees = sight.word(s0 + 32 * k) & bits_below(end - s0 - 32 * k);
#pragma unroll
                    for (int j = 0; j < 32; ++j) s[32 * k + j] = (sees >> j) & 1 ? s[32 * k + j] : 0xFF800000u;
                }
            }
            float mx[4] = {m, m, m, m};
#pragma unroll
            for (int j = 0; j < 64; j += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mx[k] = max3(mx[k], __uint_as_float(s[j + 2 * k]), __uint_as_float(s[j + 2 * k + 1]));
            const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
            // (NaN while both are -inf: no move)
            const bool move = (mt - m) * c > kAhead;
            const float f = move ? ex2((m - mt) * c) : 1.f;
            if (move) m = mt;
            const float base = m == -INFINITY ? 0.f : m * c;
            const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float2 x = ffma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, b2);
                // (2^-kAhead as a factor: in the exponent it would cost the low bits of small ones)
                const float2 e = ffma2(make_float2(ex2(x.x), ex2(x.y)), make_float2(kWeight, kWeight), make_float2(0.f, 0.f));
                sum = fadd2(sum, e);
                s[2 * j] = __float_as_uint(e.x);
                s[2 * j + 1] = __float_as_uint(e.y);
            }
            if (t > 0) {
                add((t - 1) & 1);   // P and O are free then
                if (!ok) break;
            }
            if (__any_sync(0xffffffffu, move)) {
                const float2 f2 = make_float2(f, f);
#pragma unroll
                for (int j = 0; j < D / 2; ++j) {
                    acc[j].x *= f2.x;
                    acc[j].y *= f2.y;
                }
            }
            l = l * f + (sum.x + sum.y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // 16 keys: 8 columns of each part
                uint32_t h[8], mi[8], lw[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    three_parts(make_float2(__uint_as_float(s[16 * k + 2 * j]), __uint_as_float(s[16 * k + 2 * j + 1])), h[j], mi[j], lw[j]);
                tmem_st8(tp + 8 * k, h);
                tmem_st8(tp + 32 + 8 * k, mi);
                tmem_st8(tp + 64 + 8 * k, lw);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        if (ok) add((nt - 1) & 1);
        if (ok) {
            if (misc[1]) {
                // (rare) non-finite values, for the rows that see them
#pragma unroll
                for (int j = 0; j < D; ++j) {
                    float& x = j & 1 ? acc[j / 2].y : acc[j / 2].x;
                    if (over[j] <= lim) x += INFINITY;
                    if (over[D + j] <= lim) x -= INFINITY;
                    if (over[2 * D + j] <= lim) x = __int_as_float(0x7FC00000);
                }
            }
            if constexpr (M::kind != 0) {
                if (*edge_bad) {
                    // (rare) the same for slots that not every row sees, one after the other
                    const RowSight<M> sight(mask, g, first + (min(row, rows - 1) >> a.gshift), seen0, nq, lim);
                    for (int32_t s = lo; s < end; ++s) {
                        if (all_see(s, 1)) continue;
                        const float* p = reinterpret_cast<const float*>(slot_row(v, u, key_slot<M>(s, gap, shift), true));
                        if (!p || !(sight.word(s) & 1)) continue;
#pragma unroll
                        for (int j = 0; j < D / 2; ++j) {
                            const float2 x = reinterpret_cast<const float2*>(p)[j];
                            if (non_finite(x.x)) acc[j].x += x.x;
                            if (non_finite(x.y)) acc[j].y += x.y;
                        }
                    }
                }
            }
            const bool wide = splits > 1 || (((uintptr_t)a.out.p | a.out.ts | a.out.hs) & 31) == 0;
            float inv = splits > 1 ? 1.f : 1.0f / l;
            if constexpr (M::kind == 2) {
                if (splits == 1 && l == 0.f &&
                    RowSight<M>(mask, g, first + (min(row, rows - 1) >> a.gshift), seen0, nq, lim).blind())
                    inv = 0.f;   // (the sums are zero)
            }
            const int32_t row4 = row & ~3;
            const int32_t pt = M::kind != 0 ? part_token(a, i) : 0;   // of a token in the partial results, from its packed row
            uint8_t* dst[4];   // lane k of each four writes the k-th 32 bytes of four rows' 128
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t tok = first + ((row4 + j) >> a.gshift);
                const int32_t h = (g << a.gshift) + ((row4 + j) & ((1 << a.gshift) - 1));
                dst[j] = (splits > 1 ? reinterpret_cast<uint8_t*>(
                                           a.part + ((int64_t)split * a.part_rows + (int64_t)(tok + pt) * v.hq + h) * D)
                                     : a.out.row(tok, h)) +
                         32 * (lane & 3);
            }
#pragma unroll
            for (int j = 0; j < D; j += 32) {
                uint32_t x[4][8];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    x[k / 4][2 * k % 8] = __float_as_uint(acc[j / 2 + k].x * inv);
                    x[k / 4][2 * k % 8 + 1] = __float_as_uint(acc[j / 2 + k].y * inv);
                }
                quad_transpose(x, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (row4 + k < rows) store32(dst[k] + 4 * j, x[k], wide);
            }
            if (splits > 1 && row < rows) {
                const int32_t tok = first + (row >> a.gshift), h = (g << a.gshift) + (row & ((1 << a.gshift) - 1));
                const int64_t pr = (int64_t)split * a.part_rows + (int64_t)(tok + pt) * v.hq + h;
                *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m * c, l);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp < 12) {
            // ---------------- parts of K and V ----------------
            constexpr int CHUNKS = D / 8;   // groups of eight elements of a row
            // a row's group of eight within a part: 128-byte rows of 64 columns, 16-byte pieces swizzled by the row
            auto place = [&](int chunk, int r, int block) {
                return (chunk >> 3) * block + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
            };
            auto done = [&](uint64_t* bar) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            // warps 4-7 take the keys, 8-11 the values: a tile's rows wait in
            // registers while the products of the tile before run
            const bool is_v = warp >= 8;
            constexpr int STEP = kConvert / 2 / CHUNKS, PER = kKeys / STEP;   // rows a pass, rows of a thread
            const int ct = (threadIdx.x - 128) % (kConvert / 2), chunk = ct % CHUNKS, row_t = ct / CHUNKS;
            uint8_t* tiles0 = sm + (is_v ? C::OFF_V : C::OFF_K);
            float x[PER][8];
            auto load = [&](int32_t s0) {
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int32_t s = s0 + row_t + j * STEP;
                    const uint8_t* p = s < end ? slot_row(v, u, key_slot<M>(s, gap, shift), is_v) : nullptr;
                    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4*>(x[j]) = p ? reinterpret_cast<const float4*>(p)[2 * chunk] : z;
                    *reinterpret_cast<float4*>(x[j] + 4) = p ? reinterpret_cast<const float4*>(p)[2 * chunk + 1] : z;
                }
            };
            bool ok = run;
            if (run) load(lo);
            for (int32_t t = 0; ok && t < nt; ++t) {
                const int32_t s0 = lo + t * kKeys;
                if (t > 1) ok = warp_wait((is_v ? v_empty : k_empty) + (t & 1), ((t - 2) >> 1) & 1, where, 0x802 + is_v);
                if (!ok) break;
                uint8_t* tile = tiles0 + (t & 1) * C::TILE;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int r = row_t + j * STEP;
                    auto mend = [&](float* y) {
                        if (!is_v) return mark_nan(y);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (!non_finite(y[k])) continue;
                            const int kind = y[k] != y[k] ? 2 : (y[k] < 0.f ? 1 : 0);
                            y[k] = 0.f;
                            if (M::kind != 0 && !all_see(s0 + r, 1)) {
                                *edge_bad = 1;
                                continue;
                            }
                            atomicMin(&over[kind * D + 8 * chunk + k], M::kind == 0 ? s0 + r : -1);
                            misc[1] = 1;
                        }
                        __threadfence_block();
                    };
                    put_parts(tile + place(chunk, r, C::KBLOCK), C::KPART, x[j], mend);
                }
                done((is_v ? v_full : k_full) + (t & 1));
                if (t + 1 < nt) load(s0 + kKeys);
            }
        } else if (warp == 12) {
            // ---------------- products ----------------
            if (elect_one()) {
                constexpr uint32_t id_qk = idesc_of(128, kKeys, false), id_pv = idesc_of(128, D, true);
                const uint64_t dk = sdesc(smem_u32(sm + C::OFF_K), 16, 1024), dv = sdesc(smem_u32(sm + C::OFF_V), C::KBLOCK, 1024);
                // the parts of the two operands, smallest products first (0: h, 1: m, 2: l)
                constexpr int PA[6] = {1, 0, 2, 0, 1, 0}, PB[6] = {1, 2, 0, 1, 0, 0};
                bool ok = run;
                auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t index) {
                    ok = ok && attend_wait(bar, parity, where, index);
                };
                auto qk = [&](int32_t t) {   // S of tile t
                    const uint64_t b = dk + (t & 1) * (C::TILE >> 4);
                    wait(&k_full[t & 1], (t >> 1) & 1, 0x804);
                    if (t > 0) wait(s_read, (t - 1) & 1, 0x809);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int p = 0; p < 6; ++p)
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ts(tmem + kTmS, tmem + kTmQ + PA[p] * (D / 2) + 8 * k,
                                   b + ((PB[p] * C::KPART + (k / 4) * C::KBLOCK + (k % 4) * 32) >> 4), id_qk, p + k > 0);
                    mma_commit(s_full);
                    mma_commit(&k_empty[t & 1]);
                };
                wait(q_full, 0, 0x805);
                if (ok) qk(0);
                for (int32_t t = 0; ok && t < nt; ++t) {
                    if (t + 1 < nt) qk(t + 1);
                    const uint64_t b = dv + (t & 1) * (C::TILE >> 4);
                    wait(&v_full[t & 1], (t >> 1) & 1, 0x806);
                    wait(p_full, t & 1, 0x807);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int p = 0; p < 6; ++p)
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            mma_ts(tmem + kTmO, tmem + kTmP + 32 * PA[p] + 8 * k, b + ((PB[p] * C::KPART + k * 2048) >> 4), id_pv,
                                   p + k > 0);
                    mma_commit(o_full);
                    mma_commit(&v_empty[t & 1]);
                }
                // nothing is in flight when the CTA ends, after a wait that gave up neither
                mma_commit(drained);
                attend_wait(drained, 0, where, 0x808);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) attend_record(v.err, *where);
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int D, class M>
cudaError_t launch_masked(const AttendArgs& a, const M& m, cudaStream_t s) {
    const cudaError_t e = func_smem_optin((const void*)k_attend_f32<D, M>, F3<D>::BYTES);
    if (e != cudaSuccess) return e;
    return launch_overlapped(k_attend_f32<D, M>, a.items, kThreads, F3<D>::BYTES, s, a, m);
}

}  // namespace
}  // namespace hikv
