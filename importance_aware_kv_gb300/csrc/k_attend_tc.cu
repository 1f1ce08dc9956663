// Causal attention of packed queries over the paged cache on the tensor cores
// (bf16).
//
//   o_i = sum_{s <= lim_i} 2^(t_is - m_i) v_s / sum_{s <= lim_i} 2^(t_is - m_i),
//   t_is = scale log2(e) q_i . k_s,
//
// in one pass over the keys.  The exponent's reference m_i lies up to 24 (in
// powers of two) above the running maximum and moves only when a tile's
// maximum passes it: until then the accumulator needs no rescaling.  The
// largest weight of a row is then in [2^-24, 1], so that sums of n weighted
// values stay below n max |v|, as with a reference at the maximum, and bf16 and
// fp32 hold weights and sums at their full relative precision (a product of a
// weight and a value below 2^-126, |v| < 2^-102, may be lost).  (A step of 8
// moves it in one tile of twenty for heavy-tailed logits, and one row that
// moves holds up its whole tile: 2650 us against 2575 for 16K tokens of 64/8
// heads.)
//
// A CTA takes one work item after the other, 256 query rows x one KV head: two
// tiles of 128 rows that share every key tile, so that the tensor cores work
// on one while the softmax of the other runs.
//   warps 0-3, 4-7  softmax of row tile 0 and 1, one thread a row: logits from
//                   tensor memory, probabilities back over them as bf16
//   warp 8          TMA: the query tiles, then K and V tiles of 128 keys
//                   through a ring of stages (boxes of at most one page)
//   warps 9, 11     one thread each issues the products of row tile 0 and 1: S = Q K^T
//                   (both operands in shared memory), O += P V (P in tensor memory)
//   warp 10         the V tiles at the end of what rows see: rows past the last
//                   visible key become zero, non-finite values are
//                   taken out and added back only for the rows that see them
// Tensor memory: S/P of tile 0 and 1 in columns [0, 128) and [128, 256), O in
// [256, 256 + D) and [384, 384 + D).  The products of one thread execute in
// the order they are issued -- O += P V(t), S = Q K(t+1) -- so S(t+1) lands
// after P(t) was read, and a tile's S being complete means its O is up to
// date.
//
// Probabilities enter the product with V as bf16 (relative error 2^-8 each,
// averaged over the keys).  The sums l are of the fp32 values, but for a row's
// largest probability (the largest between two moves of the reference), which
// enters rounded there too: a row that sees little else returns that key's value
// as it is, wherever in [2^-24, 1] the reference has left its
// probability.  (Against 64 bits the 8K prompt is off by 0.0019 norm-wise,
// 0.0023 without this; summing every rounded value gives 0.0019 too and takes
// 358 us instead of 350.)
//
// Measured: 16K tokens with 64/8 heads, d = 128, 2.65 ms, 1.66 PFLOP/s; 8K with
// 32/8 345 us, 1.59; five tokens over eight 8K-32K caches 119 us, 6.1 TB/s of
// keys and values.  What bounds a long prompt: a row tile's step takes about
// 2,450 cycles (softmax 770 to the first half of P, waking the issuing thread
// 400, the products 1,024, their latency 340) where the products of both
// tiles need 2,048, and the chip runs at its power limit.  256 rows an item
// because each key tile is then read from L2 once for two row tiles (64 KB a
// step and SM; one row tile would double that to more than L2 delivers).
#include "hikv_tcgen05.cuh"

namespace hikv {
namespace {

constexpr int kThreads = 384;
// Registers a thread: 168 at launch (384 x 168 of the SM's 64 K); the softmax
// warps, which hold a row of 128 logits each, take what the others give up:
// 256 x 216 + 128 x 72 = 384 x 168.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr int kKeys = kTcKeys, kRows = kTcRows;
constexpr float kAhead = 24.f;   // the reference above the maximum that it was set at

template <int D>
struct Tc {
    static constexpr int HALVES = D / 64;                 // 128-byte columns blocks of a row
    static constexpr int BLOCK = 128 * 128;               // 128 rows x 128 bytes
    static constexpr int TILE = HALVES * BLOCK;           // a tile of Q, K or V
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int OFF_Q = 0;                       // two tiles
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_BAR = OFF_KV + STAGES * TILE;
    // barriers: kv_full[STAGES], kv_empty[STAGES], v_ok[STAGES], q_full, q_empty, s_full[2], p_full[2][2], o_full[2],
    // drained, answer, item_full[2], item_empty[2]
    static constexpr int NBAR = 3 * STAGES + 16;
    static constexpr int OFF_ANSWER = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;   // of the work distributor, 16 bytes
    static constexpr int OFF_ITEM = OFF_ANSWER + 16;      // two work items
    static constexpr int OFF_MISC = OFF_ITEM + 2 * 64;    // tensor memory address, epilogue count, overlay item, turn
    static constexpr int OFF_WHERE = OFF_MISC + 16;       // where a wait gave up
    static constexpr int OFF_OVER = OFF_WHERE + 16;       // [3][D] first slots of +inf, -inf, NaN
    static constexpr int BYTES = OFF_OVER + 3 * D * 4 + 1024;
};

// position in a ring of N stages and the parity of its fill
template <int N>
struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
        if (++st == N) {
            st = 0;
            ph ^= 1;
        }
    }
};

// A work item, the same in every warp
struct __align__(16) Item {
    int32_t some;            // 0: there is none left
    int32_t g, first, rows;  // KV head, first packed row, query rows of the sequence
    int32_t r0, seen0, lim0; // first row; slots before the first query's own; last slot the first row sees
    int32_t lo, end;         // keys [lo, end) of this split that any row sees
    int32_t nt0, nt1, ntiles;   // key tiles of each row tile, and of the item
    int32_t split;           // of the keys, -1: not split
    int32_t u, pad[2];
};
static_assert(sizeof(Item) == 64, "two items in OFF_ITEM");
// item number `it` of the grid; false if it has nothing to do
__device__ __forceinline__ bool load_item(const AttendArgs& a, int32_t it, Item& w) {
    const View& v = a.v;
    const int32_t i = prefix_find(a.item0, a.nseq, it);
    const int32_t nq = a.nq[i];
    w.some = 1;
    w.rows = nq << a.gshift;
    const int32_t tiles = (w.rows + kRows - 1) / kRows;
    const int32_t rem = it - a.item0[i], x = a.hkv_shift >= 0 ? rem >> a.hkv_shift : rem / v.hkv;
    w.g = rem - x * v.hkv;
    w.u = a.u0 + a.brow[i] * v.hkv + w.g;
    const int32_t n = unit_len(a, i, w.u);
    const int32_t splits = a.parts[i];
    const int32_t tile = splits > 1 ? x / splits : x;
    w.split = splits > 1 ? x - tile * splits : -1;
    w.r0 = (tiles - 1 - tile) * kRows;
    w.first = a.start[i];
    if (n < nq || n > v.cap) {
        if ((threadIdx.x & 31) == 0) atomicOr(v.err, DEVERR_STATE);
        return false;
    }
    w.seen0 = n - nq;
    w.lim0 = w.seen0 + (w.r0 >> a.gshift);
    w.lo = splits > 1 ? w.split * a.chunk : 0;
    auto keys_end = [&](int32_t a0) {   // one past the last key that the row tile from row a0 on sees
        if (a0 >= w.rows) return 0;
        const int32_t hi = w.seen0 + ((min(a0 + 128, w.rows) - 1) >> a.gshift) + 1;
        return splits > 1 ? min(hi, w.lo + a.chunk) : hi;
    };
    const int32_t e0 = keys_end(w.r0), e1 = keys_end(w.r0 + 128);
    w.nt0 = max(e0 - w.lo + kKeys - 1, 0) / kKeys;
    w.nt1 = max(e1 - w.lo + kKeys - 1, 0) / kKeys;
    w.end = max(e0, e1);
    w.ntiles = max(w.nt0, w.nt1);
    return w.ntiles > 0;
}
// tile t holds slots that the item's first row does not see, or that do not exist
__device__ __forceinline__ bool edge_tile(const Item& w, int32_t t) { return w.lo + t * kKeys + kKeys - 1 > w.lim0; }

// The work items of a CTA.  The grid has a CTA per item; a CTA that has
// started takes the numbers of CTAs that have not, so the items go out one by
// one, in order, to whoever is free.  Warp 8 asks for the next number while
// it loads an item, works out what the item is and hands it to the other
// roles through shared memory, one item ahead of them.
constexpr int kReaders = 11;   // softmax warps, both issuing threads, warp 10
struct Items {
    uint64_t* full;
    uint64_t* empty;
    const Item* slot;
    volatile uint32_t* where;
    uint32_t n = 0;   // number of the next item to take
    // the next item, false if there is none left; a whole warp
    __device__ __forceinline__ bool take(Item& w) {
        const uint32_t s = n & 1;
        if (!warp_wait(&full[s], (n >> 1) & 1, where, 0x700)) return false;
        w = slot[s];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
        ++n;
        return w.some != 0;
    }
    // the same for one thread
    __device__ __forceinline__ bool take_one(Item& w) {
        const uint32_t s = n & 1;
        if (!attend_wait(&full[s], (n >> 1) & 1, where, 0x701)) return false;
        w = slot[s];
        mbar_arrive(&empty[s]);
        ++n;
        return w.some != 0;
    }
};
// ask for the number of a CTA that has not started; answered on `bar`
__device__ __forceinline__ void ask_next(uint32_t answer, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
        "r"(smem_u32(bar))
        : "memory");
}
// the answer: a number, or -1 if every CTA has started
__device__ __forceinline__ int32_t read_next(uint32_t answer) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(answer)
        : "memory");
    fence_proxy_async_smem();   // before the next answer is written over it
    return ok ? (int32_t)x : -1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend_tc(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kvmap) {
    using C = Tc<D>;
    extern __shared__ __align__(128) uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
    uint64_t* kv_empty = kv_full + C::STAGES;
    uint64_t* v_ok = kv_empty + C::STAGES;
    uint64_t* q_full = v_ok + C::STAGES;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = p_full + 4;   // p_full: [tile][half of the keys]
    uint64_t* drained = o_full + 2;
    uint64_t* answer = drained + 1;
    uint64_t* item_full = answer + 1;
    uint64_t* item_empty = item_full + 2;
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_MISC);
    volatile uint32_t* where = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_WHERE);
    int32_t* over = reinterpret_cast<int32_t*>(sm + C::OFF_OVER);
    const View& v = a.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 3);   // both tiles' products are complete, and warp 10
            mbar_init(&v_ok[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        mbar_init(drained, 2);
        mbar_init(answer, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);   // one lane of each softmax warp
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], kReaders);
        }
        misc[1] = 0;                      // epilogues done, in warps
        misc[3] = 0;                      // a row tile is issuing the products between two of its softmaxes
        *where = 0;
        misc[2] = 0;                      // the item that `over` belongs to, from 1 on
        fence_mbar_init();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kvmap);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(sm + C::OFF_MISC))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const bool gave_up = warp == 8 && attend_gave_up(v);
    griddep_wait();   // what the kernel before writes is there: lengths, pages, q
    Item w0;
    if (warp == 8) {
        if (!load_item(a, blockIdx.x, w0)) w0.ntiles = 0;
        w0.some = !gave_up;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    Items items{item_full, item_empty, reinterpret_cast<Item*>(sm + C::OFF_ITEM), where};
    Item w;

    if (warp < 8) {
        // ---------------- softmax ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int tile = warp >> 2;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lane_base + 128 * tile, to = tmem + lane_base + 256 + 128 * tile;
        uint32_t sphase = 0, ophase = 0;
        const float c = a.qscale;
        const bool wide = (((uintptr_t)a.out.p | a.out.ts | a.out.hs) & 31) == 0;
        bool ok = true;
        while (ok && items.take(w)) {
            const int32_t row = w.r0 + 128 * tile + 32 * (warp & 3) + lane;
            const int32_t rc = min(row, w.rows - 1);
            const int32_t lim = w.seen0 + (rc >> a.gshift);   // this row sees slots [0, lim]
            const int32_t lim_w = w.seen0 + (min(w.r0 + 128 * tile + 32 * (warp & 3), w.rows - 1) >> a.gshift);
            const int32_t nt = tile ? w.nt1 : w.nt0;
            float m = -INFINITY, l = 0.f;   // m: the maximum at the reference's last move
            float top = -INFINITY;          // the largest logit since
            auto reference = [&] { return m == -INFINITY ? 0.f : fmaf(m, c, kAhead); };
            auto settle = [&] {             // top's probability in l as the product took it
                const float pt = ex2(fmaf(top, c, -reference()));
                l += __uint_as_float(pack_bf16x2(pt, 0.f) << 16) - pt;
            };
            for (int32_t t = 0; t < nt; ++t) {
                if (!warp_wait(&s_full[tile], sphase, where, 0x100 + t)) { ok = false; break; }
                sphase ^= 1;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld32(s + 32 * j, ts + 32 * j);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) held(s + 32 * j);
                const int32_t s0 = w.lo + t * kKeys;
                if (s0 + kKeys - 1 > lim_w) {
                    const int32_t left = lim - s0;   // columns [0, left] are seen
#pragma unroll
                    for (int j = 0; j < 128; ++j) s[j] = j <= left ? s[j] : 0xFF800000u;
                }
                float mx[4] = {m, m, m, m};
#pragma unroll
                for (int j = 0; j < 128; j += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = max3(mx[k], __uint_as_float(s[j + 2 * k]), __uint_as_float(s[j + 2 * k + 1]));
                const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                // (mt - m is NaN while both are -inf: no move)
                const bool move = (mt - m) * c > kAhead;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = m == mt ? 1.f : ex2((m - mt) * c);
                    if (t > 0) {
#pragma unroll
                        for (int j = 0; j < D; j += 8) {
                            uint32_t o[8];
                            tmem_ld8(o, to + j);
                            tmem_wait_ld();
                            held8(o);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st8(to + j, o);
                        }
                    }
                    settle();
                    l *= f;
                    top = m = mt;
                }
                top = fmaxf(top, mt);
                const float base = reference();
                const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const uint32_t* y = s + 32 * k + 2 * j;
                        const float2 x = ffma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), c2, b2);
                        const float2 e = make_float2(ex2(x.x), ex2(x.y));
                        sum = fadd2(sum, e);
                        p[j] = pack_bf16x2(e.x, e.y);
                    }
                    tmem_st16(ts + 16 * k, p);
                    if (k & 1) {   // half of the keys: their product with V may start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[2 * tile + k / 2]);
                    }
                }
                l += sum.x + sum.y;
            }
            if (!ok) break;
            settle();
            if (nt > 0) {
                if (!warp_wait(&o_full[tile], ophase, where, 0x200)) { ok = false; break; }
                ophase ^= 1;
                tc_fence_after();
                if (misc[2] == items.n) {
                    // (rare) non-finite values of the edge tiles, for the rows that see them
#pragma unroll 1
                    for (int j = 0; j < D; ++j) {
                        uint32_t o;
                        tmem_ld1(o, to + j);
                        float x = __uint_as_float(o);
                        if (over[j] <= lim) x += INFINITY;
                        if (over[D + j] <= lim) x -= INFINITY;
                        if (over[2 * D + j] <= lim) x = __int_as_float(0x7FC00000);
                        tmem_st1(to + j, __float_as_uint(x));
                    }
                    tmem_wait_st();
                }
                const float inv = w.split < 0 ? 1.0f / l : 1.f;
                // lane i of each four ends up with the i-th 32 bytes of four rows' 128
                const int32_t row4 = row & ~3;
                uint8_t* dst[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t tok = w.first + ((row4 + j) >> a.gshift);
                    const int32_t h = (w.g << a.gshift) + ((row4 + j) & ((1 << a.gshift) - 1));
                    dst[j] = (w.split < 0 ? a.out.row(tok, h)
                                          : reinterpret_cast<uint8_t*>(
                                                a.part + ((int64_t)w.split * a.part_rows + (int64_t)tok * v.hq + h) * D)) +
                             32 * (lane & 3);
                }
                // (not unrolled: an item runs this once, from a cold instruction cache)
                if (w.split < 0) {
#pragma unroll 1
                    for (int j = 0; j < D; j += 64) {
                        uint32_t o[64], x[4][8];
                        tmem_ld32(o, to + j);
                        tmem_ld32(o + 32, to + j + 32);
                        tmem_wait_ld();
                        held(o);
                        held(o + 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i / 8][i % 8] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                        quad_transpose(x, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row4 + i < w.rows) store32(dst[i] + 2 * j, x[i], wide);
                    }
                } else {
#pragma unroll 1
                    for (int j = 0; j < D; j += 32) {
                        uint32_t x[4][8];
                        tmem_ld32(&x[0][0], to + j);
                        tmem_wait_ld();
                        held(&x[0][0]);
                        quad_transpose(x, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row4 + i < w.rows) store32(dst[i] + 4 * j, x[i], true);
                    }
                }
                if (w.split >= 0 && row < w.rows) {
                    const int32_t tok = w.first + (row >> a.gshift), h = (w.g << a.gshift) + (row & ((1 << a.gshift) - 1));
                    const int64_t pr = (int64_t)w.split * a.part_rows + (int64_t)tok * v.hq + h;
                    *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m == -INFINITY ? m : reference(), l);
                }
            }
            __syncwarp();
            if (lane == 0) atomicAdd(const_cast<uint32_t*>(&misc[1]), 1u);
        }
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
        // ---------------- TMA ----------------
        const int bx = min(v.page_tokens, 128), nb = 128 / bx;   // rows of a box, boxes of a tile
        const uint32_t ans = smem_u32(sm + C::OFF_ANSWER);
        uint32_t fill = 0, n = 0, asked = 0, read = 0;   // n: items handed out
        bool ok = true;
        auto hand_out = [&](const Item& x) {
            const uint32_t s = n & 1;
            if (n >= 2) ok = ok && warp_wait(&item_empty[s], ((n - 2) >> 1) & 1, where, 0x702);
            if (!ok) return;
            if (lane == 0) {
                *reinterpret_cast<Item*>(sm + C::OFF_ITEM + 64 * s) = x;
                mbar_arrive(&item_full[s]);
            }
            ++n;
        };
        auto ask = [&] {
            if (lane == 0) ask_next(ans, answer);
            ++asked;
        };
        // the next item that has something to do; asks on until then
        auto next_item = [&](Item& x) {
            x.some = 0;
            while (ok) {
                ok = warp_wait(answer, read & 1, where, 0x703);
                if (!ok) return;
                ++read;
                const int32_t it = read_next(ans);
                __syncwarp();
                if (it < 0 || load_item(a, it, x)) {
                    x.some = it >= 0;
                    return;
                }
                ask();
            }
        };
        w = w0;
        if (w.some && w.ntiles == 0) {
            ask();
            next_item(w);
        }
        uint32_t loaded = 0;
        if (ok) hand_out(w);
        while (ok && w.some) {
            Item next;
            const int32_t fills = 2 * w.ntiles, when = min(4, fills);
            for (int32_t x = 0; ok && x <= fills; ++x) {
                if (x == when) {
                    next_item(next);
                    if (ok) hand_out(next);
                }
                if (x == fills || !ok) break;
                if (x == 1) {   // the first keys wait for nothing
                    if (loaded > 0) ok = warp_wait(q_empty, (loaded - 1) & 1, where, 0x300);
                    if (!ok) break;
                    ++loaded;
                    const int tiles = w.r0 + 128 < w.rows ? 2 : 1;
                    if (lane == 0) mbar_arrive_expect_tx(q_full, tiles * C::TILE);
                    __syncwarp();
                    if (lane < tiles * C::HALVES) {
                        const int t = lane / C::HALVES, hf = lane % C::HALVES;
                        tma_load_3d(sm + C::OFF_Q + t * C::TILE + hf * C::BLOCK, &qmap, 64 * hf, w.g << a.gshift,
                                    w.first + ((w.r0 + 128 * t) >> a.gshift), q_full);
                    }
                    if (asked == read) ask();
                }
                const int st = fill % C::STAGES;
                const uint32_t use = fill / C::STAGES;
                if (use > 0 && !warp_wait(&kv_empty[st], (use - 1) & 1, where, 0x400 + st)) { ok = false; break; }
                ++fill;
                const bool is_v = x & 1;
                const int32_t s0 = w.lo + (x >> 1) * kKeys;
                // lane -> (box, half); a box wholly past the last visible slot is not loaded
                const int box = lane / C::HALVES, hf = lane % C::HALVES;
                const int32_t s = s0 + box * bx;
                int32_t pg = -1;
                if (box < nb && s < w.end) {
                    pg = unit_page(v, w.u, s);
                    if (pg < 0 || pg >= v.pool_pages) {
                        atomicOr(v.err, DEVERR_PAGE);
                        pg = -1;
                    }
                }
                const uint32_t cnt = __popc(__ballot_sync(0xffffffffu, pg >= 0));
                if (lane == 0) mbar_arrive_expect_tx(&kv_full[st], cnt * bx * 128);
                __syncwarp();
                if (pg >= 0)
                    tma_load_2d(sm + C::OFF_KV + st * C::TILE + hf * C::BLOCK + box * bx * 128, &kvmap, 64 * hf,
                                (int32_t)((2 * (int64_t)pg + (is_v ? 1 : 0)) * v.page_tokens + (s & (v.page_tokens - 1))),
                                &kv_full[st]);
            }
            w = next;
        }
        // every answer and copy has landed and every commit arrived before the CTA ends
        if (asked > read) warp_wait(answer, read & 1, where, 0x704);
        if (loaded > 0) {
            if (ok) warp_wait(q_empty, (loaded - 1) & 1, where, 0x301);
            else warp_wait(q_full, (loaded - 1) & 1, where, 0x302);
        }
        for (uint32_t f = fill > C::STAGES ? fill - C::STAGES : 0; f < fill; ++f) {
            const int st = f % C::STAGES;
            const uint32_t par = (f / C::STAGES) & 1;
            if (ok) warp_wait(&kv_empty[st], par, where, 0x401);
            else warp_wait(&kv_full[st], par, where, 0x402);
        }
    } else if (warp == 9 || warp == 11) {
        // ---------------- products of row tile 0 (warp 9) and 1 (warp 11) ----------------
        // One thread each.  What it waits for besides P it waits for while
        // products it has issued are still running: about four products
        // queue, so a late issue is idle time.
        if (elect_one()) {
            constexpr uint32_t id_qk = idesc_of(128, kKeys, false), id_pv = idesc_of(128, D, true);
            const int tile = warp == 9 ? 0 : 1;
            const uint64_t dq = sdesc(smem_u32(sm + C::OFF_Q + tile * C::TILE), 16, 1024);
            const uint64_t dk = sdesc(smem_u32(sm + C::OFF_KV), 16, 1024), dv = sdesc(smem_u32(sm + C::OFF_KV), C::BLOCK, 1024);
            const uint32_t ts = tmem + 128 * tile, to = tmem + 256 + 128 * tile;
            uint32_t qphase = 0, pphase = 0, vuse = 0;
            Ring<C::STAGES> r;   // the fill in turn
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t index) {
                ok = ok && (mbar_try_wait(bar, parity) || attend_wait(bar, parity, where, index));
            };
            auto qk = [&](int st) {   // S = Q K^T
                const uint64_t k = dk + st * (C::TILE >> 4);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t off = ((i / 4) * C::BLOCK + (i % 4) * 32) >> 4;
                    mma_ss(ts, dq + off, k + off, id_qk, i > 0);
                }
                mma_commit(&s_full[tile]);
            };
            auto pv = [&](int st, int half, bool first) {   // O += P V of half of the tile's keys
                const uint64_t b = dv + st * (C::TILE >> 4);
#pragma unroll
                for (int j = 0; j < kKeys / 32; ++j) {
                    const int i = half * (kKeys / 32) + j;
                    mma_ts(to, ts + 8 * i, b + i * (2048 >> 4), id_pv, !(first && i == 0));
                }
            };
            bool have = items.take_one(w);
            while (have) {
                const int32_t nt = tile ? w.nt1 : w.nt0;
                wait(q_full, qphase, 0x501);
                qphase ^= 1;
                wait(&kv_full[r.st], r.ph, 0x500);
                if (!ok) break;
                tc_fence_after();
                if (nt > 0) qk(r.st);
                mma_commit(&kv_empty[r.st]);
                if (w.ntiles == 1) mma_commit(q_empty);
                r.step();
                for (int32_t t = 0; t < w.ntiles; ++t) {
                    const bool more = t + 1 < w.ntiles;
                    const int sv = r.st;   // V(t)
                    wait(&kv_full[sv], r.ph, 0x505);
                    if (edge_tile(w, t)) {
                        wait(&v_ok[sv], (vuse >> sv) & 1, 0x502);
                        vuse ^= 1u << sv;
                    }
                    r.step();
                    if (more) wait(&kv_full[r.st], r.ph, 0x506);   // K(t + 1)
                    if (t < nt) {
                        wait(&p_full[2 * tile], pphase, 0x503);
                        if (!ok) break;
                        tc_fence_after();
                        pv(sv, 0, t == 0);
                        wait(&p_full[2 * tile + 1], pphase, 0x507);
                        pphase ^= 1;
                        // One row tile at a time from here to its next S: sharing the
                        // tensor cores, two tiles in step would stay in step, their
                        // softmaxes at once and then their products at once.
                        ok = ok && turn_begin(const_cast<uint32_t*>(&misc[3]), where);
                        if (!ok) break;
                        tc_fence_after();
                        pv(sv, 1, false);
                        if (t + 1 < nt) qk(r.st);
                        else mma_commit(&o_full[tile]);
                        turn_end(const_cast<uint32_t*>(&misc[3]));
                    }
                    if (!ok) break;
                    mma_commit(&kv_empty[sv]);
                    if (more) {
                        mma_commit(&kv_empty[r.st]);
                        if (t + 2 == w.ntiles) mma_commit(q_empty);
                        r.step();
                    }
                }
                if (!ok) break;
                have = items.take_one(w);
            }
            // nothing is in flight when the CTA ends, after a wait that gave up neither
            mma_commit(drained);
            attend_wait(drained, 0, where, 0x504);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ---------------- the edge of what rows see ----------------
        uint32_t fill = 0, seen = 0;
        bool ok = true;
        while (ok && items.take(w)) {
            for (int32_t x = 0; x < 2 * w.ntiles; ++x, ++fill) {
                const int st = fill % C::STAGES;
                ok = warp_wait(&kv_full[st], (fill / C::STAGES) & 1, where, 0x600);
                if (!ok) break;
                if ((x & 1) && edge_tile(w, x >> 1)) {
                    const int32_t s0 = w.lo + (x >> 1) * kKeys;
                    const int32_t rv = min(kKeys, w.end - s0);   // rows that hold visible tokens
                    uint8_t* tile = sm + C::OFF_KV + st * C::TILE;
                    uint32_t top = 0;   // largest magnitude in either half of the words
                    for (int hf = 0; hf < C::HALVES; ++hf) {
                        uint4* p = reinterpret_cast<uint4*>(tile + hf * C::BLOCK);
#pragma unroll 8
                        for (int i = lane; i < rv * 8; i += 32) {
                            const uint4 y = p[i];
                            top = __vmaxu2(top, __vmaxu2(__vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu),
                                                         __vmaxu2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu)));
                        }
                        for (int i = rv * 8 + lane; i < kKeys * 8; i += 32) p[i] = make_uint4(0, 0, 0, 0);
                    }
                    const bool bad = (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u;
                    if (__any_sync(0xffffffffu, bad)) {
                        if (misc[2] != items.n) {
                            // `over` is free once every epilogue before this item has read it
                            const uint64_t t0 = global_ns();
                            while (misc[1] < 8 * seen) {
                                if (global_ns() - t0 > kWaitLimitNs) {
                                    *where = 0x601;
                                    ok = false;
                                    break;
                                }
                            }
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            for (int i = lane; i < 3 * D; i += 32) over[i] = 0x7FFFFFFF;
                            __syncwarp();
                        }
                        for (int hf = 0; hf < C::HALVES; ++hf)
                            for (int i = lane; i < rv * 64; i += 32) {
                                uint16_t* e = reinterpret_cast<uint16_t*>(tile + hf * C::BLOCK) + i;
                                const uint16_t y = *e;
                                if ((y & 0x7F80) != 0x7F80) continue;
                                const int r = i >> 6, col = 64 * hf + ((((i >> 3) & 7) ^ (r & 7)) << 3) + (i & 7);
                                const int kind = (y & 0x7F) ? 2 : (y >> 15);
                                atomicMin(&over[kind * D + col], s0 + r);
                                *e = 0;
                            }
                        __syncwarp();
                        __threadfence_block();
                        if (lane == 0) misc[2] = items.n;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_ok[st]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_empty[st]);
            }
            ++seen;
        }
    }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) attend_record(v.err, *where);
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int D>
cudaError_t launch(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kvmap, cudaStream_t s) {
    const void* f = (const void*)k_attend_tc<D>;
    cudaError_t e = func_smem_optin(f, Tc<D>::BYTES);
    if (e != cudaSuccess) return e;
    return launch_overlapped(k_attend_tc<D>, a.items, kThreads, Tc<D>::BYTES, s, a, qmap, kvmap);
}

}  // namespace

cudaError_t launch_attend_tc(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kvmap, int d,
                             cudaStream_t s) {
    return d == 128 ? launch<128>(a, qmap, kvmap, s) : launch<64>(a, qmap, kvmap, s);
}

}  // namespace hikv
