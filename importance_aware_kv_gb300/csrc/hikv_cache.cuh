// The cache object of the C ABI and the host helpers its entry points share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <vector>

#include "../../include/hikv.h"
#include "hikv_internal.cuh"

struct hikv_cache {
    using View = hikv::View;
    // configuration
    int L = 0, B = 0, Hq = 0, Hkv = 0, G = 0, d = 0, dtype = 0, esz = 0;
    int S = 0, W = 0, cap = 0, P = 0, page_shift = 0, max_pages = 0, max_wq = 0;
    int units = 0, per_layer = 0;
    int64_t pool_pages = 0;
    float scale = 0.f;
    std::vector<int32_t> budget_unit;   // [units]
    // device
    int device = 0, sm_count = 0;
    size_t smem_optin = 0;
    int max_smem_chunk = 0;             // decode smem path limit (tokens per CTA)
    int dec_occ = 2;                    // decode CTAs per SM
    View v{};
    int32_t* d_append_base = nullptr;
    float* d_logits = nullptr;          // long-chunk decode logits; packed attention's partial results
    // of d_logits for packed attention's partial results, in floats: every SM's
    // three work items of 256 query rows, or the longest unit's keys in parts of 256
    int64_t attend_room = 0;
    unsigned long long* d_cand = nullptr;
    int32_t* d_cand_slot = nullptr;
    int32_t* d_holes = nullptr;
    int64_t* d_hole_off = nullptr;
    float* d_wpart = nullptr;
    int wchunks = 0;
    int32_t* d_order_all = nullptr;
    int32_t* d_order_layer = nullptr;
    std::vector<int32_t> order_all, order_layer;   // host copies: units by budget, descending
    // balanced unit-to-cluster assignment of ragged decode calls (device copy
    // [units] list + [clusters + 1] offsets), recomputed when its inputs change
    // Device layout: [units] lists (a call over units [u0, u0 + nu) keeps its
    // list at [u0, ...)) + per first layer of a call an offsets region, so the
    // per-layer calls of a step each keep theirs and re-upload nothing while
    // their lengths repeat.
    int32_t* d_assign = nullptr;        // clusters: [units] + [L][max clusters + 1]
    std::vector<int32_t> asg;
    std::vector<uint64_t> asg_key;      // [L]
    // the same for the warp-per-unit kernel's per-warp unit lists
    int32_t* d_sassign = nullptr;       // [units] + [L][4 * max CTAs + 1]
    std::vector<int32_t> sasg;
    std::vector<uint64_t> sasg_key;     // [L]
    int small_mode = 1;                 // HIKV_DECODE_SMALL (tuning): 0 never, 1 auto, 2 always when eligible
    int first_burst = 4;                // one tile per consumer warp first (HIKV_DECODE_BURST: tuning)
    int prefetch_override = -1;         // HIKV_DECODE_PREFETCH (tuning): L2 prefetch distance in tiles, -1 auto
    CUtensorMap tmap;                   // the pool as rows of d elements, 16 x 128-byte swizzled boxes
    CUtensorMap tmap_page;              // the same with boxes of min(P, 128) rows (bf16: packed attention)
    std::vector<void*> allocs;
    // host mirror
    std::vector<int32_t> len, next_pos, mapped;
    std::vector<uint8_t> fresh;         // decode ran since the last state change
    // newest tokens of each unit that sit in its last slots in position order:
    // all of them until a cut moves survivors, then those appended since
    std::vector<int32_t> tail;
    int64_t pages_in_use = 0;
    int cs_override = 0;                // HIKV_DECODE_CS (tuning)
    int64_t launches = 0;               // kernels launched through this cache
    // the cluster launches of the latest decode call (at most two): units,
    // cluster size, clusters, logits in shared memory
    int32_t last_cfg[2][4] = {};
    int last_ncfg = 0;
    int pool_k = 0;                     // SnapKV pooling of the prompt scores (> 1: on)
    // HiKV Stage II element-level decode (elem > 0: on)
    int elem = 0;
    int elem_stride = 0;                // row stride of its order / logit buffers
    int32_t* d_eorder = nullptr;        // [units][elem_stride]
    float* d_elg = nullptr;             // [units][G][elem_stride]
    float* d_epart = nullptr;           // [units][max spans][G][d + 2]
    unsigned long long* d_erows = nullptr;   // V rows the element-level steps read
    float* d_eqmask = nullptr;          // [units][G][d]
    int32_t* d_edone = nullptr;         // [units]
    // HiKV banded prefill scores (band_scoring): one layer's per-query softmax statistics
    float2* d_band = nullptr;           // [per_layer][G][cap]
    // Programmatic dependent launch: the units [pdl_lo, pdl_hi) the latest
    // kernel this cache launched may write, and its stream (pdl_valid: that
    // latest launch is known); a decode launch on disjoint units of the same
    // stream may load its pages before waiting for it
    bool pdl_on = true;                 // HIKV_PDL=0 (tuning) turns it off
    bool pdl_valid = false;
    int pdl_lo = 0, pdl_hi = 0;
    hikv_stream_t pdl_stream = nullptr;
};

namespace hikv {

// NVTX range around an entry point (seen by nsys / ncu timelines; a no-op
// when no tool is attached)
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

// Set hikv_last_error() and return `s`.
hikv_status fail(hikv_status s, const char* fmt, ...);
hikv_status cuda_fail(cudaError_t e, const char* what);
hikv_status cuda_fail(cudaError_t e, const char* who, const char* part);
void set_last_error(const char* msg);

// cuTensorMapEncodeTiled from the driver, or null.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline void pdl_forget(hikv_cache* c) { if (c) c->pdl_valid = false; }

inline bool range_ok(const hikv_cache* c, int32_t layer0, int32_t nl) {
    return c && layer0 >= 0 && layer0 < c->L && nl > 0 && nl <= c->L - layer0;   // (their sum can pass 32 bits)
}

// The cache's device made current for the length of a call.
struct DeviceGuard {
    int prev = -1;
    cudaError_t status;
    explicit DeviceGuard(int device) {
        status = cudaGetDevice(&prev);
        if (status == cudaSuccess && prev != device) status = cudaSetDevice(device);
        else prev = -1;
    }
    ~DeviceGuard() { if (prev >= 0) cudaSetDevice(prev); }
};

}  // namespace hikv
