// Attention of trees of drafted tokens on the tensor cores (bf16).
#include "k_attend_tc.cuh"

namespace hikv {

cudaError_t launch_attend_tc_tree(const AttendArgs& a, const TreeMask& m, const CUtensorMap& qmap,
                                  const CUtensorMap& kvmap, int d, cudaStream_t s) {
    return d == 128 ? launch_masked<128>(a, m, qmap, kvmap, s) : launch_masked<64>(a, m, qmap, kvmap, s);
}

}  // namespace hikv
