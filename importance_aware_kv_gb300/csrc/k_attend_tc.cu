// Causal attention of packed queries on the tensor cores (bf16).
#include "k_attend_tc.cuh"

namespace hikv {

cudaError_t launch_attend_tc(const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kvmap, int d,
                             cudaStream_t s) {
    return d == 128 ? launch_masked<128>(a, CausalMask{}, qmap, kvmap, s) : launch_masked<64>(a, CausalMask{}, qmap, kvmap, s);
}

}  // namespace hikv
