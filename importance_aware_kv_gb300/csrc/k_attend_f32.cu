// Causal attention of packed queries, fp32.
#include "k_attend_f32.cuh"

namespace hikv {

cudaError_t launch_attend_f32(const AttendArgs& a, int d, cudaStream_t s) {
    return d == 128 ? launch_masked<128>(a, CausalMask{}, s) : launch_masked<64>(a, CausalMask{}, s);
}

}  // namespace hikv
