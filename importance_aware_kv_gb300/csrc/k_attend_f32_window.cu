// Attention over a sliding window a head and the first tokens, fp32.
#include "k_attend_f32.cuh"

namespace hikv {

cudaError_t launch_attend_f32_window(const AttendArgs& a, const WindowMask& m, int d, cudaStream_t s) {
    return d == 128 ? launch_masked<128>(a, m, s) : launch_masked<64>(a, m, s);
}

}  // namespace hikv
