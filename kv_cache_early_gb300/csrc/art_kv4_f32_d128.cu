// art_kv4_f32_d128.cu -- attention over a cache in 4 bits: f32, head_dim 128.
#include "art_attend_kv4.cuh"

namespace art {

cudaError_t launch_kv4_f32_d128(const AttendKv4Params& p, int ng, cudaStream_t st) {
    if (ng == 1) return launch_kv4<false, 128, 1>(p, st);
    if (ng == 2) return launch_kv4<false, 128, 2>(p, st);
    return launch_kv4<false, 128, 4>(p, st);
}

}  // namespace art
