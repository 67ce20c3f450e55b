// art_kv4_bf16_d64.cu -- attention over a cache in 4 bits: bf16, head_dim 64.
#include "art_attend_kv4.cuh"

namespace art {

cudaError_t launch_kv4_bf16_d64(const AttendKv4Params& p, int ng, cudaStream_t st) {
    if (ng == 1) return launch_kv4<true, 64, 1>(p, st);
    return launch_kv4<true, 64, 2>(p, st);
}

}  // namespace art
