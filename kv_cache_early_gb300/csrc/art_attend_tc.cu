// art_attend_tc.cu -- launch of the bf16 segment kernel (art_attend_tc.cuh).
#include "art_attend_tc.cuh"
#include "art_kernel.cuh"

namespace art {

// The cache as 8-row groups: {64 columns, 8 rows, column halves, groups}; a copy takes
// a page's rows (at most a tile's) and lands as [group][half][8 rows][128 bytes].
static cudaError_t make_group_map(CUtensorMap* m, const void* base, long long groups, int D, int rows) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)(D / 64), (cuuint64_t)groups};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)(D / 64), (cuuint32_t)(rows / 8)};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
static cudaError_t launch_tc(const AttendParams& p, cudaStream_t st) {
    CUtensorMap tk, tv;
    const long long groups = (long long)p.num_pages * p.Hkv * p.Ps / 8;
    const int rows = p.Ps < kKeyTile ? p.Ps : kKeyTile;
    cudaError_t e;
    if ((e = make_group_map(&tk, p.k, groups, D, rows)) != cudaSuccess) return e;
    if ((e = make_group_map(&tv, p.v, groups, D, rows)) != cudaSuccess) return e;
    constexpr size_t smem = tc_smem<D>();
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    if ((e = cudaFuncSetAttribute(art_attend_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
        cudaSuccess)
        return e;
    return launch_after(art_attend_tc_kernel<D>, dim3(p.ctas), dim3(kTcThreads), smem, st, p, tk, tv);
}

cudaError_t launch_attend_tc(const AttendParams& p, cudaStream_t st) {
    return p.D == 128 ? launch_tc<128>(p, st) : launch_tc<64>(p, st);
}

}  // namespace art
