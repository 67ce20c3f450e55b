// art_kv4.cuh -- the layout of a KV cache that is held in 4 bits (art.h, "A cache in 4 bits").
//
// The bytes of one page of one KV head: slabs of S = min(page, 64) tokens, each with the keys'
// codes, the values' codes, the keys' scales and the values' scales. Eight tokens x 32 columns of
// codes are 128 bytes, [8 tokens][16 bytes]: an 8 x 8 matrix of 16-bit units to ldmatrix, whose
// rows lie in all banks. Read as it is, it gives a lane 8 columns of one key; transposed, 4
// columns of two neighbouring tokens: both are operands of a matrix product after a mask and a
// shift (art_attend_kv4.cuh). A slab is one run of memory, so one bulk copy brings the whole of a
// page of up to 64 tokens, or 64 tokens of a larger one.
#pragma once

#include "art_common.cuh"

namespace art {

constexpr int kSlabTokens = 64;  // tokens of a slab at most

struct Kv4Layout {
    int slab, slab_log2;  // tokens of a slab
    int slab_bytes, page_bytes;
};
inline Kv4Layout kv4_layout(int page_size, int head_dim, int group) {
    Kv4Layout l;
    const int token = head_dim + 8 * (head_dim / group);
    l.slab = page_size < kSlabTokens ? page_size : kSlabTokens;
    l.slab_log2 = 0;
    while (1 << l.slab_log2 < l.slab) ++l.slab_log2;
    l.slab_bytes = l.slab * token;
    l.page_bytes = page_size * token;
    return l;
}
inline bool kv4_group_ok(int head_dim, int group) {
    return (group == 32 || group == 64 || group == 128) && group <= head_dim;
}

// Reads the whole cache of the sequences that have new tokens (by q_offsets) into a pool of max_pages_per_seq pages for
// each, whose block table `map` it writes: -1 for a page outside the cache (art_read_kv4.cu).
cudaError_t read_kv4_pool(const art_shape& s, int group, const void* cache, const int32_t* block_table,
                          const int32_t* seq_lens, const int32_t* q_offsets, int32_t* map, void* k_out, void* v_out,
                          int sms, cudaStream_t st);

// Place of a token in its slab's arrays: u is its number in the slab.
template <int D>
__device__ __forceinline__ int kv4_code_at(int u, int chunk) {  // 16 bytes: columns 32 chunk ..
    return (((u >> 3) * (D / 32) + chunk) * 8 + (u & 7)) * 16;
}
template <int NG>
__device__ __forceinline__ int kv4_scale_at(int u, int g) {  // 4 bytes: step, lowest
    return (((u >> 3) * NG + g) * 8 + (u & 7)) * 4;
}

}  // namespace art
