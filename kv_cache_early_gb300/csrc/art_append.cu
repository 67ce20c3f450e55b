// art_append.cu -- appending new tokens to the paged cache, with the position
// rotation applied on the way.
//
// For token t of sequence b, the i-th of its n_b new tokens, with cache place
// s = seq_len_b - n_b + i (seq_lens count the new tokens already) and position
// pos (s, or the caller's):
//     angle_j = pos * inv_freq_j                              j < rot_dim / 2
//     (x_j, x_j') -> scale * (x_j cos - x_j' sin, x_j' cos + x_j sin)
// for every query head (into q_out) and every key head (into the cache); the
// pairs are (j, j + rot_dim / 2) or, interleaved, (2j, 2j + 1); columns from
// rot_dim on and the values are copied. The cache row of KV head g is
// (page(s / Ps) * Hkv + g) * Ps + s % Ps.
//
// pos * inv_freq reaches 1e5..1e6 radians, where a 32-bit product is off by hundredths
// of a radian: the angle is formed and reduced to one turn with more than 32 bits
// (turn_of). Sine, cosine and the rotation are 32-bit; a bf16 result is rounded once
// at the store.
//
// Bound: HBM, 2 (Hq + 2 Hkv) d bytes in and as many out a token. A CTA takes one
// token, or two: their first rows are loaded (independent of the position) before
// the chain offsets -> seq_len -> page id -> angles, so a decode step waits for the
// longer of the two and not for their sum. One more CTA (block 0) checks the device
// data of the call and stores the status word, so that no memset precedes the
// kernel; every token's CTA checks what it uses by itself. Measured: prompts of 36727
// tokens (32/8 heads, d 128, bf16) 136 us, 98 % of the copy rate; a step of 1 or 128
// tokens 2.9 us.
#include "art_append.cuh"

namespace art {

// Up to these many tokens a CTA takes one (four CTAs an SM: all run at once and a step
// waits for one chain of loads), beyond it two (which share the chain). Measured, one
// against two (us): 128 tokens 3.5 / 4.2, 512 4.4 / 4.7, 1024 7.3 / 6.1, 4096 24.0 / 21.3.
constexpr int kFewTokens = 608;

template <bool kBF16, int D, bool kVec, int kTok>
__global__ void __launch_bounds__(kAppendThreads) art_append_kernel(const AppendParams p) {
    if (blockIdx.x == 0) {
        append_check(p);
        return;
    }
    append_rows<kBF16, D, kVec, kTok>(p, p.Hkv, blockIdx.x - 1);
}

int append_setup(AppendParams& p, const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                 int64_t v_stride, const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions,
                 const int32_t* block_table, const int32_t* seq_lens, const float* inv_freq, const art_rope* rope,
                 void* q_out, const void* cache, const void* cache2, const art_shape* shape, void* workspace,
                 size_t workspace_bytes) {
    const int rc = check_cache_shape(shape);
    if (rc != ART_OK) return rc;
    const art_shape& s = *shape;
    if (!block_table || !seq_lens || !cache || !cache2 || !workspace || !rope) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (!k || !v)) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (q != nullptr) != (q_out != nullptr)) return ART_ERR_INVALID_ARG;
    if (num_tokens < 0 || (!q_offsets && num_tokens != s.batch)) return ART_ERR_INVALID_ARG;
    if (num_tokens == 0x7fffffff) return ART_ERR_UNSUPPORTED;  // one block more than tokens
    for (int i = 0; i < 5; ++i)
        if (rope->reserved[i] != 0) return ART_ERR_INVALID_ARG;
    if (rope->rot_dim < 0 || rope->rot_dim > s.head_dim || (rope->rot_dim & 1)) return ART_ERR_INVALID_ARG;
    if (rope->interleaved != 0 && rope->interleaved != 1) return ART_ERR_INVALID_ARG;
    if (rope->rot_dim > 0 && !inv_freq) return ART_ERR_INVALID_ARG;
    const int elt = s.dtype == ART_DTYPE_BF16 ? 2 : 4, chunk = 16 / elt;
    auto bad = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) != 0; };
    if (bad(q) || bad(k) || bad(v) || bad(q_out) || bad(cache) || bad(cache2) || bad(workspace))
        return ART_ERR_INVALID_ARG;
    const int64_t kvw = (int64_t)s.num_kv_heads * s.head_dim;
    if ((q && (q_stride < (int64_t)s.num_q_heads * s.head_dim || q_stride % chunk)) || k_stride < kvw ||
        k_stride % chunk || v_stride < kvw || v_stride % chunk)
        return ART_ERR_INVALID_ARG;
    // in place only row by row: another token's row would be overwritten before it is read
    if (q && q == q_out && num_tokens > 1 && q_stride != (int64_t)s.num_q_heads * s.head_dim) return ART_ERR_INVALID_ARG;
    if (2 * ((int64_t)s.num_q_heads + 2 * (int64_t)s.num_kv_heads) * s.head_dim > (1LL << 30)) return ART_ERR_UNSUPPORTED;
    if (workspace_bytes < sizeof(WsHeader)) return ART_ERR_WORKSPACE;

    p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_offsets = q_offsets;
    p.positions = positions;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.inv_freq = inv_freq;
    p.q_out = q_out;
    p.hdr = static_cast<WsHeader*>(workspace);
    p.B = s.batch;
    p.T = num_tokens;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.Ps = s.page_size;
    p.max_pages = s.max_pages_per_seq;
    p.num_pages = s.num_pages_total;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved;
    p.scale = rope->scale;
    return ART_OK;
}

}  // namespace art

using namespace art;

extern "C" {

size_t art_append_workspace_bytes(const art_shape* shape) { return shape ? sizeof(WsHeader) : 0; }

int art_append_kv(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                  const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions, const int32_t* block_table,
                  const int32_t* seq_lens, const float* inv_freq, const art_rope* rope, void* q_out, void* k_cache,
                  void* v_cache, const art_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
    AppendParams p;
    const int rc = append_setup(p, q, k, v, q_stride, k_stride, v_stride, q_offsets, num_tokens, positions, block_table,
                                seq_lens, inv_freq, rope, q_out, k_cache, v_cache, shape, workspace, workspace_bytes);
    if (rc != ART_OK) return rc;
    const art_shape& s = *shape;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    const int chunk = s.dtype == ART_DTYPE_BF16 ? 8 : 4;
    const bool bf = s.dtype == ART_DTYPE_BF16;
    const bool vec = (p.interleaved ? p.rot : p.rot / 2) % chunk == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int tok = num_tokens <= kFewTokens ? 1 : 2;
    const unsigned grid = (unsigned)((num_tokens + tok - 1) / tok) + 1u;
#define ART_APPEND(BF, DD, VEC)                                                               \
    (tok == 1 ? art_append_kernel<BF, DD, VEC, 1><<<grid, kAppendThreads, 0, st>>>(p)         \
              : art_append_kernel<BF, DD, VEC, 2><<<grid, kAppendThreads, 0, st>>>(p))
    if (bf && s.head_dim == 128) { if (vec) ART_APPEND(true, 128, true); else ART_APPEND(true, 128, false); }
    else if (bf) { if (vec) ART_APPEND(true, 64, true); else ART_APPEND(true, 64, false); }
    else if (s.head_dim == 128) { if (vec) ART_APPEND(false, 128, true); else ART_APPEND(false, 128, false); }
    else { if (vec) ART_APPEND(false, 64, true); else ART_APPEND(false, 64, false); }
#undef ART_APPEND
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ART_OK : cuda_fail(e);
}

}  // extern "C"
