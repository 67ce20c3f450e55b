// art_attend_kv4.cu -- dense_extend_kv4: argument checks and the choice of the kernel.
#include <cmath>

#include "art_attend_kv4.cuh"

namespace art {

// Cost units of items and of their tiles of 128 keys, by rows (8, more).
constexpr CostRule kCostKv4 = {13, 5, 13, 8, 13, 8};

static void kv4_shape(AttendParams& p, const art_shape& s) {
    attend_shape(p, s);
    p.rt = kRowsKv4;
    p.kt_log2 = 7;
    p.small_rows = 8;
    p.cost = kCostKv4;
}

static cudaError_t launch_attend_kv4(const AttendParams& p, const void* more, cudaStream_t st) {
    AttendKv4Params pp = *static_cast<const AttendKv4Params*>(more);
    pp.a = p;
    const int ng = (pp.page_bytes / p.Ps - p.D) / 8;
    const bool bf = pp.bf16 != 0;
    if (p.D == 128) return bf ? launch_kv4_bf16_d128(pp, ng, st) : launch_kv4_f32_d128(pp, ng, st);
    return bf ? launch_kv4_bf16_d64(pp, ng, st) : launch_kv4_f32_d64(pp, ng, st);
}

static bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace art

using namespace art;

extern "C" {

size_t dense_extend_kv4_workspace_bytes(const art_shape* shape, int32_t num_tokens, int32_t group) {
    if (check_cache_shape(shape) != ART_OK || num_tokens < 0 || !kv4_group_ok(shape->head_dim, group)) return 0;
    // a call without offsets, and one with them
    AttendParams p = {}, d = {};
    kv4_shape(p, *shape);
    p.T = num_tokens;
    const size_t with = attend_layout(p, nullptr);
    if (num_tokens != shape->batch) return with;
    kv4_shape(d, *shape);
    d.shared = 1;
    const size_t without = attend_layout(d, nullptr);
    return with == 0 || without == 0 ? 0 : with > without ? with : without;
}

int dense_extend_kv4(const void* q, const void* cache, int32_t group, const int32_t* block_table, const int32_t* seq_lens,
                     const int32_t* q_offsets, int32_t num_tokens, int32_t causal, void* out, const art_shape* shape,
                     void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_cache_shape(shape);
    if (rc != ART_OK) return rc;
    const art_shape& s = *shape;
    if (!cache || !block_table || !seq_lens || !workspace) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (!q || !out)) return ART_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(cache) || misaligned(out) || misaligned(workspace)) return ART_ERR_INVALID_ARG;
    if (num_tokens < 0 || (causal != 0 && causal != 1) || (!q_offsets && num_tokens != s.batch)) return ART_ERR_INVALID_ARG;
    if (!kv4_group_ok(s.head_dim, group)) return ART_ERR_UNSUPPORTED;
    AttendKv4Params pp = {};
    const Kv4Layout l = kv4_layout(s.page_size, s.head_dim, group);
    pp.cache = static_cast<const unsigned char*>(cache);
    pp.slab = l.slab;
    pp.slab_bytes = l.slab_bytes;
    pp.page_bytes = l.page_bytes;
    pp.bf16 = s.dtype == ART_DTYPE_BF16;
    pp.f16_1024 = 0x64006400u;
    AttendParams p = {};
    kv4_shape(p, s);
    p.q = q;
    p.out = out;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    if (q_offsets) {
        p.offsets = q_offsets;
        p.causal = causal;
        p.T = num_tokens;
    } else {
        p.shared = 1;  // one row group a sequence, nothing shared; the one new token sees all keys
    }
    return attend_run(p, s, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), launch_attend_kv4, &pp);
}

}  // extern "C"
