// art_attend_kv4.cu -- dense_extend_kv4: argument checks and the choice of the kernels.
//
// Two paths. Path 0 attends over the codes (art_attend_kv4.cuh): 16 rows of queries at a time, bound by the
// cache's bytes for few rows and by the taking apart of codes and the small products for many. Path 1, for prompt chunks
// in bf16, reads the cache back to bf16 in the workspace and calls the tensor-memory kernel of dense_extend
// on it, whose products are several times faster.
#include <cmath>

#include "art_attend_kv4.cuh"

namespace art {

// Cost units of items and of their tiles of 128 keys, by rows (8, more). Five drafts of 16 sequences (20 rows of 4 heads,
// 16 and 4): tiles of 16 rows at 5, 6, 8, 10, 14 units 71.2, 68.0, 65.4, 68.0, 71.7 us (items at 20); at 8 and 10 units with
// items at 32 65.8 and 67.7; items at 20 67.6, at 44 68.2. 64 decoding sequences: items at 13, 17, 21 units 66.0, 65.8, 66.4 us.
constexpr CostRule kCostKv4 = {17, 5, 32, 8, 32, 8};

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
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of a key head and sequence, in the mean, and rows of all heads together, from which the cache is read back.
// Measured, codes against read back (us; 32/8 heads, d 128, context 2048, 8 sequences): 64 rows 48 / 50, 96 rows
// 62 / 54, 256 rows 127 / 69; context 4096, 32 sequences: 64 rows 217 / 239, 96 rows 313 / 243. One sequence of
// 8192 tokens leaves most SMs idle on path 1's large tiles: 192 rows (1536 in all) 57 / 74, 256 (2048) 69 / 73,
// 384 92 / 62. 8/8 heads, d 64, 8 sequences of 8192: 64 rows 69 / 86, 96 rows 97 / 87.
constexpr int kReadBackRows = 96, kReadBackAll = 2048;
constexpr size_t kReadBackMost = 4ull << 30;  // bytes of a pool at most

// What a call needs of the workspace, by its path. Path 1: dense_extend's part, the pool's block table, the pool.
struct Kv4Workspace {
    size_t codes;  // path 0; 0 where its sizes are not supported
    size_t least;  // of a call with so many tokens or fewer, those without offsets (a token a sequence) among them
    size_t table, pool, whole;  // path 1: offsets of the last two and the bytes, whole 0 where it is not offered
};
static Kv4Workspace kv4_workspace(const art_shape& s, int num_tokens, bool offsets) {
    Kv4Workspace w = {};
    AttendParams p = {};
    kv4_shape(p, s);
    p.T = num_tokens;
    p.shared = !offsets;
    w.codes = w.least = attend_layout(p, nullptr);
    if (offsets && w.codes != 0 && num_tokens >= s.batch) {
        const size_t step = kv4_workspace(s, s.batch, false).codes;  // 0 where it is not supported
        if (step > w.least) w.least = step;
    }
    const int G = s.num_q_heads / s.num_kv_heads;
    if (!offsets || s.dtype != ART_DTYPE_BF16 || (long long)num_tokens * G < (long long)kReadBackRows * s.batch ||
        (long long)num_tokens * s.num_q_heads < kReadBackAll)
        return w;
    const unsigned long long pages = (unsigned long long)s.batch * s.max_pages_per_seq;
    const unsigned long long page = 2ull * s.num_kv_heads * s.page_size * s.head_dim;  // of keys, or values
    if (pages > 0x7fffffffull || pages * page > kReadBackMost / 2) return w;
    AttendParams t = {};
    attend_shape(t, s);
    t.T = num_tokens;
    const size_t need = attend_layout(t, nullptr);
    if (need == 0) return w;
    w.table = up256(need > w.least ? need : w.least);  // so that the least workspace never holds path 1
    w.pool = up256(w.table + pages * sizeof(int32_t));
    w.whole = w.pool + 2 * pages * page;
    return w;
}

}  // namespace art

using namespace art;

extern "C" {

static size_t kv4_bytes(const art_shape* shape, int32_t num_tokens, int32_t group, bool least) {
    if (check_cache_shape(shape) != ART_OK || num_tokens < 0 || !kv4_group_ok(shape->head_dim, group)) return 0;
    const Kv4Workspace w = kv4_workspace(*shape, num_tokens, true);
    return !least && w.whole != 0 ? w.whole : w.least;
}

size_t dense_extend_kv4_workspace_bytes(const art_shape* shape, int32_t num_tokens, int32_t group) {
    return kv4_bytes(shape, num_tokens, group, false);
}

size_t dense_extend_kv4_min_workspace_bytes(const art_shape* shape, int32_t num_tokens, int32_t group) {
    return kv4_bytes(shape, num_tokens, group, true);
}

int dense_extend_kv4_path(const art_shape* shape, int32_t num_tokens, int32_t group, size_t workspace_bytes) {
    if (check_cache_shape(shape) != ART_OK || num_tokens < 0 || !kv4_group_ok(shape->head_dim, group)) return 0;
    const Kv4Workspace w = kv4_workspace(*shape, num_tokens, true);
    return w.whole != 0 && workspace_bytes >= w.whole;
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
    const Kv4Workspace w = kv4_workspace(s, num_tokens, q_offsets != nullptr);
    if (w.codes == 0) return ART_ERR_UNSUPPORTED;
    if (workspace_bytes < w.codes) return ART_ERR_WORKSPACE;
    AttendParams p = {};
    if (w.whole != 0 && workspace_bytes >= w.whole) {
        int dev = 0, sms = 0;
        cudaError_t e;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e);
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return cuda_fail(e);
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        int32_t* map = reinterpret_cast<int32_t*>(ws + w.table);
        unsigned char *k = ws + w.pool, *v = k + (w.whole - w.pool) / 2;
        e = read_kv4_pool(s, group, cache, block_table, seq_lens, q_offsets, map, k, v, sms, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_fail(e);
        art_shape plain = s;
        plain.num_pages_total = s.batch * s.max_pages_per_seq;
        attend_shape(p, plain);
        p.num_pages = plain.num_pages_total;
        p.k = k;
        p.v = v;
        p.q = q;
        p.out = out;
        p.block_table = map;
        p.seq_lens = seq_lens;
        p.offsets = q_offsets;
        p.causal = causal;
        p.T = num_tokens;
        return attend_run(p, plain, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    }
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
