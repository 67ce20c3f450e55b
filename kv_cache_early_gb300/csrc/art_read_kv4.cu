// art_read_kv4.cu -- reading a cache that is held in 4 bits back into rows or into the pages of a
// plain cache: a column's value is lowest + step * code, formed by one fused product in fp32 and
// rounded once more to bf16 there.
//
// Bound: HBM, d / 2 + 4 d / group bytes of a key or value head in and 2 d (bf16) out a token. The
// work is the 8-token units of the places read, sequence by sequence, cut into equal runs, one for
// each CTA, which finds its run by a sum over the sequences. A warp takes a unit of a head: a
// lane has 8 columns of one token, so a load is 128 bytes of codes and a store eight runs of 64 bytes.
// One more CTA (block 0) checks the call's device data and stores the status word; the others
// check what they use by themselves.
#include "art_common.cuh"
#include "art_kv4.cuh"

namespace art {

constexpr int kReadThreads = 256;
constexpr int kReadCtas = 4;  // an SM; 139k tokens into pages: 2, 3, 4, 6, 8 of them 107, 92, 91, 101, 89 us, small reads 4.4 .. 5.2 from 4 to 8

struct ReadKv4Params {
    const unsigned char* cache;
    const int32_t *block_table, *seq_lens;
    const int32_t* q_offsets;  // null: every token, or (one) the last one of each sequence
    const int32_t* out_table;  // null: rows
    // a pool with max_pages pages for each sequence, and its block table, which is written, -1 for bad pages; the
    // sequences with new tokens by q_offsets only
    int32_t* map;
    void *k_out, *v_out;
    WsHeader* hdr;
    int B, T, Hkv, Ps, max_pages, num_pages, out_pages;
    int slab, slab_log2, page_log2, slab_bytes, page_bytes;
};

// Sequence b: its places [lo, hi) to read; false where its offsets or its length are bad.
__device__ __forceinline__ bool read_span(const ReadKv4Params& p, int b, int& lo, int& hi, int& row0, int& err) {
    const int len = p.seq_lens[b];
    lo = hi = row0 = 0;
    int n = len;
    if (p.map) {
        if (p.q_offsets[b] == p.q_offsets[b + 1]) return false;
    } else if (!p.out_table) {
        const int a = p.q_offsets ? p.q_offsets[b] : b, z = p.q_offsets ? p.q_offsets[b + 1] : b + 1;
        if (a < 0 || z < a || z > p.T) {
            err |= ART_STATUS_BAD_OFFSETS;
            return false;
        }
        row0 = a;
        n = z - a;
    }
    if (len < 0 || len < n || (long long)len > (long long)p.max_pages * p.Ps) {
        err |= ART_STATUS_BAD_SEQLEN;
        // its rows are zero
        hi = p.out_table || p.map ? 0 : n;
        return false;
    }
    lo = len - n;
    hi = len;
    return true;
}

__device__ void read_check(const ReadKv4Params& p) {
    __shared__ int s_err;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s_err = 0;
    __syncthreads();
    int err = 0;
    for (int b0 = 0; b0 < p.B; b0 += kReadThreads) {
        const int b = b0 + tid;
        int lo = 0, hi = 0, row0, first = 0, np = 0;
        if (b < p.B && read_span(p, b, lo, hi, row0, err) && hi > lo) {
            first = lo / p.Ps;
            np = (hi - 1) / p.Ps - first + 1;
        }
        auto check = [&](int row, int col) {
            const size_t at = (size_t)row * p.max_pages + col;
            const int pg = p.block_table[at];
            if (pg < 0 || pg >= p.num_pages) err |= ART_STATUS_BAD_PAGE;
            if (p.out_table) {
                const int to = p.out_table[at];
                if (to < 0 || to >= p.out_pages) err |= ART_STATUS_BAD_PAGE;
            }
        };
        const bool few = np <= 4;
        if (few)
            for (int k = 0; k < np; ++k) check(b, first + k);
        unsigned many = __ballot_sync(0xffffffffu, !few);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            const int f = __shfl_sync(0xffffffffu, first, src), n = __shfl_sync(0xffffffffu, np, src);
            for (int k = lane; k < n; k += 32) check(b0 + (tid & ~31) + src, f + k);
        }
    }
    if (err) atomicOr(&s_err, err);
    __syncthreads();
    if (tid == 0) p.hdr->status = s_err;
}

struct ReadRun {  // units [u0, u1) of a sequence, counted from its first
    int b, lo, hi, row0, u0, u1, ok;
};

// A unit of a head: 8 tokens at places 8 * oct .. of sequence r.b.
template <bool kBF16, int D, int NG>
__device__ __forceinline__ void read_unit(const ReadKv4Params& p, const ReadRun& r, int oct, int g, int lane) {
    constexpr int NC = D / 32, ROWB = D * (kBF16 ? 2 : 4);
    const int i = lane >> 2, w = lane & 3, place = oct * 8 + i;
    const int in_page = place & (p.Ps - 1);
    const size_t at = (size_t)r.b * p.max_pages + (place >> p.page_log2);
    const bool here = place >= r.lo && place < r.hi;
    const int page = r.ok && here ? p.block_table[at] : -1;
    const bool good = page >= 0 && page < p.num_pages;
    size_t row = 0;
    bool to = here;
    if (p.map) {
        row = (at * p.Hkv + g) * p.Ps + in_page;
        to = good;
        if (here && g == 0 && w == 0) p.map[at] = good ? (int)at : -1;
    } else if (p.out_table) {
        const int o = here ? p.out_table[at] : -1;
        to = o >= 0 && o < p.out_pages;
        row = ((size_t)(to ? o : 0) * p.Hkv + g) * p.Ps + in_page;
    } else {
        row = (size_t)(r.row0 + place - r.lo) * p.Hkv + g;
    }
    const unsigned char* slab = p.cache + ((size_t)(good ? page : 0) * p.Hkv + g) * (size_t)p.page_bytes +
                                (size_t)(in_page >> p.slab_log2) * p.slab_bytes;
    const int u = in_page & (p.slab - 1);
    uint32_t code[2][NC], scale[2][NG];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            code[kv][c] = good ? __ldg(reinterpret_cast<const uint32_t*>(slab + kv * p.slab * (D / 2) + kv4_code_at<D>(u, c) + w * 4)) : 0u;
#pragma unroll
        for (int n = 0; n < NG; ++n)
            scale[kv][n] = good ? __ldg(reinterpret_cast<const uint32_t*>(slab + p.slab * (D + kv * 4 * NG) + kv4_scale_at<NG>(u, n))) : 0u;
    }
    if (!to) return;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        char* dst = static_cast<char*>(kv ? p.v_out : p.k_out) + row * ROWB;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint32_t s = scale[kv][c * NG / NC];
            const float step = bf16_lo_f(s), low = bf16_hi_f(s);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // a code as the last bits of 2^23 + code: no conversion
                const float f = __uint_as_float(0x4b000000u | ((code[kv][c] >> (4 * e)) & 15u)) - 8388608.f;
                x[e] = fmaf(step, f, low);
            }
            if constexpr (kBF16) {
                *reinterpret_cast<uint4*>(dst + c * 64 + w * 16) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                                             pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            } else {
                float4* o = reinterpret_cast<float4*>(dst + c * 128 + w * 32);
                o[0] = make_float4(x[0], x[1], x[2], x[3]);
                o[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

template <bool kBF16, int D, int NG>
__global__ void __launch_bounds__(kReadThreads) art_read_kv4_kernel(const ReadKv4Params p) {
    if (blockIdx.x == 0) {
        if (!p.map) read_check(p);
        return;
    }
    constexpr int WARPS = kReadThreads / 32;
    __shared__ int s_sum[WARPS], s_n;
    __shared__ ReadRun s_run[kReadThreads];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int ctas = gridDim.x - 1, c = blockIdx.x - 1;
    const int rounds = (p.B + kReadThreads - 1) / kReadThreads;
    // a first sweep for the whole work where one round does not hold it
    long long total = 0, start = 0, lo_u = 0, hi_u = 0;
    bool bad = false;
    for (int k = rounds == 1 ? rounds : 0; k < 2 * rounds; ++k) {
        const int b = (k % rounds) * kReadThreads + tid;
        ReadRun r;
        int err = 0, units = 0;
        r.ok = 0;
        if (b < p.B) {
            r.b = b;
            r.ok = read_span(p, b, r.lo, r.hi, r.row0, err);
            units = r.hi > r.lo ? (r.hi + 7) / 8 - r.lo / 8 : 0;
        }
        bad |= __syncthreads_or(err & ART_STATUS_BAD_OFFSETS) != 0;
        int z = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += y;
        }
        if (lane == 31) s_sum[w] = z;
        if (tid == 0) s_n = 0;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            if (i < w) before += s_sum[i];
            all += s_sum[i];
        }
        if (k < rounds || rounds == 1) total += all;
        if (k >= rounds) {
            if (k == rounds) {
                if (bad) return;
                const long long quota = (total + ctas - 1) / ctas;
                lo_u = quota * c;
                hi_u = lo_u + quota;
            }
            const long long first = start + before + z - units;
            if (units > 0 && first < hi_u && first + units > lo_u) {
                r.u0 = (int)max(lo_u - first, 0LL);
                r.u1 = (int)min(hi_u - first, (long long)units);
                s_run[atomicAdd(&s_n, 1)] = r;
            }
            start += all;
            __syncthreads();
            const int n = s_n;
            for (int i = 0; i < n; ++i) {
                const ReadRun q = s_run[i];
                for (int x = w; x < (q.u1 - q.u0) * p.Hkv; x += WARPS) {
                    // heads of an 8-token unit one after the other: rows of a token side by side
                    const int o = x / p.Hkv;
                    read_unit<kBF16, D, NG>(p, q, q.lo / 8 + q.u0 + o, x - o * p.Hkv, lane);
                }
            }
        }
        __syncthreads();
    }
}

static void launch_read_kv4(const ReadKv4Params& p, const art_shape& s, int group, unsigned grid, cudaStream_t st) {
    const int ng = s.head_dim / group;
    const bool bf = s.dtype == ART_DTYPE_BF16;
#define ART_READ4(DD, NN)                                                              \
    (bf ? art_read_kv4_kernel<true, DD, NN><<<grid, kReadThreads, 0, st>>>(p)          \
        : art_read_kv4_kernel<false, DD, NN><<<grid, kReadThreads, 0, st>>>(p))
    if (s.head_dim == 128) {
        if (ng == 1) ART_READ4(128, 1);
        else if (ng == 2) ART_READ4(128, 2);
        else ART_READ4(128, 4);
    } else {
        if (ng == 1) ART_READ4(64, 1);
        else ART_READ4(64, 2);
    }
#undef ART_READ4
}

static void read_params(ReadKv4Params& p, const art_shape& s, int group) {
    p.B = s.batch;
    p.Hkv = s.num_kv_heads;
    p.Ps = s.page_size;
    p.max_pages = s.max_pages_per_seq;
    p.num_pages = s.num_pages_total;
    const Kv4Layout l = kv4_layout(s.page_size, s.head_dim, group);
    p.slab = l.slab;
    p.slab_log2 = l.slab_log2;
    p.page_log2 = 0;
    while (1 << p.page_log2 < s.page_size) ++p.page_log2;
    p.slab_bytes = l.slab_bytes;
    p.page_bytes = l.page_bytes;
}

cudaError_t read_kv4_pool(const art_shape& s, int group, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* q_offsets, int32_t* map, void* k_out, void* v_out, int sms, cudaStream_t st) {
    ReadKv4Params p = {};
    read_params(p, s, group);
    p.cache = static_cast<const unsigned char*>(cache);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.q_offsets = q_offsets;
    p.map = map;
    p.k_out = k_out;
    p.v_out = v_out;
    launch_read_kv4(p, s, group, (unsigned)(kReadCtas * sms) + 1u, st);
    return cudaGetLastError();
}

int check_cache_shape(const art_shape* s);  // art_attend.cu

}  // namespace art

using namespace art;

extern "C" {

size_t art_read_kv4_workspace_bytes(const art_shape* shape) { return shape ? sizeof(WsHeader) : 0; }

int art_read_kv4(const void* cache, int32_t group, const int32_t* block_table, const int32_t* seq_lens,
                 const int32_t* q_offsets, int32_t num_tokens, const int32_t* out_table, int32_t out_pages, void* k_out,
                 void* v_out, const art_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_cache_shape(shape);
    if (rc != ART_OK) return rc;
    const art_shape& s = *shape;
    if (!cache || !block_table || !seq_lens || !workspace) return ART_ERR_INVALID_ARG;
    if (out_table ? (q_offsets || num_tokens != 0 || out_pages < 1) : (out_pages != 0 || num_tokens < 0)) return ART_ERR_INVALID_ARG;
    if (!out_table && !q_offsets && num_tokens != s.batch) return ART_ERR_INVALID_ARG;
    if ((out_table || num_tokens != 0) && (!k_out || !v_out)) return ART_ERR_INVALID_ARG;
    auto bad = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) != 0; };
    if (bad(cache) || bad(k_out) || bad(v_out) || bad(workspace)) return ART_ERR_INVALID_ARG;
    if (!kv4_group_ok(s.head_dim, group)) return ART_ERR_UNSUPPORTED;
    // counts of 8-token units have 32 bits, and so do a CTA's units times heads
    const long long row = (long long)s.max_pages_per_seq * s.page_size;
    if (row > (1LL << 30) || (out_table && s.batch * row > (1LL << 33))) return ART_ERR_UNSUPPORTED;
    if ((out_table ? s.batch * row : (long long)num_tokens) > (1LL << 40) / s.num_kv_heads) return ART_ERR_UNSUPPORTED;
    if (workspace_bytes < sizeof(WsHeader)) return ART_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e);
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return cuda_fail(e);
    ReadKv4Params p = {};
    read_params(p, s, group);
    p.cache = static_cast<const unsigned char*>(cache);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.q_offsets = q_offsets;
    p.out_table = out_table;
    p.out_pages = out_pages;
    p.k_out = k_out;
    p.v_out = v_out;
    p.hdr = static_cast<WsHeader*>(workspace);
    p.T = num_tokens;
    // no more CTAs than there may be units of rows
    long long ctas = (long long)kReadCtas * sms;
    if (!out_table) {
        const long long units = (long long)num_tokens / 8 + 2LL * (num_tokens < s.batch ? num_tokens : s.batch);
        if (units < ctas) ctas = units > 0 ? units : 1;
    }
    const unsigned grid = (unsigned)ctas + 1u;
    launch_read_kv4(p, s, group, grid, static_cast<cudaStream_t>(stream));
    e = cudaGetLastError();
    return e == cudaSuccess ? ART_OK : cuda_fail(e);
}

}  // extern "C"
