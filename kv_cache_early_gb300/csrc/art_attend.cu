// art_attend.cu -- dense_extend and dense_decode_shared: argument checks and the merge
// kernel (the work and its shares: art_attend.cuh).
#include <cmath>
#include <cstdlib>

#include "art_attend.cuh"

namespace art {

constexpr int kMergeBlock = 256;

// Columns 4 ch .. 4 ch + 3 of a finished row.
template <bool kBF16, int D>
__device__ __forceinline__ void put_row4(const AttendParams& p, size_t row, int ch, const float4& o, float l) {
    const float inv = l > 0.f ? 1.f / l : l;  // no key seen: 0; NaN stays
    if constexpr (kBF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + ch * 4) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * D + ch * 4) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

// One row's pieces joined: a lane holds one piece's (m, l), up to 16 of each of two items
// at a time, then the pieces' columns are read side by side (no load waits for another).
template <bool kBF16, int D>
struct MergeRow {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    int lane;
    int nr, r;  // this half warp's item: its rows, the row's place among them
    // n: the item's pieces; at(k, prow): piece k's first partial row, false where it is empty
    template <class F>
    __device__ __forceinline__ void add(const AttendParams& p, int n, F at) {
        const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 16));
        for (int k0 = 0; k0 < most; k0 += 16) {
            int prow = 0;
            const int k = k0 + (lane & 15);
            const bool some = k < n && at(k, prow);
            const float2 ml = some ? __ldcg(&p.part_ml[prow + r]) : make_float2(-INFINITY, 0.f);
            unsigned todo = __ballot_sync(0xffffffffu, some), saw = 0;
            float w = 0.f;
            bool fresh = true;
            do {
                float4 v[4];
                unsigned use = todo;
#pragma unroll
                for (int u = 0; u < 4; ++u) {  // the first columns come beside the (m, l)
                    const int from = __ffs(todo) - 1;
                    const int pr = __shfl_sync(0xffffffffu, prow, from);
                    const int n1 = __shfl_sync(0xffffffffu, nr, from), r1 = __shfl_sync(0xffffffffu, r, from);
                    if (todo && lane < D / 4)
                        v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (size_t)pr * D) + (size_t)lane * n1 + r1);
                    todo &= todo - 1;
                }
                if (fresh) {
                    fresh = false;
                    const bool live = ml.y != 0.f;  // saw a key (or a NaN)
                    saw = __ballot_sync(0xffffffffu, live);
                    float top = live ? ml.x : -INFINITY;
#pragma unroll
                    for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float mn = fmaxf(m, top);
                    const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
                    w = live ? exp2f(ml.x - mn) : 0.f;
                    float sum = live ? ml.y * w : 0.f;
#pragma unroll
                    for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                    l = l * a + sum;
                    o.x *= a;
                    o.y *= a;
                    o.z *= a;
                    o.w *= a;
                    m = mn;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float f = __shfl_sync(0xffffffffu, w, __ffs(use) - 1);
                    const bool skip = !(use & -use & saw);
                    use &= use - 1;
                    if (skip) continue;
                    o.x += v[u].x * f;
                    o.y += v[u].y * f;
                    o.z += v[u].z * f;
                    o.w += v[u].w * f;
                }
            } while (todo);
        }
    }
    __device__ __forceinline__ void store(const AttendParams& p, size_t row) {
        if (lane < D / 4) put_row4<kBF16, D>(p, row, lane, o, l);
    }
};

// Whether a page of sequence b's own tokens, or of the prefix that group j's first
// sequence (lead) holds, lies outside the pool: only asked when some CTA met such a page.
static __device__ __noinline__ bool seq_bad(const AttendParams& p, int b, int lead, int lane) {
    bool bad = false;
    for (int c = 0; c < p.ctas; ++c) {
        if (!(p.cta_status[c] & ART_STATUS_BAD_PAGE)) continue;
        const int2 r = p.cta_segs[c];
        for (int i = r.x + lane; i < r.y; i += 32) {
            const Seg& s = p.seg[i];
            if (s.nrow > 0 && s.bad) bad |= s.kind == kLimSeq ? s.table_row == lead : s.table_row == b;
        }
    }
    return __any_sync(0xffffffffu, bad);
}

// kMany (dense_decode_shared): more rows than three blocks an SM take at once. Four need 64
// registers, and then a row's first columns wait for its (m, l): 128 x 32 rows 138 us with
// three blocks against 134 with four; 64 x 32 rows 50.7 against 52.8, 89 x 28 rows 91.1
// against 93.5. dense_extend at five blocks: drafts 66.7, encoder 30.5; at three 65.5, 31.3.
template <bool kBF16, int D, bool kShared, bool kMany>
__global__ void __launch_bounds__(kMergeBlock, !kShared ? 5 : kMany ? 4 : 3) art_attend_merge_kernel(const AttendParams p) {
    constexpr int WPB = kMergeBlock / 32;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the first loads all at once
    const int first = kShared ? min(blockIdx.x * WPB + w, p.B * p.Hq - 1) / p.Hq : 0;
    const int j0 = kShared ? p.group_of[first] : -1, lim0 = kShared ? p.row_lim[first] : 0;
    const int quota = p.info->quota, computed = p.info->ok;
    const MergeItem it0 = p.merge[kShared ? 0 : min((int)blockIdx.x, p.ctas - 1)];
    __shared__ int s_status;
    if (tid == 0) s_status = 0;
    const int mine = tid < p.ctas ? p.cta_status[tid] : 0;
    if (__syncthreads_or(mine)) {
        if (mine) atomicOr(&s_status, mine);
        __syncthreads();
    }
    const int status = s_status;
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) p.hdr->status = status;
    if (!computed) return;
    const bool slow = (status & ART_STATUS_BAD_PAGE) != 0;
    if constexpr (kShared) {
        for (int row = blockIdx.x * WPB + w; row < p.B * p.Hq; row += gridDim.x * WPB) {
            const int b = row / p.Hq, h = row - b * p.Hq, g = h / p.G, hg = h - g * p.G;
            const int j = b == first ? j0 : p.group_of[b], lim = b == first ? lim0 : p.row_lim[b];
            MergeRow<kBF16, D> m;
            m.lane = lane;
            const int lead = j >= 0 ? p.offsets[j] : -1;
            if (lim >= 0 && !(slow && seq_bad(p, b, lead, lane))) {
                // the items that hold the row, of its group (lanes 0 to 15) and its own: their
                // pieces by the plan's arithmetic
                const bool own = lane >= 16;
                const EntityPlace q = p.place[!own && lim > 0 ? j : p.NG + b];
                const int R = own ? hg : (b - lead) * p.G + hg, t = R / p.rt;
                const int nrow = min(p.rt, q.nrows - t * p.rt), tiles = tiles_of(p, q.k0, q.k1);
                const int base = item_cost_base(p, nrow), per = item_cost_tile(p, nrow);
                const int x = q.start + g * q.hc + t * (item_cost_base(p, p.rt) + item_cost_tile(p, p.rt) * tiles);
                const int end = x + base + per * tiles, c0 = x / quota;
                const int np = q.nrows != 0 && (own || lim > 0) ? (end - 1) / quota - c0 + 1 : 0;
                m.nr = nrow;
                m.r = R - t * p.rt;
                m.add(p, np, [&](int k, int& prow) {
                    const int c = c0 + k, a = max(c * quota, x), y = min((c + 1) * quota, end);
                    prow = q.prow + g * q.nrows + t * p.rt + c * p.rt;
                    return tiles_before(y - x, base, per, tiles) > tiles_before(a - x, base, per, tiles);
                });
            }
            m.store(p, row);
        }
    } else {
        MergeRow<kBF16, D> z;
        z.lane = lane;
        // the items that go over a border between shares: a thread takes four columns of a row
        __shared__ int s_prow[kAttendCtas];
        for (int c = blockIdx.x; c < p.ctas; c += gridDim.x) {
            const MergeItem it = c == (int)blockIdx.x ? it0 : p.merge[c];
            if (it.np == 0 || (slow && seq_bad(p, it.seq, -1, lane))) continue;
            if (tid < it.np) {  // the pieces' first partial rows, -1 where one is empty
                const int base = item_cost_base(p, it.nrow), per = item_cost_tile(p, it.nrow);
                const int from = tid == 0 ? 0 : tiles_before(it.off + (tid - 1) * quota, base, per, it.tiles);
                const int to = tid == it.np - 1 ? it.tiles : tiles_before(it.off + tid * quota, base, per, it.tiles);
                s_prow[tid] = to > from ? piece_row_extend(it.c0 + tid, tid == 0, p.rt) : -1;
            }
            __syncthreads();
            for (int u = blockIdx.y * kMergeBlock + tid; u < it.nrow * (D / 4); u += gridDim.y * kMergeBlock) {
                const int r = u / (D / 4), ch = u - r * (D / 4);
                float m = -INFINITY, l = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int k = 0; k < it.np; ++k) {
                    const int pr = s_prow[k];
                    if (pr < 0) continue;
                    const float2 e = __ldcg(&p.part_ml[pr + r]);
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + (size_t)pr * D) + ch * it.nrow + r);
                    if (e.y == 0.f) continue;  // saw no key
                    const float mn = fmaxf(m, e.x), a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(e.x - mn);
                    l = l * a + e.y * w;
                    o.x = o.x * a + v.x * w;
                    o.y = o.y * a + v.y * w;
                    o.z = o.z * a + v.z * w;
                    o.w = o.w * a + v.w * w;
                    m = mn;
                }
                const int R = it.r0 + r, t = R / p.G;
                put_row4<kBF16, D>(p, (size_t)(it.tok0 + t) * p.Hq + it.g * p.G + (R - t * p.G), ch, o, l);
            }
            __syncthreads();
        }
        // sequences without keys, and bad ones: zero
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const int lo = p.offsets[b], hi = p.offsets[b + 1];
            if (lo == hi || !(p.place[b].nrows == 0 || (slow && seq_bad(p, b, -1, lane)))) continue;
            for (size_t row = (size_t)lo * p.Hq + blockIdx.y * WPB + w; row < (size_t)hi * p.Hq; row += gridDim.y * WPB)
                z.store(p, row);
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int check_cache_shape(const art_shape* s) {
    if (!s) return ART_ERR_INVALID_ARG;
    if (s->batch < 1 || s->num_q_heads < 1 || s->num_kv_heads < 1 || s->head_dim < 1 || s->page_size < 1 ||
        s->block_size < 1 || s->max_pages_per_seq < 1 || s->num_pages_total < 1)
        return ART_ERR_INVALID_ARG;
    if (s->num_q_heads % s->num_kv_heads != 0) return ART_ERR_INVALID_ARG;
    if (s->dtype != ART_DTYPE_BF16 && s->dtype != ART_DTYPE_F32) return ART_ERR_INVALID_ARG;
    if ((long long)s->batch * s->num_kv_heads > (1LL << 30)) return ART_ERR_UNSUPPORTED;
    const int G = s->num_q_heads / s->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 7 && G != 8) return ART_ERR_UNSUPPORTED;
    if (s->head_dim != 64 && s->head_dim != 128) return ART_ERR_UNSUPPORTED;
    if (s->block_size != kBK) return ART_ERR_UNSUPPORTED;
    if ((s->page_size & (s->page_size - 1)) != 0 || s->page_size < 8 || s->page_size > 4096) return ART_ERR_UNSUPPORTED;
    return ART_OK;
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t attend_layout(AttendParams& p, unsigned char* base) {
    p.G = p.Hq / p.Hkv;
    p.NE = p.shared ? p.NG + p.B : p.B;
    const long long rows = (long long)(p.shared ? p.B : p.T) * p.G;  // of one KV head
    // items and partial rows at most
    long long items = (rows / p.rt + (p.shared ? p.NG : p.B)) * p.Hkv;
    if (p.shared) items += (long long)p.B * p.Hkv;
    const long long prows =
        p.shared ? 2 * rows * p.Hkv + (long long)(kAttendCtas + 1) * p.rt : 2LL * kAttendCtas * p.rt;
    // 32-bit row and key counts in the work list
    if (rows > (1LL << 30) || items > (1LL << 28) || prows > (1LL << 30) || p.NG > kMaxGroups ||
        (long long)p.max_pages * p.Ps > (1LL << 30))
        return 0;
    // cost units fit 31 bits, with room for sums of one share beyond the end
    const long long tiles = (((long long)p.max_pages * p.Ps) >> p.kt_log2) + 1;
    const long long per = p.cost.two_tile > p.cost.small_tile ? p.cost.two_tile : p.cost.small_tile;
    if (items * (per * tiles + p.cost.two_item) > (1LL << 30)) p.cost = {0, 1, 0, 1, 0, 1};
    if (items * tiles > (1LL << 30)) return 0;
    size_t o = sizeof(WsHeader);
    auto take = [&](size_t bytes) {
        const size_t at = up256(o);
        o = at + bytes;
        return base ? base + at : nullptr;
    };
    p.hdr = reinterpret_cast<WsHeader*>(base);
    p.info = reinterpret_cast<PlanInfo*>(take(sizeof(PlanInfo)));
    p.place = reinterpret_cast<EntityPlace*>(take(sizeof(EntityPlace) * (size_t)p.NE));
    p.row_lim = reinterpret_cast<int*>(take(sizeof(int) * (size_t)p.B));
    p.group_of = reinterpret_cast<int*>(take(sizeof(int) * (size_t)p.B));
    p.cta_status = reinterpret_cast<int*>(take(sizeof(int) * kAttendCtas));
    p.cta_segs = reinterpret_cast<int2*>(take(sizeof(int2) * kAttendCtas));
    p.merge = reinterpret_cast<MergeItem*>(take(sizeof(MergeItem) * kAttendCtas));
    p.seg = reinterpret_cast<Seg*>(take(sizeof(Seg) * ((size_t)items + kAttendCtas)));
    p.part_ml = reinterpret_cast<float2*>(take(sizeof(float2) * (size_t)prows));
    p.part_o = reinterpret_cast<float*>(take(sizeof(float) * (size_t)prows * p.D));
    return up256(o);
}

// Cost units (about 0.15 us): what segments and key tiles of each kind take beside their
// neighbours, fitted to the CTAs' timelines at head_dim 128. They set the shares only. Tiles
// alone at one cost: chunks of 1-2k tokens 527 us against 362, 128 sequences behind a
// document 159 against 134, 64 behind a prompt 61 against 52. At head_dim 64, where a tile has half the
// bytes and products, the same numbers hold: with tiles at {4, 7, 9} instead of {7, 11, 13}
// chunks 299 us against 297, a document 125 against 116, a mixed batch 62.2 against 60.8; with
// items at {9, 20, 30} instead of {13, 35, 50} chunks 315, a document 117, mixed 60.7.
constexpr CostRule kCostBf16 = {13, 7, 35, 11, 50, 13}, kCostF32 = {10, 8, 10, 16, 10, 16};

void attend_shape(AttendParams& p, const art_shape& s) {
    p.B = s.batch;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.D = s.head_dim;
    const int G = s.num_q_heads / s.num_kv_heads;
    p.g_mul = ((1ull << 34) + G - 1) / G;
    p.Ps = s.page_size;
    p.max_pages = s.max_pages_per_seq;
    p.num_pages = s.num_pages_total;
    p.rt = s.dtype == ART_DTYPE_BF16 ? kRowsTc : kItemRows;
    p.kt_log2 = s.dtype == ART_DTYPE_BF16 ? 7 : 6;
    p.small_rows = s.dtype == ART_DTYPE_BF16 ? kSmallRows : kSmallRowsF32;
    static_assert(kKeyTile == 1 << 7 && kKeyTileF32 == 1 << 6, "tiles");
    p.cost = s.dtype == ART_DTYPE_BF16 ? kCostBf16 : kCostF32;
    p.scale_log2 = (float)(1.4426950408889634074 / std::sqrt((double)s.head_dim));
}

int attend_run(AttendParams& p, const art_shape& s, void* workspace, size_t workspace_bytes, cudaStream_t st,
               AttendLaunch launch, const void* more) {
    const size_t need = attend_layout(p, nullptr);
    if (need == 0) return ART_ERR_UNSUPPORTED;
    if (workspace_bytes < need) return ART_ERR_WORKSPACE;
    attend_layout(p, static_cast<unsigned char*>(workspace));
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e);
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return cuda_fail(e);
    p.ctas = sms < kAttendCtas ? sms : kAttendCtas;
    // the failure-path test hook of art_decode (ART_TEST_STALL_NS)
    p.wait_ns = kWaitLimitNs;
    p.stall = 0;
    if (const char* es = std::getenv("ART_TEST_STALL_NS")) {
        const long long ns = std::atoll(es);
        if (ns > 0) {
            p.stall = 1;
            p.wait_ns = (unsigned long long)(ns < (long long)kWaitLimitNs ? ns : (long long)kWaitLimitNs);
        }
    }
    const bool bf = s.dtype == ART_DTYPE_BF16;
    if (launch) e = launch(p, more, st);
    else e = bf ? launch_attend_tc(p, st) : launch_attend_simt(p, st);
    if (e != cudaSuccess) return cuda_fail(e);
    // the merge kernel's launch overlaps the main kernel's end
    const long long blocks = p.shared ? ((long long)p.B * p.Hq + kMergeBlock / 32 - 1) / (kMergeBlock / 32) : p.ctas;
    const dim3 grid((unsigned)(blocks < 8LL * p.ctas ? blocks : 8LL * p.ctas), p.shared ? 1 : p.rt / 16);
    const bool many = blocks > 3LL * p.ctas;
#define ART_MERGE(BF, DD)                                                                                              \
    e = !p.shared ? launch_after(art_attend_merge_kernel<BF, DD, false, false>, grid, dim3(kMergeBlock), 0, st, p)    \
        : many    ? launch_after(art_attend_merge_kernel<BF, DD, true, true>, grid, dim3(kMergeBlock), 0, st, p)      \
                  : launch_after(art_attend_merge_kernel<BF, DD, true, false>, grid, dim3(kMergeBlock), 0, st, p)
    if (bf && p.D == 128) ART_MERGE(true, 128);
    else if (bf) ART_MERGE(true, 64);
    else if (p.D == 128) ART_MERGE(false, 128);
    else ART_MERGE(false, 64);
#undef ART_MERGE
    if (e != cudaSuccess) return cuda_fail(e);
    return ART_OK;
}

static bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace art

using namespace art;

extern "C" {

size_t dense_extend_workspace_bytes(const art_shape* shape, int32_t num_tokens) {
    if (check_cache_shape(shape) != ART_OK || num_tokens < 0) return 0;
    AttendParams p = {};
    attend_shape(p, *shape);
    p.T = num_tokens;
    return attend_layout(p, nullptr);
}

int dense_extend(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                 const int32_t* seq_lens, const int32_t* q_offsets, int32_t num_tokens, int32_t causal, void* out,
                 const art_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_cache_shape(shape);
    if (rc != ART_OK) return rc;
    if (!k_cache || !v_cache || !block_table || !seq_lens || !q_offsets || !workspace) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (!q || !out)) return ART_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out) || misaligned(workspace))
        return ART_ERR_INVALID_ARG;
    if (num_tokens < 0 || (causal != 0 && causal != 1)) return ART_ERR_INVALID_ARG;
    AttendParams p = {};
    attend_shape(p, *shape);
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    p.out = out;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.offsets = q_offsets;
    p.causal = causal;
    p.T = num_tokens;
    return attend_run(p, *shape, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

size_t dense_decode_shared_workspace_bytes(const art_shape* shape, int32_t num_groups) {
    if (check_cache_shape(shape) != ART_OK || num_groups < 0) return 0;
    AttendParams p = {};
    attend_shape(p, *shape);
    p.shared = 1;
    p.NG = num_groups;
    return attend_layout(p, nullptr);
}

int dense_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                        const int32_t* seq_lens, const int32_t* group_offsets, const int32_t* prefix_lens,
                        int32_t num_groups, void* out, const art_shape* shape, void* workspace,
                        size_t workspace_bytes, void* stream) {
    const int rc = check_cache_shape(shape);
    if (rc != ART_OK) return rc;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace) return ART_ERR_INVALID_ARG;
    if (num_groups < 0 || (num_groups > 0 && (!group_offsets || !prefix_lens))) return ART_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out) || misaligned(workspace))
        return ART_ERR_INVALID_ARG;
    AttendParams p = {};
    attend_shape(p, *shape);
    p.shared = 1;
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    p.out = out;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.offsets = group_offsets;
    p.prefix = prefix_lens;
    p.NG = num_groups;
    return attend_run(p, *shape, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
