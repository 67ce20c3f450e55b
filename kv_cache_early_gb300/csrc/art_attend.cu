// art_attend.cu -- dense_extend and dense_decode_shared: argument checks, the plan
// kernel that builds the work list (art_attend.cuh), and the merge kernel.
#include <cmath>
#include <cstdlib>

#include "art_attend.cuh"

namespace art {

int check_shape(const art_shape* s);  // art_api.cu

constexpr int kPlanBlock = 512;
constexpr int kMergeBlock = 256;
constexpr int kEntSmem = 2048;  // entities whose first items are searched in shared memory

// Inclusive sums over the block; returns the exclusive one, `total` the block's.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    if (w == 0) {
        long long t = lane < kPlanBlock / 32 ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        if (lane < kPlanBlock / 32) s_warp[lane] = t;
    }
    __syncthreads();
    total = s_warp[kPlanBlock / 32 - 1];
    const long long before = w > 0 ? s_warp[w - 1] : 0;
    __syncthreads();
    return before + x - v;
}

// Another CTA's entity: read past the L1.
__device__ __forceinline__ Entity load_entity(const Entity* e) {
    const int4 a = __ldcg(reinterpret_cast<const int4*>(e)), b = __ldcg(reinterpret_cast<const int4*>(e) + 1);
    Entity r;
    r.table_row = a.x;
    r.tok0 = a.y;
    r.nrows = a.z;
    r.k0 = a.w;
    r.k1 = b.x;
    r.lim0 = b.y;
    r.kind = b.z;
    r.bad = b.w;
    return r;
}

struct Item {
    int e, g, rt;   // entity, KV head, row tile
    int r0, nrow;
    int k0, k1;     // keys of the tile's last row
    int t0, tiles;  // first key tile, number of key tiles
};

__device__ __forceinline__ Item item_of(const AttendParams& p, const int* item0, int i) {
    int lo = 0, hi = p.NE - 1;  // the last entity with item0 <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (item0[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    const Entity en = load_entity(&p.ent[lo]);
    Item it;
    it.e = lo;
    const int nrt = (en.nrows + p.rt - 1) / p.rt, j = i - item0[lo];
    it.g = j / nrt;
    it.rt = j - it.g * nrt;
    it.r0 = it.rt * p.rt;
    it.nrow = min(p.rt, en.nrows - it.r0);
    it.k0 = en.k0;
    it.k1 = en.k1;
    if (en.kind == kLimCausal && !en.bad) it.k1 = en.lim0 + (it.r0 + it.nrow - 1) / p.G;
    it.t0 = it.k0 / kKeyTile;
    it.tiles = it.k1 > it.k0 ? (it.k1 + kKeyTile - 1) / kKeyTile - it.t0 : 0;
    return it;
}

// Whether the block-table entries [c0, c1) of a row all lie in the pool (block-wide).
__device__ __forceinline__ bool pages_bad(const AttendParams& p, int row, int c0, int c1) {
    int bad = 0;
    const int32_t* t = p.block_table + (size_t)row * p.max_pages;
    for (int c = c0 + (int)threadIdx.x; c < c1; c += kPlanBlock) {
        const int pg = t[c];
        bad |= pg < 0 || pg >= p.num_pages;
    }
    return __syncthreads_or(bad) != 0;
}

__device__ __forceinline__ int pages_of(int tokens, int Ps) { return (tokens + Ps - 1) / Ps; }

// dense_extend, CTA b: sequence b's rows, keys and checks.
__device__ void plan_extend(const AttendParams& p, int b, int& err) {
    const int lo = p.offsets[b], hi = p.offsets[b + 1], len = p.seq_lens[b];
    const bool off_ok = lo >= 0 && hi >= lo && hi <= p.T;
    const int n = off_ok ? hi - lo : 0;
    bool ok = len >= 0 && (long long)len <= (long long)p.max_pages * p.Ps && (!p.causal || len >= n);
    if (!ok && off_ok) err |= ART_STATUS_BAD_SEQLEN;
    if (ok && n > 0 && pages_bad(p, b, 0, pages_of(len, p.Ps))) {
        err |= ART_STATUS_BAD_PAGE;
        ok = false;
    }
    if (threadIdx.x == 0) {
        Entity e;
        e.table_row = b;
        e.tok0 = lo;
        e.nrows = n * p.G;
        e.k0 = 0;
        e.k1 = ok ? len : 0;
        e.lim0 = len - n + 1;
        e.kind = p.causal ? kLimCausal : kLimAll;
        e.bad = !ok;
        p.ent[b] = e;
    }
}

// dense_decode_shared, CTA j < NG: group j's prefix.
__device__ void plan_group(const AttendParams& p, int j, int& err) {
    __shared__ int s_top;
    const int lo = p.offsets[j], hi = p.offsets[j + 1], pre = p.prefix[j];
    const long long cap = (long long)p.max_pages * p.Ps;
    const bool off_ok = lo >= 0 && hi >= lo && hi <= p.B;
    bool ok = pre >= 0 && pre <= cap;
    if (threadIdx.x == 0) s_top = 0;
    __syncthreads();
    int top = 0;  // keys that the farthest member sees of the prefix
    if (off_ok && ok)
        for (int b = lo + (int)threadIdx.x; b < hi; b += kPlanBlock) {
            const int len = p.seq_lens[b];
            if (len >= 0 && len <= cap) top = max(top, min(len, pre));
        }
    if (top) atomicMax(&s_top, top);
    __syncthreads();
    top = s_top;
    if (off_ok && hi > lo) {
        if (!ok) err |= ART_STATUS_BAD_SEQLEN;
        else if (pages_bad(p, lo, 0, pages_of(top, p.Ps))) {
            err |= ART_STATUS_BAD_PAGE;
            ok = false;
        }
    }
    if (threadIdx.x == 0) {
        Entity e;
        e.table_row = lo;
        e.tok0 = lo;
        e.nrows = off_ok && ok && top > 0 ? (hi - lo) * p.G : 0;
        e.k0 = 0;
        e.k1 = top;
        e.lim0 = 0;
        e.kind = kLimSeq;
        e.bad = !ok;
        p.ent[j] = e;
    }
}

// dense_decode_shared, CTA NG + b: sequence b's own tokens.
__device__ void plan_own(const AttendParams& p, int b, int& err) {
    int cnt = 0;  // group offsets at or below b
    for (int i0 = 0; i0 <= p.NG; i0 += kPlanBlock) {
        const int i = i0 + (int)threadIdx.x;
        cnt += __syncthreads_count(i <= p.NG && p.NG > 0 && p.offsets[i] <= b);
    }
    const int j = cnt >= 1 && cnt <= p.NG ? cnt - 1 : -1;
    const int len = p.seq_lens[b];
    bool ok = len >= 0 && (long long)len <= (long long)p.max_pages * p.Ps;
    if (!ok) err |= ART_STATUS_BAD_SEQLEN;
    const int pre = ok && j >= 0 ? max(0, min(len, p.prefix[j])) : 0;
    if (ok && pages_bad(p, b, pre / p.Ps, len > pre ? pages_of(len, p.Ps) : 0)) {
        err |= ART_STATUS_BAD_PAGE;
        ok = false;
    }
    if (threadIdx.x == 0) {
        Entity e;
        e.table_row = b;
        e.tok0 = b;
        e.nrows = ok && len > pre ? p.G : 0;
        e.k0 = pre;
        e.k1 = ok ? len : 0;
        e.lim0 = 0;
        e.kind = kLimAll;
        e.bad = !ok;
        p.ent[p.NG + b] = e;
        p.group_of[b] = j;
        p.row_lim[b] = ok ? pre : 0;
    }
}

// One CTA per entity checks its device data; the last one to finish lays out the
// work: items, their tiles end to end, the CTAs' shares and segments.
__global__ void __launch_bounds__(kPlanBlock) art_attend_plan_kernel(const AttendParams p) {
    __shared__ long long s_warp[kPlanBlock / 32];
    __shared__ int s_item0[kEntSmem + 1];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31;
    int err = 0;
    if (!p.shared) plan_extend(p, blockIdx.x, err);
    else if ((int)blockIdx.x < p.NG) plan_group(p, blockIdx.x, err);
    else plan_own(p, blockIdx.x - p.NG, err);
    if (tid == 0) {
        if (err) atomicOr(&p.hdr->status, err);
        __threadfence();
        s_last = atomicAdd(&p.hdr->plan_done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();

    // offsets that do not rise from 0 to their end: nothing is computed or written
    const int noff = p.shared ? p.NG : p.B, top = p.shared ? p.B : p.T;
    int bad = 0;
    if (noff > 0)
        for (int i = tid; i <= noff; i += kPlanBlock) {
            const int o = p.offsets[i];
            bad |= o < 0 || o > top || (i < noff && p.offsets[i + 1] < o);
        }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (tid == 0) {
            atomicOr(&p.hdr->status, ART_STATUS_BAD_OFFSETS);
            p.hdr->n_units = -1;  // the merge kernel writes nothing either
            *p.merge_n = 0;
        }
        for (int c = tid; c <= p.ctas; c += kPlanBlock) p.cta_first[c] = 0;
        return;
    }
    // a group whose prefix is bad takes its sequences with it
    if (p.shared)
        for (int b = tid; b < p.B; b += kPlanBlock) {
            const int j = __ldcg(&p.group_of[b]);
            if (j >= 0 && __ldcg(&p.ent[j].bad)) {
                p.ent[p.NG + b].nrows = 0;
                p.row_lim[b] = 0;
            }
        }
    __syncthreads();
    // items and partial rows before each entity
    int* item0 = p.NE <= kEntSmem ? s_item0 : p.item0;
    long long items = 0, prows = 0;
    for (int e0 = 0; e0 < p.NE; e0 += kPlanBlock) {
        const int e = e0 + tid;
        const int nrows = e < p.NE ? __ldcg(&p.ent[e].nrows) : 0;
        const long long mine = (long long)((nrows + p.rt - 1) / p.rt) * p.Hkv;
        long long tot;
        const long long before = block_scan(mine, s_warp, tot);
        long long rtot;
        const long long rbefore = block_scan((long long)nrows * p.Hkv, s_warp, rtot);
        if (e < p.NE) {
            item0[e] = (int)(items + before);
            p.item0[e] = (int)(items + before);
            p.prow0[e] = (int)(prows + rbefore);
        }
        items += tot;
        prows += rtot;
    }
    const int NI = (int)items;
    if (tid == 0) {
        p.item0[p.NE] = NI;
        *p.merge_n = 0;
    }
    __syncthreads();
    // the whole work and a CTA's share of it
    long long part = 0;
    for (int i = tid; i < NI; i += kPlanBlock) part += item_of(p, item0, i).tiles;
    long long W;
    (void)block_scan(part, s_warp, W);
    const long long quota = W > p.ctas ? (W + p.ctas - 1) / p.ctas : 1;
    // segments: piece c of item i is segment i + c (both rise along the work; where an
    // item ends at the end of a share one number stays free and is marked empty)
    const int c_end = W > 0 ? (int)((W - 1) / quota) : 0;
    for (int c = tid; c <= p.ctas; c += kPlanBlock)
        if ((long long)c * quota >= W) p.cta_first[c] = W > 0 ? NI + c_end : 0;
    Seg none;
    none.table_row = none.tok0 = none.r0 = none.nrow = none.g = none.k0 = none.k1 = none.lim0 = none.kind = 0;
    none.prow = -1;
    none.pad[0] = none.pad[1] = 0;
    long long start = 0;
    for (int i0 = 0; i0 < NI; i0 += kPlanBlock) {
        const int i = i0 + tid;
        Item it;
        it.tiles = 0;
        if (i < NI) it = item_of(p, item0, i);
        long long tot;
        const long long s = start + block_scan(it.tiles, s_warp, tot);
        start += tot;
        int c0 = 0, np = 0;
        Seg sg = none;
        if (i < NI) {
            c0 = (int)(s / quota);
            const Entity en = load_entity(&p.ent[it.e]);
            sg.table_row = en.table_row;
            sg.tok0 = en.tok0;
            sg.r0 = it.r0;
            sg.nrow = it.nrow;
            sg.g = it.g;
            sg.lim0 = en.lim0;
            sg.kind = en.kind;
            if (it.tiles == 0) {
                p.seg[i + c0] = none;
            } else {
                np = (int)((s + it.tiles - 1) / quota) - c0 + 1;
                if ((s + it.tiles) % quota == 0) p.seg[i + c0 + np] = none;
            }
            p.item_c[i] = make_int2(c0, np);
            if (!p.shared && np != 1) {  // split, or no keys: the merge kernel writes its rows
                MergeItem m;
                m.tok0 = en.tok0;
                m.r0 = it.r0;
                m.nrow = it.nrow;
                m.g = it.g;
                m.c0 = c0;
                m.np = np;
                m.pad[0] = m.pad[1] = 0;
                p.merge[atomicAdd(p.merge_n, 1)] = m;
            }
        }
        const int prow_i = i < NI && p.shared ? p.prow0[it.e] + it.g * __ldcg(&p.ent[it.e].nrows) + it.r0 : 0;
        auto emit = [&](const Seg& base, int idx, long long s0, int t0, int tiles, int k0, int k1, int cf, int n, int c,
                        int prow) {
            Seg o = base;
            const long long a = max(s0, (long long)c * quota) - s0, z = min(s0 + tiles, (long long)(c + 1) * quota) - s0;
            o.k0 = max(k0, (t0 + (int)a) * kKeyTile);
            o.k1 = min(k1, (t0 + (int)z) * kKeyTile);
            o.prow = p.shared ? prow + c * p.rt : (n == 1 ? -1 : piece_row_extend(c, c == cf, p.rt));
            p.seg[idx + c] = o;
            if (s0 <= (long long)c * quota) p.cta_first[c] = idx + c;
        };
        const bool few = np <= 2;
        if (few)
            for (int c = c0; c < c0 + np; ++c) emit(sg, i, s, it.t0, it.tiles, it.k0, it.k1, c0, np, c, prow_i);
        unsigned many = __ballot_sync(0xffffffffu, !few);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            Seg b;
            b.table_row = __shfl_sync(0xffffffffu, sg.table_row, src);
            b.tok0 = __shfl_sync(0xffffffffu, sg.tok0, src);
            b.r0 = __shfl_sync(0xffffffffu, sg.r0, src);
            b.nrow = __shfl_sync(0xffffffffu, sg.nrow, src);
            b.g = __shfl_sync(0xffffffffu, sg.g, src);
            b.lim0 = __shfl_sync(0xffffffffu, sg.lim0, src);
            b.kind = __shfl_sync(0xffffffffu, sg.kind, src);
            b.pad[0] = b.pad[1] = 0;
            const long long s0 = __shfl_sync(0xffffffffu, s, src);
            const int t0 = __shfl_sync(0xffffffffu, it.t0, src), tiles = __shfl_sync(0xffffffffu, it.tiles, src);
            const int k0 = __shfl_sync(0xffffffffu, it.k0, src), k1 = __shfl_sync(0xffffffffu, it.k1, src);
            const int cf = __shfl_sync(0xffffffffu, c0, src), n = __shfl_sync(0xffffffffu, np, src);
            const int pr = __shfl_sync(0xffffffffu, prow_i, src);
            for (int c = cf + lane; c < cf + n; c += 32)
                emit(b, i0 + (tid & ~31) + src, s0, t0, tiles, k0, k1, cf, n, c, pr);
        }
    }
}

// One warp per output row: joins the row's partial results and rounds once.
template <bool kBF16, int D>
__device__ __forceinline__ void merge_row(const AttendParams& p, float4 o, float l, size_t out_row, int lane) {
    constexpr int PER = D / 32;  // columns of a lane: 4 or 2
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key seen: 0; NaN stays
    const float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if constexpr (kBF16) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + out_row * D + lane * PER);
        dst[0] = pack_bf16(x[0], x[1]);
        if constexpr (PER == 4) dst[1] = pack_bf16(x[2], x[3]);
    } else {
        float* dst = static_cast<float*>(p.out) + out_row * D + lane * PER;
#pragma unroll
        for (int k = 0; k < PER; ++k) dst[k] = x[k];
    }
}

// Adds the partial row `pr` into the running (m, l, o).
template <int D>
__device__ __forceinline__ void merge_add(const AttendParams& p, int pr, float& m, float& l, float4& o, int lane) {
    constexpr int PER = D / 32;
    const float2 ml = __ldcg(&p.part_ml[pr]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = p.part_o + (size_t)pr * D + lane * PER;
    if constexpr (PER == 4) {
        x = __ldcg(reinterpret_cast<const float4*>(src));
    } else {
        const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
        x.x = t.x;
        x.y = t.y;
    }
    if (ml.y == 0.f) return;  // saw no key
    const float mn = fmaxf(m, ml.x);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float b = exp2f(ml.x - mn);
    l = l * a + ml.y * b;
    o.x = o.x * a + x.x * b;
    o.y = o.y * a + x.y * b;
    o.z = o.z * a + x.z * b;
    o.w = o.w * a + x.w * b;
    m = mn;
}

template <bool kBF16, int D>
__global__ void __launch_bounds__(kMergeBlock) art_attend_merge_kernel(const AttendParams p) {
    constexpr int WPB = kMergeBlock / 32;
    const int lane = threadIdx.x & 31;
    const int warp = blockIdx.x * WPB + (threadIdx.x >> 5), warps = gridDim.x * WPB;
    if (p.shared) {
        if (p.hdr->n_units < 0) return;  // bad offsets
        for (int row = warp; row < p.B * p.Hq; row += warps) {
            const int b = row / p.Hq, h = row - b * p.Hq, g = h / p.G, hg = h - g * p.G;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            const int j = p.group_of[b];
            auto add_item = [&](int e, int R) {
                const Entity en = p.ent[e];
                if (en.nrows == 0) return;
                const int nrt = (en.nrows + p.rt - 1) / p.rt, t = R / p.rt;
                const int2 c = p.item_c[p.item0[e] + g * nrt + t];
                const int pr = p.prow0[e] + g * en.nrows + R;
                for (int k = 0; k < c.y; ++k) merge_add<D>(p, pr + (c.x + k) * p.rt, m, l, o, lane);
            };
            if (j >= 0 && p.row_lim[b] > 0) add_item(j, (b - p.ent[j].tok0) * p.G + hg);
            add_item(p.NG + b, hg);
            merge_row<kBF16, D>(p, o, l, row, lane);
        }
        return;
    }
    const long long n = (long long)*p.merge_n * p.rt;
    for (long long w = warp; w < n; w += warps) {
        const MergeItem it = p.merge[w / p.rt];
        const int r = (int)(w % p.rt);
        if (r >= it.nrow) continue;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < it.np; ++k) merge_add<D>(p, piece_row_extend(it.c0 + k, k == 0, p.rt) + r, m, l, o, lane);
        const int R = it.r0 + r, t = R / p.G;
        merge_row<kBF16, D>(p, o, l, (size_t)(it.tok0 + t) * p.Hq + it.g * p.G + (R - t * p.G), lane);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Sizes and workspace layout of a call; returns the bytes, or 0 where they pass the
// supported range. `base` null: only the bytes.
static size_t attend_layout(AttendParams& p, unsigned char* base) {
    p.G = p.Hq / p.Hkv;
    p.NE = p.shared ? p.NG + p.B : p.B;
    const long long rows = (long long)(p.shared ? p.B : p.T) * p.G;  // of one KV head
    // rows of an item's tile; items and partial rows at most
    const long long ent = p.shared ? p.NG : p.B;
    long long items = (rows / p.rt + ent) * p.Hkv;
    if (p.shared) items += (long long)p.B * p.Hkv;
    const long long prows =
        p.shared ? 2 * rows * p.Hkv + (long long)(kAttendCtas + 1) * p.rt : 2LL * kAttendCtas * p.rt;
    // 32-bit row and key counts in the work list
    if (rows > (1LL << 30) || items > (1LL << 28) || prows > (1LL << 30) ||
        (long long)p.max_pages * p.Ps > (1LL << 30))
        return 0;
    p.max_items = (int)items;
    p.part_rows = (int)prows;
    size_t o = sizeof(WsHeader);
    auto take = [&](size_t bytes) {
        const size_t at = up256(o);
        o = at + bytes;
        return base ? base + at : nullptr;
    };
    p.hdr = reinterpret_cast<WsHeader*>(base);
    p.ent = reinterpret_cast<Entity*>(take(sizeof(Entity) * (size_t)p.NE));
    p.row_lim = reinterpret_cast<int*>(take(sizeof(int) * (size_t)p.B));
    p.group_of = reinterpret_cast<int*>(take(sizeof(int) * (size_t)p.B));
    p.item0 = reinterpret_cast<int*>(take(sizeof(int) * ((size_t)p.NE + 1)));
    p.prow0 = reinterpret_cast<int*>(take(sizeof(int) * (size_t)p.NE));
    p.item_c = reinterpret_cast<int2*>(take(sizeof(int2) * (size_t)items));
    p.cta_first = reinterpret_cast<int*>(take(sizeof(int) * (kAttendCtas + 1)));
    p.seg = reinterpret_cast<Seg*>(take(sizeof(Seg) * ((size_t)items + kAttendCtas + 2)));
    p.merge = reinterpret_cast<MergeItem*>(take(sizeof(MergeItem) * (size_t)(p.shared ? 1 : items)));
    p.merge_n = reinterpret_cast<int*>(take(sizeof(int)));
    p.part_ml = reinterpret_cast<float2*>(take(sizeof(float2) * (size_t)prows));
    p.part_o = reinterpret_cast<float*>(take(sizeof(float) * (size_t)prows * p.D));
    return up256(o);
}

static void fill_shape(AttendParams& p, const art_shape& s) {
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
    p.scale_log2 = (float)(1.4426950408889634074 / std::sqrt((double)s.head_dim));
}

static int attend_run(AttendParams& p, const art_shape& s, void* workspace, size_t workspace_bytes, cudaStream_t st) {
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
    if ((e = cudaMemsetAsync(p.hdr, 0, sizeof(WsHeader), st)) != cudaSuccess) return cuda_fail(e);
    art_attend_plan_kernel<<<p.NE, kPlanBlock, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e);
    const bool bf = s.dtype == ART_DTYPE_BF16;
    if ((e = bf ? launch_attend_tc(p, st) : launch_attend_simt(p, st)) != cudaSuccess) return cuda_fail(e);
    const long long rows = p.shared ? (long long)p.B * p.Hq : (long long)p.ctas * p.rt;
    const long long want = (rows + kMergeBlock / 32 - 1) / (kMergeBlock / 32);
    const unsigned grid = (unsigned)(want < 4LL * p.ctas ? (want > 0 ? want : 1) : 4LL * p.ctas);
    if (bf && p.D == 128) art_attend_merge_kernel<true, 128><<<grid, kMergeBlock, 0, st>>>(p);
    else if (bf) art_attend_merge_kernel<true, 64><<<grid, kMergeBlock, 0, st>>>(p);
    else if (p.D == 128) art_attend_merge_kernel<false, 128><<<grid, kMergeBlock, 0, st>>>(p);
    else art_attend_merge_kernel<false, 64><<<grid, kMergeBlock, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e);
    return ART_OK;
}

static bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace art

using namespace art;

extern "C" {

size_t dense_extend_workspace_bytes(const art_shape* shape, int32_t num_tokens) {
    if (check_shape(shape) != ART_OK || num_tokens < 0) return 0;
    AttendParams p = {};
    fill_shape(p, *shape);
    p.T = num_tokens;
    return attend_layout(p, nullptr);
}

int dense_extend(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                 const int32_t* seq_lens, const int32_t* q_offsets, int32_t num_tokens, int32_t causal, void* out,
                 const art_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_shape(shape);
    if (rc != ART_OK) return rc;
    if (!k_cache || !v_cache || !block_table || !seq_lens || !q_offsets || !workspace) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (!q || !out)) return ART_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out) || misaligned(workspace))
        return ART_ERR_INVALID_ARG;
    if (num_tokens < 0 || (causal != 0 && causal != 1)) return ART_ERR_INVALID_ARG;
    AttendParams p = {};
    fill_shape(p, *shape);
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
    if (check_shape(shape) != ART_OK || num_groups < 0) return 0;
    AttendParams p = {};
    fill_shape(p, *shape);
    p.shared = 1;
    p.NG = num_groups;
    return attend_layout(p, nullptr);
}

int dense_decode_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                        const int32_t* seq_lens, const int32_t* group_offsets, const int32_t* prefix_lens,
                        int32_t num_groups, void* out, const art_shape* shape, void* workspace,
                        size_t workspace_bytes, void* stream) {
    const int rc = check_shape(shape);
    if (rc != ART_OK) return rc;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace) return ART_ERR_INVALID_ARG;
    if (num_groups < 0 || (num_groups > 0 && (!group_offsets || !prefix_lens))) return ART_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out) || misaligned(workspace))
        return ART_ERR_INVALID_ARG;
    AttendParams p = {};
    fill_shape(p, *shape);
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
