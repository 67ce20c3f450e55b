// art_attend_plan.cuh -- plan_share: a CTA of the main kernel finds its share of the
// work and writes its segments (art_attend.cuh).
#pragma once

#include "art_attend.cuh"

namespace art {

// R / G for R < 2^30: g_mul = ceil(2^34 / G)
__device__ __forceinline__ int token_of(const AttendParams& p, int R) {
    return (int)((unsigned long long)R * p.g_mul >> 34);
}

// An entity with its place in the work.
struct alignas(16) PlanEntity {
    Entity en;
    int nrt;           // row tiles (0: no work)
    int hc, start;     // cost of one KV head, first cost unit
    int item0, prow;   // first item, first partial row
};
static_assert(sizeof(PlanEntity) == 48, "three 16-byte words");

struct PlanScratch {  // shared memory; may be reused once plan_share has returned
    int4 warp_sum[12];
    int first, last, status, listed;
    PlanEntity list[384];
    int offs[kMaxGroups + 1];  // dense_decode_shared: group_offsets
    int top[kMaxGroups];       // ... and the keys that the farthest member sees of the prefix
};

// The code below runs once in a CTA's life, and most of its time is the fetch of its
// instructions: loops stay rolled, functions are not repeated, counts have 32 bits (the
// host bounds them, attend_layout).

__device__ __forceinline__ void scan3(int (&v)[3]) {  // inclusive, over a warp
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int y = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += y;
        }
}

// Exclusive sums of three values over the block, and their totals.
template <int NT>
__device__ __forceinline__ void plan_scan(int (&v)[3], int (&total)[3], int4* s_warp) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int own[3] = {v[0], v[1], v[2]};
    scan3(v);
    if (lane == 31) s_warp[w] = make_int4(v[0], v[1], v[2], 0);
    named_bar_sync(1, NT);
    const int4 t = lane < NT / 32 ? s_warp[lane] : make_int4(0, 0, 0, 0);
    int u[3] = {t.x, t.y, t.z};
    scan3(u);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int before = __shfl_sync(0xffffffffu, u[i], w > 0 ? w - 1 : 0);
        total[i] = __shfl_sync(0xffffffffu, u[i], NT / 32 - 1);
        v[i] += (w > 0 ? before : 0) - own[i];
    }
    named_bar_sync(1, NT);
}

// Whether sequence b's length is one that its table row can hold.
__device__ __forceinline__ bool len_ok(const AttendParams& p, int len) {
    return len >= 0 && (long long)len <= (long long)p.max_pages * p.Ps;
}

// Entity e; `err` collects status bits. Keys none (k1 <= k0) where it has no work. A
// group's needs the tops, which the own tokens of its members set.
static __device__ __noinline__ Entity entity_of(const AttendParams& p, PlanScratch* s, int e, int& err) {
    Entity en;
    en.k0 = en.lim0 = 0;
    if (p.shared && e < p.NG) {
        en.table_row = en.tok0 = s->offs[e];
        en.nrows = (s->offs[e + 1] - s->offs[e]) * p.G;
        en.k1 = s->top[e];
        en.kind = kLimSeq;
        return en;
    }
    const int b = p.shared ? e - p.NG : e;
    const int len = p.seq_lens[b];
    bool ok = len_ok(p, len);
    en.table_row = en.tok0 = b;
    en.nrows = p.G;
    en.k1 = len;
    en.kind = kLimAll;
    if (!p.shared) {
        const int lo = p.offsets[b], n = p.offsets[b + 1] - lo;
        ok = ok && (!p.causal || len >= n);
        en.tok0 = lo;
        en.nrows = n * p.G;
        en.lim0 = len - n + 1;
        if (p.causal) en.kind = kLimCausal;
        if (n == 0) en.k1 = 0;
    } else if (p.NG > 0 && b >= s->offs[0] && b < s->offs[p.NG]) {
        int lo = 0, hi = p.NG;  // its group: the last that starts at or before b
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s->offs[mid] <= b) lo = mid;
            else hi = mid;
        }
        const int pre = p.prefix[lo];
        ok = ok && len_ok(p, pre);
        en.k0 = min(len, pre);
        if (ok && en.k0 > 0) atomicMax(&s->top[lo], en.k0);
        if (blockIdx.x == 0) p.group_of[b] = lo;
    } else if (blockIdx.x == 0) {
        p.group_of[b] = -1;
    }
    if (!ok) {
        err |= ART_STATUS_BAD_SEQLEN;
        en.k0 = en.k1 = 0;
    }
    if (p.shared && blockIdx.x == 0) p.row_lim[b] = ok ? en.k0 : -1;
    return en;
}

__device__ __forceinline__ int entity_tiles(const AttendParams& p, const Entity& en, int r) {  // row tile r's key tiles
    int k1 = en.k1;
    if (en.kind == kLimCausal) k1 = en.lim0 + token_of(p, min((r + 1) * p.rt, en.nrows) - 1);
    return tiles_of(p, en.k0, k1);
}
__device__ __forceinline__ int item_cost(const AttendParams& p, const Entity& en, int r, int& tiles) {
    const int n = min(p.rt, en.nrows - r * p.rt);
    tiles = entity_tiles(p, en, r);
    return item_cost_base(p, n) + item_cost_tile(p, n) * tiles;
}

// The segments of a listed entity that lie in CTA c's share [lo, hi): one warp, an item
// a lane.
static __device__ void emit_entity(const AttendParams& p, PlanScratch* s, const PlanEntity& q, int lo, int hi, int quota,
                                   int slack, int c) {
    const int lane = threadIdx.x & 31;
    const Entity en = q.en;
    const int g0 = q.start >= lo ? 0 : (int)((unsigned)(lo - q.start) / (unsigned)q.hc), items = p.Hkv * q.nrt;
    int x0 = q.start + g0 * q.hc;  // first unit of the items that follow
#pragma unroll 1
    for (int i0 = g0 * q.nrt; i0 < items && x0 < hi; i0 += 32) {
        const int i = i0 + lane, g = (int)((unsigned)i / (unsigned)q.nrt), r = i - g * q.nrt;
        int tiles = 0;
        const int cost = i < items ? item_cost(p, en, r, tiles) : 0;
        int z = cost;  // inclusive sum, then the item's end
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += y;
        }
        z += x0;
        const int x = z - cost;
        x0 = __shfl_sync(0xffffffffu, z, 31);
        if (i >= items || x >= hi || z <= lo) continue;
        const int n = min(p.rt, en.nrows - r * p.rt);
        const int base = item_cost_base(p, n), per = item_cost_tile(p, n), t0 = en.k0 >> p.kt_log2;
        // the CTAs that hold its first and its last unit; nearly always this one. Where little
        // of it lies on one side of a border between shares, it moves to the other whole:
        // a split costs the partial results' way through memory.
        int c0 = x >= lo ? c : (int)((unsigned)x / (unsigned)quota), c1 = z <= hi ? c : (int)((unsigned)(z - 1) / (unsigned)quota);
        if (c0 < c1 && (c0 + 1) * quota - x <= slack) ++c0;
        if (c0 < c1 && z - c1 * quota <= slack) --c1;
        if (c < c0 || c > c1) continue;
        const int ta = c == c0 ? 0 : tiles_before(lo - x, base, per, tiles);
        const int tz = c == c1 ? tiles : tiles_before(hi - x, base, per, tiles);
        int k1 = en.k1;
        if (en.kind == kLimCausal) k1 = en.lim0 + token_of(p, r * p.rt + n - 1);
        Seg o;
        o.table_row = en.table_row;
        o.tok0 = en.tok0;
        o.r0 = r * p.rt;
        o.nrow = tz > ta ? n : 0;
        o.g = g;
        o.k0 = max(en.k0, (t0 + ta) << p.kt_log2);
        o.k1 = min(k1, (t0 + tz) << p.kt_log2);
        o.lim0 = en.lim0;
        o.kind = en.kind;
        o.prow = p.shared ? q.prow + g * en.nrows + r * p.rt + c * p.rt : (c0 == c1 ? -1 : piece_row_extend(c, c == c0, p.rt));
        o.bad = o.pad = 0;
        p.seg[q.item0 + i + c] = o;
        atomicMin(&s->first, q.item0 + i + c);
        atomicMax(&s->last, q.item0 + i + c + 1);
        if (!p.shared && c == c0 + 1) {
            MergeItem m;
            m.tok0 = en.tok0;
            m.r0 = o.r0;
            m.nrow = n;
            m.g = g;
            m.c0 = c0;
            m.np = c1 - c0 + 1;
            m.tiles = tiles;
            m.off = lo - x;
            m.seq = en.table_row;
            m.pad[0] = m.pad[1] = m.pad[2] = 0;
            p.merge[c] = m;
        }
    }
}

// The CTA's segments are seg[s0 .. s1). The first NT threads of the block (named
// barrier 1).
template <int NT>
__device__ void plan_share(const AttendParams& p, PlanScratch* s, int& s0, int& s1) {
    static_assert(NT <= 384, "list");
    const int tid = threadIdx.x, c = blockIdx.x;
    if (tid == 0) {
        s->first = 0x7fffffff;
        s->last = s->listed = 0;
        s->status = 0;
        p.merge[c].np = 0;
    }
    named_bar_sync(1, NT);
    // offsets that do not rise within 0 .. their end: nothing is computed or written
    const int noff = p.shared ? p.NG : p.B, end = p.shared ? p.B : p.T;
    int bad = 0;
#pragma unroll 1
    for (int i = tid; i <= noff && noff > 0; i += NT) {
        const int o = p.offsets[i], prev = i > 0 ? p.offsets[i - 1] : 0;
        bad |= o < prev || o > end || o < 0;
        if (p.shared) s->offs[i] = o;
        if (p.shared && i < noff) s->top[i] = 0;
    }
    if (bad) atomicOr(&s->status, ART_STATUS_BAD_OFFSETS);
    named_bar_sync(1, NT);
    if (s->status) {
        if (tid == 0) {
            p.cta_status[c] = ART_STATUS_BAD_OFFSETS;
            p.cta_segs[c] = make_int2(0, 0);
            if (c == 0) p.info->ok = 0;
        }
        s0 = s1 = 0;
        return;
    }
    // Rounds over the entities, as many as threads in each: with more than one, a first
    // sweep for the tops, a second for the whole work, and the last lays it out.
    const int rounds = (p.NE + NT - 1) / NT;
    int err = 0, W = 0, quota = 1, lo = 0, hi = 0, start = 0, items = 0, prows = 0;
    int v[3], tot[3];
    PlanEntity q;
#pragma unroll 1
    for (int k = rounds == 1 ? 2 * rounds : 0; k < 3 * rounds; ++k) {
        const int sweep = k / rounds, e = (k - sweep * rounds) * NT + tid;
        const bool own = !p.shared || e >= p.NG;
        q.en.nrows = 0;
        if (e < p.NE && own) q.en = entity_of(p, s, e, err);
        if (p.shared) named_bar_sync(1, NT);  // the tops of a single round
        if (sweep == 0 && rounds > 1) continue;
        if (e < p.NE && !own) q.en = entity_of(p, s, e, err);
        q.nrt = e < p.NE && q.en.nrows > 0 && q.en.k1 > q.en.k0 ? (q.en.nrows + p.rt - 1) / p.rt : 0;
        q.hc = 0;
#pragma unroll 1
        for (int r = 0; r < q.nrt; ++r) {
            int tiles;
            const int cost = item_cost(p, q.en, r, tiles);
            // equal row tiles but the last, where the keys do not go by the row
            const int skip = q.en.kind != kLimCausal && r == 0 && q.nrt > 2 ? q.nrt - 2 : 0;
            q.hc += cost * (skip + 1);
            r += skip;
        }
        v[0] = q.hc * p.Hkv;
        v[1] = q.nrt * p.Hkv;
        v[2] = p.shared && q.nrt > 0 ? q.en.nrows * p.Hkv : 0;
        plan_scan<NT>(v, tot, s->warp_sum);
        if (sweep == 1 || rounds == 1) {
            W += tot[0];
            quota = W > p.ctas ? (W + p.ctas - 1) / p.ctas : 1;
            lo = min(c * quota, W);
            hi = min(lo + quota, W);
            if (rounds > 1) continue;
        }
        q.start = start + v[0];
        q.item0 = items + v[1];
        q.prow = prows + v[2];
        start += tot[0];
        items += tot[1];
        prows += tot[2];
        if (c == 0 && e < p.NE) {
            EntityPlace pl;
            pl.nrows = q.nrt > 0 ? q.en.nrows : 0;
            pl.k0 = q.en.k0;
            pl.k1 = q.en.k1;
            pl.start = q.start;
            pl.prow = q.prow;
            pl.hc = q.hc;
            pl.pad[0] = pl.pad[1] = 0;
            p.place[e] = pl;
        }
        if (q.nrt > 0 && q.start < hi && q.start + q.hc * p.Hkv > lo) s->list[atomicAdd(&s->listed, 1)] = q;
        named_bar_sync(1, NT);
        const int n = s->listed, slack = p.shared ? 0 : quota / kSplitSlack;
#pragma unroll 1
        for (int i = tid >> 5; i < n; i += NT / 32) emit_entity(p, s, s->list[i], lo, hi, quota, slack, c);
        named_bar_sync(1, NT);
        if (tid == 0) s->listed = 0;
    }
    if (err) atomicOr(&s->status, err);
    named_bar_sync(1, NT);
    s1 = s->last;
    s0 = min(s->first, s1);
    if (tid == 0) {
        p.cta_status[c] = s->status;
        p.cta_segs[c] = make_int2(s0, s1);
        if (c == 0) {
            p.info->quota = quota;
            p.info->ok = 1;
        }
    }
    named_bar_sync(1, NT);  // the segments are written, the scratch is free
}

// Segments are written by the same kernel: not through the read-only path.
__device__ __forceinline__ Seg load_seg(const Seg* s) {
    Seg r;
    const int4 a = __ldcg(reinterpret_cast<const int4*>(s)), b = __ldcg(reinterpret_cast<const int4*>(s) + 1),
               c = __ldcg(reinterpret_cast<const int4*>(s) + 2);
    r.table_row = a.x;
    r.tok0 = a.y;
    r.r0 = a.z;
    r.nrow = a.w;
    r.g = b.x;
    r.k0 = b.y;
    r.k1 = b.z;
    r.lim0 = b.w;
    r.kind = c.x;
    r.prow = c.y;
    r.bad = r.pad = 0;
    return r;
}

// A row's place in q and out.
__device__ __forceinline__ size_t row_index(const AttendParams& p, const Seg& sg, int r) {
    const int R = sg.r0 + r, t = token_of(p, R);
    return (size_t)(sg.tok0 + t) * p.Hq + sg.g * p.G + (R - t * p.G);
}
// What sequence b's rows see of the prefix [.., k1): as its own entity has it.
__device__ __forceinline__ int seq_limit(const AttendParams& p, int b, int k1) {
    const int len = p.seq_lens[b];
    return len_ok(p, len) ? min(len, k1) : 0;
}
// Keys that row r sees lie below this.
__device__ __forceinline__ int row_limit(const AttendParams& p, const Seg& sg, int r) {
    if (r >= sg.nrow) return sg.k0;
    if (sg.kind == kLimAll) return sg.k1;
    const int t = token_of(p, sg.r0 + r);
    return min(sg.k1, sg.kind == kLimCausal ? sg.lim0 + t : seq_limit(p, sg.tok0 + t, sg.k1));
}
// Column c of row r of a segment's partial results.
__device__ __forceinline__ float* part_at(const AttendParams& p, const Seg& sg, int r, int c) {
    return p.part_o + (size_t)sg.prow * p.D + ((size_t)(c >> 2) * sg.nrow + r) * 4 + (c & 3);
}

}  // namespace art
