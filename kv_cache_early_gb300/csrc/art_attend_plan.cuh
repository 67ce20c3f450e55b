// art_attend_plan.cuh -- plan_share: a CTA of the main kernel finds its share of the
// work and writes its segments (art_attend.cuh).
#pragma once

#include "art_attend.cuh"

namespace art {

// R / G for R < 2^30: g_mul = ceil(2^34 / G)
__device__ __forceinline__ int token_of(const AttendParams& p, int R) {
    return (int)((unsigned long long)R * p.g_mul >> 34);
}

struct PlanScratch {  // shared memory; may be reused once plan_share has returned
    long long warp_sum[32];
    int first, last, status;
    int pad;
    int offs[kMaxGroups + 1];  // dense_decode_shared: group_offsets
    int top[kMaxGroups];       // ... and the keys that the farthest member sees of the prefix
};

template <int NT>
__device__ __forceinline__ long long plan_scan(long long v, long long* s_warp, long long& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        const long long t = s_warp[i];
        before += i < w ? t : 0;
        all += t;
    }
    total = all;
    __syncthreads();
    return before + x - v;
}

// Whether sequence b's length is one that its table row can hold.
__device__ __forceinline__ bool len_ok(const AttendParams& p, int len) {
    return len >= 0 && (long long)len <= (long long)p.max_pages * p.Ps;
}

// Entity e; `err` collects status bits. Keys none (k1 <= k0) where it has no work.
__device__ __forceinline__ Entity entity_of(const AttendParams& p, const PlanScratch* s, int e, int& err) {
    Entity en;
    if (!p.shared) {
        const int lo = p.offsets[e], n = p.offsets[e + 1] - lo, len = p.seq_lens[e];
        const bool ok = len_ok(p, len) && (!p.causal || len >= n);
        if (!ok) err |= ART_STATUS_BAD_SEQLEN;
        en.table_row = e;
        en.tok0 = lo;
        en.nrows = n * p.G;
        en.k0 = 0;
        en.k1 = ok && n > 0 ? len : 0;
        en.lim0 = len - n + 1;
        en.kind = p.causal ? kLimCausal : kLimAll;
    } else if (e < p.NG) {
        en.table_row = en.tok0 = s->offs[e];
        en.nrows = (s->offs[e + 1] - s->offs[e]) * p.G;
        en.k0 = 0;
        en.k1 = en.nrows > 0 ? s->top[e] : 0;
        en.lim0 = 0;
        en.kind = kLimSeq;
    } else {
        const int b = e - p.NG, len = p.seq_lens[b];
        int lo = -1, hi = p.NG;  // offs[lo] <= b < offs[hi], as far as there are such
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s->offs[mid] <= b) lo = mid;
            else hi = mid;
        }
        const int j = lo >= 0 && p.NG > 0 && b < s->offs[p.NG] ? lo : -1;
        bool ok = len_ok(p, len);
        if (!ok) err |= ART_STATUS_BAD_SEQLEN;
        int pre = 0;
        if (j >= 0) {
            pre = p.prefix[j];
            if (!len_ok(p, pre)) {
                err |= ART_STATUS_BAD_SEQLEN;
                ok = false;
            }
        }
        en.table_row = en.tok0 = b;
        en.nrows = p.G;
        en.k0 = ok ? min(len, pre) : 0;
        en.k1 = ok ? len : 0;
        en.lim0 = ok ? en.k0 : -1;  // what its rows see of the prefix
        en.kind = kLimAll;
        if (blockIdx.x == 0) {
            p.group_of[b] = j;
        }
    }
    return en;
}

__device__ __forceinline__ int entity_tiles(const AttendParams& p, const Entity& en, int r) {  // row tile r's key tiles
    int k1 = en.k1;
    if (en.kind == kLimCausal) k1 = en.lim0 + token_of(p, min((r + 1) * p.rt, en.nrows) - 1);
    return (k1 + kKeyTile - 1) / kKeyTile - en.k0 / kKeyTile;
}

// The cost of one KV head of an entity (0: no keys), and its row tiles.
__device__ __forceinline__ long long head_cost(const AttendParams& p, const Entity& en, int& nrt) {
    nrt = 0;
    if (en.nrows <= 0 || en.k1 <= en.k0) return 0;
    nrt = (en.nrows + p.rt - 1) / p.rt;
    long long c = 0;
    if (en.kind != kLimCausal) {
        const int tiles = entity_tiles(p, en, 0), last = en.nrows - (nrt - 1) * p.rt;
        c = (long long)(nrt - 1) * (item_cost_base(p, p.rt) + (long long)item_cost_tile(p, p.rt) * tiles);
        return c + item_cost_base(p, last) + (long long)item_cost_tile(p, last) * tiles;
    }
    for (int r = 0; r < nrt; ++r) {
        const int n = min(p.rt, en.nrows - r * p.rt);
        c += item_cost_base(p, n) + (long long)item_cost_tile(p, n) * entity_tiles(p, en, r);
    }
    return c;
}

// The segments of entity en (first item item0, first cost unit start, first partial row
// prow) that lie in CTA c's share [lo, hi).
static __device__ void emit_entity(const AttendParams& p, PlanScratch* s, const Entity& en, long long hc, int nrt, int item0,
                            long long start, long long prow, long long lo, long long hi, long long quota, int c) {
    int g = start >= lo ? 0 : (int)((lo - start) / hc);
    for (; g < p.Hkv && start + g * hc < hi; ++g) {
        long long x = start + g * hc;  // first unit of the row tile
        int r = 0;
        if (en.kind != kLimCausal && x < lo) {  // equal row tiles but the last: skip by division
            const long long ic = item_cost_base(p, p.rt) + (long long)item_cost_tile(p, p.rt) * entity_tiles(p, en, 0);
            r = (int)min((lo - x) / ic, (long long)(nrt - 1));
            x += r * ic;
        }
        for (; r < nrt && x < hi; ++r) {
            const int n = min(p.rt, en.nrows - r * p.rt), tiles = entity_tiles(p, en, r);
            const int base = item_cost_base(p, n), per = item_cost_tile(p, n);
            const long long z = x + base + (long long)per * tiles;
            if (z > lo) {
                const int i = item0 + g * nrt + r;
                const int ta = tiles_before(lo - x, base, per, tiles), tz = tiles_before(min(z, hi) - x, base, per, tiles);
                const int t0 = en.k0 / kKeyTile;
                const int c0 = (int)(x / quota), np = (int)((z - 1) / quota) - c0 + 1;
                int k1 = en.k1;
                if (en.kind == kLimCausal) k1 = en.lim0 + token_of(p, r * p.rt + n - 1);
                Seg o;
                o.table_row = en.table_row;
                o.tok0 = en.tok0;
                o.r0 = r * p.rt;
                o.nrow = tz > ta ? n : 0;
                o.g = g;
                o.k0 = max(en.k0, (t0 + ta) * kKeyTile);
                o.k1 = min(k1, (t0 + tz) * kKeyTile);
                o.lim0 = en.lim0;
                o.kind = en.kind;
                o.prow = p.shared ? (int)(prow + (long long)g * en.nrows + r * p.rt) + c * p.rt
                                  : (np == 1 ? -1 : piece_row_extend(c, c == c0, p.rt));
                o.bad = o.pad = 0;
                p.seg[i + c] = o;
                if (x <= lo) s->first = i + c;
                if (z >= hi) s->last = i + c + 1;
                if (!p.shared && x < lo && c == c0 + 1) {
                    MergeItem m;
                    m.tok0 = en.tok0;
                    m.r0 = o.r0;
                    m.nrow = n;
                    m.g = g;
                    m.c0 = c0;
                    m.np = np;
                    m.tiles = tiles;
                    m.off = (int)(lo - x);  // less than a share
                    m.seq = en.table_row;
                    m.pad[0] = m.pad[1] = m.pad[2] = 0;
                    p.merge[c] = m;
                }
            }
            x = z;
        }
    }
}

// The CTA's segments are seg[s0 .. s1). All threads of the block.
template <int NT>
__device__ void plan_share(const AttendParams& p, PlanScratch* s, int& s0, int& s1) {
    const int tid = threadIdx.x, c = blockIdx.x;
    if (tid == 0) {
        s->first = s->last = 0;
        s->status = 0;
        p.merge[c].np = 0;
    }
    // offsets that do not rise within 0 .. their end: nothing is computed or written
    const int noff = p.shared ? p.NG : p.B, end = p.shared ? p.B : p.T;
    int bad = 0;
    for (int i = tid; i <= noff && noff > 0; i += NT) {
        const int o = p.offsets[i], prev = i > 0 ? p.offsets[i - 1] : 0;
        bad |= o < prev || o > end || o < 0;
        if (p.shared) s->offs[i] = o;
        if (p.shared && i < noff) s->top[i] = 0;
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (tid == 0) {
            p.cta_status[c] = ART_STATUS_BAD_OFFSETS;
            p.cta_segs[c] = make_int2(0, 0);
            if (c == 0) p.info->ok = 0;
        }
        s0 = s1 = 0;
        return;
    }
    // the whole work: own tokens first (they tell how much of the prefixes is seen)
    int err = 0;
    long long W = 0, tot;
    if (p.shared) {
        for (int b = tid; b < p.B; b += NT) {
            const Entity en = entity_of(p, s, p.NG + b, err);
            if (c == 0) p.row_lim[b] = en.lim0;
            if (en.lim0 > 0) {
                int lo = 0, hi = p.NG;  // its group
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s->offs[mid] <= b) lo = mid;
                    else hi = mid;
                }
                atomicMax(&s->top[lo], en.lim0);
            }
        }
        __syncthreads();
    }
    for (int e0 = 0; e0 < p.NE; e0 += NT) {
        long long cost = 0;
        int nrt;
        if (e0 + tid < p.NE) cost = head_cost(p, entity_of(p, s, e0 + tid, err), nrt) * p.Hkv;
        (void)plan_scan<NT>(cost, s->warp_sum, tot);
        W += tot;
    }
    const long long quota = W > p.ctas ? (W + p.ctas - 1) / p.ctas : 1;
    const long long lo = (long long)c * quota, hi = min(lo + quota, W);
    long long start = 0, items = 0, prows = 0;
    for (int e0 = 0; e0 < p.NE && (lo < hi || c == 0); e0 += NT) {
        const int e = e0 + tid;
        long long hc = 0;
        int nrt = 0;
        Entity en;
        en.nrows = 0;
        if (e < p.NE) {
            en = entity_of(p, s, e, err);
            hc = head_cost(p, en, nrt);
        }
        const long long x = start + plan_scan<NT>(hc * p.Hkv, s->warp_sum, tot);
        start += tot;
        const int i0 = (int)(items + plan_scan<NT>((long long)nrt * p.Hkv, s->warp_sum, tot));
        items += tot;
        long long pr = 0;
        if (p.shared) {
            pr = prows + plan_scan<NT>(nrt > 0 ? (long long)en.nrows * p.Hkv : 0, s->warp_sum, tot);
            prows += tot;
        }
        if (c == 0 && e < p.NE) {
            EntityPlace q;
            q.nrows = nrt > 0 ? en.nrows : 0;
            q.k0 = en.k0;
            q.k1 = en.k1;
            q.item0 = i0;
            q.start = x;
            q.prow = pr;
            p.place[e] = q;
        }
        if (hc > 0 && x < hi && x + hc * p.Hkv > lo) emit_entity(p, s, en, hc, nrt, i0, x, pr, lo, hi, quota, c);
    }
    if (err) atomicOr(&s->status, err);
    __syncthreads();
    if (tid == 0) {
        p.cta_status[c] = s->status;
        if (c == 0) {
            p.info->quota = quota;
            p.info->total = W;
            p.info->ok = 1;
        }
    }
    s0 = s->first;
    s1 = s->last;
    if (tid == 0) p.cta_segs[c] = make_int2(s0, s1);
    __syncthreads();  // the segments are written, the scratch is free
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
