// art_attend_kv4.cuh -- the segments of art_attend.cuh over a cache that is held in 4 bits.
//
// With K = low + step c in each group of columns (c the codes) the products need the codes only:
//     q . k_t = sum_g step_tg (sum_{j in g} q_j c_tj) + low_tg (sum_{j in g} q_j)
//     o_j     = sum_t (p_t step_tg) c_tj + p_t low_tg
// so codes are never turned into values: they enter the matrix product as fp16, where the four
// bits of a code, moved to the lowest bits, ARE the number code * 2^-24 (a denormal), and moved to
// the next four code * 2^-20. Eight codes of a 32-bit word become four operand registers by four
// masks and one shift; 2^24 and the 16 of the odd ones go into queries and results.
//
// S^T = C Q^T and O^T = C^T W^T, keys or columns in the 16 rows of mma.sync 16 x 8 x 16, up to
// eight query rows in its columns, so no row of the product is padding where eight rows attend
// (GQA with 8 heads; 4 heads leave half). Keys' codes come by ldmatrix as they lie (a lane has 8
// columns of one key), values' codes by its transposed form (4 columns of two neighbouring
// tokens): both are operands after the masks. W = p step is rounded to fp16 (11 bits; fp32 calls
// take a second part for what is left, and split the queries too, so about 22 bits). Scores,
// weights, their sums and what is multiplied by low are fp32.
//
// Range: a row's reference follows the maximum of score + log2(step), not of the score alone, so W
// stays within fp16's range whatever the values' scales are, and the row's sum l is brought to
// [1, 2) before parts meet. Queries are scaled by a power of two to fp16's range.
//
// One CTA per SM: a producer warp (page ids 32 at a time, one bulk copy for each slab of a page,
// art_kv4.cuh) fills a ring of tiles of 128 keys; 8 consumer warps in two groups of four take
// alternate tiles, a warp 32 keys of each. Up to 8 rows: 32 keys at a time, two chains of
// products; up to 16: two column tiles. 17 to 32 rows: the groups take 16 rows each, and every tile.
// Each warp has its own reference, sums and O; they meet at the segment's end.
//
// Keys and values outside a segment's keys may be anything: codes are always finite numbers, and
// scales of keys that a row does not see are not used for it.
#pragma once

#include "art_attend_tc.cuh"
#include "art_kv4.cuh"

namespace art {

constexpr int kRowsKv4 = 32;  // rows of an item's tile
constexpr int kKv4Consumers = 8, kKv4Threads = (kKv4Consumers + 1) * 32;
// A row's reference is set so that its largest weight times step is about 2^kKv4Lift, and moves when
// one passes 2^kKv4Most: fp16 holds 11 bits of whatever is within 2^-19 of the largest.
constexpr float kKv4Lift = 5.f, kKv4Most = 14.f;

struct AttendKv4Params {
    AttendParams a;
    const unsigned char* cache;
    int slab, slab_bytes, page_bytes, bf16;
};

template <int D, int NG>
struct Kv4Cfg {
    static constexpr int TILE = kKeyTile * (D + 8 * NG);  // bytes of a tile
    static constexpr int EXROW = D + 4;                   // floats of a row in the exchange area
    static constexpr int EX = kKv4Consumers * 8 * EXROW * 4;
    static constexpr int NS = (220 * 1024 - EX) / TILE < 16 ? (220 * 1024 - EX) / TILE : 16;  // ring stages
    static constexpr int EXOFF = NS * TILE;
    static constexpr int CTRL = EXOFF + EX;
};

template <int NS>
struct alignas(16) Kv4Ctrl {
    uint64_t full[NS], empty[NS], cons, stall;
    float2 ml[kKv4Consumers][8];
    int abort, seg0, seg1;
};

template <int D, int NG>
constexpr size_t kv4_smem() {
    return (size_t)Kv4Cfg<D, NG>::CTRL + sizeof(Kv4Ctrl<Kv4Cfg<D, NG>::NS>);
}

// d[0..3] += A(16x16 fp16, row) * B(16x8 fp16, col)
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
    float lo, hi;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
    return make_float2(lo, hi);
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ---------------------------------------------------------------------------
// producer warp
// ---------------------------------------------------------------------------
template <int D, int NG>
__device__ void kv4_producer(const AttendKv4Params& pp, unsigned char* gen, Kv4Ctrl<Kv4Cfg<D, NG>::NS>* c, int s0, int s1) {
    using C = Kv4Cfg<D, NG>;
    const AttendParams& p = pp.a;
    const int lane = threadIdx.x & 31;
    const int ppt = kKeyTile / pp.slab;  // slabs of a tile (2 .. 16)
    const int tpb = 32 / ppt;            // tiles whose page ids the warp holds
    auto ids_of = [&](const Seg& sg, int bt) -> int {  // of this lane's slab of batch bt, -1 where it has none
        const int key = (sg.k0 / kKeyTile + bt * tpb) * kKeyTile + lane * pp.slab;
        if (sg.nrow == 0 || key >= sg.k1 || key + pp.slab <= sg.k0) return -1;
        const int pg = __ldg(&p.block_table[(size_t)sg.table_row * p.max_pages + key / p.Ps]);
        return pg < 0 || pg >= p.num_pages ? -2 : pg;
    };
    Stage<C::NS> st;
    uint32_t used = 0, ph = 0, filled_ph = 0;  // per stage: filled once; parity to wait for
    Seg sg = load_seg(&p.seg[s0]);
    int ids = ids_of(sg, 0);
    bool ok = true;
    for (int si = s0; si < s1 && ok; ++si) {
        Seg nx = sg;
        nx.nrow = 0;
        if (si + 1 < s1) nx = load_seg(&p.seg[si + 1]);
        if (sg.nrow == 0) {
            sg = nx;
            ids = ids_of(sg, 0);
            continue;
        }
        const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
        for (int bt = 0; bt * tpb < nt && ok; ++bt) {
            const int more = (bt + 1) * tpb < nt ? ids_of(sg, bt + 1) : ids_of(nx, 0);
            const int nb = min(tpb, nt - bt * tpb);
            if (__any_sync(0xffffffffu, ids == -2)) {  // outside the pool: page 0 instead, the merge kernel zeroes the rows
                if (lane == 0) {
                    p.seg[si].bad = 1;
                    atomicOr(&p.cta_status[blockIdx.x], ART_STATUS_BAD_PAGE);
                }
                if (ids == -2) ids = 0;
            }
            for (int t = 0; t < nb; ++t) {
                const bool mine = lane / ppt == t && ids >= 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * pp.slab_bytes;
                const int in_tile = lane - t * ppt;  // this lane's slab in the tile
                const int key = (t0 + bt * tpb + t) * kKeyTile + in_tile * pp.slab;
                const uint32_t bit = 1u << st.s;
                if (used & bit) {
                    if (!wait_tc(&c->empty[st.s], (ph & bit) ? 1u : 0u, &c->abort, p)) {
                        ok = false;
                        break;
                    }
                    ph ^= bit;
                }
                used |= bit;
                filled_ph = st.ph ? filled_ph | bit : filled_ph & ~bit;
                if (lane == 0) mbar_arrive_expect_tx(&c->full[st.s], bytes);
                __syncwarp();
                if (mine)
                    bulk_g2s(gen + st.s * C::TILE + in_tile * pp.slab_bytes,
                             pp.cache + ((size_t)ids * p.Hkv + sg.g) * (size_t)pp.page_bytes +
                                 (size_t)((key & (p.Ps - 1)) / pp.slab) * pp.slab_bytes,
                             (uint32_t)pp.slab_bytes, &c->full[st.s]);
                st.next();
            }
            ids = more;
        }
        sg = nx;
    }
    // no copy of this CTA may be in flight when it ends
    for (int s = 0; s < C::NS; ++s)
        if (used & (1u << s)) {
            const unsigned long long w0 = global_ns();
            while (!__all_sync(0xffffffffu, mbar_try_wait(&c->full[s], (filled_ph >> s) & 1u)))
                if (__any_sync(0xffffffffu, lane == 0 && global_ns() - w0 > kWaitLimitNs)) break;
        }
}

// ---------------------------------------------------------------------------
// consumer warps
// ---------------------------------------------------------------------------
template <bool kBF16, int D, int NG>
struct Kv4Consumer {
    using C = Kv4Cfg<D, NG>;
    static constexpr int NC = D / 32;       // 32-column chunks
    static constexpr int CPG = NC / NG;     // ... of a group
    static constexpr int KP = kBF16 ? 1 : 2;  // fp16 parts of a query and of a weight
    const AttendKv4Params& pp;
    const AttendParams& p;
    Kv4Ctrl<C::NS>* c;
    uint32_t smem;
    unsigned char* gen;
    int w, lane;
    uint32_t ph_c = 0;
    int odd = 0;  // which group of warps takes the next tile
    Stage<C::NS> st;

    __device__ __forceinline__ bool wait(uint64_t* b, uint32_t ph) { return wait_tc(b, ph, &c->abort, p); }
    __device__ __forceinline__ bool sync() {  // all consumer warps
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->cons);
        const bool ok = wait(&c->cons, ph_c);
        ph_c ^= 1u;
        return ok;
    }
    // codes of 8 tokens: a word a chunk of 32 columns. `o`: offset in shared memory of the octets' codes
    template <bool kTrans>
    __device__ __forceinline__ void codes(uint32_t oa, uint32_t ob, uint32_t (&wa)[NC], uint32_t (&wb)[NC]) const {
        if constexpr (NC == 4) {
            if constexpr (kTrans) {
                ldsm_x4_t(oa + lane * 16, wa[0], wa[1], wa[2], wa[3]);
                ldsm_x4_t(ob + lane * 16, wb[0], wb[1], wb[2], wb[3]);
            } else {
                ldsm_x4(oa + lane * 16, wa[0], wa[1], wa[2], wa[3]);
                ldsm_x4(ob + lane * 16, wb[0], wb[1], wb[2], wb[3]);
            }
        } else {
            const uint32_t o = lane < 16 ? oa + lane * 16 : ob + (lane - 16) * 16;
            if constexpr (kTrans) ldsm_x4_t(o, wa[0], wa[1], wb[0], wb[1]);
            else ldsm_x4(o, wa[0], wa[1], wb[0], wb[1]);
        }
    }

    // The rows r0 .. r0 + 8 NT - 1 of a segment, by this warp, over its tiles. dual: the other group
    // of warps has other rows and takes every tile, too. KM: steps of 16 keys taken together.
    template <int NT, int KM>
    __device__ bool rows(const Seg& sg, int r0, bool dual, int t0, int nt) {
        const int gq = lane >> 2, tq = lane & 3;
        const int grp = w >> 2, sub = w & 3;
        constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;

        // queries: lane (gq, tq) has row gq of each column tile, columns 32 chunk + 8 tq ..
        uint32_t qb[KP][NT][NC][4];
        uint64_t F2[NT], qs2[NT][NG];  // of rows 2 tq and 2 tq + 1: factor of the products, the groups' sums of q
        int lim[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[NC][8];
            const size_t row = row_index(p, sg, min(r0 + n * 8 + gq, sg.nrow - 1));
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                if constexpr (kBF16) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row * D + ch * 32) + tq);
                    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[ch][2 * i] = bf16_lo_f(v[i]);
                        x[ch][2 * i + 1] = bf16_hi_f(v[i]);
                    }
                } else {
                    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + row * D + ch * 32) + 2 * tq;
                    const float4 u = __ldg(q), v = __ldg(q + 1);
                    x[ch][0] = u.x; x[ch][1] = u.y; x[ch][2] = u.z; x[ch][3] = u.w;
                    x[ch][4] = v.x; x[ch][5] = v.y; x[ch][6] = v.z; x[ch][7] = v.w;
                }
            }
            float qs[NG], top = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) qs[g] = 0.f;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    qs[ch / CPG] += x[ch][e];
                    top = fmaxf(top, fabsf(x[ch][e]));
                }
#pragma unroll
            for (int k = 1; k <= 2; k <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
#pragma unroll
                for (int g = 0; g < NG; ++g) qs[g] += __shfl_xor_sync(0xffffffffu, qs[g], k);
            }
            // the row times 2^-e lies below 2^14
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127 - 13, -100), 113);
            const float down = pow2i(-e), F = pow2i(e) * p.scale_log2;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch)
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // columns i and i + 4; the odd ones meet codes times 16
                    const float f = i & 1 ? down * 0.0625f : down;
                    const float a = x[ch][i] * f, b = x[ch][i + 4] * f;
                    qb[0][n][ch][i] = pack_f16(a, b);
                    if constexpr (KP == 2) {
                        const float2 h = unpack_f16(qb[0][n][ch][i]);
                        qb[1][n][ch][i] = pack_f16(a - h.x, b - h.y);
                    }
                }
            // what the lanes of the results need: rows 2 tq, 2 tq + 1 (lanes 8 tq and 8 tq + 4 have them)
            F2[n] = pk2(__shfl_sync(0xffffffffu, F, 8 * tq) * 16777216.f, __shfl_sync(0xffffffffu, F, 8 * tq + 4) * 16777216.f);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float s = qs[g] * p.scale_log2;
                qs2[n][g] = pk2(__shfl_sync(0xffffffffu, s, 8 * tq), __shfl_sync(0xffffffffu, s, 8 * tq + 4));
            }
            lim[n][0] = row_limit(p, sg, r0 + n * 8 + 2 * tq);
            lim[n][1] = row_limit(p, sg, r0 + n * 8 + 2 * tq + 1);
        }
        // keys beyond khi nobody sees; below klo + 1 everybody (of the rows that are there)
        int khi = sg.k0, klo = sg.k1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                khi = max(khi, lim[n][i]);
                if (r0 + n * 8 + 2 * tq + i < sg.nrow) klo = min(klo, lim[n][i]);
            }
        khi = __reduce_max_sync(0xffffffffu, khi);
        klo = __reduce_min_sync(0xffffffffu, klo);

        float R[NT][2], l[NT][2], L[NT][NG][2], o[NT][2 * NC][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                R[n][i] = -INFINITY;
                l[n][i] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) L[n][g][i] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        // the octets of this warp's 32 keys in a tile
        uint32_t at[4];
        {
            const int per = pp.slab >> 3;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int oct = sub * 4 + k;
                at[k] = (uint32_t)(oct / per * pp.slab_bytes) | ((uint32_t)(oct % per) << 20);
            }
        }
        const uint32_t v_codes = pp.slab * (D / 2), scales = pp.slab * D, v_scales = pp.slab * 4 * NG;

#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
            const bool own = dual || odd == grp;
            odd ^= 1;
            if (!own) {
                st.next();
                continue;
            }
            if (!wait(&c->full[st.s], st.ph)) return false;
            const uint32_t tile = st.s * C::TILE;
            const int kw = (t0 + j) * kKeyTile + sub * 32;  // first key of this warp's slice
#pragma unroll 1
            for (int h = 0; h < 2; h += KM) {
                const int kb = kw + h * 16;
                if (kb >= khi || kb + 16 * KM <= sg.k0) continue;
                const bool whole = kb >= sg.k0 && kb + 16 * KM <= klo;
                float s[KM][NT][4];
                uint32_t pv[KM][2][NG];  // (step, lowest) of the values of keys gq and gq + 8
                bool vis[KM][NT][4];
                uint32_t base_a[KM], base_b[KM];
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    // octets 2 (h + m) and 2 (h + m) + 1 of the slice
                    const uint32_t xa = KM == 2 ? at[2 * m] : h ? at[2] : at[0], xb = KM == 2 ? at[2 * m + 1] : h ? at[3] : at[1];
                    const uint32_t sa = smem + tile + (xa & 0xfffffu), sb = smem + tile + (xb & 0xfffffu);
                    const uint32_t ia = xa >> 20, ib = xb >> 20;
                    base_a[m] = sa + ia * (8 * D / 2);
                    base_b[m] = sb + ib * (8 * D / 2);
                    uint32_t pk[2][NG];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const uint32_t ka = sa + scales + (ia * NG + g) * 32 + gq * 4, kb2 = sb + scales + (ib * NG + g) * 32 + gq * 4;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(pk[0][g]) : "r"(ka));
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(pk[1][g]) : "r"(kb2));
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(pv[m][0][g]) : "r"(ka + v_scales));
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(pv[m][1][g]) : "r"(kb2 + v_scales));
                    }
                    uint32_t wa[NC], wb[NC];
                    codes<false>(base_a[m], base_b[m], wa, wb);
                    uint64_t tot[NT][2], lo2[NT][2];  // of keys gq, gq + 8: rows 2 tq, 2 tq + 1
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float acc[NT][4];
#pragma unroll
                        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
                        for (int ch = g * CPG; ch < (g + 1) * CPG; ++ch) {
                            const uint32_t ua = wa[ch] >> 8, ub = wb[ch] >> 8;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int k = 0; k < KP; ++k) {
                                    mma_f16(acc[n], wa[ch] & M0, wb[ch] & M0, wa[ch] & M1, wb[ch] & M1, qb[k][n][ch][0], qb[k][n][ch][1]);
                                    mma_f16(acc[n], ua & M0, ub & M0, ua & M1, ub & M1, qb[k][n][ch][2], qb[k][n][ch][3]);
                                }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float step = bf16_lo_f(pk[i][g]), low = bf16_hi_f(pk[i][g]);
                            const uint64_t step2 = pk2(step, step), low2 = pk2(low, low);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint64_t a2 = pk2(acc[n][2 * i], acc[n][2 * i + 1]);
                                tot[n][i] = g == 0 ? mul2(a2, step2) : fma2(a2, step2, tot[n][i]);
                                lo2[n][i] = g == 0 ? mul2(low2, qs2[n][g]) : fma2(low2, qs2[n][g], lo2[n][i]);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) up2(fma2(tot[n][i], F2[n], lo2[n][i]), s[m][n][2 * i], s[m][n][2 * i + 1]);
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int key = kb + m * 16 + i * 8 + gq;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    vis[m][n][2 * i + e] = key >= sg.k0 && key < lim[n][e];
                                    if (!vis[m][n][2 * i + e]) s[m][n][2 * i + e] = -INFINITY;
                                }
                        }
                    }
                }
                // references: above score + log2 of the values' step (the largest of the groups')
                bool rise = false;
                float ev[KM][2];
#pragma unroll
                for (int m = 0; m < KM; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t x = pv[m][i][0] & 0x7f80u;
#pragma unroll
                        for (int g = 1; g < NG; ++g) x = max(x, pv[m][i][g] & 0x7f80u);
                        x = min(max(x >> 7, 27u), 227u);  // 2^-100 .. 2^100
                        ev[m][i] = __uint_as_float(0x4b000000u | x) - (8388608.f + 127.f);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) rise |= s[m][n][2 * i + e] + ev[m][i] > R[n][e] + kKv4Most;
                    }
                if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = -INFINITY;
#pragma unroll
                            for (int m = 0; m < KM; ++m)
                                top = fmaxf(top, fmaxf(s[m][n][e] + ev[m][0], s[m][n][2 + e] + ev[m][1]));
#pragma unroll
                            for (int k = 4; k <= 16; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                            if (top > R[n][e] + kKv4Most) {  // the same for all lanes of the row
                                top = ceilf(top) - kKv4Lift;
                                const float f = ex2(R[n][e] - top);
                                R[n][e] = top;
                                l[n][e] *= f;
#pragma unroll
                                for (int g = 0; g < NG; ++g) L[n][g][e] *= f;
#pragma unroll
                                for (int k = 0; k < 2 * NC; ++k) {
                                    o[n][k][e] *= f;
                                    o[n][k][2 + e] *= f;
                                }
                            }
                        }
                }
                // weights, and the products with the values' codes
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    uint32_t wf[KP][NT][NG][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float xr0 = R[n][0] == -INFINITY ? 0.f : R[n][0], xr1 = R[n][1] == -INFINITY ? 0.f : R[n][1];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float p0 = ex2(s[m][n][2 * i] - xr0), p1 = ex2(s[m][n][2 * i + 1] - xr1);
                            l[n][0] += p0;
                            l[n][1] += p1;
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                const float step = bf16_lo_f(pv[m][i][g]), low = bf16_hi_f(pv[m][i][g]);
                                float w0 = p0 * step, w1 = p1 * step;
                                if (whole) {
                                    L[n][g][0] = fmaf(p0, low, L[n][g][0]);
                                    L[n][g][1] = fmaf(p1, low, L[n][g][1]);
                                } else {  // scales that a row does not see may be no numbers
                                    if (vis[m][n][2 * i]) L[n][g][0] = fmaf(p0, low, L[n][g][0]);
                                    else w0 = 0.f;
                                    if (vis[m][n][2 * i + 1]) L[n][g][1] = fmaf(p1, low, L[n][g][1]);
                                    else w1 = 0.f;
                                }
                                const uint32_t u = pack_f16(w0, w1);
                                wf[0][n][g][i] = movm_t(u);
                                if constexpr (KP == 2) {
                                    const float2 hi = unpack_f16(u);
                                    wf[1][n][g][i] = movm_t(pack_f16(w0 - hi.x, w1 - hi.y));
                                }
                            }
                        }
                    }
                    uint32_t wa[NC], wb[NC];
                    codes<true>(base_a[m] + v_codes, base_b[m] + v_codes, wa, wb);
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch) {
                        const uint32_t ua = wa[ch] >> 8, ub = wb[ch] >> 8;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < KP; ++k) {
                                const uint32_t b0 = wf[k][n][ch / CPG][0], b1 = wf[k][n][ch / CPG][1];
                                mma_f16(o[n][2 * ch], wa[ch] & M0, wa[ch] & M1, wb[ch] & M0, wb[ch] & M1, b0, b1);
                                mma_f16(o[n][2 * ch + 1], ua & M0, ua & M1, ub & M0, ub & M1, b0, b1);
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_n(&c->empty[st.s], dual ? 1 : 2);
            st.next();
        }

        // the warps' parts meet, eight rows at a time
        float* ex = reinterpret_cast<float*>(gen + C::EXOFF);
#pragma unroll 1
        for (int n = 0; n < NT; ++n) {
            if (!sync()) return false;  // the exchange area is free
#pragma unroll
            for (int n2 = 0; n2 < NT; ++n2) {
                if (n2 != n) continue;
                uint64_t f2[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[n2][e];
#pragma unroll
                    for (int k = 4; k <= 16; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
                    // sums of any size come to [1, 2)
                    const int k = min(max((int)((__float_as_uint(sum) >> 23) & 255u) - 127, -100), 120);
                    const float f = sum > 0.f ? pow2i(-k) : 1.f;
                    f2[e] = pk2(f * 16777216.f, f * 1048576.f);
                    if (gq == 0) c->ml[w][2 * tq + e] = make_float2(sum > 0.f ? R[n2][e] + (float)k : R[n2][e], sum * f);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float x = L[n2][g][e];
#pragma unroll
                        for (int k2 = 4; k2 <= 16; k2 <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k2);
                        L[n2][g][e] = x * f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float fa, fb;
                    up2(f2[e], fa, fb);
                    float* row = ex + (w * 8 + 2 * tq + e) * C::EXROW + gq * 4;
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch) {
                        const float lw = L[n2][ch / CPG][e];
                        *reinterpret_cast<float4*>(row + ch * 32) =
                            make_float4(fmaf(o[n2][2 * ch][e], fa, lw), fmaf(o[n2][2 * ch][2 + e], fb, lw),
                                        fmaf(o[n2][2 * ch + 1][e], fa, lw), fmaf(o[n2][2 * ch + 1][2 + e], fb, lw));
                    }
                }
            }
            if (!sync()) return false;
            // dual: the rows of each group are its own
            const int wa = dual ? grp * 4 : 0, wn = dual ? 4 : kKv4Consumers;
            const int tid = (w - wa) * 32 + lane;
            for (int u = tid; u < 8 * (D / 4); u += wn * 32) {
                const int r = u / (D / 4), col = (u - r * (D / 4)) * 4, rr = r0 + n * 8 + r;
                if (rr >= sg.nrow) continue;
                float mm = -INFINITY, ll = 0.f;
                for (int k = wa; k < wa + wn; ++k) mm = fmaxf(mm, c->ml[k][r].x);
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                for (int k = wa; k < wa + wn; ++k) {
                    const float2 e = c->ml[k][r];
                    if (e.y == 0.f) continue;  // saw no key
                    const float f = e.x == mm ? 1.f : ex2(e.x - mm);
                    const float4 v = *reinterpret_cast<const float4*>(ex + (k * 8 + r) * C::EXROW + col);
                    ll += e.y * f;
                    acc[0] += v.x * f;
                    acc[1] += v.y * f;
                    acc[2] += v.z * f;
                    acc[3] += v.w * f;
                }
                put4(sg, rr, col, acc, ll);
                if (col == 0 && sg.prow >= 0) p.part_ml[sg.prow + rr] = make_float2(mm, ll);
            }
        }
        return true;
    }

    __device__ __forceinline__ void put4(const Seg& sg, int r, int col, const float* o, float l) {
        if (sg.prow >= 0) {
            *reinterpret_cast<float4*>(part_at(p, sg, r, col)) = make_float4(o[0], o[1], o[2], o[3]);
            return;
        }
        const float inv = l > 0.f ? 1.f / l : l;  // no key seen: 0; NaN stays
        const size_t at = row_index(p, sg, r) * D + col;
        if constexpr (kBF16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
                make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    }

    __device__ void run(int s0, int s1) {
        Seg nx = load_seg(&p.seg[s0]);
        for (int si = s0; si < s1; ++si) {
            const Seg sg = nx;
            if (si + 1 < s1) nx = load_seg(&p.seg[si + 1]);
            if (sg.nrow == 0) continue;
            const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
            bool ok;
            if (sg.nrow <= 8) ok = rows<1, 2>(sg, 0, false, t0, nt);
            else ok = rows<2, 1>(sg, sg.nrow > 16 ? (w >> 2) * 16 : 0, sg.nrow > 16, t0, nt);
            if (!ok) return;
        }
    }
};

template <bool kBF16, int D, int NG>
__global__ void __launch_bounds__(kKv4Threads, 1) art_attend_kv4_kernel(const __grid_constant__ AttendKv4Params pp) {
    using C = Kv4Cfg<D, NG>;
    extern __shared__ __align__(1024) unsigned char gen[];
    const AttendParams& p = pp.a;
    Kv4Ctrl<C::NS>* c = reinterpret_cast<Kv4Ctrl<C::NS>*>(gen + C::CTRL);
    const int w = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&c->full[i], 1);
            mbar_init(&c->empty[i], kKv4Consumers);
        }
        mbar_init(&c->cons, kKv4Consumers);
        mbar_init(&c->stall, 1);
        c->abort = 0;
        fence_mbar_init();
    }
    static_assert(sizeof(PlanScratch) <= C::CTRL, "the scratch lies in the tiles");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what ran before on the stream has ended
    if (w < kKv4Consumers) {
        int a, z;
        plan_share<kKv4Consumers * 32>(p, reinterpret_cast<PlanScratch*>(gen), a, z);
        if (threadIdx.x == 0) {
            c->seg0 = a;
            c->seg1 = z;
        }
    }
    fence_proxy_async_smem();  // the scratch's accesses before the copies over it
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel may be set up; it waits for this grid's end
    const int s0 = c->seg0, s1 = c->seg1;
    if (s0 >= s1) return;
    if (w == kKv4Consumers) {
        kv4_producer<D, NG>(pp, gen, c, s0, s1);
    } else if (!p.stall || wait_tc(&c->stall, 0u, &c->abort, p)) {
        Kv4Consumer<kBF16, D, NG> k{pp, p, c, smem_addr(gen), gen, w, lane};
        k.run(s0, s1);
    }
}

template <bool kBF16, int D, int NG>
cudaError_t launch_kv4(const AttendKv4Params& p, cudaStream_t st) {
    constexpr size_t smem = kv4_smem<D, NG>();
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    auto kernel = art_attend_kv4_kernel<kBF16, D, NG>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(p.a.ctas), dim3(kKv4Threads), smem, st, p);
}

// One translation unit for each head_dim and type.
cudaError_t launch_kv4_bf16_d128(const AttendKv4Params& p, int ng, cudaStream_t st);
cudaError_t launch_kv4_bf16_d64(const AttendKv4Params& p, int ng, cudaStream_t st);
cudaError_t launch_kv4_f32_d128(const AttendKv4Params& p, int ng, cudaStream_t st);
cudaError_t launch_kv4_f32_d64(const AttendKv4Params& p, int ng, cudaStream_t st);

}  // namespace art
