// art_attend_kv4.cuh -- the segments of art_attend.cuh over a cache that is held in 4 bits.
//
// With K = low + step c in each group of columns (c the codes) the products need the codes only:
//     q . k_t = sum_g step_tg (sum_{j in g} q_j c_tj) + low_tg (sum_{j in g} q_j)
//     o_j     = sum_t (p_t step_tg) c_tj + p_t low_tg
// so codes are never turned into values: they enter the matrix product as fp16. Four bits moved to
// the lowest ones ARE the number code * 2^-24 (a denormal), moved to the next four code * 2^-20, so
// eight codes of a 32-bit word become four operand registers by four masks and a shift: the keys'
// of bf16 calls; 2^24 and the 16 of the odd ones go into queries and results. The products'
// sums take a denormal's place for that of 2^-14 and cut off what lies 2^24 below, which leaves
// about 17 bits beside the row's largest query column. The values' codes, and fp32 calls' keys', are taken less 8 (and low more by 8 step)
// by one more fp16 sum: all of one sign, their sums over many tokens are far larger than what is
// left of them (an fp32 decode of 100 to 4000 tokens was 3.9e-5 from the exact result without it,
// 8e-6 with denormals less 8, 2.2e-7 so).
//
// S^T = C Q^T and O^T = C^T W^T, keys or columns in the 16 rows of mma.sync 16 x 8 x 16, up to
// eight query rows in its columns, so no row of the product is padding where eight rows attend
// (GQA with 8 heads; 4 heads leave half). Keys' codes come by ldmatrix as they lie (a lane has 8
// columns of one key), values' codes by its transposed form (4 columns of two neighbouring
// tokens): both are operands after the masks. W = p step is rounded to fp16 (11 bits; fp32 calls
// take a second part for what is left, and split the queries too, so about 22 bits). Scores,
// weights, their sums and what is multiplied by low are fp32.
//
// Range: a row has a reference for its weights and one for each group's W. The weights' own, R, follows the scores:
// weights stay below 2^-20, so that sums of weights times lowest stay finite (kWeightLift). W's, a power of two F
// beside it (W = p F step), follows the maximum of score + log2(the group's step), so that W stays within fp16's range and
// keeps its bits in every group, however small beside the others; values without a step need no W. Parts meet with R
// and the sums as they are: a sum's exponent added to R would be lost where scores are beyond 2^24. Queries are scaled by a
// power of two to fp16's range.
//
// One CTA per SM, of 16 (decode) or 12 warps, which meet at barriers in shared memory only:
//   2 producers: page ids 32 at a time, one bulk copy for each slab of a page (art_kv4.cuh), into a ring of
//              tiles of 128 keys
//   queries    turns the next segment's queries into operands, in shared memory
//   consumers  12 (decode) or 8, in groups of four that take the tiles in turn, a warp 32 keys of each, with a
//              reference, sums and O of its own. Up to 8 rows: the queries in registers; up to 16: two column
//              tiles, for which the codes are taken apart once
//   a merger   joins the consumers' parts of a segment, eight rows at a time, and stores them, while the
//              consumers are at the next one
//
// Keys and values outside a segment's keys may be anything: codes are always finite numbers, and
// scales of keys that a row does not see are not used for it.
//
// Measured on a GB300 (32/8 heads, d 128, pages of 16, groups of 64): 64 sequences of 1 to 8192 tokens 66 us a call, the
// cache's bytes at 5.0 TB/s while the main kernel streams; 8 sequences of 30k to 131k (28/4 heads, pages of 64, groups of
// 128) 81 us, 5.7 TB/s. 16 keys of 8 rows take about 230 instructions of a warp (70 to take codes apart, 32 to centre,
// 16 products), which 12 warps issue in 0.47 us a tile of 128 keys; its bytes take 0.42. What made it fast (64 sequences, in
// the order of the steps; those between them are not listed):
//   a ring of whole groups' stages, 12 consumers instead of 8          97 -> 88 us
//   producer lanes side by side instead of a tile after the other      88 -> 80
//   helper warps that sleep, masks only in steps with an edge, 2^10 from a register  80 -> 74
//   two producer warps                                                76 -> 66
// References of their own for the weights and for each group's W, without which large and small groups went wrong, cost
// 65.2 -> 65.8 us (81 against 80 for the long ones, 65.8 against 62.8 for five drafts of 16 sequences with groups of 32).
// Without effect: more consumers (16), 32 keys at a time with 12, products in two chains, a longer ring.
#pragma once

#include <type_traits>

#include "art_attend_tc.cuh"
#include "art_kv4.cuh"

namespace art {

constexpr int kRowsKv4 = 16;  // rows of an item's tile
constexpr int kKv4Producers = 2;
// W's factor is set so that a row's largest W is 2^5 to 2^6, and moves when one reaches 2^14: fp16 holds 11 bits of
// whatever is within 2^-19 of the largest.
constexpr int kKv4Lift = 5;
constexpr uint32_t kMostW = 0x7400u;  // 2^14 in fp16
// A row's reference is set 28 to 29 above its largest score (in log2), and moves when one comes within 20: sums of weights
// times lowest are finite for 2^20 keys of whatever size, and for 2^30 of up to 2^117.
constexpr float kWeightLift = 28.f;
constexpr float kMostWeight = 0x1p-20f;
constexpr int kMostFactor = 126;        // F = 2^126 at most: its inverse is a normal number
constexpr float kNoReference = -3.40282347e38f;  // of a row that has seen no key, no score is lower: any key's weight passes the limit

struct AttendKv4Params {
    AttendParams a;
    const unsigned char* cache;
    int slab, slab_bytes, page_bytes, bf16;
    uint32_t f16_1024;  // 2^10 in fp16, twice
};

// kCons: consumer warps.
template <bool kBF16, int D, int NG, int kCons>
struct Kv4Cfg {
    static constexpr int THREADS = (kCons + 2 + kKv4Producers) * 32;
    static constexpr int NC = D / 32;                     // 32-column chunks
    static constexpr int KP = kBF16 ? 1 : 2;              // fp16 parts of a query and of a weight
    static constexpr int TILE = kKeyTile * (D + 8 * NG);  // bytes of a tile
    static constexpr int EXROW = D + 4;                   // floats of a row in the exchange area
    static constexpr int EX = kCons * 8 * EXROW * 4;
    static constexpr int QTILE = KP * NC * 512;           // bytes of the operands of 8 rows
    static constexpr int Q = kRowsKv4 / 8 * QTILE;
    static constexpr int NS0 = (224 * 1024 - EX - 2 * Q) / TILE;
    // Ring stages: a multiple of the groups, so that a group of warps always has the same stages. Copies land out
    // of order; a group that saw every other use of a stage would take the one before for its own.
    static constexpr int GROUPS = kCons / 4, NS = (NS0 < 16 ? NS0 : 16) / GROUPS * GROUPS;
    static constexpr int EXOFF = NS * TILE, QOFF = EXOFF + EX, CTRL = QOFF + 2 * Q;
};

template <int NS, int NG, int kCons>
struct alignas(16) Kv4Ctrl {
    uint64_t full[NS], empty[NS], q_full[2], q_free[2], ex_full, ex_free, stall;
    struct Rows {  // of a segment's queries: factor of the products, the groups' sums, limit
        float f[kRowsKv4], sum[NG][kRowsKv4];
        int lim[kRowsKv4];
    } rows[2];
    float2 ml[kCons][8];
    float f[NG < 4 || kCons > 8 ? 1 : kCons][2 * NG][8];  // F of a warp's rows, fp32 (Kv4Consumer::rows)
    int abort, seg0, seg1;
};

template <bool kBF16, int D, int NG, int kCons>
constexpr size_t kv4_smem() {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    return (size_t)C::CTRL + sizeof(Kv4Ctrl<C::NS, NG, kCons>);
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
__device__ __forceinline__ uint32_t add_f16(uint32_t a, uint32_t c) {  // two sums
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t max_f16(uint32_t a, uint32_t b) {  // of two pairs; no numbers are left out
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_s16(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint64_t lds64(uint32_t a) {
    uint64_t r;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void sts64(uint32_t a, uint64_t v) {
    asm volatile("st.shared.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
// wait_tc for warps that mostly wait: asleep between the looks, so that they leave the issue slots to others (with
// wait_tc's looks, a fifth of the kernel's instructions were theirs).
static __device__ __noinline__ bool wait_asleep(uint64_t* bar, uint32_t parity, int* abort, unsigned most, unsigned long long wait_ns,
                                                int* status) {
    const unsigned long long t0 = global_ns();
    for (unsigned nap = 32;;) {
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
        __nanosleep(nap);
        nap = min(nap * 2, most);
        const bool late = (threadIdx.x & 31) == 0 && global_ns() - t0 > wait_ns;
        if (__any_sync(0xffffffffu, late)) {
            if ((threadIdx.x & 31) == 0) {
                st_volatile_shared(abort, 1);
                atomicOr(status, ART_STATUS_TIMEOUT);
            }
            return false;
        }
        if (__any_sync(0xffffffffu, ld_volatile_shared(abort) != 0)) return false;
    }
}
__device__ __forceinline__ bool wait_asleep(uint64_t* bar, uint32_t parity, int* abort, unsigned most, const AttendParams& p) {
    return wait_asleep(bar, parity, abort, most, p.wait_ns, &p.cta_status[blockIdx.x]);
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ---------------------------------------------------------------------------
// producer warp
// ---------------------------------------------------------------------------
// A lane has a slab of a batch of tiles: it waits for its tile's stage and issues its copy, side by side
// with the others. (One tile after the other, a warp of few instructions, each waiting for the one
// before, was what bound the kernel: 0.4 us a tile alone, 0.7 beside busy consumers.) The copies of a warp are issued one
// after the other all the same, so kKv4Producers warps share a tile's: with pages of 16 tokens, eight copies a
// tile, 64 sequences of 4096 tokens took 76 us with
// one warp and 66 with two.
template <bool kBF16, int D, int NG, int kCons>
__device__ void kv4_producer(const AttendKv4Params& pp, unsigned char* gen, Kv4Ctrl<Kv4Cfg<kBF16, D, NG, kCons>::NS, NG, kCons>* c,
                             int s0, int s1, int which) {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    const AttendParams& p = pp.a;
    const int lane = threadIdx.x & 31;
    const int ppt = kKeyTile / pp.slab / kKv4Producers;  // slabs of a tile that are this warp's (1 .. 8)
    const int tpb = min(32 / ppt, C::NS);                // tiles of a batch: no two of them in one stage
    const int t = lane / ppt, in_tile = (lane - t * ppt) * kKv4Producers + which;  // this lane's tile of a batch, its slab of the tile
    const uint32_t dst0 = in_tile * pp.slab_bytes;
    auto ids_of = [&](const Seg& sg, int bt) -> int {  // page of this lane's slab of batch bt, -1 where it has none
        const int key = (sg.k0 / kKeyTile + bt * tpb + t) * kKeyTile + in_tile * pp.slab;
        if (t >= tpb || sg.nrow == 0 || key >= sg.k1 || key + pp.slab <= sg.k0) return -1;
        const int pg = __ldg(&p.block_table[(size_t)sg.table_row * p.max_pages + key / p.Ps]);
        return pg < 0 || pg >= p.num_pages ? -2 : pg;
    };
    int stage = 0, use = 0, tiles = 0;  // of the batch's first tile
    unsigned issued = 0;                // lanes that issued copies of a batch that was given up
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
            int s = stage + t, u = use;
            if (s >= C::NS) {
                s -= C::NS;
                ++u;
            }
            const int key = (t0 + bt * tpb + t) * kKeyTile + in_tile * pp.slab;
            const unsigned char* src = pp.cache + ((size_t)max(ids, 0) * p.Hkv + sg.g) * (size_t)pp.page_bytes +
                                       (size_t)((key & (p.Ps - 1)) / pp.slab) * pp.slab_bytes;
            bool todo = t < nb;
            for (int polls = 0;;) {
                // the lanes of a tile go by what the first of them sees: all of a tile's copies are issued, or none
                const bool mine = t < nb && (u == 0 || mbar_test_wait(&c->empty[s], (uint32_t)(u - 1) & 1u));  // no stage else
                const bool room = __shfl_sync(0xffffffffu, (int)mine, t * ppt) != 0;
                if (todo && room) {
                    if (ids >= 0) {
                        mbar_arrive_expect_tx(&c->full[s], (uint32_t)pp.slab_bytes);
                        bulk_g2s(gen + s * C::TILE + dst0, src, (uint32_t)pp.slab_bytes, &c->full[s]);
                    } else {
                        mbar_arrive(&c->full[s]);  // no key of the segment in this slab
                    }
                    todo = false;
                }
                const unsigned left = __ballot_sync(0xffffffffu, todo);
                if (!left) break;
                if (++polls == 2) {  // the long wait, by the whole warp for one lane's stage
                    polls = 0;
                    const int from = __ffs(left) - 1;
                    const int ls = __shfl_sync(0xffffffffu, s, from), lu = __shfl_sync(0xffffffffu, u, from);
                    if (!wait_asleep(&c->empty[ls], (uint32_t)(lu - 1) & 1u, &c->abort, 64u, p)) {
                        ok = false;
                        issued = __ballot_sync(0xffffffffu, t < nb && !todo);
                        break;
                    }
                }
            }
            if (!ok) break;
            tiles += nb;
            stage += nb;
            if (stage >= C::NS) {
                stage -= C::NS;
                ++use;
            }
            ids = more;
        }
        sg = nx;
    }
    // no copy of this CTA may be in flight when it ends: a lane waits for the last tile of its stage
    {
        const int back = (stage - 1 - lane + 2 * C::NS) % C::NS;  // tiles between the stage's last whole one and the last
        int k = tiles - 1 - back;
        const int given = (lane - stage + C::NS) % C::NS;  // its tile of the batch that was given up
        if (given < tpb && (issued >> (given * ppt) & 1u)) k = tiles + given;
        bool open = lane < C::NS && k >= 0;
        const unsigned long long w0 = global_ns();
        while (__any_sync(0xffffffffu, open)) {
            if (open && mbar_test_wait(&c->full[lane], (uint32_t)(k / C::NS) & 1u)) open = false;
            if (__any_sync(0xffffffffu, lane == 0 && global_ns() - w0 > kWaitLimitNs)) break;
        }
    }
}

// ---------------------------------------------------------------------------
// query warp
// ---------------------------------------------------------------------------
template <bool kBF16, int D, int NG, int kCons>
__device__ void kv4_queries(const AttendParams& p, unsigned char* gen, Kv4Ctrl<Kv4Cfg<kBF16, D, NG, kCons>::NS, NG, kCons>* c, int s0, int s1) {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    constexpr int NC = C::NC, CPG = NC / NG;
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    int k = 0;
    for (int si = s0; si < s1; ++si) {
        const Seg sg = load_seg(&p.seg[si]);
        if (sg.nrow == 0) continue;
        const int buf = k & 1;
        if (k >= 2 && !wait_asleep(&c->q_free[buf], (uint32_t)((k >> 1) - 1) & 1u, &c->abort, 128u, p)) return;
        ++k;
#pragma unroll 1
        for (int n = 0; n * 8 < sg.nrow; ++n) {
            // lane (gq, tq): row gq of the tile, columns 32 chunk + 8 tq ..
            float x[NC][8];
            const size_t row = row_index(p, sg, min(n * 8 + gq, sg.nrow - 1));
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
                    x[ch][0] = u.x, x[ch][1] = u.y, x[ch][2] = u.z, x[ch][3] = u.w;
                    x[ch][4] = v.x, x[ch][5] = v.y, x[ch][6] = v.z, x[ch][7] = v.w;
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
            for (int o = 1; o <= 2; o <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
                for (int g = 0; g < NG; ++g) qs[g] += __shfl_xor_sync(0xffffffffu, qs[g], o);
            }
            // the row times 2^-e lies below 2^14
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127 - 13, -100), 113);
            const float down = pow2i(-e);
            uint4* dst = reinterpret_cast<uint4*>(gen + C::QOFF + buf * C::Q + n * C::QTILE) + lane;
#pragma unroll
            for (int ch = 0; ch < NC; ++ch) {
                uint32_t u[C::KP][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // columns i and i + 4; the odd ones meet codes times 16
                    const float f = i & 1 ? down * 0.0625f : down;
                    const float a = x[ch][i] * f, b = x[ch][i + 4] * f;
                    u[0][i] = pack_f16(a, b);
                    if constexpr (C::KP == 2) {
                        const float2 h = unpack_f16(u[0][i]);
                        u[1][i] = pack_f16(a - h.x, b - h.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < C::KP; ++i) dst[(i * NC + ch) * 32] = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
            }
            if (tq == 0) {
                const int r = n * 8 + gq;
                c->rows[buf].f[r] = pow2i(e) * p.scale_log2 * (kBF16 ? 16777216.f : 1.f);
#pragma unroll
                for (int g = 0; g < NG; ++g) c->rows[buf].sum[g][r] = qs[g] * p.scale_log2;
                c->rows[buf].lim[r] = row_limit(p, sg, r);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->q_full[buf]);
    }
}

// ---------------------------------------------------------------------------
// merger warp
// ---------------------------------------------------------------------------
template <bool kBF16, int D, int NG, int kCons>
__device__ void kv4_merger(const AttendParams& p, unsigned char* gen, Kv4Ctrl<Kv4Cfg<kBF16, D, NG, kCons>::NS, NG, kCons>* c, int s0, int s1) {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    // A lane has a row and every fourth four columns (every eighth, where there are four rows or fewer): the eight lanes
    // that read side by side have the same columns of eight rows, which lie in different banks, and store 128 bytes
    // of a partial result.
    const int lane = threadIdx.x & 31;
    uint32_t ph = 0;
    Seg nx = load_seg(&p.seg[s0]);
    for (int si = s0; si < s1; ++si) {
        const Seg sg = nx;
        if (si + 1 < s1) nx = load_seg(&p.seg[si + 1]);
#pragma unroll 1
        for (int n = 0; n * 8 < sg.nrow; ++n) {
            if (!wait_asleep(&c->ex_full, ph, &c->abort, 128u, p)) return;
            ph ^= 1u;
            const int rl = sg.nrow - n * 8 <= 4 ? 2 : 3, r = lane & ((1 << rl) - 1), c0 = lane >> rl, rr = n * 8 + r;
            const float* ex = reinterpret_cast<const float*>(gen + C::EXOFF) + r * C::EXROW + c0 * 4;
            float f[kCons], mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int k = 0; k < kCons; ++k) mm = fmaxf(mm, c->ml[k][r].x);
#pragma unroll
            for (int k = 0; k < kCons; ++k) {
                const float2 ml = c->ml[k][r];
                f[k] = ml.y == 0.f ? 0.f : ex2(ml.x - mm);  // saw no key: its sums are zero
                ll = fmaf(ml.y, f[k], ll);
            }
            const float inv = ll > 0.f ? 1.f / ll : ll;  // no key seen: 0; NaN stays
            const bool mine = rr < sg.nrow, part = sg.prow >= 0;
            float* to = part && mine ? part_at(p, sg, rr, c0 * 4) : nullptr;
            const size_t row = mine && !part ? row_index(p, sg, rr) * D + c0 * 4 : 0;
            if (mine && part && c0 == 0) p.part_ml[sg.prow + rr] = make_float2(mm, ll);
#pragma unroll 2
            for (int i = 0; i < D / 4; i += 32 >> rl) {  // four columns each
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kCons; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(ex + k * 8 * C::EXROW + i * 4);
                    acc[0] = fmaf(v.x, f[k], acc[0]);
                    acc[1] = fmaf(v.y, f[k], acc[1]);
                    acc[2] = fmaf(v.z, f[k], acc[2]);
                    acc[3] = fmaf(v.w, f[k], acc[3]);
                }
                if (!mine) continue;
                if (part) {
                    *reinterpret_cast<float4*>(to + (size_t)i * 4 * sg.nrow) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                } else if constexpr (kBF16) {
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row + i * 4) =
                        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row + i * 4) =
                        make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->ex_free);
        }
    }
}

// ---------------------------------------------------------------------------
// consumer warps
// ---------------------------------------------------------------------------
template <bool kBF16, int D, int NG, int kCons>
struct Kv4Consumer {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    static constexpr int NC = C::NC, CPG = NC / NG, KP = C::KP;
    const AttendKv4Params& pp;
    const AttendParams& p;
    Kv4Ctrl<C::NS, NG, kCons>* c;
    uint32_t smem;
    unsigned char* gen;
    int w, lane;
    uint32_t k1024;
    uint32_t ph_ex = 0;
    int turn = 0;   // which group of four warps takes the next tile
    int segs = 0;   // segments so far
    bool ex_used = false;
    Stage<C::NS> st;

    __device__ __forceinline__ bool wait(uint64_t* b, uint32_t ph) { return wait_tc(b, ph, &c->abort, p); }

    // codes of two octets of tokens: a word a chunk of 32 columns. `oa`, `ob`: shared-memory addresses, this lane's
    // 16 bytes of each (head_dim 64: of one of them)
    template <bool kTrans>
    __device__ __forceinline__ static void codes(uint32_t oa, uint32_t ob, uint32_t (&wa)[NC], uint32_t (&wb)[NC]) {
        if constexpr (NC == 4) {
            if constexpr (kTrans) {
                ldsm_x4_t(oa, wa[0], wa[1], wa[2], wa[3]);
                ldsm_x4_t(ob, wb[0], wb[1], wb[2], wb[3]);
            } else {
                ldsm_x4(oa, wa[0], wa[1], wa[2], wa[3]);
                ldsm_x4(ob, wb[0], wb[1], wb[2], wb[3]);
            }
        } else {
            const uint32_t o = (threadIdx.x & 16) ? ob : oa;
            if constexpr (kTrans) ldsm_x4_t(o, wa[0], wa[1], wb[0], wb[1]);
            else ldsm_x4(o, wa[0], wa[1], wb[0], wb[1]);
        }
    }
    // the operand registers of a chunk: codes 0 | 1 (times 16) of octets a, b, then codes 2 | 3, as code * 2^-24, or
    // (kLess) less 8: 2^10 + code, by its bits, less 2^10 + 8. The bits of 2^10 come from a register (of the call's
    // parameters), since an instruction holds one constant only: a mask and they would be two.
    template <bool kLess>
    __device__ __forceinline__ void apart(uint32_t wa, uint32_t wb, uint32_t (&a0)[4], uint32_t (&a1)[4]) const {
        constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
        const uint32_t ua = wa >> 8, ub = wb >> 8, K = kLess ? k1024 : 0u;
        a0[0] = wa & M0 | K, a0[1] = wa & M1 | K, a0[2] = wb & M0 | K, a0[3] = wb & M1 | K;
        a1[0] = ua & M0 | K, a1[1] = ua & M1 | K, a1[2] = ub & M0 | K, a1[3] = ub & M1 | K;
        if constexpr (kLess)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a0[i] = add_f16(a0[i], i & 1 ? 0xe480e480u : 0xe408e408u);  // -1152, -1032
                a1[i] = add_f16(a1[i], i & 1 ? 0xe480e480u : 0xe408e408u);
            }
    }

    // A segment's rows, eight to each of NT tiles, by this warp over its keys. KM: steps of 16 keys taken together.
    template <int NT, int KM>
    __device__ bool rows(const Seg& sg, int t0, int nt) {
        const int gq = lane >> 2, tq = lane & 3, grp = w >> 2, sub = w & 3;
        const int buf = segs & 1;
        if (!wait(&c->q_full[buf], (uint32_t)(segs >> 1) & 1u)) return false;
        const uint32_t qaddr = smem + C::QOFF + buf * C::Q + lane * 16;
        constexpr bool kQRegs = NT == 1;  // the queries stay in registers
        uint32_t qr[kQRegs ? KP : 1][kQRegs ? NC : 1][4];
        if constexpr (kQRegs)
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int ch = 0; ch < NC; ++ch) lds128(qaddr + (k * NC + ch) * 512, qr[k][ch]);
        // Of several new tokens and four groups the queries' sums, and in fp32 the factors F, are read from shared memory.
        // Five drafts of 16 sequences, a pass in a graph: bf16 75.2 us with the sums in registers, 65.9 so, 3 more with F read
        // too; fp32 123 with F in registers, 101 so.
        constexpr bool kSums = NG < 4 || kCons > 8, kFRegs = kSums || kBF16;
        uint64_t F2[NT], qs2[kSums ? NT : 1][kSums ? NG : 1];  // of rows 2 tq and 2 tq + 1
        const uint32_t sum_addr = smem_addr(&c->rows[buf].sum[0][2 * tq]);
        int lim[NT][2], khi = sg.k0, klo = sg.k1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + 2 * tq;
            F2[n] = *reinterpret_cast<const uint64_t*>(&c->rows[buf].f[r]);
#pragma unroll
            for (int g = 0; g < (kSums ? NG : 0); ++g) qs2[n][g] = *reinterpret_cast<const uint64_t*>(&c->rows[buf].sum[g][r]);
            lim[n][0] = c->rows[buf].lim[r];
            lim[n][1] = c->rows[buf].lim[r + 1];
            // keys from khi on nobody sees; those below klo everybody (of the rows that are there)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                khi = max(khi, lim[n][i]);
                if (r + i < sg.nrow) klo = min(klo, lim[n][i]);
            }
        }
        khi = __reduce_max_sync(0xffffffffu, khi);
        klo = __reduce_min_sync(0xffffffffu, klo);

        float R[NT][2], l[NT][2], o[NT][2 * NC][4];
        const uint32_t f_addr = smem_addr(&c->f[kFRegs ? 0 : w][0][2 * tq]);
        uint64_t L2[NT][NG], W2[kFRegs ? NT : 1][kFRegs ? NG : 1];  // of rows 2 tq, 2 tq + 1: sums of weights times lowest; F
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                R[n][i] = kNoReference;
                l[n][i] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) L2[n][g] = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint64_t f = pk2(pow2i(kMostFactor), pow2i(kMostFactor));
                if constexpr (kFRegs) W2[n][g] = f;
                else if (gq == 0) sts64(f_addr + (n * NG + g) * 32, f);
            }
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        __syncwarp();
        // the octets of this warp's 32 keys in a tile, two to each 16 keys: its bytes of the keys' codes, and its
        // keys' scales; the second 16 keys lie dk, ds bytes on whatever the slab
        uint32_t kc[2], sc[2], dk, ds;
        {
            const int per = pp.slab >> 3;
            auto codes_at = [&](int oct) { return oct / per * pp.slab_bytes + oct % per * (4 * D); };
            auto scales_at = [&](int oct) { return oct / per * pp.slab_bytes + oct % per * (32 * NG); };
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                kc[i] = smem + codes_at(sub * 4 + i) + (NC == 4 ? lane : lane & 15) * 16;
                sc[i] = smem + pp.slab * D + scales_at(sub * 4 + i) + gq * 4;
            }
            dk = codes_at(sub * 4 + 2) - codes_at(sub * 4);
            ds = scales_at(sub * 4 + 2) - scales_at(sub * 4);
        }
        const uint32_t v_codes = pp.slab * (D / 2), v_scales = pp.slab * 4 * NG;

        // 16 KM keys from kb on. whole: every row sees all of them. ka .. sb: addresses of their first octets
        auto step = [&](auto whole_, int kb, const uint32_t ka0, const uint32_t kb0, const uint32_t sa0, const uint32_t sb0) {
            constexpr bool whole = decltype(whole_)::value;
            float s[KM][NT][4];
            uint32_t pv[KM][2][NG];  // (step, lowest) of the values of keys gq and gq + 8
            bool vis[KM][NT][4];
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                const uint32_t ka = ka0 + m * dk, kb2 = kb0 + m * dk, sa = sa0 + m * ds, sb = sb0 + m * ds;
                uint32_t pk[2][NG], wa[NC], wb[NC];
                codes<false>(ka, kb2, wa, wb);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    pk[0][g] = lds32(sa + g * 32);
                    pk[1][g] = lds32(sb + g * 32);
                    pv[m][0][g] = lds32(sa + v_scales + g * 32);
                    pv[m][1][g] = lds32(sb + v_scales + g * 32);
                }
                uint64_t tot[NT][2], lo2[NT][2];  // of keys gq, gq + 8: rows 2 tq, 2 tq + 1
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float acc[KP][NT][4];  // the parts apart: sums of the second are far smaller
#pragma unroll
                    for (int k = 0; k < KP; ++k)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[k][n][0] = acc[k][n][1] = acc[k][n][2] = acc[k][n][3] = 0.f;
#pragma unroll
                    for (int ch = g * CPG; ch < (g + 1) * CPG; ++ch) {
                        uint32_t a0[4], a1[4];
                        apart<!kBF16>(wa[ch], wb[ch], a0, a1);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < KP; ++k) {
                                uint32_t q4[4];
                                if constexpr (kQRegs) {
#pragma unroll
                                    for (int i = 0; i < 4; ++i) q4[i] = qr[k][ch][i];
                                } else {
                                    lds128(qaddr + n * C::QTILE + (k * NC + ch) * 512, q4);
                                }
                                mma_f16(acc[k][n], a0[0], a0[2], a0[1], a0[3], q4[0], q4[1]);
                                mma_f16(acc[k][n], a1[0], a1[2], a1[1], a1[3], q4[2], q4[3]);
                            }
                    }
                    uint64_t sum2[kSums ? 1 : NT];
                    if constexpr (!kSums)
#pragma unroll
                        for (int n = 0; n < NT; ++n) sum2[n] = lds64(sum_addr + (g * kRowsKv4 + n * 8) * 4);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float step = bf16_lo_f(pk[i][g]);
                        const float low = kBF16 ? bf16_hi_f(pk[i][g]) : fmaf(8.f, step, bf16_hi_f(pk[i][g]));
                        const uint64_t step2 = pk2(step, step), low2 = pk2(low, low);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float x = acc[0][n][2 * i], y = acc[0][n][2 * i + 1];
                            if constexpr (KP == 2) {
                                x += acc[1][n][2 * i];
                                y += acc[1][n][2 * i + 1];
                            }
                            const uint64_t a2 = pk2(x, y), qs = kSums ? qs2[kSums ? n : 0][kSums ? g : 0] : sum2[kSums ? 0 : n];
                            tot[n][i] = g == 0 ? mul2(a2, step2) : fma2(a2, step2, tot[n][i]);
                            lo2[n][i] = g == 0 ? mul2(low2, qs) : fma2(low2, qs, lo2[n][i]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) up2(fma2(tot[n][i], F2[n], lo2[n][i]), s[m][n][2 * i], s[m][n][2 * i + 1]);
                if constexpr (!whole) {
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
            // Weights, and weights times steps, against the references as they are; where one goes too far, the
            // references move and they are formed once more.
            float pr[KM][NT][4];
            auto factor = [&](int n, int g) -> uint64_t {
                if constexpr (kFRegs) return W2[n][g];
                else return lds64(f_addr + (n * NG + g) * 32);
            };
            auto weight = [&](int m, int n, int g, int i, float p0, float p1, float& w0, float& w1) {
                const float step = bf16_lo_f(pv[m][i][g]);
                up2(mul2(mul2(pk2(p0, p1), factor(n, g)), pk2(step, step)), w0, w1);
                if constexpr (!whole) {  // scales that a row does not see may be no numbers
                    if (!vis[m][n][2 * i]) w0 = 0.f;
                    if (!vis[m][n][2 * i + 1]) w1 = 0.f;
                }
            };
#pragma unroll 1
            for (bool again = false;; again = true) {
                float most = 0.f;
                uint32_t most_w = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < KM; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float p0 = ex2(s[m][n][2 * i] - R[n][0]), p1 = ex2(s[m][n][2 * i + 1] - R[n][1]);
                            pr[m][n][2 * i] = p0;
                            pr[m][n][2 * i + 1] = p1;
                            most = max3(most, p0, p1);  // no number: left out
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                float w0, w1;
                                weight(m, n, g, i, p0, p1, w0, w1);
                                most_w = max_f16(most_w, pack_f16(w0, w1));
                            }
                        }
                // a half of most_w that is kMostW or more comes to its sign
                const bool far = most > kMostWeight || ((most_w + (0x80008000u - kMostW * 0x10001u)) & 0x80008000u);
                if (again || !__any_sync(0xffffffffu, far)) break;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float up[2], a[2];  // R's move, 2 to the opposite of it
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = -INFINITY;
#pragma unroll
                        for (int m = 0; m < KM; ++m) top = fmaxf(top, fmaxf(s[m][n][e], s[m][n][2 + e]));
#pragma unroll
                        for (int k = 4; k <= 16; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                        const float r = fmaxf(R[n][e], ceilf(top) + kWeightLift);  // the same for all lanes of the row
                        up[e] = r - R[n][e];
                        a[e] = ex2(-up[e]);
                        R[n][e] = r;
                        l[n][e] *= a[e];
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g) L2[n][g] = mul2(L2[n][g], pk2(a[0], a[1]));
                    // F: up with R, which leaves W as it is, and down where the largest W would be too large
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float top[2] = {0.f, 0.f};  // weight times step
#pragma unroll
                        for (int m = 0; m < KM; ++m)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (whole || vis[m][n][2 * i + e])
                                        top[e] = fmaxf(top[e], ex2(s[m][n][2 * i + e] - R[n][e]) * bf16_lo_f(pv[m][i][g]));
                        uint32_t both = pack_bf16(top[0], top[1]);
#pragma unroll
                        for (int k = 4; k <= 16; k <<= 1) both = max_s16(both, __shfl_xor_sync(0xffffffffu, both, k));
                        float f[2], fix[2];
                        up2(factor(n, g), f[0], f[1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int x = e ? both >> 23 : both >> 7 & 255u;  // its exponent
                            const float most = __uint_as_float((uint32_t)min(kKv4Lift + 254 - x, kMostFactor + 127) << 23);
                            const float now = fminf(f[e] * ex2(up[e]), most);
                            const int by = (int)(__float_as_uint(now) - __float_as_uint(f[e])) >> 23;
                            fix[e] = ex2((float)by - up[e]);  // 1 where W stays
                            f[e] = now;
                        }
                        if constexpr (kFRegs) W2[n][g] = pk2(f[0], f[1]);
                        else {
                            __syncwarp();
                            if (gq == 0) sts64(f_addr + (n * NG + g) * 32, pk2(f[0], f[1]));
                            __syncwarp();
                        }
#pragma unroll
                        for (int k = 2 * CPG * g; k < 2 * CPG * (g + 1); ++k) {
                            o[n][k][0] *= fix[0];
                            o[n][k][1] *= fix[1];
                            o[n][k][2] *= fix[0];
                            o[n][k][3] *= fix[1];
                        }
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < KM; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float p0 = pr[m][n][2 * i], p1 = pr[m][n][2 * i + 1];
                        l[n][0] += p0;
                        l[n][1] += p1;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const float low = fmaf(8.f, bf16_lo_f(pv[m][i][g]), bf16_hi_f(pv[m][i][g]));
                            if constexpr (whole) {
                                L2[n][g] = fma2(pk2(p0, p1), pk2(low, low), L2[n][g]);
                            } else {
                                float x, y;
                                up2(L2[n][g], x, y);
                                if (vis[m][n][2 * i]) x = fmaf(p0, low, x);
                                if (vis[m][n][2 * i + 1]) y = fmaf(p1, low, y);
                                L2[n][g] = pk2(x, y);
                            }
                        }
                    }
            // the products with the values' codes
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                uint32_t wa[NC], wb[NC];
                codes<true>(ka0 + m * dk + v_codes, kb0 + m * dk + v_codes, wa, wb);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t wf[KP][NT][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float w0, w1;
                            weight(m, n, g, i, pr[m][n][2 * i], pr[m][n][2 * i + 1], w0, w1);
                            const uint32_t u = pack_f16(w0, w1);
                            wf[0][n][i] = movm_t(u);
                            if constexpr (KP == 2) {
                                const float2 hi = unpack_f16(u);
                                wf[KP - 1][n][i] = movm_t(pack_f16(w0 - hi.x, w1 - hi.y));
                            }
                        }
#pragma unroll
                    for (int ch = g * CPG; ch < (g + 1) * CPG; ++ch) {
                        uint32_t a0[4], a1[4];
                        apart<true>(wa[ch], wb[ch], a0, a1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(o[n][2 * ch], a0[0], a0[1], a0[2], a0[3], wf[0][n][0], wf[0][n][1]);
                            mma_f16(o[n][2 * ch + 1], a1[0], a1[1], a1[2], a1[3], wf[0][n][0], wf[0][n][1]);
                            if constexpr (KP == 2) {  // apart, as above
                                float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(x, a0[0], a0[1], a0[2], a0[3], wf[KP - 1][n][0], wf[KP - 1][n][1]);
                                mma_f16(y, a1[0], a1[1], a1[2], a1[3], wf[KP - 1][n][0], wf[KP - 1][n][1]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    o[n][2 * ch][i] += x[i];
                                    o[n][2 * ch + 1][i] += y[i];
                                }
                            }
                        }
                    }
                }
            }
        };

        // this group's tiles of the segment
        constexpr int GROUPS = C::GROUPS;
        int j = grp - turn + (grp < turn ? GROUPS : 0);
        Stage<C::NS> at = st;
        at.skip(j);
#pragma unroll 1
        for (; j < nt; j += GROUPS) {
            if (!wait(&c->full[at.s], at.ph)) return false;
            const uint32_t tile = at.s * C::TILE;
            const int kw = (t0 + j) * kKeyTile + sub * 32;  // first key of this warp's slice
            if (kw >= sg.k0 && kw + 32 <= klo) {
#pragma unroll 1
                for (int h = 0; h < 2; h += KM) {
                    const uint32_t ok = tile + h * dk, os = tile + h * ds;
                    step(std::true_type(), 0, kc[0] + ok, kc[1] + ok, sc[0] + os, sc[1] + os);
                }
            } else {
#pragma unroll 1
                for (int h = 0; h < 2; h += KM) {
                    const int kb = kw + h * 16;
                    if (kb >= khi || kb + 16 * KM <= sg.k0) continue;
                    const uint32_t ok = tile + h * dk, os = tile + h * ds;
                    step(std::false_type(), kb, kc[0] + ok, kc[1] + ok, sc[0] + os, sc[1] + os);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->empty[at.s]);
            at.s += GROUPS;
            if (at.s >= C::NS) {
                at.s -= C::NS;
                at.ph ^= 1u;
            }
        }
        st.skip(nt);
        turn = (turn + nt) % GROUPS;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->q_free[buf]);
        ++segs;

        // this warp's part, eight rows at a time
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n * 8 >= sg.nrow) break;
            float fa[NG][2], L[NG][2];
#pragma unroll
            for (int g = 0; g < NG; ++g) up2(L2[n][g], L[g][0], L[g][1]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if constexpr (kFRegs) up2(W2[n][g], fa[g][0], fa[g][1]);
                else up2(lds64(f_addr + (n * NG + g) * 32), fa[g][0], fa[g][1]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], k);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    fa[g][e] = __uint_as_float((254u << 23) - __float_as_uint(fa[g][e]));  // 1 / F
#pragma unroll
                    for (int k = 4; k <= 16; k <<= 1) L[g][e] += __shfl_xor_sync(0xffffffffu, L[g][e], k);
                }
            }
            if (ex_used) {
                if (!wait(&c->ex_free, ph_ex)) return false;
                ph_ex ^= 1u;
            }
            ex_used = true;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (gq == 0) c->ml[w][2 * tq + e] = make_float2(R[n][e], l[n][e]);
                float* row = reinterpret_cast<float*>(gen + C::EXOFF) + (w * 8 + 2 * tq + e) * C::EXROW + gq * 4;
#pragma unroll
                for (int ch = 0; ch < NC; ++ch) {
                    const float lw = L[ch / CPG][e], f = fa[ch / CPG][e], f16 = f * 0.0625f;
                    *reinterpret_cast<float4*>(row + ch * 32) =
                        make_float4(fmaf(o[n][2 * ch][e], f, lw), fmaf(o[n][2 * ch][2 + e], f16, lw),
                                    fmaf(o[n][2 * ch + 1][e], f, lw), fmaf(o[n][2 * ch + 1][2 + e], f16, lw));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->ex_full);
        }
        return true;
    }

    template <int KM, bool kDecode>
    __device__ void run(int s0, int s1) {
        Seg nx = load_seg(&p.seg[s0]);
        for (int si = s0; si < s1; ++si) {
            const Seg sg = nx;
            if (si + 1 < s1) nx = load_seg(&p.seg[si + 1]);
            if (sg.nrow == 0) continue;
            const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
            bool ok;
            if (kDecode || sg.nrow <= 8) ok = rows<1, KM>(sg, t0, nt);
            else if constexpr (!kDecode) ok = rows<2, 1>(sg, t0, nt);
            if (!ok) return;
        }
    }
};

// kDecode: one token of each sequence, so no item has more than 8 rows.
template <bool kBF16, int D, int NG, int kCons, int KM, bool kDecode>
__global__ void __launch_bounds__((kCons + 2 + kKv4Producers) * 32, 1) art_attend_kv4_kernel(const __grid_constant__ AttendKv4Params pp) {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    extern __shared__ __align__(1024) unsigned char gen[];
    const AttendParams& p = pp.a;
    auto* c = reinterpret_cast<Kv4Ctrl<C::NS, NG, kCons>*>(gen + C::CTRL);
    const int w = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&c->full[i], kKeyTile / pp.slab);
            mbar_init(&c->empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->q_full[i], 1);
            mbar_init(&c->q_free[i], kCons);
        }
        mbar_init(&c->ex_full, kCons);
        mbar_init(&c->ex_free, 1);
        mbar_init(&c->stall, 1);
        c->abort = 0;
        fence_mbar_init();
    }
    static_assert(sizeof(PlanScratch) <= C::CTRL, "the scratch lies in the tiles");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what ran before on the stream has ended
    if (w < 8) {
        int a, z;
        plan_share<256>(p, reinterpret_cast<PlanScratch*>(gen), a, z);
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
    if (w < kCons) {
        if (p.stall && !wait_tc(&c->stall, 0u, &c->abort, p)) return;
        Kv4Consumer<kBF16, D, NG, kCons> k{pp, p, c, smem_addr(gen), gen, w, lane, pp.f16_1024};
        k.template run<KM, kDecode>(s0, s1);
    } else if (w == kCons) {
        kv4_merger<kBF16, D, NG, kCons>(p, gen, c, s0, s1);
    } else if (w == kCons + 1) {
        kv4_queries<kBF16, D, NG, kCons>(p, gen, c, s0, s1);
    } else {
        kv4_producer<kBF16, D, NG, kCons>(pp, gen, c, s0, s1, w - kCons - 2);
    }
}

template <bool kBF16, int D, int NG, int kCons, int KM, bool kDecode>
cudaError_t launch_kv4_as(const AttendKv4Params& p, cudaStream_t st) {
    using C = Kv4Cfg<kBF16, D, NG, kCons>;
    constexpr size_t smem = kv4_smem<kBF16, D, NG, kCons>();
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    auto kernel = art_attend_kv4_kernel<kBF16, D, NG, kCons, KM, kDecode>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(p.a.ctas), dim3(C::THREADS), smem, st, p);
}
template <bool kBF16, int D, int NG>
cudaError_t launch_kv4(const AttendKv4Params& p, cudaStream_t st) {
    return p.a.shared ? launch_kv4_as<kBF16, D, NG, 12, 1, true>(p, st) : launch_kv4_as<kBF16, D, NG, 8, 2, false>(p, st);
}

// One translation unit for each head_dim and type.
cudaError_t launch_kv4_bf16_d128(const AttendKv4Params& p, int ng, cudaStream_t st);
cudaError_t launch_kv4_bf16_d64(const AttendKv4Params& p, int ng, cudaStream_t st);
cudaError_t launch_kv4_f32_d128(const AttendKv4Params& p, int ng, cudaStream_t st);
cudaError_t launch_kv4_f32_d64(const AttendKv4Params& p, int ng, cudaStream_t st);

}  // namespace art
