// art_attend_tc.cuh -- the segments of art_attend.cuh for bf16, on the tensor cores.
//
// One CTA per SM, 12 warps, and one shared-memory ring that K and V tiles of 128
// keys stream through without a pause from segment to segment:
//
//   producer warp   resolves the tiles' pages (the ids of 32 pages at a time, one
//                   batch ahead) and copies each page by one tensor copy
//   issuer warp     one thread issues the tcgen05 products of large segments
//   8 consumer warps: softmax, and the whole computation of small segments
//
// Large segments (more than 16 rows): 128 rows are one stream; S = Q K^T (128 x 128)
// and O (128 x d) are accumulators in tensor memory, and the weights P go back there
// as the bf16 operand of O += P V, over the first half of their S. A thread owns a
// row, so maximum and sum need no shuffles. Two streams run at once, one in the
// tensor cores while the other is in the softmax: the two row tiles of a segment
// with more than 128 rows, else the even and the odd key tiles of its one row tile
// (their O meet in the epilogue: equal rows lie in equal lanes of tensor memory).
//
// Small segments (16 rows or fewer: one sequence's own tokens, drafted tokens) are
// bound by the copies; the tensor memory path would spend 128 rows on them. Each
// consumer warp takes 16 keys of every tile by itself (mma.sync 16 x 8 x 16 on the
// swizzled tile) with its own running maximum, sum and O, and the eight meet at the
// segment's end.
//
// Softmax: p = 2^(s c - m) with c = log2(e) / sqrt(d), s and the sums in fp32; m
// follows the row's maximum only when that has risen by more than 2^8 (p and l stay
// far from overflow, and O need not be rescaled for each new maximum). p is rounded
// to bf16 for the product, as V is bf16 and both operands have one type; its sum is
// taken before the rounding.
//
// Layout: a page's copy lands as [8-row group][64-column half][8 rows][128 bytes],
// 128B-swizzled. So 8-row groups follow one another at d * 16 bytes whatever the
// page size, and the same bytes are a K-major operand for Q K^T (rows = keys) and an
// MN-major one for P V (rows = columns of V).
//
// Rows of V outside the segment's keys are zeroed in shared memory before they meet
// p = 0 (they may hold NaN), and 16-key steps without a key are skipped.
//
// Every wait is bounded (AttendParams::wait_ns); see wait_tc.
#pragma once

#include "art_attend.cuh"

namespace art {

template <int D>
struct TcCfg {
    static constexpr int NH = D / 64;              // 128-byte halves of a row
    static constexpr int GRP = NH * 1024;          // bytes of an 8-row group
    static constexpr int TILE = kKeyTile * D * 2;  // bytes of a tile of K or V, and of 128 rows of Q
    static constexpr int NS = D == 128 ? 5 : 12;   // ring stages
    static constexpr int RING = 2 * TILE;          // after the two tiles of Q
    static constexpr int CTRL = RING + NS * TILE;
};

constexpr int kTcConsumers = 8, kTcThreads = (kTcConsumers + 4) * 32;  // three warpgroups
// Registers: 12 warps at 168 at launch (64512); then the two consumer warpgroups take
// 208 each (a row's 128 scores live in registers) and the third keeps 80: 63488.
constexpr int kRegConsumer = 208, kRegHelper = 80;
static_assert(128 * (2 * kRegConsumer + kRegHelper) <= kTcThreads * 168, "no more than the launch's registers");
constexpr int kSmallRows = 16;   // rows of a segment that the consumer warps take by themselves
constexpr float kRescale = 8.f;  // log2 units by which a row's maximum may lead its reference

template <int NS>
struct alignas(16) TcCtrl {
    uint64_t full[NS], empty_t[NS], empty_s[NS];  // empty: after a large / a small segment's use
    uint64_t s_full[2], p_full[2], o_full[2], q_full, cons, fin, stall;
    float2 ml[kTcConsumers * kSmallRows > 128 ? kTcConsumers * kSmallRows : 128];  // (m, l) exchanged between warps
    float2 ml2[128];
    uint32_t tmem;
    int abort;
};

template <int D>
constexpr size_t tc_smem() {
    return (size_t)TcCfg<D>::CTRL + sizeof(TcCtrl<TcCfg<D>::NS>);
}

// ---------------------------------------------------------------------------
// PTX wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int group, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(group), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tc_alloc(uint32_t* dst) {  // all 512 columns, whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t t) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// arrives on `bar` when every product issued so far by this thread has finished
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((int)acc)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((int)acc)
        : "memory");
}

#define ART_R8(a, o) "=f"(a[o]), "=f"(a[o + 1]), "=f"(a[o + 2]), "=f"(a[o + 3]), "=f"(a[o + 4]), "=f"(a[o + 5]), "=f"(a[o + 6]), "=f"(a[o + 7])
#define ART_F8(a, o) "f"(a[o]), "f"(a[o + 1]), "f"(a[o + 2]), "f"(a[o + 3]), "f"(a[o + 4]), "f"(a[o + 5]), "f"(a[o + 6]), "f"(a[o + 7])
#define ART_U8(a, o) "r"(a[o]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])

// 32 columns of the warp's 32 lanes: thread = lane, register = column
__device__ __forceinline__ void tc_ld32(uint32_t t, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
        "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : ART_R8(r, 0), ART_R8(r, 8), ART_R8(r, 16), ART_R8(r, 24)
        : "r"(t));
}
__device__ __forceinline__ void tc_st32(uint32_t t, const float* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
        "%24, %25, %26, %27, %28, %29, %30, %31};" ::ART_F8(r, 0),
        ART_F8(r, 8), ART_F8(r, 16), ART_F8(r, 24), "r"(t)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t t, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::ART_U8(r, 0),
        ART_U8(r, 8), "r"(t)
        : "memory");
}

// 2^x, flushing results below the normal range to zero (relative error 2^-22)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Shared-memory operand descriptor: 128B swizzle; lead, stride in bytes.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, int lead, int stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 operands, fp32 accumulator, M = 128; B K-major or MN-major.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Waits, the whole warp, for the phase with `parity`. Gives up after wait_ns (setting
// the status bit and the CTA's abort flag) or when another warp has: every warp then
// leaves its loop, and none is left in a barrier, since all waits are of this kind.
__device__ __forceinline__ bool wait_tc(uint64_t* bar, uint32_t parity, int* abort, const AttendParams& p) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        for (int k = 0; k < 16; ++k)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool late = (threadIdx.x & 31) == 0 && global_ns() - t0 > p.wait_ns;
        if (__any_sync(0xffffffffu, late)) {
            if ((threadIdx.x & 31) == 0) {
                st_volatile_shared(abort, 1);
                atomicOr(&p.hdr->status, ART_STATUS_TIMEOUT);
            }
            return false;
        }
        if (__any_sync(0xffffffffu, ld_volatile_shared(abort) != 0)) return false;
    }
}

__device__ __forceinline__ Seg load_seg(const Seg* s) {
    Seg r;
    const int4 a = __ldg(reinterpret_cast<const int4*>(s)), b = __ldg(reinterpret_cast<const int4*>(s) + 1),
               c = __ldg(reinterpret_cast<const int4*>(s) + 2);
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
    return r;
}

template <int NS>
struct Stage {  // position in the ring
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == NS) {
            s = 0;
            ph ^= 1u;
        }
    }
    __device__ __forceinline__ void skip(int n) {
        s += n % NS;
        ph ^= (uint32_t)(n / NS) & 1u;
        if (s >= NS) {
            s -= NS;
            ph ^= 1u;
        }
    }
};

// A row's place in q and out.
__device__ __forceinline__ size_t row_index(const AttendParams& p, const Seg& sg, int r) {
    const int R = sg.r0 + r, t = R / p.G;
    return (size_t)(sg.tok0 + t) * p.Hq + sg.g * p.G + (R - t * p.G);
}
// Keys that row r sees lie below this.
__device__ __forceinline__ int row_limit(const AttendParams& p, const Seg& sg, int r) {
    if (r >= sg.nrow) return sg.k0;
    if (sg.kind == kLimAll) return sg.k1;
    const int t = (sg.r0 + r) / p.G;
    return min(sg.k1, sg.kind == kLimCausal ? sg.lim0 + t : __ldg(&p.row_lim[sg.tok0 + t]));
}

// ---------------------------------------------------------------------------
// producer warp
// ---------------------------------------------------------------------------
template <int D>
__device__ void tc_producer(const AttendParams& p, uint32_t smem, TcCtrl<TcCfg<D>::NS>* c, const CUtensorMap* tk,
                            const CUtensorMap* tv, int s0, int s1) {
    using C = TcCfg<D>;
    const int lane = threadIdx.x & 31;
    const int prow = p.Ps < kKeyTile ? p.Ps : kKeyTile;  // rows of one copy
    const int ppt = kKeyTile / prow;                     // pages of a tile (16 at most)
    const int tpb = 32 / ppt;                            // tiles whose page ids the warp holds
    // this lane's page id of batch `bt` of a segment, -1 where it has none
    auto ids_of = [&](const Seg& sg, int bt) -> int {
        const int key = (sg.k0 / kKeyTile + bt * tpb) * kKeyTile + lane * prow;
        if (sg.nrow == 0 || key >= sg.k1 || key + prow <= sg.k0) return -1;
        return __ldg(&p.block_table[(size_t)sg.table_row * p.max_pages + key / p.Ps]);
    };
    Stage<C::NS> st;
    uint32_t used = 0, small_use = 0, ph_t = 0, ph_s = 0;  // per stage: filled once; last use; parities to wait for
    uint32_t filled_ph = 0;
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
        const bool small = sg.nrow <= kSmallRows;
        const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
        for (int bt = 0; bt * tpb < nt && ok; ++bt) {
            const int more = (bt + 1) * tpb < nt ? ids_of(sg, bt + 1) : ids_of(nx, 0);
            const int nb = min(tpb, nt - bt * tpb);
            for (int t = 0; t < nb && ok; ++t) {
                const bool mine = lane / ppt == t && ids >= 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * prow * (D * 2);
                const int tb = (t0 + bt * tpb + t) * kKeyTile;
                const int in_tile = (lane - t * ppt) * prow;  // first row of this lane's page in the tile
                const int group = mine ? (int)((((long long)ids * p.Hkv + sg.g) * p.Ps + ((tb + in_tile) & (p.Ps - 1))) >> 3)
                                       : 0;
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t bit = 1u << st.s;
                    if (used & bit) {
                        uint64_t* e = (small_use & bit) ? &c->empty_s[st.s] : &c->empty_t[st.s];
                        uint32_t& ph = (small_use & bit) ? ph_s : ph_t;
                        if (!wait_tc(e, (ph & bit) ? 1u : 0u, &c->abort, p)) {
                            ok = false;
                            break;
                        }
                        ph ^= bit;
                    }
                    used |= bit;
                    small_use = small ? small_use | bit : small_use & ~bit;
                    filled_ph = st.ph ? filled_ph | bit : filled_ph & ~bit;
                    if (lane == 0) mbar_arrive_expect_tx(&c->full[st.s], bytes);
                    __syncwarp();
                    if (mine)
                        tma_load_4d(smem + C::RING + st.s * C::TILE + (in_tile >> 3) * C::GRP, kv ? tv : tk, group,
                                    &c->full[st.s]);
                    st.next();
                }
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
// issuer warp (large segments)
// ---------------------------------------------------------------------------
template <int D>
__device__ void tc_issuer(const AttendParams& p, uint32_t smem, unsigned char* gen, TcCtrl<TcCfg<D>::NS>* c,
                          uint32_t tmem, int s0, int s1) {
    using C = TcCfg<D>;
    constexpr uint32_t kIdQK = tc_idesc(kKeyTile, false), kIdPV = tc_idesc(D, true);
    const int lane = threadIdx.x & 31;
    Stage<C::NS> st;           // next stage to take
    uint32_t ph_q = 0, ph_p = 0;  // ph_p: a bit per stream
    bool issued = false;
    auto wait = [&](uint64_t* b, uint32_t ph) { return wait_tc(b, ph, &c->abort, p); };
    // S_x = Q_(tile) K^T
    auto qk = [&](int x, int qt, const Stage<C::NS>& k) {
        if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 32;
                tc_mma_ss(tmem + 256 + x * 128, tc_desc(smem + qt * C::TILE + off, 16, C::GRP),
                          tc_desc(smem + C::RING + k.s * C::TILE + off, 16, C::GRP), kIdQK, kk > 0);
            }
            tc_commit(&c->s_full[x]);
        }
        issued = true;
    };
    // O_x += P_x V over the 16-key steps [a, z)
    auto pv = [&](int x, const Stage<C::NS>& v, int a, int z, bool acc) {
        if (lane == 0)
            for (int kk = a; kk < z; ++kk)
                tc_mma_ts(tmem + x * 128, tmem + 256 + x * 128 + kk * 8,
                          tc_desc(smem + C::RING + v.s * C::TILE + kk * 2 * C::GRP, 1024, C::GRP), kIdPV, acc || kk > a);
    };
    // rows of V of the first and last step that lie outside [lo, hi) of the tile
    auto zero_edges = [&](const Stage<C::NS>& v, int a, int z, int lo, int hi) {
        unsigned char* base = gen + C::RING + v.s * C::TILE;
        for (int i = lane; i < 32 * C::NH * 8; i += 32) {
            const int row = (i / (C::NH * 8)) < 16 ? a * 16 + i / (C::NH * 8) : (z - 1) * 16 + i / (C::NH * 8) - 16;
            if (row >= lo && row < hi) continue;
            const int col = i % (C::NH * 8);
            *reinterpret_cast<uint4*>(base + (row >> 3) * C::GRP + (col >> 3) * 1024 + (row & 7) * 128 + (col & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
    };
    for (int si = s0; si < s1; ++si) {
        const Seg sg = load_seg(&p.seg[si]);
        if (sg.nrow == 0) continue;
        const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
        if (sg.nrow <= kSmallRows) {
            st.skip(2 * nt);
            continue;
        }
        const bool dual = sg.nrow > 128;
        if (!wait(&c->q_full, ph_q)) break;
        ph_q ^= 1u;
        tc_fence_after();
        // K of tile j is at ring place 2j of the segment, V at 2j + 1
        auto at = [&](int n) {
            Stage<C::NS> x = st;
            x.skip(n);
            return x;
        };
        bool ok = true;
        const int ahead = dual ? 1 : 2;  // tiles whose S may be under way
        for (int j = 0; j < min(ahead, nt) && ok; ++j) {
            const Stage<C::NS> k = at(2 * j);
            if (!(ok = wait(&c->full[k.s], k.ph))) break;
            if (dual) {
                qk(0, 0, k);
                qk(1, 1, k);
            } else {
                qk(j, 0, k);
            }
            if (lane == 0) tc_commit(&c->empty_t[k.s]);
        }
        for (int j = 0; j < nt && ok; ++j) {
            const Stage<C::NS> v = at(2 * j + 1);
            if (!(ok = wait(&c->full[v.s], v.ph))) break;
            const int lo = max(sg.k0 - (t0 + j) * kKeyTile, 0), hi = min(sg.k1 - (t0 + j) * kKeyTile, kKeyTile);
            const int a = lo >> 4, z = (hi + 15) >> 4;
            if ((lo | hi) & 15) zero_edges(v, a, z, lo, hi);
            const int jn = j + ahead;
            const Stage<C::NS> k = at(2 * jn);
            for (int x = dual ? 0 : (j & 1); x < (dual ? 2 : (j & 1) + 1) && ok; ++x) {
                if (!(ok = wait(&c->p_full[x], (ph_p >> x) & 1u))) break;
                ph_p ^= 1u << x;
                tc_fence_after();
                pv(x, v, a, z, j >= (dual ? 1 : 2));
                if ((!dual || x == 1) && lane == 0) tc_commit(&c->empty_t[v.s]);
                if (jn < nt) {
                    if ((!dual || x == 0) && !(ok = wait(&c->full[k.s], k.ph))) break;
                    qk(x, dual ? x : 0, k);
                    if ((!dual || x == 1) && lane == 0) tc_commit(&c->empty_t[k.s]);
                } else if (dual && lane == 0) {
                    tc_commit(&c->o_full[x]);
                }
            }
        }
        if (!ok) break;
        if (!dual && lane == 0) {
            tc_commit(&c->o_full[0]);
            tc_commit(&c->o_full[1]);
        }
        st.skip(2 * nt);
    }
    // the products have finished before the tensor memory is given back
    if (issued) {
        if (lane == 0) tc_commit(&c->fin);
        const unsigned long long w0 = global_ns();
        while (!__all_sync(0xffffffffu, mbar_try_wait(&c->fin, 0u)))
            if (__any_sync(0xffffffffu, lane == 0 && global_ns() - w0 > kWaitLimitNs)) break;
    }
}

// ---------------------------------------------------------------------------
// consumer warps
// ---------------------------------------------------------------------------
template <int D>
struct TcConsumer {
    using C = TcCfg<D>;
    const AttendParams& p;
    TcCtrl<C::NS>* c;
    uint32_t smem;
    unsigned char* gen;
    uint32_t tmem;
    int w, lane;
    uint32_t ph_c = 0, ph_s = 0, ph_o = 0;
    Stage<C::NS> st;

    __device__ __forceinline__ bool wait(uint64_t* b, uint32_t ph) { return wait_tc(b, ph, &c->abort, p); }
    // all consumer warps
    __device__ __forceinline__ bool sync() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->cons);
        const bool ok = wait(&c->cons, ph_c);
        ph_c ^= 1u;
        return ok;
    }

    // N columns of output row r, from column col: finished, or a partial result
    template <int N>
    __device__ __forceinline__ void put(const Seg& sg, int r, int col, const float* o, float l) {
        if (sg.prow >= 0) {
            float* dst = p.part_o + (size_t)(sg.prow + r) * D + col;
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            return;
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key seen: 0; NaN stays
        uint16_t* dst = static_cast<uint16_t*>(p.out) + row_index(p, sg, r) * D + col;
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 8)
                *reinterpret_cast<uint4*>(dst + i) =
                    make_uint4(pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                               pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
        } else {
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
        }
    }

    __device__ bool large(const Seg& sg, int t0, int nt) {
        const bool dual = sg.nrow > 128;
        const int x = w >> 2, quad = w & 3;
        if (!sync()) return false;  // the tiles of Q are free (small segments use them too)
        // Q: 16 bytes a lane, whole rows side by side
        {
            const int rows = dual ? 32 : 16, first = w * rows;
            constexpr int CPR = D / 8;
            for (int i = lane; i < rows * CPR; i += 32) {
                const int r = first + i / CPR, ch = i % CPR;
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (r < sg.nrow)
                    u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row_index(p, sg, r) * D) + ch);
                *reinterpret_cast<uint4*>(gen + (r >> 3) * C::GRP + (ch >> 3) * 1024 + (r & 7) * 128 +
                                          (((ch & 7) ^ (r & 7)) << 4)) = u;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->q_full);
        }
        const int r = (dual ? x * 128 : 0) + quad * 32 + lane;  // this thread's row
        const bool live = (dual ? x * 128 : 0) + quad * 32 < sg.nrow;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lanes + 256 + x * 128, tO = tmem + lanes + x * 128;
        const int lim = row_limit(p, sg, r);
        const int wlim = (int)__reduce_min_sync(0xffffffffu, (unsigned)(r < sg.nrow ? lim : 0x7fffffff));
        float m = -INFINITY, l = 0.f;
        bool first = true;
        for (int j = dual ? 0 : x; j < nt; j += dual ? 1 : 2) {
            if (!wait(&c->s_full[x], ph_s)) return false;
            ph_s ^= 1u;
            if (live) {
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int k = 0; k < 128; k += 32) tc_ld32(tS + k, s + k);
                tc_wait_ld();
                const int tb = (t0 + j) * kKeyTile;
                if (tb < sg.k0 || tb + kKeyTile > wlim) {
                    const int lo = sg.k0 - tb, hi = lim - tb;
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k < lo || k >= hi) s[k] = -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int k = 4; k < 128; ++k) mx[k & 3] = fmaxf(mx[k & 3], s[k]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                const bool up = top > m + kRescale || (m == -INFINITY && top > m);
                const float f = up ? ex2(m - top) : 1.f;
                if (up) {
                    m = top;
                    l *= f;
                }
                if (!first && __any_sync(0xffffffffu, up)) {
                    float o[32];
                    for (int k = 0; k < D; k += 32) {
                        tc_ld32(tO + k, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= f;
                        tc_st32(tO + k, o);
                    }
                }
                const float nb = m == -INFINITY ? 0.f : -m;
                const uint64_t c2 = pk2(p.scale_log2, p.scale_log2), b2 = pk2(nb, nb), one = pk2(1.f, 1.f);
                uint64_t sum0 = pk2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int k = 0; k < 128; k += 32) {
                    uint32_t pw[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float e0, e1;
                        up2(fma2(pk2(s[k + 2 * i], s[k + 2 * i + 1]), c2, b2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        if (i & 1) sum1 = fma2(pk2(e0, e1), one, sum1);
                        else sum0 = fma2(pk2(e0, e1), one, sum0);
                        pw[i] = pack_bf16(e0, e1);
                    }
                    tc_st16(tS + k / 2, pw);
                }
                float a0, a1, b0, b1;
                up2(sum0, a0, a1);
                up2(sum1, b0, b1);
                l += (a0 + a1) + (b0 + b1);
                tc_wait_st();
                tc_fence_before();
            }
            first = false;
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->p_full[x]);
        }
        if (!wait(&c->o_full[x], ph_o)) return false;
        ph_o ^= 1u;
        tc_fence_after();
        if (dual) {
            if (live) {
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    tc_ld32(tO + k, o);
                    tc_wait_ld();
                    if (r < sg.nrow) put<32>(sg, r, k, o, l);
                }
                if (r < sg.nrow && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(m, l);
                tc_fence_before();
            }
        } else {
            // the even and the odd tiles' results of a row meet; each stream writes half of the columns
            (x ? c->ml2 : c->ml)[quad * 32 + lane] = make_float2(m, l);
            if (!sync()) return false;
            if (live) {
                const float2 e = c->ml[quad * 32 + lane], d = c->ml2[quad * 32 + lane];
                const float mm = fmaxf(e.x, d.x);
                const float fe = e.x == -INFINITY ? 0.f : ex2(e.x - mm), fd = d.x == -INFINITY ? 0.f : ex2(d.x - mm);
                const float ll = (e.y == 0.f ? 0.f : e.y * fe) + (d.y == 0.f ? 0.f : d.y * fd);
                const bool odd = nt > 1;  // otherwise the odd stream's O holds nothing
                for (int k = x * (D / 2); k < (x + 1) * (D / 2); k += 32) {
                    float o[32], o2[32];
                    tc_ld32(tmem + lanes + k, o);
                    if (odd) tc_ld32(tmem + lanes + 128 + k, o2);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = odd ? o[i] * fe + o2[i] * fd : o[i] * fe;
                    if (r < sg.nrow) put<32>(sg, r, k, o, ll);
                }
                if (x == 0 && r < sg.nrow && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(mm, ll);
                tc_fence_before();
            }
        }
        return true;
    }

    __device__ bool small(const Seg& sg, int t0, int nt) {
        constexpr int KS = D / 16, NT = D / 8;
        const int ra = lane >> 2, rb = ra + 8, cq = (lane & 3) * 2;
        uint32_t q[KS][4];
        {
            const uint16_t* base = static_cast<const uint16_t*>(p.q);
            const uint32_t *qa = reinterpret_cast<const uint32_t*>(base + row_index(p, sg, min(ra, sg.nrow - 1)) * D + cq),
                           *qb = reinterpret_cast<const uint32_t*>(base + row_index(p, sg, min(rb, sg.nrow - 1)) * D + cq);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                q[k][0] = __ldg(qa + k * 8);
                q[k][1] = __ldg(qb + k * 8);
                q[k][2] = __ldg(qa + k * 8 + 4);
                q[k][3] = __ldg(qb + k * 8 + 4);
            }
        }
        const int la = row_limit(p, sg, ra), lb = row_limit(p, sg, rb);
        float ma = -INFINITY, mb = -INFINITY, suma = 0.f, sumb = 0.f;
        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        const int mat = lane >> 3, mr = lane & 7;
        for (int j = 0; j < nt; ++j) {
            const int kb = (t0 + j) * kKeyTile + w * 16;  // first key of this warp's slice
            const bool any = kb + 16 > sg.k0 && kb < sg.k1;
            if (!wait(&c->full[st.s], st.ph)) return false;
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            if (any) {
                // matrices: keys 0-7 and 8-15 of the slice (mat / 2), column chunks 2k and 2k + 1 (mat % 2)
                const uint32_t base = smem + C::RING + st.s * C::TILE + (w * 2 + (mat >> 1)) * C::GRP + mr * 128;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t b0, b1, b2, b3;
                    const int ch = 2 * k + (mat & 1);
                    ldsm_x4(base + (ch >> 3) * 1024 + (((ch & 7) ^ mr) << 4), b0, b1, b2, b3);
                    mma_bf16(s[0], q[k][0], q[k][1], q[k][2], q[k][3], b0, b1);
                    mma_bf16(s[1], q[k][0], q[k][1], q[k][2], q[k][3], b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->empty_s[st.s]);
            st.next();
            uint32_t pa[4];
            if (any) {
                float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = kb + n * 8 + cq + e;
                        s[n][e] = key >= sg.k0 && key < la ? s[n][e] * p.scale_log2 : -INFINITY;
                        s[n][2 + e] = key >= sg.k0 && key < lb ? s[n][2 + e] * p.scale_log2 : -INFINITY;
                        ta = fmaxf(ta, s[n][e]);
                        tb = fmaxf(tb, s[n][2 + e]);
                    }
#pragma unroll
                for (int k = 1; k <= 2; k <<= 1) {
                    ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, k));
                    tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, k));
                }
                const bool ua = ta > ma + kRescale || (ma == -INFINITY && ta > ma);
                const bool ub = tb > mb + kRescale || (mb == -INFINITY && tb > mb);
                if (__any_sync(0xffffffffu, ua || ub)) {
                    const float fa = ua ? ex2(ma - ta) : 1.f, fb = ub ? ex2(mb - tb) : 1.f;
                    if (ua) ma = ta;
                    if (ub) mb = tb;
                    suma *= fa;
                    sumb *= fb;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        o[i][0] *= fa;
                        o[i][1] *= fa;
                        o[i][2] *= fb;
                        o[i][3] *= fb;
                    }
                }
                const float xa = ma == -INFINITY ? 0.f : ma, xb = mb == -INFINITY ? 0.f : mb;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float e0 = ex2(s[n][0] - xa), e1 = ex2(s[n][1] - xa), e2 = ex2(s[n][2] - xb), e3 = ex2(s[n][3] - xb);
                    suma += e0 + e1;
                    sumb += e2 + e3;
                    pa[2 * n] = pack_bf16(e0, e1);
                    pa[2 * n + 1] = pack_bf16(e2, e3);
                }
            }
            if (!wait(&c->full[st.s], st.ph)) return false;
            if (any) {
                const uint32_t tile = C::RING + st.s * C::TILE + w * 2 * C::GRP;
                if (kb < sg.k0 || kb + 16 > sg.k1) {  // values of no key: zero
                    for (int i = lane; i < 16 * C::NH * 8; i += 32) {
                        const int r = i / (C::NH * 8), col = i % (C::NH * 8);
                        if (kb + r >= sg.k0 && kb + r < sg.k1) continue;
                        *reinterpret_cast<uint4*>(gen + tile + (r >> 3) * C::GRP + (col >> 3) * 1024 + (r & 7) * 128 +
                                                  (col & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();  // before the copy that takes the stage next
                    __syncwarp();
                }
                // matrices: keys 0-7 and 8-15 (mat % 2), column chunks 2i and 2i + 1 (mat / 2), transposed
                const uint32_t base = smem + tile + (mat & 1) * C::GRP + mr * 128;
#pragma unroll
                for (int i = 0; i < NT / 2; ++i) {
                    uint32_t b0, b1, b2, b3;
                    const int ch = 2 * i + (mat >> 1);
                    ldsm_x4_t(base + (ch >> 3) * 1024 + (((ch & 7) ^ mr) << 4), b0, b1, b2, b3);
                    mma_bf16(o[2 * i], pa[0], pa[1], pa[2], pa[3], b0, b1);
                    mma_bf16(o[2 * i + 1], pa[0], pa[1], pa[2], pa[3], b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->empty_s[st.s]);
            st.next();
        }
#pragma unroll
        for (int k = 1; k <= 2; k <<= 1) {
            suma += __shfl_xor_sync(0xffffffffu, suma, k);
            sumb += __shfl_xor_sync(0xffffffffu, sumb, k);
        }
        if (!sync()) return false;  // the exchange area (the tiles of Q) is free
        float* ex = reinterpret_cast<float*>(gen) + w * (kSmallRows * D);
        if ((lane & 3) == 0) {
            c->ml[w * kSmallRows + ra] = make_float2(ma, suma);
            c->ml[w * kSmallRows + rb] = make_float2(mb, sumb);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (ra < sg.nrow) *reinterpret_cast<float2*>(ex + ra * D + i * 8 + cq) = make_float2(o[i][0], o[i][1]);
            if (rb < sg.nrow) *reinterpret_cast<float2*>(ex + rb * D + i * 8 + cq) = make_float2(o[i][2], o[i][3]);
        }
        if (!sync()) return false;
        for (int u = w * 32 + lane; u < sg.nrow * (D / 4); u += kTcConsumers * 32) {
            const int r = u / (D / 4), col = (u - r * (D / 4)) * 4;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int k = 0; k < kTcConsumers; ++k) mm = fmaxf(mm, c->ml[k * kSmallRows + r].x);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kTcConsumers; ++k) {
                const float2 e = c->ml[k * kSmallRows + r];
                if (e.y == 0.f) continue;  // saw no key
                const float f = ex2(e.x - mm);
                const float4 v = *reinterpret_cast<const float4*>(gen + ((size_t)k * kSmallRows * D + r * D + col) * 4);
                ll += e.y * f;
                acc[0] += v.x * f;
                acc[1] += v.y * f;
                acc[2] += v.z * f;
                acc[3] += v.w * f;
            }
            put<4>(sg, r, col, acc, ll);
            if (col == 0 && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(mm, ll);
        }
        return true;
    }

    __device__ void run(int s0, int s1) {
        for (int si = s0; si < s1; ++si) {
            const Seg sg = load_seg(&p.seg[si]);
            if (sg.nrow == 0) continue;
            const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
            if (sg.nrow <= kSmallRows) {
                if (!small(sg, t0, nt)) return;
            } else {
                if (!large(sg, t0, nt)) return;
                st.skip(2 * nt);
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    art_attend_tc_kernel(const AttendParams p, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv) {
    using C = TcCfg<D>;
    extern __shared__ __align__(1024) unsigned char gen[];  // no static shared memory: the window's start
    const int s0 = p.cta_first[blockIdx.x], s1 = p.cta_first[blockIdx.x + 1];
    if (s0 >= s1) return;
    const uint32_t smem = smem_addr(gen);
    if (smem & 1023u) {  // the swizzle goes by address bits
        if (threadIdx.x == 0) atomicOr(&p.hdr->status, ART_STATUS_INTERNAL);
        return;
    }
    TcCtrl<C::NS>* c = reinterpret_cast<TcCtrl<C::NS>*>(gen + C::CTRL);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&c->full[i], 1);
            mbar_init(&c->empty_t[i], 1);
            mbar_init(&c->empty_s[i], kTcConsumers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->s_full[i], 1);
            mbar_init(&c->p_full[i], 4);
            mbar_init(&c->o_full[i], 1);
        }
        mbar_init(&c->q_full, kTcConsumers);
        mbar_init(&c->cons, kTcConsumers);
        mbar_init(&c->fin, 1);
        mbar_init(&c->stall, 1);
        c->abort = 0;
        fence_mbar_init();
    }
    if (w == kTcConsumers + 1) tc_alloc(&c->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem;
    if (w >= kTcConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegHelper));
        if (w == kTcConsumers) tc_producer<D>(p, smem, c, &tk, &tv, s0, s1);
        else if (w == kTcConsumers + 1) tc_issuer<D>(p, smem, gen, c, tmem, s0, s1);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegConsumer));
        if (!p.stall || wait_tc(&c->stall, 0u, &c->abort, p)) {
            TcConsumer<D> k{p, c, smem, gen, tmem, w, lane};
            k.run(s0, s1);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == kTcConsumers + 1) tc_dealloc(tmem);
}

}  // namespace art
