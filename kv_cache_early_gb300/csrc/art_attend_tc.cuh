// art_attend_tc.cuh -- the segments of art_attend.cuh for bf16, on the tensor cores.
//
// One CTA per SM, 12 warps (168 registers a thread at most), and one shared-memory ring
// that K and V tiles of 128 keys stream through without a pause from segment to segment:
//
//   producer warp   resolves the tiles' pages (the ids of 32 pages at a time, one
//                   batch ahead) and copies each page by one tensor copy
//   issuer warp     issues the tcgen05 products of large segments
//   edge warp       zeroes rows of V in shared memory that are no keys of a segment
//   8 consumer warps: softmax, and the whole computation of small segments
//
// Large segments (more than 16 rows): 128 rows are one stream; S = Q K^T (128 x 128)
// and O (128 x d) are accumulators in tensor memory, and the weights P go back there
// as the bf16 operand of O += P V, over the first half of their S. A thread owns a
// row, so sums need no shuffles. Two streams run at once, one in the tensor cores
// while the other is in the softmax: the two row tiles of a segment with more than
// 128 rows, else the two halves of each key tile for its one row tile (their O meet
// in the epilogue: equal rows lie in equal lanes of tensor memory).
//
// Small segments (16 rows or fewer: one sequence's own tokens, drafted tokens) are
// bound by the copies; the tensor memory path would spend 128 rows on them. Each
// consumer warp takes 16 keys of every tile by itself (mma.sync 16 x 8 x 16 on the
// swizzled tile) with its own running maximum, sum and O, and the eight meet at the
// segment's end.
//
// Softmax: p = 2^(s c - m) with c = log2(e) / sqrt(d), s and the sums in fp32; m
// follows the row's maximum only when that has risen by far (small segments: by more
// than 2^8; large ones: when 64 weights add up to more than 2^16): p and l stay far
// from overflow, and O need not be rescaled for each new maximum.
//
// V is bf16 and both operands have one type, so p enters the product in bf16; its sum is
// taken before. With eight rows or fewer (a sequence's one token, a few drafted ones)
// what the rounding left of p takes the product's eight rows of padding: about 16 bits of p,
// as in the decode kernel, at no product more (64 sequences of one row 175.8 us without
// and 175.7 with it, 16 x 3-4 drafts 62.9 and 63.1). With more rows p is rounded once: a
// second product for 9 to 16 rows took 2 to 6 % (d 64, 2 to 16 rows: 50.1 us without, 51.1
// unrolled, 53.2 in a loop), for large segments 35 % on chunks of 1-2k tokens (360 and
// 488 us) and 18 % on a 32k prefix for 128 sequences (136 and 161). Against 64 bits on
// random data a result's error (rms, relative) is then 2.0e-3 to 2.3e-3; the output's own
// rounding alone makes 1.65e-3.
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
//
// Measured on a GB300: chunks of 1-2k tokens behind 0-8k (32/8 heads, d 128) 362 us a
// call, the tensor pipe 59 % active: a stream's chain softmax (1580 cycles) -> P V and
// Q K^T (1024) -> hand-overs (300) is 2900 cycles a tile of two streams, whose products
// take 2048. A 32k prefix for 128 sequences with 64-2047 own tokens each: 136 us,
// 5.5 TB/s over the main kernel. Drafts of 5 tokens for 16 sequences behind 1k-8k:
// 67 us, 5.7 TB/s while it streams.
#pragma once

#include "art_attend_plan.cuh"

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
constexpr float kRescale = 8.f;  // small segments: log2 units by which a row's maximum may lead its reference
constexpr float kMaxSum = 65536.f;  // large segments: the sum of 64 weights from which it moves

template <int NS>
struct alignas(16) TcCtrl {
    uint64_t full[NS], empty_t[NS], empty_s[NS];  // empty: after a large / a small segment's use
    uint64_t s_full[2], p_full[2], o_full[2], q_full, edge_go, edge_done, cons, fin, stall;
    float2 ml[kTcConsumers * kSmallRows > 128 ? kTcConsumers * kSmallRows : 128];  // (m, l) exchanged between warps
    float2 ml2[128];
    uint32_t tmem;
    int abort, seg0, seg1;
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

#define ART_IO8(a, o) "+f"(a[o]), "+f"(a[o + 1]), "+f"(a[o + 2]), "+f"(a[o + 3]), "+f"(a[o + 4]), "+f"(a[o + 5]), "+f"(a[o + 6]), "+f"(a[o + 7])

// 32 columns of the warp's 32 lanes: thread = lane, register = column. The registers
// are valid after tc_wait_ld on them (which no use of theirs can then pass).
__device__ __forceinline__ void tc_ld32(uint32_t t, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
        "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : ART_R8(r, 0), ART_R8(r, 8), ART_R8(r, 16), ART_R8(r, 24)
        : "r"(t));
}
// 16 columns, waited for
__device__ __forceinline__ void tc_ld16(uint32_t t, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : ART_R8(r, 0), ART_R8(r, 8)
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld(float* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : ART_IO8(r, 0), ART_IO8(r, 8), ART_IO8(r, 16), ART_IO8(r, 24)
                 :
                 : "memory");
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

template <int N>
__device__ __forceinline__ float row_max(const float* s) {
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < N; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[i], s[i + 1]);
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
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
// The long wait is a function of its own: inlined at every use it made the kernel
// several times larger than the instruction cache.
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* abort, unsigned long long wait_ns,
                                              int* status) {
    const unsigned long long t0 = global_ns();
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 64; ++k)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
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
__device__ __forceinline__ bool wait_tc(uint64_t* bar, uint32_t parity, int* abort, const AttendParams& p) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_long(bar, parity, abort, p.wait_ns, &p.cta_status[blockIdx.x]);
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
        const int pg = __ldg(&p.block_table[(size_t)sg.table_row * p.max_pages + key / p.Ps]);
        return pg < 0 || pg >= p.num_pages ? -2 : pg;
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
            if (__any_sync(0xffffffffu, ids == -2)) {  // outside the pool: page 0 instead, the merge kernel zeroes the rows
                if (lane == 0) {
                    p.seg[si].bad = 1;
                    atomicOr(&p.cta_status[blockIdx.x], ART_STATUS_BAD_PAGE);
                }
                if (ids == -2) ids = 0;
            }
            for (int t = 0; t < nb && ok; ++t) {
                const bool mine = lane / ppt == t && ids >= 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * prow * (D * 2);
                const int tb = (t0 + bt * tpb + t) * kKeyTile;
                const int in_tile = (lane - t * ppt) * prow;  // first row of this lane's page in the tile
                const int group = mine ? (int)((((long long)ids * p.Hkv + sg.g) * p.Ps + ((tb + in_tile) & (p.Ps - 1))) >> 3)
                                       : 0;
#pragma unroll 1
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
// The whole warp runs the loop on warp-uniform values and one elected lane issues.
// Written so, the descriptors stay in uniform registers and 8 products are issued in
// 70 cycles (the queue then holds them); issued by one lane of a divergent branch they
// take 400, and many times that when the consumer warps leave few issue slots.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// The keys of tile t of a segment, as rows [lo, hi) of the tile; where a border lies
// inside a 16-key step, that step's rows of V beyond it are zeroed.
__device__ __forceinline__ bool tile_rows(const Seg& sg, int t, int& lo, int& hi) {
    lo = max(sg.k0 - t * kKeyTile, 0);
    hi = min(sg.k1 - t * kKeyTile, kKeyTile);
    return ((lo | hi) & 15) != 0;
}

template <int D>
__device__ void tc_issuer(const AttendParams& p, uint32_t smem, TcCtrl<TcCfg<D>::NS>* c, uint32_t tmem_, int s0, int s1) {
    using C = TcCfg<D>;
    constexpr uint32_t kIdQK = tc_idesc(kKeyTile, false), kIdHalf = tc_idesc(kKeyTile / 2, false), kIdPV = tc_idesc(D, true);
    const uint32_t tmem = (uint32_t)uniform((int)tmem_);
    Stage<C::NS> st;  // first stage of the segment: K of tile j lies 2j stages on, V of tile j 2j + 1
    uint32_t ph_q = 0, ph_p = 0, ph_e = 0;  // ph_p: a bit per stream
    bool issued = false, ok = true;
    auto wait = [&](uint64_t* b, uint32_t ph) { return ok = wait_tc(b, ph, &c->abort, p); };
    // The descriptors of all stages follow from that of the first by addition (the
    // addresses stay below 2^18).
    const uint64_t qd0 = tc_desc(smem, 16, C::GRP), kd0 = tc_desc(smem + C::RING, 16, C::GRP),
                   vd0 = tc_desc(smem + C::RING, 1024, C::GRP);
    // two row tiles: S_x = Q_x K^T; one: S_x = Q_0 K^T over the keys of half x
    auto qk = [&](int x, bool dual, int stage) {
        const uint64_t qd = qd0 + (uint64_t)(dual ? x * (C::TILE >> 4) : 0);
        const uint64_t kd = kd0 + (uint64_t)(stage * (C::TILE >> 4) + (dual ? 0 : x * (8 * C::GRP >> 4)));
        const uint32_t d = tmem + 256 + x * 128, id = dual ? kIdQK : kIdHalf;
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int off = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
                tc_mma_ss(d, qd + off, kd + off, id, kk > 0);
            }
            tc_commit(&c->s_full[x]);
        }
        __syncwarp();
    };
    // O_x += P_x V over the 16-key steps [a, z) of the tile; P's columns start at step p0
    auto pv = [&](int x, int stage, int a, int z, int p0, bool acc) {
        const uint64_t vd = vd0 + (uint64_t)(stage * (C::TILE >> 4));
        const uint32_t d = tmem + x * 128, pp = tmem + 256 + x * 128 - p0 * 8;
        if (elect_one()) {
            if (a == 0 && z == kKeyTile / 16) {
#pragma unroll
                for (int kk = 0; kk < kKeyTile / 16; ++kk)
                    tc_mma_ts(d, pp + kk * 8, vd + (uint64_t)(kk * (2 * C::GRP >> 4)), kIdPV, acc || kk > 0);
            } else {
#pragma unroll 1
                for (int kk = a; kk < z; ++kk)
                    tc_mma_ts(d, pp + kk * 8, vd + (uint64_t)(kk * (2 * C::GRP >> 4)), kIdPV, acc || kk > a);
            }
        }
        __syncwarp();
    };
    auto commit = [&](uint64_t* b) {
        if (elect_one()) tc_commit(b);
        __syncwarp();
    };
    for (int si = s0; si < s1 && ok; ++si) {
        Seg sg = load_seg(&p.seg[si]);
        sg.nrow = uniform(sg.nrow);
        sg.k0 = uniform(sg.k0);
        sg.k1 = uniform(sg.k1);
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
        issued = true;
        Stage<C::NS> ks = st, vs = st;
        vs.next();
        if (!wait(&c->full[ks.s], ks.ph)) break;
        qk(0, dual, ks.s);
        qk(1, dual, ks.s);
        commit(&c->empty_t[ks.s]);
        uint32_t acc = 0;  // streams whose O holds something
        for (int j = 0; j < nt && ok; ++j) {
            ks.next();
            ks.next();
            int lo, hi;
            const bool edge = tile_rows(sg, t0 + j, lo, hi);
            const bool more = j + 1 < nt;
            // the operands first: they are seldom what is waited for
            if (!wait(&c->full[vs.s], vs.ph)) break;
            if (edge) {
                if (elect_one()) mbar_arrive(&c->edge_go);
                __syncwarp();
                if (!wait(&c->edge_done, ph_e)) break;
                ph_e ^= 1u;
            }
            if (more && !wait(&c->full[ks.s], ks.ph)) break;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (!wait(&c->p_full[x], (ph_p >> x) & 1u)) break;
                ph_p ^= 1u << x;
                tc_fence_after();
                int a = lo >> 4, z = (hi + 15) >> 4;
                if (!dual) {
                    a = max(a, x * 4);
                    z = min(z, x * 4 + 4);
                }
                pv(x, vs.s, a, z, dual ? 0 : x * 4, (acc >> x) & 1u);
                if (z > a) acc |= 1u << x;
                if (more) qk(x, dual, ks.s);
                else commit(&c->o_full[x]);
            }
            if (!ok) break;
            commit(&c->empty_t[vs.s]);
            if (more) commit(&c->empty_t[ks.s]);
            vs.next();
            vs.next();
        }
        if (!ok) break;
        st.skip(2 * nt);
    }
    // the products have finished before the tensor memory is given back
    if (issued) {
        commit(&c->fin);
        const unsigned long long w0 = global_ns();
        while (!__all_sync(0xffffffffu, mbar_try_wait(&c->fin, 0u)))
            if (__any_sync(0xffffffffu, global_ns() - w0 > kWaitLimitNs)) break;
    }
}

// ---------------------------------------------------------------------------
// edge warp (large segments): zeroes rows of V that are no keys of the segment, when
// the issuer, which has seen the tile arrive, asks for it
// ---------------------------------------------------------------------------
template <int D>
__device__ void tc_edges(const AttendParams& p, unsigned char* gen, TcCtrl<TcCfg<D>::NS>* c, int s0, int s1) {
    using C = TcCfg<D>;
    const int lane = threadIdx.x & 31;
    Stage<C::NS> st;
    uint32_t ph = 0;
    for (int si = s0; si < s1; ++si) {
        const Seg sg = load_seg(&p.seg[si]);
        if (sg.nrow == 0) continue;
        const int t0 = sg.k0 / kKeyTile, nt = (sg.k1 + kKeyTile - 1) / kKeyTile - t0;
        for (int j = 0; sg.nrow > kSmallRows && j < nt; j += nt > 1 ? nt - 1 : 1) {  // the first and the last tile
            int lo, hi;
            if (!tile_rows(sg, t0 + j, lo, hi)) continue;
            Stage<C::NS> v = st;
            v.skip(2 * j + 1);
            if (!wait_tc(&c->edge_go, ph, &c->abort, p)) return;
            ph ^= 1u;
            const int a = lo >> 4, z = (hi + 15) >> 4;  // steps with a key
            unsigned char* base = gen + C::RING + v.s * C::TILE;
            for (int i = lane; i < 32 * C::NH * 8; i += 32) {
                const int k = i / (C::NH * 8), col = i % (C::NH * 8);
                const int row = k < 16 ? a * 16 + k : (z - 1) * 16 + k - 16;
                if (row >= lo && row < hi) continue;
                *reinterpret_cast<uint4*>(base + (row >> 3) * C::GRP + (col >> 3) * 1024 + (row & 7) * 128 +
                                          (col & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->edge_done);
        }
        st.skip(2 * nt);
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

    __device__ __forceinline__ static float inverse(float l) { return l > 0.f ? 1.f / l : l; }  // 0 stays, NaN stays

    // Four columns of row r: finished, or a partial result.
    __device__ __forceinline__ void put4(const Seg& sg, int r, int col, const float* o, float l) {
        if (sg.prow >= 0) {
            *reinterpret_cast<float4*>(part_at(p, sg, r, col)) = make_float4(o[0], o[1], o[2], o[3]);
            return;
        }
        const float inv = inverse(l);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row_index(p, sg, r) * D + col) =
            make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    }

    // 32 columns of the warp's 32 rows, a row a thread. Partial results lie row by row for
    // each four columns, so that a warp's store is one run. Of finished rows, four lanes
    // exchange their 16-byte chunks and store 64 bytes of one row after the other.
    __device__ __forceinline__ void put32(const Seg& sg, int row0, int col, const float* o, float l) {
        if (sg.prow >= 0) {
            if (row0 + lane < sg.nrow)
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(part_at(p, sg, row0 + lane, col + i)) =
                        make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            return;
        }
        const float inv = inverse(l);
        uint32_t u[4][4];  // chunk, word
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[k][i] = pack_bf16(o[8 * k + 2 * i] * inv, o[8 * k + 2 * i + 1] * inv);
        // 4 x 4 transposition within the quad: lane q gets chunk q of its four rows
#pragma unroll
        for (int step = 1; step <= 2; step <<= 1) {
            const bool high = (lane & step) != 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k & step) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? u[k][i] : u[k + step][i], step);
                    if (high) u[k][i] = got;
                    else u[k + step][i] = got;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = row0 + (lane & ~3) + k;
            if (r < sg.nrow)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row_index(p, sg, r) * D + col + (lane & 3) * 8) =
                    make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
        }
    }

    // The row's 64 weights at t, and its D sums at t, times f (seldom). References are integers,
    // so f is a power of two and the weights are not rounded a second time.
    __device__ __noinline__ static void scale_weights(uint32_t t, float f) {
#pragma unroll 1
        for (int k = 0; k < 32; k += 16) {
            float v[16];
            tc_ld16(t + k, v);
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                u[i] = __float_as_uint(v[i]);
                u[i] = pack_bf16(bf16_lo_f(u[i]) * f, bf16_hi_f(u[i]) * f);
            }
            tc_st16(t + k, u);
        }
    }
    __device__ __noinline__ static void scale_sums(uint32_t t, float f) {
#pragma unroll 1
        for (int k = 0; k < D; k += 16) {
            float v[16];
            tc_ld16(t + k, v);
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i] * f);
            tc_st16(t + k, u);
        }
    }

    __device__ bool large(const Seg& sg, int t0, int nt) {
        const bool dual = sg.nrow > 128;
        const int x = w >> 2, quad = w & 3;
        if (!sync()) return false;  // the tiles of Q are free (small segments use them too)
        // Q: 16 bytes a lane, whole rows side by side
        {
            constexpr int CPR = D / 8, RPI = 32 / CPR, NB = 16;  // chunks of a row; rows of a warp's load; loads at once
            const int rows = dual ? 32 : 16, ch = lane % CPR;
#pragma unroll 1
            for (int i0 = 0; i0 < rows; i0 += NB * RPI) {
                uint4 u[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int r = w * rows + i0 + i * RPI + lane / CPR;
                    u[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (i0 + i * RPI < rows && r < sg.nrow)
                        u[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row_index(p, sg, r) * D) + ch);
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int r = w * rows + i0 + i * RPI + lane / CPR;
                    if (i0 + i * RPI < rows) *reinterpret_cast<uint4*>(gen + (r >> 3) * C::GRP + (ch >> 3) * 1024 + (r & 7) * 128 +
                                              (((ch & 7) ^ (r & 7)) << 4)) = u[i];
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->q_full);
        }
        const int first_row = (dual ? x * 128 : 0) + quad * 32, r = first_row + lane;  // the warp's, this thread's row
        const bool live = first_row < sg.nrow;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lanes + 256 + x * 128, tO = tmem + lanes + x * 128;
        // a row that sees no key here is computed as if it saw all, and reported as empty
        const int rlim = row_limit(p, sg, r);
        const bool none = rlim <= sg.k0;
        const int lim = none ? sg.k1 : rlim;
        const int wlim = (int)__reduce_min_sync(0xffffffffu, (unsigned)lim);
        float m = -INFINITY, l = 0.f, fO = 1.f;
        bool first = true;  // O holds nothing yet
        const int cols = dual ? kKeyTile : kKeyTile / 2;  // of S and P
        const uint64_t c2 = pk2(p.scale_log2, p.scale_log2), one = pk2(1.f, 1.f);
        for (int j = 0; j < nt; ++j) {
            if (!wait(&c->s_full[x], ph_s)) return false;
            ph_s ^= 1u;
            if (live) {
                tc_fence_after();
                const int tb = (t0 + j) * kKeyTile + (dual ? 0 : x * 64);  // the key of column 0
                const bool edge = tb < sg.k0 || tb + cols > wlim;
                const int lo = sg.k0 - tb, hi = lim - tb;
                // 64 columns at a time, one loop body for both halves (the instruction cache feeds
                // eight warps from it)
#pragma unroll 1
                for (int h = 0; h < cols; h += 64) {
                    float s[64];
                    tc_ld32(tS + h, s);
                    tc_ld32(tS + h + 32, s + 32);
                    tc_wait_ld(s);
                    tc_wait_ld(s + 32);
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (h + k < lo || h + k >= hi) s[k] = -INFINITY;
                        if (hi <= h && m == -INFINITY) m = 0.f;  // no key in this stream: any reference will do
                    }
                    // Steady state: no maximum is formed. Weights and their sum are taken against the
                    // row's reference m. A row that has none yet takes these columns' maximum beforehand
                    // (again 1); where a sum passes kMaxSum (or is not a number), m moves to it and the
                    // weights are formed once more (again 2). The sums are looked at after the first pass
                    // of either kind: a row without a reference must not hold its neighbours'. One
                    // correction is enough, what it moves has a sum of 64 at most.
                    float rowsum = m == -INFINITY ? INFINITY : 0.f;
                    for (int again = __any_sync(0xffffffffu, m == -INFINITY);;) {
                        if (again) {
                            const float top = ceilf(row_max<64>(s) * p.scale_log2);  // an integer: scale_weights
                            if (!(rowsum <= kMaxSum) && top > m) {
                                // a row that had a reference: what it has summed is scaled down
                                const float f = ex2(m - top);
                                l *= f;
                                fO *= f;
                                m = top;
                            }
                        }
                        const float nb = m == -INFINITY ? 0.f : -m;
                        const uint64_t b2 = pk2(nb, nb);
                        uint64_t sum[4] = {pk2(0.f, 0.f), pk2(0.f, 0.f), pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
                        for (int k = 0; k < 64; k += 32) {
                            uint32_t pw[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float e0, e1;
                                up2(fma2(pk2(s[k + 2 * i], s[k + 2 * i + 1]), c2, b2), e0, e1);
                                e0 = ex2(e0);
                                e1 = ex2(e1);
                                sum[i & 3] = fma2(pk2(e0, e1), one, sum[i & 3]);
                                pw[i] = pack_bf16(e0, e1);
                            }
                            tc_st16(tS + (h + k) / 2, pw);
                        }
                        float a[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) up2(sum[i], a[2 * i], a[2 * i + 1]);
                        rowsum = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
                        if (again == 2 || !__any_sync(0xffffffffu, !(rowsum <= kMaxSum))) break;
                        // a row that is not a number stays so: it asks for this once, and has a reference then
                        if (!__any_sync(0xffffffffu, !(rowsum <= kMaxSum) && l == l)) break;
                        if (rowsum != rowsum && m == -INFINITY) m = 0.f;
                        tc_wait_st();
                        again = 2;
                    }
                    l += rowsum;
                    if (__any_sync(0xffffffffu, fO != 1.f)) {
                        // what the row has summed: O, and the weights of the first half of this tile
                        tc_wait_st();
                        if (h) scale_weights(tS, fO);
                        if (!first) scale_sums(tO, fO);
                        fO = 1.f;
                    }
                }
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
        if (none) {
            m = -INFINITY;
            l = 0.f;
        }
        if (dual) {
            if (live) {
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    tc_ld32(tO + k, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i];
                    put32(sg, first_row, k, o, l);
                }
                if (r < sg.nrow && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(m, l);
                tc_fence_before();
            }
        } else {
            // the two halves' results of a row meet; each stream writes half of the columns. What a
            // warp has seen of its own stream's products must hold for the other stream's warps, which
            // read this O too: the fences on both sides of the barrier.
            (x ? c->ml2 : c->ml)[quad * 32 + lane] = make_float2(m, l);
            tc_fence_before();
            if (!sync()) return false;
            tc_fence_after();
            if (live) {
                const float2 e = c->ml[quad * 32 + lane], d = c->ml2[quad * 32 + lane];
                const bool he = e.y != 0.f, hd = d.y != 0.f;  // saw a key; otherwise O may hold anything
                const float mm = fmaxf(he ? e.x : -INFINITY, hd ? d.x : -INFINITY);
                const float fe = he ? ex2(e.x - mm) : 0.f, fd = hd ? ex2(d.x - mm) : 0.f;
                const float ll = (he ? e.y * fe : 0.f) + (hd ? d.y * fd : 0.f);
#pragma unroll 1
                for (int k = x * (D / 2); k < (x + 1) * (D / 2); k += 32) {
                    float o[32], o2[32];
                    tc_ld32(tmem + lanes + k, o);
                    tc_ld32(tmem + lanes + 128 + k, o2);
                    tc_wait_ld(o);
                    tc_wait_ld(o2);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = (he ? o[i] * fe : 0.f) + (hd ? o2[i] * fd : 0.f);
                    put32(sg, first_row, k, o, ll);
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
        const bool few = sg.nrow <= 8;  // the product's rows 8 to 15 hold what the weights' rounding left
#pragma unroll 1
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
                    const float fa = ua ? ex2(ma - ta) : 1.f, fb = few ? fa : ub ? ex2(mb - tb) : 1.f;
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
                    const uint32_t rest = pack_bf16(e0 - bf16_lo_f(pa[2 * n]), e1 - bf16_hi_f(pa[2 * n]));
                    if (few) pa[2 * n + 1] = rest;
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
            if (few) {
                o[i][0] += o[i][2];
                o[i][1] += o[i][3];
            }
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
            put4(sg, r, col, acc, ll);
            if (col == 0 && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(mm, ll);
        }
        return true;
    }

    // Brings a segment's queries into the L2, a row a thread: under the load of the copies
    // they take microseconds from memory.
    __device__ __forceinline__ void prefetch(const Seg& sg) {
        const int r = w * 32 + lane;
        if (r >= sg.nrow) return;
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + row_index(p, sg, r) * D;
#pragma unroll
        for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i));
    }

    __device__ void run(int s0, int s1) {
        Seg nx = load_seg(&p.seg[s0]);
        for (int si = s0; si < s1; ++si) {
            const Seg sg = nx;
            if (si + 1 < s1) {
                nx = load_seg(&p.seg[si + 1]);
                prefetch(nx);
            }
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
    const uint32_t smem = smem_addr(gen);
    if (smem & 1023u) {  // the swizzle goes by address bits
        if (threadIdx.x == 0) {
            p.cta_status[blockIdx.x] = ART_STATUS_INTERNAL;
            if (blockIdx.x == 0) p.info->ok = 0;
        }
        return;
    }
    TcCtrl<C::NS>* c = reinterpret_cast<TcCtrl<C::NS>*>(gen + C::CTRL);
    const int w = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
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
        mbar_init(&c->edge_go, 1);
        mbar_init(&c->edge_done, 1);
        mbar_init(&c->cons, kTcConsumers);
        mbar_init(&c->fin, 1);
        mbar_init(&c->stall, 1);
        c->abort = 0;
        fence_mbar_init();
    }
    static_assert(sizeof(PlanScratch) <= C::CTRL, "the scratch lies in the tiles");
    // the tensor memory takes some microseconds to be had: beside the plan
    if (w == kTcConsumers + 1) tc_alloc(&c->tmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what ran before on the stream has ended
    if (w < kTcConsumers) {
        int a, z;
        plan_share<kTcConsumers * 32>(p, reinterpret_cast<PlanScratch*>(gen), a, z);
        if (threadIdx.x == 0) {
            c->seg0 = a;
            c->seg1 = z;
        }
    }
    fence_proxy_async_smem();  // the scratch's accesses before the copies over it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel may be set up; it waits for this grid's end
    const uint32_t tmem = c->tmem;
    const int s0 = c->seg0, s1 = c->seg1;
    if (s0 >= s1) {
        // nothing to do
    } else if (w >= kTcConsumers) {
        if (w == kTcConsumers) tc_producer<D>(p, smem, c, &tk, &tv, s0, s1);
        else if (w == kTcConsumers + 1) tc_issuer<D>(p, smem, c, tmem, s0, s1);
        else if (w == kTcConsumers + 2) tc_edges<D>(p, gen, c, s0, s1);
    } else {
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
