// art_attend_simt.cu -- the segments of art_attend.cuh for fp32, on CUDA cores (the
// tensor cores would round the operands).
//
// A CTA takes the segments of its share one after another, 64 keys at a time in shared
// memory, the next 64 on their way in registers. Two forms:
//
//   more than 8 rows: 64 rows against the 64 keys. Thread (ty, tx) of 16 x 16 forms the
//   scores of rows 4 ty .. 4 ty + 3 and keys tx + 16 j, and the output columns 4 tx + 64 j
//   of the same rows; the running maximum and sum of a row live in the 16 threads of a
//   half warp, so the weights need no block-wide barrier. Bound by FMAs and the shared
//   memory that feeds them (64 FMAs for 8 loads of 16 bytes).
//
//   8 rows or fewer (a sequence's own tokens): 64 rows would be padding. Each warp takes
//   8 of the 64 keys with its own running maximum, sum and outputs; four lanes share a
//   key's product, and the eight warps meet at the segment's end. Bound by the loads.
//
// Measured: 24 sequences behind a 4096-token prefix with up to 1024 own tokens (32/8
// heads, d 128) 130 us, with the first form alone 190; chunks of 300-500 tokens behind
// 0.1-3k (8/2 heads, d 128) 243 us, half of the FMA rate.
#include "art_attend_plan.cuh"

namespace art {

constexpr int kSimtThreads = 256;
constexpr int kSimtWarps = kSimtThreads / 32;
constexpr int kSimtKeys = kKeyTileF32;
constexpr int kPStride = kSimtKeys + 4;

template <int D>
constexpr size_t simt_smem() {
    const size_t tiles = sizeof(float) * (size_t)(kItemRows * (D + 4) + 2 * kSimtKeys * (D + 4) + kItemRows * kPStride);
    return tiles > sizeof(PlanScratch) ? tiles : sizeof(PlanScratch);
}

__device__ __forceinline__ float f4(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int D>
struct Simt {
    static constexpr int S = D + 4, CH = D / 4, LD = kSimtKeys * CH / kSimtThreads;
    const AttendParams& p;
    float *sq, *sk, *sv, *sp;
    int ps_log2;

    // This thread's part of 64 keys and values: rows tid / CH + i * (256 / CH), chunk tid % CH.
    // Their pages are read a step before them, so that no load waits for another.
    __device__ __forceinline__ void pages(const Seg& sg, int kb, int (&pg)[LD]) const {
        const int32_t* trow = p.block_table + (size_t)sg.table_row * p.max_pages;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int key = kb + (int)threadIdx.x / CH + i * (kSimtThreads / CH);
            pg[i] = key >= sg.k0 && key < sg.k1 ? __ldg(&trow[key >> ps_log2]) : 0;
        }
    }
    __device__ __forceinline__ void fetch(const Seg& sg, int kb, int (&pg)[LD], float4 (&nk)[LD], float4 (&nv)[LD],
                                          int& bad) const {
        const int ch = threadIdx.x % CH;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int key = kb + (int)threadIdx.x / CH + i * (kSimtThreads / CH);
            nk[i] = nv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (key >= sg.k0 && key < sg.k1) {
                const bool out = pg[i] < 0 || pg[i] >= p.num_pages;
                bad |= out;  // the merge kernel zeroes the rows
                const size_t row = (((size_t)(out ? 0 : pg[i]) * p.Hkv + sg.g) << ps_log2) + (key & (p.Ps - 1));
                nk[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.k) + row * D) + ch);
                nv[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.v) + row * D) + ch);
            }
        }
        pages(sg, kb + kSimtKeys, pg);
    }
    // Puts the fetched keys and values in place and fetches the next ones. Block-wide.
    __device__ __forceinline__ void step(const Seg& sg, int kb, int (&pg)[LD], float4 (&nk)[LD], float4 (&nv)[LD],
                                         int& bad) const {
        __syncthreads();
        const int r0 = threadIdx.x / CH, ch = threadIdx.x % CH;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int r = r0 + i * (kSimtThreads / CH);
            *reinterpret_cast<float4*>(sk + r * S + ch * 4) = nk[i];
            *reinterpret_cast<float4*>(sv + r * S + ch * 4) = nv[i];
        }
        __syncthreads();
        if (kb + kSimtKeys < sg.k1) fetch(sg, kb + kSimtKeys, pg, nk, nv, bad);
    }
    __device__ __forceinline__ void load_rows(const Seg& sg, int rows) const {
        for (int c = threadIdx.x; c < rows * CH; c += kSimtThreads) {
            const int r = c / CH, ch = c - r * CH;
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < sg.nrow)
                u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + row_index(p, sg, r) * D) + ch);
            *reinterpret_cast<float4*>(sq + r * S + ch * 4) = u;
        }
    }
    // Four columns of a row: finished, or a partial result.
    __device__ __forceinline__ void put(const Seg& sg, int r, int col, const float4& o, float l) const {
        if (sg.prow >= 0) {
            *reinterpret_cast<float4*>(part_at(p, sg, r, col)) = o;
            return;
        }
        const float inv = l > 0.f ? 1.f / l : l;  // no key seen: 0; NaN stays
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row_index(p, sg, r) * D + col) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }

    __device__ __forceinline__ void large(const Seg& sg, int& bad) const {
        float4 nk[LD], nv[LD];
        int pg[LD];
        pages(sg, sg.k0 / kSimtKeys * kSimtKeys, pg);
        fetch(sg, sg.k0 / kSimtKeys * kSimtKeys, pg, nk, nv, bad);
        __syncthreads();  // the segment before has done with the shared memory
        constexpr int OC = D / 64;
        const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
        int lim[4];
        float m[4], l[4];
        float4 o[4][OC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lim[i] = row_limit(p, sg, ty * 4 + i);
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < OC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        load_rows(sg, kItemRows);
#pragma unroll 1
        for (int kb = sg.k0 / kSimtKeys * kSimtKeys; kb < sg.k1; kb += kSimtKeys) {
            step(sg, kb, pg, nk, nv, bad);
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (ty * 4 + i) * S + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * S + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                        s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                        s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                        s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                    }
            }
            __syncwarp();  // the half warp's reads of the weights before have finished
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = kb + tx + 16 * j;
                    s[i][j] = key >= sg.k0 && key < lim[i] ? s[i][j] * p.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
                const float a = m[i] == -INFINITY ? 0.f : exp2f(m[i] - base);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = exp2f(s[i][j] - base);
                    sum += w;
                    sp[(ty * 4 + i) * kPStride + tx + 16 * j] = w;
                }
                l[i] = l[i] * a + sum;  // this thread's keys; the half warp's are added at the end
                m[i] = mn;
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    o[i][c].x *= a;
                    o[i][c].y *= a;
                    o[i][c].z *= a;
                    o[i][c].w *= a;
                }
            }
            __syncwarp();
#pragma unroll 2
            for (int k = 0; k < kSimtKeys; k += 4) {
                float4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(sp + (ty * 4 + i) * kPStride + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int c = 0; c < OC; ++c) {
                        const float4 v = *reinterpret_cast<const float4*>(sv + (k + kk) * S + c * 64 + tx * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x = f4(w[i], kk);
                            o[i][c].x = fmaf(x, v.x, o[i][c].x);
                            o[i][c].y = fmaf(x, v.y, o[i][c].y);
                            o[i][c].z = fmaf(x, v.z, o[i][c].z);
                            o[i][c].w = fmaf(x, v.w, o[i][c].w);
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            if (r >= sg.nrow) continue;
            if (tx == 0 && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(m[i], l[i]);
#pragma unroll
            for (int c = 0; c < OC; ++c) put(sg, r, c * 64 + tx * 4, o[i][c], l[i]);
        }
    }

    // R: rows computed (those from nrow on are zero)
    template <int R>
    __device__ __forceinline__ void small(const Seg& sg, int& bad) const {
        float4 nk[LD], nv[LD];
        int pg[LD];
        pages(sg, sg.k0 / kSimtKeys * kSimtKeys, pg);
        fetch(sg, sg.k0 / kSimtKeys * kSimtKeys, pg, nk, nv, bad);
        __syncthreads();  // the segment before has done with the shared memory
        constexpr int C = D / 32;  // columns of a lane
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, kk = lane >> 2, part = lane & 3, n = sg.nrow;
        float m[R], l[R], o[R][C];
        int lim[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            lim[r] = row_limit(p, sg, r);
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) o[r][c] = 0.f;
        }
        load_rows(sg, R);
#pragma unroll 1
        for (int kb = sg.k0 / kSimtKeys * kSimtKeys; kb < sg.k1; kb += kSimtKeys) {
            step(sg, kb, pg, nk, nv, bad);
            const int key = kb + w * 8 + kk;
            if (kb + w * 8 >= sg.k1 || kb + w * 8 + 8 <= sg.k0) continue;  // none of this warp's keys
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = 0.f;
            const float *krow = sk + (w * 8 + kk) * S + part * 4, *qrow = sq + part * 4;
#pragma unroll 2
            for (int d = 0; d < D; d += 16) {
                const float4 b = *reinterpret_cast<const float4*>(krow + d);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 a = *reinterpret_cast<const float4*>(qrow + r * S + d);
                    s[r] = fmaf(a.x, b.x, s[r]);
                    s[r] = fmaf(a.y, b.y, s[r]);
                    s[r] = fmaf(a.z, b.z, s[r]);
                    s[r] = fmaf(a.w, b.w, s[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
                s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
                s[r] = key >= sg.k0 && key < lim[r] ? s[r] * p.scale_log2 : -INFINITY;
                float mx = s[r];
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
                const float a = m[r] == -INFINITY ? 0.f : exp2f(m[r] - base);
                s[r] = exp2f(s[r] - base);
                l[r] = l[r] * a + s[r];  // of this lane's key, four times over; added up at the end
                m[r] = mn;
#pragma unroll
                for (int c = 0; c < C; ++c) o[r][c] *= a;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float v[C];
                const float* vrow = sv + (w * 8 + k) * S + lane * C;
#pragma unroll
                for (int c = 0; c < C; ++c) v[c] = vrow[c];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float x = __shfl_sync(0xffffffffu, s[r], k * 4);
#pragma unroll
                    for (int c = 0; c < C; ++c) o[r][c] = fmaf(x, v[c], o[r][c]);
                }
            }
        }
        __syncthreads();  // the last keys and values have been read: their place holds the warps' results
        float* ex = sk;   // [warp][row][D], then (m, l) of [warp][row]
        float2* ml = reinterpret_cast<float2*>(sp);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
            if (r >= n) continue;
            if (lane == 0) ml[w * R + r] = make_float2(m[r], l[r]);
#pragma unroll
            for (int c = 0; c < C; ++c) ex[(w * R + r) * D + lane * C + c] = o[r][c];
        }
        __syncthreads();
        for (int u = threadIdx.x; u < n * (D / 4); u += kSimtThreads) {
            const int r = u / (D / 4), col = (u - r * (D / 4)) * 4;
            float mm = -INFINITY, ll = 0.f;
            for (int k = 0; k < kSimtWarps; ++k) mm = fmaxf(mm, ml[k * R + r].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < kSimtWarps; ++k) {
                const float2 e = ml[k * R + r];
                if (e.y == 0.f) continue;  // saw no key
                const float f = exp2f(e.x - mm);
                const float4 v = *reinterpret_cast<const float4*>(ex + (k * R + r) * D + col);
                ll += e.y * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            put(sg, r, col, acc, ll);
            if (col == 0 && sg.prow >= 0) p.part_ml[sg.prow + r] = make_float2(mm, ll);
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kSimtThreads, 1) art_attend_simt_kernel(const AttendParams p) {
    static_assert(kSimtWarps * kSmallRowsF32 * D <= 2 * kSimtKeys * (D + 4), "the small form's exchange fits the tiles");
    extern __shared__ __align__(16) unsigned char smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what ran before on the stream has ended
    int s_begin, s_end;
    plan_share<kSimtThreads>(p, reinterpret_cast<PlanScratch*>(smem), s_begin, s_end);
    asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel may be set up; it waits for this grid's end
    float* f = reinterpret_cast<float*>(smem);
    const Simt<D> k{p, f, f + kItemRows * (D + 4), f + (kItemRows + kSimtKeys) * (D + 4), f + (kItemRows + 2 * kSimtKeys) * (D + 4),
              31 - __clz(p.Ps)};
    for (int si = s_begin; si < s_end; ++si) {
        const Seg sg = load_seg(&p.seg[si]);
        if (sg.nrow == 0) continue;
        int bad = 0;
        if (sg.nrow <= 4) k.template small<4>(sg, bad);
        else if (sg.nrow <= kSmallRowsF32) k.template small<kSmallRowsF32>(sg, bad);
        else k.large(sg, bad);
        if (bad) {
            p.seg[si].bad = 1;
            atomicOr(&p.cta_status[blockIdx.x], ART_STATUS_BAD_PAGE);
        }
    }
}

template <int D>
static cudaError_t launch_one(const AttendParams& p, cudaStream_t st) {
    constexpr size_t smem = simt_smem<D>();
    const cudaError_t e = cudaFuncSetAttribute(art_attend_simt_kernel<D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_after(art_attend_simt_kernel<D>, dim3(p.ctas), dim3(kSimtThreads), smem, st, p);
}

cudaError_t launch_attend_simt(const AttendParams& p, cudaStream_t st) {
    return p.D == 128 ? launch_one<128>(p, st) : launch_one<64>(p, st);
}

}  // namespace art
