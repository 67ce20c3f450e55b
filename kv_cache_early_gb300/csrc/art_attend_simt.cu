// art_attend_simt.cu -- the segments of art_attend.cuh for fp32, on CUDA cores (the
// tensor cores would round the operands).
//
// A CTA takes the segments of its share one after another: up to 64 rows against
// 64 keys at a time, all in fp32. Thread (ty, tx) of 16 x 16 forms the scores of
// rows 4 ty .. 4 ty + 3 and keys tx + 16 j, and the output columns 4 tx + 64 j of
// the same rows; the running maximum and sum of a row live in the 16 threads of a
// half warp, so the weights need no block-wide barrier.
#include "art_attend_plan.cuh"

namespace art {

constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;
constexpr int kPStride = kSimtKeys + 4;

template <int D>
constexpr size_t simt_smem() {
    const size_t tiles = sizeof(float) * (size_t)(kItemRows * (D + 4) + 2 * kSimtKeys * (D + 4) + kItemRows * kPStride);
    return tiles > sizeof(PlanScratch) ? tiles : sizeof(PlanScratch);
}

__device__ __forceinline__ float f4(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int D>
__global__ void __launch_bounds__(kSimtThreads, 1) art_attend_simt_kernel(const AttendParams p) {
    constexpr int S = D + 4, CH = D / 4, OC = D / 64;
    extern __shared__ __align__(16) unsigned char smem[];
    float* sq = reinterpret_cast<float*>(smem);
    float* sk = sq + kItemRows * S;
    float* sv = sk + kSimtKeys * S;
    float* sp = sv + kSimtKeys * S;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what ran before on the stream has ended
    int s_begin, s_end;
    plan_share<kSimtThreads>(p, reinterpret_cast<PlanScratch*>(smem), s_begin, s_end);
    asm volatile("griddepcontrol.launch_dependents;");  // the merge kernel may be set up; it waits for this grid's end
    for (int si = s_begin; si < s_end; ++si) {
        const Seg sg = load_seg(&p.seg[si]);
        if (sg.nrow == 0) continue;
        __syncthreads();
        for (int c = tid; c < kItemRows * CH; c += kSimtThreads) {
            const int r = c / CH, ch = c - r * CH;
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < sg.nrow) {
                const size_t row = row_index(p, sg, r);
                u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + row * D) + ch);
            }
            *reinterpret_cast<float4*>(sq + r * S + ch * 4) = u;
        }
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
        int bad = 0;
        const int32_t* trow = p.block_table + (size_t)sg.table_row * p.max_pages;
        // the next 64 keys and values are on their way, in registers, while these are used
        constexpr int LD = kSimtKeys * CH / kSimtThreads;
        float4 nk[LD], nv[LD];
        auto fetch = [&](int kb) {
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                const int c = tid + i * kSimtThreads, r = c / CH, ch = c - r * CH, key = kb + r;
                nk[i] = nv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (key >= sg.k0 && key < sg.k1) {
                    int pg = __ldg(&trow[key / p.Ps]);
                    if (pg < 0 || pg >= p.num_pages) {  // the merge kernel zeroes the rows
                        bad = 1;
                        pg = 0;
                    }
                    const size_t row = ((size_t)pg * p.Hkv + sg.g) * p.Ps + (key & (p.Ps - 1));
                    nk[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.k) + row * D) + ch);
                    nv[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.v) + row * D) + ch);
                }
            }
        };
        fetch(sg.k0 / kSimtKeys * kSimtKeys);
        for (int kb = sg.k0 / kSimtKeys * kSimtKeys; kb < sg.k1; kb += kSimtKeys) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                const int c = tid + i * kSimtThreads, r = c / CH, ch = c - r * CH;
                *reinterpret_cast<float4*>(sk + r * S + ch * 4) = nk[i];
                *reinterpret_cast<float4*>(sv + r * S + ch * 4) = nv[i];
            }
            __syncthreads();
            if (kb + kSimtKeys < sg.k1) fetch(kb + kSimtKeys);
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
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
#pragma unroll
                for (int x = 8; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[i] = l[i] * a + sum;
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
        if (bad) {
            p.seg[si].bad = 1;
            atomicOr(&p.cta_status[blockIdx.x], ART_STATUS_BAD_PAGE);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= sg.nrow) continue;
            if (sg.prow >= 0) {
                if (tx == 0) p.part_ml[sg.prow + r] = make_float2(m[i], l[i]);
#pragma unroll
                for (int c = 0; c < OC; ++c)
                    *reinterpret_cast<float4*>(part_at(p, sg, r, c * 64 + tx * 4)) = o[i][c];
                continue;
            }
            const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
            const size_t row = row_index(p, sg, r);
#pragma unroll
            for (int c = 0; c < OC; ++c) {
                const size_t at = row * D + c * 64 + tx * 4;
                *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
                    make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv);
            }
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
