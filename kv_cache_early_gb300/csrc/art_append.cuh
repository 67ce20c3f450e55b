// art_append.cuh -- what the kernels that append tokens to a paged cache share (art_append.cu
// has the mathematics, what bounds them and the figures): the call's parameters, its checks
// on the device, the tokens' places, the angles, and the rotation of rows.
#pragma once

#include "art_common.cuh"

namespace art {

constexpr int kAppendThreads = 256;
constexpr int kMaxRotHalf = 64;  // rot_dim / 2 at most (head_dim 128)

struct AppendParams {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // elements between tokens
    const int32_t* q_offsets;                // null: token b is sequence b's only new one
    const int32_t* positions;                // null: the token's place in the cache
    const int32_t* block_table;
    const int32_t* seq_lens;
    const float* inv_freq;
    void *q_out, *k_cache, *v_cache;
    WsHeader* hdr;
    int B, T, Hq, Hkv, Ps, max_pages, num_pages;
    int rot, interleaved;
    float scale;
};

template <bool kBF16>
struct Vec16 {  // 16 bytes of a row as fp32 values
    static constexpr int N = kBF16 ? 8 : 4;
    float x[N];
    __device__ __forceinline__ explicit Vec16(const uint4& u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kBF16) {
                x[2 * i] = bf16_lo_f(w[i]);
                x[2 * i + 1] = bf16_hi_f(w[i]);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
    __device__ __forceinline__ uint4 pack() const {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kBF16) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            else w[i] = __float_as_uint(x[i]);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The call's device data: offsets, lengths and the pages of the new tokens. One
// thread per sequence; sequences with many pages are shared out over its warp.
static __device__ void append_check(const AppendParams& p) {
    __shared__ int s_err;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s_err = 0;
    __syncthreads();
    int err = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAppendThreads) {
        const int b = b0 + tid;
        int first = 0, np = 0;
        if (b < p.B) {
            const int len = p.seq_lens[b];
            const int lo = p.q_offsets ? p.q_offsets[b] : b, hi = p.q_offsets ? p.q_offsets[b + 1] : b + 1;
            if (lo < 0 || hi < lo || hi > p.T) {
                err |= ART_STATUS_BAD_OFFSETS;
            } else if (len < hi - lo || (long long)len > (long long)p.max_pages * p.Ps) {
                err |= ART_STATUS_BAD_SEQLEN;
            } else if (hi > lo) {
                first = (len - (hi - lo)) / p.Ps;
                np = (len - 1) / p.Ps - first + 1;
            }
        }
        auto check = [&](int row, int col) {
            const int pg = p.block_table[(size_t)row * p.max_pages + col];
            if (pg < 0 || pg >= p.num_pages) err |= ART_STATUS_BAD_PAGE;
        };
        const bool few = np <= 4;
        if (few)
            for (int k = 0; k < np; ++k) check(b, first + k);
        unsigned many = __ballot_sync(0xffffffffu, !few);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            const int f = __shfl_sync(0xffffffffu, first, src), n = __shfl_sync(0xffffffffu, np, src);
            for (int k = lane; k < n; k += 32) check(b0 + (tid & ~31) + src, f + k);
        }
    }
    if (err) atomicOr(&s_err, err);
    __syncthreads();
    if (tid == 0) p.hdr->status = s_err;
}

// pos * f less whole turns as r + low, and its cosine and sine. The product is held as h + e
// (exact, by the fused product), 2 pi in three parts (Cody and Waite's reduction): with k = the nearest
// number of turns, h - k C1 is exact, k C2 is taken with its own rounding error, and what
// the sums round off (Knuth's two-sum) is kept; in 32-bit arithmetic the remainder
// r + low is within 2e-14 of the true one for products below 2^24. low enters to first order.
// Beyond, in 64 bits. (64-bit arithmetic for every angle cost 5 of 150 us: its pipe
// gives two results a clock and SM.)
__device__ __forceinline__ void turn_reduce(int pos, float f, float& r, float& low) {
    const float p = (float)pos, h = __fmul_rn(p, f);  // _rn: not contracted
    if (pos > -(1 << 24) && pos < (1 << 24) && fabsf(h) < 16777216.f) {
        constexpr float C1 = 6.2831854820251465f, C2 = -1.7484555314695172e-07f, C3 = -6.8604980400235275e-15f;
        const float e = fmaf(p, f, -h), k = rintf(h * 0.15915494f);
        const float r1 = fmaf(-k, C1, h), t = __fmul_rn(k, C2), tl = fmaf(k, C2, -t);
        const float a = r1 - t, ab = a - r1, ae = (r1 - (a - ab)) + (-t - ab);
        r = a + e;
        const float rb = r - a, re = (a - (r - rb)) + (e - rb);
        low = ((ae - tl) - k * C3) + re;
    } else {
        double y = (double)pos * (double)f;
        y -= 6.283185307179586476925 * rint(y * 0.159154943091895335769);
        r = (float)y;
        low = (float)(y - (double)r);
    }
}
__device__ __forceinline__ float2 turn_of(int pos, float f) {
    float r, low;
    turn_reduce(pos, f, r, low);
    float s, c;
    sincosf(r, &s, &c);
    return make_float2(c - low * s, s + low * c);
}

// The sequences, places and pages of tokens t0 .. t0 + ntok - 1. All threads of the block.
enum AppendState : int { kStateNone = 0, kStateBad = 1, kStateOk = 2 };
template <int kTok>
__device__ __forceinline__ void append_places(const AppendParams& p, int t0, int ntok, int* s_place, int* s_page,
                                              int* s_state) {
    const int tid = threadIdx.x;
    int b0 = t0;
    if (p.q_offsets) {
        b0 = 0;  // sequences that end at or before t0
        for (int base = 0; base < p.B; base += kAppendThreads)
            b0 += __syncthreads_count(base + tid < p.B && p.q_offsets[base + tid + 1] <= t0);
    }
    if (tid < ntok) {
        int b = p.q_offsets ? b0 : t0 + tid, i = 0, n = 1, state = kStateNone, page = -1, s = 0;
        if (p.q_offsets) {
            while (b < p.B && p.q_offsets[b + 1] <= t0 + tid) ++b;
            const int lo = b < p.B ? p.q_offsets[b] : 0, hi = b < p.B ? p.q_offsets[b + 1] : 0;
            const bool fine = lo >= 0 && hi <= p.T;  // flagged by block 0 where not
            i = t0 + tid - lo;
            n = fine ? hi - lo : 0;  // 0 too behind the last sequence
        }
        if (i >= 0 && i < n) {
            const int len = p.seq_lens[b];
            s = len - n + i;
            if (len >= n && (long long)len <= (long long)p.max_pages * p.Ps) {
                state = kStateOk;
                page = p.block_table[(size_t)b * p.max_pages + s / p.Ps];
                if (page < 0 || page >= p.num_pages) page = -1;
            } else {
                state = kStateBad;
            }
        }
        s_place[tid] = s;
        s_page[tid] = page;
        s_state[tid] = state;
    }
    __syncthreads();
}

// kVec: a row is taken in units of two 16-byte chunks: of a rotated row in pairs
// (j, j + rot_dim / 2) the chunks c and c + npair for c < npair; of what is left, and of
// other rows, a chunk of the first half and its like of the second. It needs rot_dim / 2
// (interleaved: rot_dim) to be a multiple of a chunk's elements; without it a thread takes
// an element, or a pair.
// kTok: tokens of a CTA. hkv: p.Hkv, or 0 where only the queries are rotated.
template <bool kBF16, int D, bool kVec, int kTok>
__device__ __forceinline__ void append_rows(const AppendParams& p, int hkv, int tile) {
    using E = Elem<kBF16>;
    constexpr int N = Vec16<kBF16>::N;
    constexpr int ROWB = D * E::kBytes;
    constexpr int PER = kVec ? D / N / 2 : D;          // units of a row
    constexpr int RPS = kAppendThreads / PER > 0 ? kAppendThreads / PER : 1;  // rows of a step of the CTA
    constexpr int PF = 3;                              // steps whose loads a thread has under way
    __shared__ float s_cos[kTok * kMaxRotHalf], s_sin[kTok * kMaxRotHalf];
    __shared__ int s_place[kTok], s_page[kTok], s_state[kTok];  // place in the cache; its page or -1; kState*
    const int t0 = tile * kTok, tid = threadIdx.x;
    const int ntok = min(kTok, p.T - t0);
    const int nq = p.q ? p.Hq : 0, half = p.rot / 2, rows = nq + 2 * hkv;
    const int npair = kVec && !p.interleaved ? half / N : 0;
    // row R of the CTA: token, then query heads, key heads, value heads
    auto split = [&](int R, int& tok, int& r) {
        tok = 0;
#pragma unroll
        for (int k = 1; k < kTok; ++k) tok += R >= k * rows;
        r = R - tok * rows;
    };
    auto src_of = [&](int tok, int r) -> const char* {
        const size_t t = (size_t)(t0 + tok);
        if (r < nq) return static_cast<const char*>(p.q) + (t * p.q_stride + (size_t)r * D) * E::kBytes;
        if (r < nq + hkv) return static_cast<const char*>(p.k) + (t * p.k_stride + (size_t)(r - nq) * D) * E::kBytes;
        return static_cast<const char*>(p.v) + (t * p.v_stride + (size_t)(r - nq - hkv) * D) * E::kBytes;
    };
    const int c = kVec ? tid % PER : 0;
    // the unit's chunks; neighbouring threads take neighbouring chunks, so that each access
    // of a warp is of whole 32-byte sectors (two neighbours a thread: 7 chunks of 1-4000
    // tokens, interleaved pairs in half a head, 49 us against 45)
    auto chunks = [&](bool turned, int& ca, int& cb) {
        const int n = turned ? npair : 0;
        ca = c < n ? c : c + n;
        cb = c < n ? c + n : c + PER;
    };
    uint4 a[PF], b2[PF];
    auto load = [&](int R0) {
#pragma unroll
        for (int k = 0; k < PF; ++k) {
            const int R = R0 + k * RPS;
            if (R >= ntok * rows) continue;
            int tok, r, ca, cb;
            split(R, tok, r);
            chunks(r < nq + hkv, ca, cb);
            const uint4* src = reinterpret_cast<const uint4*>(src_of(tok, r));
            a[k] = src[ca];
            b2[k] = src[cb];
        }
    };
    // before it is known which sequence holds the tokens, or whether any does: behind the loads of
    // the first and the last offset, prompts took 139.6 us against 136.2, chunks 46.4 against 44.8
    if constexpr (kVec) load(tid / PER);

    append_places<kTok>(p, t0, ntok, s_place, s_page, s_state);
    for (int x = tid; x < ntok * half; x += kAppendThreads) {
        const int tok = x / half, j = x - tok * half;
        const float2 cs = turn_of(p.positions ? p.positions[t0 + tok] : s_place[tok], p.inv_freq[j]);
        s_cos[tok * kMaxRotHalf + j] = cs.x * p.scale;
        s_sin[tok * kMaxRotHalf + j] = cs.y * p.scale;
    }
    __syncthreads();

    auto dst_of = [&](int tok, int r) -> char* {
        if (r < nq) return static_cast<char*>(p.q_out) + ((size_t)(t0 + tok) * p.Hq + r) * ROWB;
        if (s_page[tok] < 0) return nullptr;
        const int g = r < nq + hkv ? r - nq : r - nq - hkv;
        const size_t row = ((size_t)s_page[tok] * hkv + g) * p.Ps + (s_place[tok] & (p.Ps - 1));
        return static_cast<char*>(r < nq + hkv ? p.k_cache : p.v_cache) + row * ROWB;
    };
    if constexpr (kVec) {
        // a chunk rotated with itself: neighbouring pairs
        auto turn_inside = [&](Vec16<kBF16>& x, int ch, const float* cosv, const float* sinv) {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const int j = (ch * N + e) / 2;
                const float cs = cosv[j], sn = sinv[j], xe = x.x[e], ye = x.x[e + 1];
                x.x[e] = xe * cs - ye * sn;
                x.x[e + 1] = ye * cs + xe * sn;
            }
        };
        for (int R0 = tid / PER; R0 < ntok * rows; R0 += PF * RPS) {
            if (R0 != tid / PER) load(R0);
#pragma unroll
            for (int k = 0; k < PF; ++k) {
                const int R = R0 + k * RPS;
                if (R >= ntok * rows) continue;
                int tok, r, ca, cb;
                split(R, tok, r);
                const bool turned = r < nq + hkv;
                chunks(turned, ca, cb);
                const int state = s_state[tok];
                char* dst = state == kStateNone ? nullptr : dst_of(tok, r);
                if (!dst) continue;
                const float *cosv = s_cos + tok * kMaxRotHalf, *sinv = s_sin + tok * kMaxRotHalf;
                uint4 u = a[k], v = b2[k];
                if (state == kStateBad) {  // no position: queries of a bad sequence are zero
                    u = v = make_uint4(0u, 0u, 0u, 0u);
                } else if (turned && npair > 0) {
                    if (c < npair) {
                        Vec16<kBF16> x(u), y(v);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float cs = cosv[c * N + e], sn = sinv[c * N + e], xe = x.x[e], ye = y.x[e];
                            x.x[e] = xe * cs - ye * sn;
                            y.x[e] = ye * cs + xe * sn;
                        }
                        u = x.pack();
                        v = y.pack();
                    }
                } else if (turned && p.interleaved) {
                    if (ca * N < p.rot) {
                        Vec16<kBF16> x(u);
                        turn_inside(x, ca, cosv, sinv);
                        u = x.pack();
                    }
                    if (cb * N < p.rot) {
                        Vec16<kBF16> x(v);
                        turn_inside(x, cb, cosv, sinv);
                        v = x.pack();
                    }
                }
                *reinterpret_cast<uint4*>(dst + ca * 16) = u;
                *reinterpret_cast<uint4*>(dst + cb * 16) = v;
            }
        }
    } else {
        for (int x = tid; x < ntok * rows * D; x += kAppendThreads) {
            int tok, r;
            const int R = x / D, e = x - R * D;
            split(R, tok, r);
            const int state = s_state[tok];
            char* dst = state == kStateNone ? nullptr : dst_of(tok, r);
            if (!dst) continue;
            const bool turned = r < nq + hkv && e < p.rot;
            if (turned && (p.interleaved ? (e & 1) != 0 : e >= half)) continue;  // written with its partner
            const char* src = src_of(tok, r);
            auto get = [&](int i) -> float {
                if (state == kStateBad) return 0.f;
                if constexpr (kBF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(src)[i] << 16);
                else return reinterpret_cast<const float*>(src)[i];
            };
            const float v = get(e);
            if (turned) {
                const int j = p.interleaved ? e / 2 : e, e2 = p.interleaved ? e + 1 : e + half;
                const float y = get(e2), cs = s_cos[tok * kMaxRotHalf + j], sn = s_sin[tok * kMaxRotHalf + j];
                E::store(dst, e, v * cs - y * sn);
                E::store(dst, e2, y * cs + v * sn);
            } else {
                E::store(dst, e, v);
            }
        }
    }
}

int check_cache_shape(const art_shape* s);  // art_attend.cu

// Host: the argument checks of the calls that append, and their parameters without the caches.
int append_setup(AppendParams& p, const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                 int64_t v_stride, const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions,
                 const int32_t* block_table, const int32_t* seq_lens, const float* inv_freq, const art_rope* rope,
                 void* q_out, const void* cache, const void* cache2, const art_shape* shape, void* workspace,
                 size_t workspace_bytes);

}  // namespace art
