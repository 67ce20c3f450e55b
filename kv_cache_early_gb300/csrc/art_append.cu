// art_append.cu -- appending new tokens to the paged cache, with the position
// rotation applied on the way.
//
// For token t of sequence b, the i-th of its n_b new tokens, with cache place
// s = seq_len_b - n_b + i (seq_lens count the new tokens already) and position
// pos (s, or the caller's):
//     angle_j = pos * inv_freq_j                              j < rot_dim / 2
//     (x_j, x_j') -> scale * (x_j cos - x_j' sin, x_j' cos + x_j sin)
// for every query head (into q_out) and every key head (into the cache); the
// pairs are (j, j + rot_dim / 2) or, interleaved, (2j, 2j + 1); columns from
// rot_dim on and the values are copied. The cache row of KV head g is
// (page(s / Ps) * Hkv + g) * Ps + s % Ps.
//
// pos * inv_freq reaches 1e5..1e6 radians, where a 32-bit product is off by hundredths
// of a radian: the angle is formed and reduced to one turn with more than 32 bits
// (turn_of). Sine, cosine and the rotation are 32-bit; a bf16 result is rounded once
// at the store.
//
// Bound: HBM, 2 (Hq + 2 Hkv) d bytes in and as many out a token. A CTA takes one
// token, or two: their first rows are loaded (independent of the position) before
// the chain offsets -> seq_len -> page id -> angles, so a decode step waits for the
// longer of the two and not for their sum. One more CTA (block 0) checks the device
// data of the call and stores the status word, so that no memset precedes the
// kernel; every token's CTA checks what it uses by itself. Measured: prompts of 36727
// tokens (32/8 heads, d 128, bf16) 136 us, 98 % of the copy rate; a step of 1 or 128
// tokens 2.9 us.
#include "art_common.cuh"

namespace art {

constexpr int kAppendThreads = 256;
constexpr int kMaxRotHalf = 64;  // rot_dim / 2 at most (head_dim 128)
// Up to these many tokens a CTA takes one (four CTAs an SM: all run at once and a step
// waits for one chain of loads), beyond it two (which share the chain). Measured, one
// against two (us): 128 tokens 3.5 / 4.2, 512 4.4 / 4.7, 1024 7.3 / 6.1, 4096 24.0 / 21.3.
constexpr int kFewTokens = 608;

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
__device__ void append_check(const AppendParams& p) {
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

// Cosine and sine of pos * f. The product is held as h + e (exact, by the fused
// product), 2 pi in three parts (Cody and Waite's reduction): with k = the nearest
// number of turns, h - k C1 is exact, k C2 is taken with its own rounding error, and what
// the sums round off (Knuth's two-sum) is kept; in 32-bit arithmetic the remainder
// r + low is within 2e-14 of the true one for products below 2^24. low enters to first order.
// Beyond, in 64 bits. (64-bit arithmetic for every angle cost 5 of 150 us: its pipe
// gives two results a clock and SM.)
__device__ __forceinline__ float2 turn_of(int pos, float f) {
    const float p = (float)pos, h = __fmul_rn(p, f);  // _rn: not contracted
    float r, low;
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
    float s, c;
    sincosf(r, &s, &c);
    return make_float2(c - low * s, s + low * c);
}

// kVec: a row is taken in units of two 16-byte chunks: of a rotated row in pairs
// (j, j + rot_dim / 2) the chunks c and c + npair for c < npair; of what is left, and of
// other rows, a chunk of the first half and its like of the second. It needs rot_dim / 2
// (interleaved: rot_dim) to be a multiple of a chunk's elements; without it a thread takes
// an element, or a pair.
// kTok: tokens of a CTA.
template <bool kBF16, int D, bool kVec, int kTok>
__global__ void __launch_bounds__(kAppendThreads) art_append_kernel(const AppendParams p) {
    using E = Elem<kBF16>;
    constexpr int N = Vec16<kBF16>::N;
    constexpr int ROWB = D * E::kBytes;
    constexpr int PER = kVec ? D / N / 2 : D;          // units of a row
    constexpr int RPS = kAppendThreads / PER > 0 ? kAppendThreads / PER : 1;  // rows of a step of the CTA
    constexpr int PF = 3;                              // steps whose loads a thread has under way
    __shared__ float s_cos[kTok * kMaxRotHalf], s_sin[kTok * kMaxRotHalf];
    __shared__ int s_place[kTok], s_page[kTok], s_state[kTok];  // place in the cache; its page or -1; kState*
    enum { kStateNone = 0, kStateBad = 1, kStateOk = 2 };
    if (blockIdx.x == 0) {
        append_check(p);
        return;
    }
    const int t0 = (blockIdx.x - 1) * kTok, tid = threadIdx.x;
    const int ntok = min(kTok, p.T - t0);
    const int nq = p.q ? p.Hq : 0, half = p.rot / 2, rows = nq + 2 * p.Hkv;
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
        if (r < nq + p.Hkv) return static_cast<const char*>(p.k) + (t * p.k_stride + (size_t)(r - nq) * D) * E::kBytes;
        return static_cast<const char*>(p.v) + (t * p.v_stride + (size_t)(r - nq - p.Hkv) * D) * E::kBytes;
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
            chunks(r < nq + p.Hkv, ca, cb);
            const uint4* src = reinterpret_cast<const uint4*>(src_of(tok, r));
            a[k] = src[ca];
            b2[k] = src[cb];
        }
    };
    // before it is known which sequence holds the tokens, or whether any does: behind the loads of
    // the first and the last offset, prompts took 139.6 us against 136.2, chunks 46.4 against 44.8
    if constexpr (kVec) load(tid / PER);

    // the tokens' sequences, places and pages
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
        const int g = r < nq + p.Hkv ? r - nq : r - nq - p.Hkv;
        const size_t row = ((size_t)s_page[tok] * p.Hkv + g) * p.Ps + (s_place[tok] & (p.Ps - 1));
        return static_cast<char*>(r < nq + p.Hkv ? p.k_cache : p.v_cache) + row * ROWB;
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
                const bool turned = r < nq + p.Hkv;
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
            const bool turned = r < nq + p.Hkv && e < p.rot;
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

}  // namespace art

using namespace art;

extern "C" {

size_t art_append_workspace_bytes(const art_shape* shape) { return shape ? sizeof(WsHeader) : 0; }

int art_append_kv(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                  const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions, const int32_t* block_table,
                  const int32_t* seq_lens, const float* inv_freq, const art_rope* rope, void* q_out, void* k_cache,
                  void* v_cache, const art_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_cache_shape(shape);
    if (rc != ART_OK) return rc;
    const art_shape& s = *shape;
    if (!block_table || !seq_lens || !k_cache || !v_cache || !workspace || !rope) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (!k || !v)) return ART_ERR_INVALID_ARG;
    if (num_tokens != 0 && (q != nullptr) != (q_out != nullptr)) return ART_ERR_INVALID_ARG;
    if (num_tokens < 0 || (!q_offsets && num_tokens != s.batch)) return ART_ERR_INVALID_ARG;
    if (num_tokens == 0x7fffffff) return ART_ERR_UNSUPPORTED;  // one block more than tokens
    for (int i = 0; i < 5; ++i)
        if (rope->reserved[i] != 0) return ART_ERR_INVALID_ARG;
    if (rope->rot_dim < 0 || rope->rot_dim > s.head_dim || (rope->rot_dim & 1)) return ART_ERR_INVALID_ARG;
    if (rope->interleaved != 0 && rope->interleaved != 1) return ART_ERR_INVALID_ARG;
    if (rope->rot_dim > 0 && !inv_freq) return ART_ERR_INVALID_ARG;
    const int elt = s.dtype == ART_DTYPE_BF16 ? 2 : 4, chunk = 16 / elt;
    auto bad = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) != 0; };
    if (bad(q) || bad(k) || bad(v) || bad(q_out) || bad(k_cache) || bad(v_cache) || bad(workspace))
        return ART_ERR_INVALID_ARG;
    const int64_t kvw = (int64_t)s.num_kv_heads * s.head_dim;
    if ((q && (q_stride < (int64_t)s.num_q_heads * s.head_dim || q_stride % chunk)) || k_stride < kvw ||
        k_stride % chunk || v_stride < kvw || v_stride % chunk)
        return ART_ERR_INVALID_ARG;
    // in place only row by row: another token's row would be overwritten before it is read
    if (q && q == q_out && num_tokens > 1 && q_stride != (int64_t)s.num_q_heads * s.head_dim) return ART_ERR_INVALID_ARG;
    if (2 * ((int64_t)s.num_q_heads + 2 * (int64_t)s.num_kv_heads) * s.head_dim > (1LL << 30)) return ART_ERR_UNSUPPORTED;
    if (workspace_bytes < sizeof(WsHeader)) return ART_ERR_WORKSPACE;

    AppendParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_offsets = q_offsets;
    p.positions = positions;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.inv_freq = inv_freq;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.hdr = static_cast<WsHeader*>(workspace);
    p.B = s.batch;
    p.T = num_tokens;
    p.Hq = s.num_q_heads;
    p.Hkv = s.num_kv_heads;
    p.Ps = s.page_size;
    p.max_pages = s.max_pages_per_seq;
    p.num_pages = s.num_pages_total;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved;
    p.scale = rope->scale;
    const bool bf = s.dtype == ART_DTYPE_BF16;
    const bool vec = (p.interleaved ? p.rot : p.rot / 2) % chunk == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int tok = num_tokens <= kFewTokens ? 1 : 2;
    const unsigned grid = (unsigned)((num_tokens + tok - 1) / tok) + 1u;
#define ART_APPEND(BF, DD, VEC)                                                               \
    (tok == 1 ? art_append_kernel<BF, DD, VEC, 1><<<grid, kAppendThreads, 0, st>>>(p)         \
              : art_append_kernel<BF, DD, VEC, 2><<<grid, kAppendThreads, 0, st>>>(p))
    if (bf && s.head_dim == 128) { if (vec) ART_APPEND(true, 128, true); else ART_APPEND(true, 128, false); }
    else if (bf) { if (vec) ART_APPEND(true, 64, true); else ART_APPEND(true, 64, false); }
    else if (s.head_dim == 128) { if (vec) ART_APPEND(false, 128, true); else ART_APPEND(false, 128, false); }
    else { if (vec) ART_APPEND(false, 64, true); else ART_APPEND(false, 64, false); }
#undef ART_APPEND
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ART_OK : cuda_fail(e);
}

}  // extern "C"
