// art_append_kv4.cu -- appending new tokens to a cache that is held in 4 bits: rotation,
// quantisation and the write in one kernel.
//
// Keys and queries are turned as in art_append.cu. A turned key is rounded to the cache's type;
// then, of the values x of a token's group of columns of a key or value head,
//     lowest = the largest bf16 that is no larger than min x
//     step   = the bf16 nearest to (max x - lowest) / 15
//     code   = the whole number nearest to (x - lowest) / step, 15 at most
// with ties to even, all as in exact arithmetic. So the cache holds the same bits on any machine
// and a test can ask for equality; a border between two codes moves by nothing. What that takes:
//   - the angle's sine and cosine as sums of two fp32 numbers (turn_exact, within 1e-11 where
//     position and angle are below 2^24; beyond, the angle is 64-bit arithmetic's, within 2e-16 of its size), the
//     products x cos and y sin with their rounding errors (by the fused product) and the sum with
//     its own (Knuth's two-sum): the turned key's rounding to fp32, and from there to bf16, is
//     then the exact one's but for about one value in 10^8 (below 2^24);
//   - x - lowest with its rounding error, and where the quotient by the rounded 1 / step comes
//     near a border, the sign of (x - lowest) - border * step, whose terms are exact (a border is
//     a half-integer up to 15, step has 8 bits).
// bf16 inputs meet ties often, since step and x lie on grids, so this is no rare matter.
//
// One kernel. Block 0 checks the call's device data and stores the status word. A tile of 8 tokens is a block's: it turns
// their queries (RotateQueries), then quantises keys and values (append_kv4_tile). A thread keeps its token and columns and
// walks the heads; the lanes of a group of columns find its least and largest value by shuffles; eight codes are one
// 32-bit store, and neighbouring lanes store to neighbouring tokens, so that a tile fills whole 128-byte units.
//
// Bound by instructions: 36,864 tokens (32/8 heads, d 128, bf16) take 176 us where their bytes take 117. Eight values of a
// row are 228 instructions, a tile's fixed part with them, two thirds of the issue slots busy (without rotation and queries
// 82 us), the rotation as in exact arithmetic 42 us more. Not by the loads' latency: a ring of eight steps of a warp's rows
// (177), rows sent for into L2 ahead (175 for the tile's own, 186 and more for later tiles') change nothing. What
// brought it from 265: 32-bit arithmetic with a bound that decides nearly always, ties resolved where they occur
// only, fixed columns a thread (the general tile of art_append.cuh spends most on addresses), places and angles of
// 8 tokens at a time.
#include "art_append.cuh"
#include "art_kv4.cuh"

namespace art {

// Up to these many tokens a CTA takes one token's keys and values, beyond it kKvTile's. One prompt, a token each against
// tiles, us: 32/8 heads, d 128: 256 tokens 5.4 / 11.2, 608 9.6 / 11.2, 700 11.1 / 11.5, 1024 14.9 / 11.6; in fp32 608
// 8.3 / 10.7, 1024 12.6 / 11.0; 16/16 heads 608 11.5 / 15.7, 1024 17.6 / 15.5; 8/2 heads, d 64: 256 4.8 / 6.4,
// 608 8.2 / 6.3. Tiles take the same time up to all SMs' worth of them: four tokens an SM, between the crossings.
constexpr int kFewTokensKv4 = 608;
// Tokens of a tile, and blocks an SM. 36,864 tokens (32/8 heads, d 128, groups of 64): 4 tokens 197 us, 8 176, 16 183; two
// blocks 195 (of 16 tokens), four 210, whose 64 registers spill.
constexpr int kKvTile = 8, kKvBlocks = 3;

struct AppendKv4Params {
    AppendParams a;
    unsigned char* cache;
    int slab, slab_log2, slab_bytes, page_bytes;
};

// sin(n pi / 32), n = 0 .. 16, as a sum of two fp32 numbers.
__device__ const float2 kSin32[17] = {
    {0.0f, 0.0f},
    {0x1.917a6cp-4f, -0x1.eb25eap-31f},
    {0x1.8f8b84p-3f, -0x1.cb2cfap-30f},
    {0x1.294062p-2f, 0x1.dab3e0p-27f},
    {0x1.87de2ap-2f, 0x1.abaa58p-28f},
    {0x1.e2b5d4p-2f, -0x1.fe4272p-28f},
    {0x1.1c73b4p-1f, -0x1.9465cep-27f},
    {0x1.44cf32p-1f, 0x1.424776p-27f},
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f},
    {0x1.8bc806p-1f, 0x1.62a2e8p-26f},
    {0x1.a9b662p-1f, 0x1.21d434p-26f},
    {0x1.c38b30p-1f, -0x1.cfe84ap-26f},
    {0x1.d906bcp-1f, 0x1.e651a8p-26f},
    {0x1.e9f416p-1f, -0x1.273a44p-26f},
    {0x1.f6297cp-1f, 0x1.feeb96p-26f},
    {0x1.fd88dap-1f, 0x1.e89292p-28f},
    {1.0f, 0.0f}};

// sin(n pi / 32), n >= 0
__device__ __forceinline__ float2 sin32(int n) {
    const int m = n & 31;
    const float2 v = kSin32[m <= 16 ? m : 32 - m];
    return n & 32 ? make_float2(-v.x, -v.y) : v;
}

// a b + c d (+ low) as a sum of two fp32 numbers
__device__ __forceinline__ float2 dot2(float a, float b, float c, float d, float low) {
    const float p = __fmul_rn(a, b), pe = fmaf(a, b, -p), q = __fmul_rn(c, d), qe = fmaf(c, d, -q);
    const float s = __fadd_rn(p, q), t = __fadd_rn(s, -p);
    const float se = __fadd_rn(__fadd_rn(p, -__fadd_rn(s, -t)), __fadd_rn(q, -t));
    const float e = se + ((pe + qe) + low), h = __fadd_rn(s, e);
    return make_float2(h, __fadd_rn(__fadd_rn(s, -h), e));
}

// Cosine and sine of pos * f times `scale`, each as a sum of two fp32 numbers (cos, cos low, sin,
// sin low). The turn r + low is n steps of pi / 32 and a rest t + tail with |t| < 0.05; n C1 is exact
// (C1 has 17 bits), and so is r - n C1. cos and sin of the rest by their series, what is above
// 2^-40 of them with its rounding errors, then the sums of angles with table values.
__device__ __forceinline__ float4 turn_exact(int pos, float f, float scale) {
    constexpr float C1 = 0x1.921fp-4f, C2 = 0x1.6a8886p-21f;  // pi / 32 = C1 + C2 - 1.03e-14
    float r, low;
    turn_reduce(pos, f, r, low);
    const bool neg = r < 0.f;
    r = fabsf(r);
    low = neg ? -low : low;
    const float k = rintf(r * 10.185916f);
    const int n = (int)k;  // turn_reduce may leave a little more than half a turn
    const float t1 = fmaf(-k, C1, r), m = __fmul_rn(k, C2), ml = fmaf(k, C2, -m);
    const float t = __fadd_rn(t1, -m), tb = __fadd_rn(t, -t1);
    const float tail = (__fadd_rn(__fadd_rn(t1, -__fadd_rn(t, -tb)), -__fadd_rn(m, tb)) - ml) + low;
    const float z = __fmul_rn(t, t), zl = fmaf(t, t, -z);
    // sin(t + tail) = t + sl, cos(t + tail) = 1 + a + al
    const float sl = fmaf(tail, 1.f - 0.5f * z, t * z * (-1.6666667e-1f + z * (8.3333333e-3f - z * 1.9841270e-4f)));
    const float a = -0.5f * z, al = fmaf(z * z, 4.1666667e-2f - z * 1.3888889e-3f, -0.5f * zl) - tail * t;
    const float2 S = sin32(n), C = sin32(n + 16);
    // C cos - S sin = C + (C a - S t + ...), S cos + C sin = S + (S a + C t + ...)
    const float2 dc = dot2(C.x, a, -S.x, t, C.x * al - S.x * sl + fmaf(C.y, a, C.y) - S.y * t);
    const float2 ds = dot2(S.x, a, C.x, t, S.x * al + C.x * sl + fmaf(S.y, a, S.y) + C.y * t);
    auto sum = [](float h, float2 d) {  // |h| may be smaller than |d.x|
        const float s = __fadd_rn(h, d.x), b = __fadd_rn(s, -h);
        const float e = __fadd_rn(__fadd_rn(h, -__fadd_rn(s, -b)), __fadd_rn(d.x, -b)) + d.y;
        return make_float2(s, e);
    };
    float2 c = sum(C.x, dc), s = sum(S.x, ds);
    if (neg) s = make_float2(-s.x, -s.y);
    if (scale != 1.f) {
        auto times = [&](float2 x) {
            const float h = __fmul_rn(x.x, scale);
            return make_float2(h, fmaf(x.y, scale, fmaf(x.x, scale, -h)));
        };
        c = times(c);
        s = times(s);
    }
    return make_float4(c.x, c.y, s.x, s.y);
}

// x cos + y sin, rounded to the cache's type. Where its fp32 rounding is the middle between two
// bf16 numbers, what that rounding left decides.
template <bool kBF16>
__device__ __forceinline__ float turned(float x, float y, const float4& cs) {
    const float2 v = dot2(x, cs.x, y, cs.z, fmaf(x, cs.y, y * cs.w));
    if constexpr (!kBF16) return v.x;
    uint32_t u = __float_as_uint(v.x);
    if ((u & 0xffffu) == 0x8000u && v.y != 0.f) u += (v.y > 0.f) == (v.x > 0.f) ? 1 : -1;
    return bf16_lo_f(pack_bf16(__uint_as_float(u), 0.f));
}

// The larger and the smaller number; not a number where one of them is none.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

constexpr float kMaxRange = 0x1.ep103f;   // 15 * 2^100: groups of such a range, and those with an infinity or NaN, become NaN
constexpr float kMinStep = 0x1p-100f;     // smaller steps are zero

// The largest bf16 number that is no larger than x.
__device__ __forceinline__ float floor_bf16(float x) {
    const uint32_t u = __float_as_uint(x);
    const uint32_t up = (u >> 31) & ((u & 0xffffu) != 0u);
    return __uint_as_float((u & 0xffff0000u) + (up << 16));
}

// The codes of the thread's 8 values, the first in the lowest bits, and (step, lowest) of its
// group of `kLanes` threads (consecutive lanes from a multiple of kLanes). kBF16: the values are bf16 numbers, so their
// least is `lowest`, and a lane sends it and the largest, negated, in one word.
template <bool kBF16, int kLanes>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t& scales) {
    float mn = min_nan(x[0], x[1]), mx = max_nan(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        mn = min_nan(mn, x[i], x[i + 1]);
        mx = max_nan(mx, x[i], x[i + 1]);
    }
    float low;
    if constexpr (kBF16) {
        uint32_t both = __byte_perm(__float_as_uint(mn), __float_as_uint(mx), 0x7632) ^ 0x80000000u;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
            const uint32_t z = __shfl_xor_sync(0xffffffffu, both, o);
            asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(both) : "r"(z));
        }
        low = bf16_lo_f(both);
        mx = bf16_hi_f(both ^ 0x80000000u);
    } else {
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
            mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        low = floor_bf16(mn);
    }
    const float d = __fadd_rn(mx, -low);
    // (d + de) / 15 = q + rest / 15: the quotient by a rounded 1 / 15, corrected once
    const float b = __fadd_rn(d, -mx);
    const float de = __fadd_rn(__fadd_rn(mx, -__fadd_rn(d, -b)), -__fadd_rn(low, b));
    const bool fine = d < kMaxRange || (d == kMaxRange && de < 0.f);  // the exact span is below it
    constexpr float kFifteenth = 0.0666666701f;
    const float q0 = __fmul_rn(d, kFifteenth), q = fmaf(fmaf(-15.f, q0, d), kFifteenth, q0);
    const float rest = fmaf(-15.f, q, d) + de;
    uint32_t u = __float_as_uint(q);
    if ((u & 0xffffu) == 0x8000u && rest != 0.f) u += rest > 0.f ? 1 : -1;
    float step = bf16_lo_f(pack_bf16(__uint_as_float(u), 0.f));
    if (step < kMinStep) step = 0.f;
    scales = (__float_as_uint(step) >> 16) | __float_as_uint(low);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
    if (step == 0.f) inv = 0.f;
    // to the nearest whole number by 1.5 * 2^23, even at ties; the codes of four make a number below 2^16
    float r[8], w[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __fadd_rn(x[i], -low);
        r[i] = __fadd_rn(fmaf(t, inv, 12582912.f), -12582912.f);
        w[i] = fmaf(t, inv, -r[i]);
        off = fmaxf(off, fabsf(w[i]));
    }
    if (off > 0.49998f) {  // t inv is within 16 * 4 * 2^-24 of (x - lowest) / step: near a border, by exact terms
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (fabsf(w[i]) <= 0.49998f) continue;
            const float t = __fadd_rn(x[i], -low), f = w[i] > 0.f ? r[i] : r[i] - 1.f, hs = (f + 0.5f) * step;  // the border
            const float bb = __fadd_rn(t, -x[i]);
            const float te = __fadd_rn(__fadd_rn(x[i], -__fadd_rn(t, -bb)), -__fadd_rn(low, bb));
            const float side = __fadd_rn(__fadd_rn(t, -hs), te);
            r[i] = side > 0.f || (side == 0.f && ((int)f & 1)) ? f + 1.f : f;
        }
    }
    const float lo4 = fmaf(r[3], 4096.f, fmaf(r[2], 256.f, fmaf(r[1], 16.f, r[0])));
    const float hi4 = fmaf(r[7], 4096.f, fmaf(r[6], 256.f, fmaf(r[5], 16.f, r[4])));
    const uint32_t codes = (__float_as_uint(lo4 + 8388608.f) & 0xffffu) | (__float_as_uint(hi4 + 8388608.f) << 16);
    if (!fine) {
        scales = 0x7fc00000u;
        return 0u;
    }
    return codes;
}

// Eight turned values x cos + y sin (y with its sign), rounded to the cache's type. bf16: from 32-bit arithmetic, which is
// within 3.5 * 2^-24 (|x| + |y|) scale; where that bound holds a border between bf16 numbers, by turned(), for which
// whole(e) gives column e's cosine and sine in full.
template <bool kBF16, class F>
__device__ __forceinline__ void turn8(const float (&x)[8], const float (&y)[8], const float2 (&cs)[8], float reach, F whole,
                                      float (&o)[8]) {
    if constexpr (kBF16) {
        uint32_t differ = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = fmaf(x[e], cs[e].x, __fmul_rn(y[e], cs[e].y)), m = fabsf(x[e]) + fabsf(y[e]);
            const uint32_t u = pack_bf16(fmaf(m, reach, v), fmaf(m, -reach, v));
            differ |= u ^ (u >> 16);
            o[e] = bf16_hi_f(u);
        }
        if ((differ & 0xffffu) == 0) return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = turned<kBF16>(x[e], y[e], whole(e));
}

// The queries of a block's kTok tokens from t0 on, whose columns turn in whole 16-byte chunks. A thread keeps a token and
// two chunks, c and c + rot_dim / 2 where they turn with one another, and walks the heads with their cosines and sines
// (angle(token, j)) in registers. load: the first heads' chunks, before the angles are there.
template <bool kBF16, int D, int kTok>
struct RotateQueries {
    static constexpr int N = Vec16<kBF16>::N, PER = D / N / 2, ELT = kBF16 ? 2 : 4;
    static constexpr int HSTEP = kAppendThreads / PER / kTok;  // heads of a step
    static constexpr int PF = 4;                               // steps whose loads are under way
    static_assert(HSTEP * PER * kTok == kAppendThreads, "a step takes whole heads of the tile");
    const AppendParams& p;
    const char* src;
    char* dst;
    int tok, h0, c, ca, cb;
    bool here;
    uint4 a[PF], b[PF];
    __device__ __forceinline__ RotateQueries(const AppendParams& p_, int t0, int ntok) : p(p_) {
        const int tid = threadIdx.x, npair = p.interleaved ? 0 : p.rot / 2 / N;
        c = tid % PER;
        tok = tid / PER % kTok;
        h0 = tid / PER / kTok;
        ca = c < npair ? c : c + npair;
        cb = c < npair ? c + npair : c + PER;
        here = tok < ntok;
        const size_t t = (size_t)(t0 + tok);
        src = static_cast<const char*>(p.q) + (t * (size_t)p.q_stride + (size_t)h0 * D) * ELT;
        dst = static_cast<char*>(p.q_out) + ((t * p.Hq + h0) * D) * ELT;
    }
    __device__ __forceinline__ void load(int hb) {
#pragma unroll
        for (int k = 0; k < PF; ++k)
            if (here && hb + k * HSTEP + h0 < p.Hq) {
                const uint4* row = reinterpret_cast<const uint4*>(src + (size_t)(hb + k * HSTEP) * (D * ELT));
                a[k] = row[ca];
                b[k] = row[cb];
            }
    }
    template <class F>
    __device__ __forceinline__ void run(int state, F angle) {
        if (state == kStateNone) return;
        const bool pairs = !p.interleaved && c < p.rot / 2 / N, in_a = p.interleaved && ca * N < p.rot, in_b = p.interleaved && cb * N < p.rot;
        float2 cs[N];  // pairs: of pair c N + e; interleaved: of chunk ca's N / 2 pairs, then of cb's
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int j = p.interleaved ? (e < N / 2 ? ca * (N / 2) + e : cb * (N / 2) + e - N / 2) : c * N + e;
            cs[e] = pairs || (e < N / 2 ? in_a : in_b) ? angle(tok, j) : make_float2(1.f, 0.f);
        }
#pragma unroll 1
        for (int hb = 0; hb < p.Hq; hb += PF * HSTEP) {
            if (hb > 0) load(hb);
#pragma unroll
            for (int k = 0; k < PF; ++k) {
                if (hb + k * HSTEP + h0 >= p.Hq) continue;
                uint4 u = a[k], v = b[k];
                if (state == kStateBad) {  // no position: queries of a bad sequence are zero
                    u = v = make_uint4(0u, 0u, 0u, 0u);
                } else if (pairs) {
                    Vec16<kBF16> x(u), y(v);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float xe = x.x[e], ye = y.x[e];
                        x.x[e] = xe * cs[e].x - ye * cs[e].y;
                        y.x[e] = ye * cs[e].x + xe * cs[e].y;
                    }
                    u = x.pack();
                    v = y.pack();
                } else if (p.interleaved) {
                    auto inside = [&](uint4& w, int e0) {
                        Vec16<kBF16> x(w);
#pragma unroll
                        for (int e = 0; e < N; e += 2) {
                            const float2 z = cs[e0 + e / 2];
                            const float xe = x.x[e], ye = x.x[e + 1];
                            x.x[e] = xe * z.x - ye * z.y;
                            x.x[e + 1] = ye * z.x + xe * z.y;
                        }
                        w = x.pack();
                    };
                    if (in_a) inside(u, 0);
                    if (in_b) inside(v, N / 2);
                }
                uint4* row = reinterpret_cast<uint4*>(dst + (size_t)(hb + k * HSTEP) * (D * ELT));
                row[ca] = u;
                row[cb] = v;
            }
        }
    }
};

// One token's queries in a block of their own.
template <bool kBF16, int D>
__device__ __forceinline__ void rotate_token(const AppendParams& p, int t0) {
    __shared__ float2 s_cs[kMaxRotHalf];
    __shared__ int s_place[1], s_page[1], s_state[1];
    RotateQueries<kBF16, D, 1> q(p, t0, 1);
    q.load(0);
    append_places<1>(p, t0, 1, s_place, s_page, s_state);
    for (int j = threadIdx.x; j < p.rot / 2; j += kAppendThreads) {
        const float2 cs = turn_of(p.positions ? p.positions[t0] : s_place[0], p.inv_freq[j]);
        s_cs[j] = make_float2(cs.x * p.scale, cs.y * p.scale);
    }
    __syncthreads();
    q.run(s_state[0], [&](int, int j) { return s_cs[j]; });
}

// Keys and values of tokens kTok * tile .., and (kQueries) their queries.
// kVec: columns turn in whole units of 8 (rot_dim, or its half where the pairs are (j, j + rot_dim / 2)).
template <bool kBF16, int D, int NG, bool kVec, bool kQueries, int kTok>
__device__ __forceinline__ void append_kv4_tile(const AppendKv4Params& pp, int tile) {
    const AppendParams& p = pp.a;
    constexpr int PER = D / 8;                       // units of a row
    constexpr int RPS = kAppendThreads / PER;        // rows of a step of the CTA
    constexpr int N = kBF16 ? 1 : 2;                 // 16-byte chunks of a unit
    __shared__ float4 s_cs[kTok][8][kMaxRotHalf / 8 + 1];  // of frequency j: [j % 8][j / 8], neighbouring units in other banks
    __shared__ int s_place[kTok], s_page[kTok], s_state[kTok];
    const int t0 = tile * kTok, tid = threadIdx.x, ntok = min(kTok, p.T - t0), half = p.rot / 2;
    // A thread keeps its columns and its token; from step to step it has other heads (keys', then values').
    static_assert(RPS % kTok == 0, "a step takes whole heads of the tile");
    constexpr int HSTEP = RPS / kTok;
    const int ch = tid % PER, e0 = ch * 8, tok = tid / PER % kTok, h0 = tid / PER / kTok, heads = 2 * p.Hkv;
    const bool turns = e0 < p.rot, second = e0 >= half;
    constexpr int ELT = kBF16 ? 2 : 4;
    const size_t t = (size_t)(t0 + tok);
    const char* k_row = static_cast<const char*>(p.k) + (t * (size_t)p.k_stride + e0) * ELT;
    const char* v_row = static_cast<const char*>(p.v) + (t * (size_t)p.v_stride + e0) * ELT;
    const int partner = (second ? -half : half) * ELT;  // kVec, pairs (j, j + rot_dim / 2): bytes to the unit's partners
    const bool paired = kVec && turns && !p.interleaved;
    uint4 a[N] = {}, b[N] = {};  // threads without a row work on what is here, and store nothing
    auto load = [&](bool key, const char* row) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = reinterpret_cast<const uint4*>(row)[i];
            if (key && paired) b[i] = reinterpret_cast<const uint4*>(row + partner)[i];
        }
    };
    // the first row's bytes before the chain offsets -> length -> page
    if (tok < ntok && h0 < heads) {
        if (h0 < p.Hkv) load(true, k_row + (size_t)h0 * (D * ELT));
        else load(false, v_row + (size_t)(h0 - p.Hkv) * (D * ELT));
    }
    append_places<kTok>(p, t0, ntok, s_place, s_page, s_state);
    for (int x = tid; x < ntok * half; x += kAppendThreads) {
        const int tk = x / half, j = x - tk * half;
        s_cs[tk][j & 7][j >> 3] = turn_exact(p.positions ? p.positions[t0 + tk] : s_place[tk], p.inv_freq[j], p.scale);
    }
    __syncthreads();
    if constexpr (kQueries) {
        if (p.q) {
            RotateQueries<kBF16, D, kTok> q(p, t0, ntok);
            q.load(0);
            q.run(q.here ? s_state[q.tok] : kStateNone, [&](int tk, int j) {
                const float4 v = s_cs[tk][j & 7][j >> 3];
                return make_float2(v.x, v.z);
            });
        }
    }
    const bool held = tok < ntok && s_state[tok] == kStateOk && s_page[tok] >= 0;
    const float reach = 0x1p-22f * fabsf(p.scale);
    // Cosine and sine of the unit's column e; the sine with the sign that the column's partner has. The high parts
    // stay in registers.
    auto whole = [&](int e) {
        const int c = e0 + e, j = min(p.interleaved ? c / 2 : c < half ? c : c - half, kMaxRotHalf - 1);
        float4 v = s_cs[tok][j & 7][j >> 3];
        if (p.interleaved ? !(c & 1) : c < half) {
            v.z = -v.z;
            v.w = -v.w;
        }
        return v;
    };
    float2 cs[8];
    if (kBF16 && kVec && turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 v = whole(e);
            cs[e] = make_float2(v.x, v.z);
        }
    }
    const int in_page = s_place[tok] & (p.Ps - 1), u = in_page & (pp.slab - 1);
    unsigned char* dst = pp.cache + (size_t)(held ? s_page[tok] : 0) * p.Hkv * (size_t)pp.page_bytes +
                         (size_t)(in_page >> pp.slab_log2) * pp.slab_bytes;
    const int code_at = kv4_code_at<D>(u, ch >> 2) + (ch & 3) * 4;
    const int scale_at = pp.slab * D + kv4_scale_at<NG>(u, ch / (PER / NG));
    const int v_codes = pp.slab * (D / 2), v_scales = pp.slab * 4 * NG;
    // The unit in a and b, of a row whose columns begin at `row`, into the head's page at `page`; `live`: it is stored.
    // Whole warps: the lanes of a group of columns exchange values.
    auto unit = [&](bool key, const char* row, unsigned char* page, bool live, auto next) {
        auto unpack = [&](const uint4 (&w)[N], float (&o)[8]) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const Vec16<kBF16> v(w[i]);
#pragma unroll
                for (int e = 0; e < Vec16<kBF16>::N; ++e) o[i * Vec16<kBF16>::N + e] = v.x[e];
            }
        };
        float x[8], y[8];
        unpack(a, x);
        if (key && turns && kVec) {
            if (p.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
            } else {
                unpack(b, y);
            }
        }
        next();  // the next unit's loads, under way while this one is worked on
        if (key && turns) {
            float o[8];
            if constexpr (kVec) {
                turn8<kBF16>(x, y, cs, reach, whole, o);
            } else {
                const char* first = row - e0 * ELT;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = e0 + e;
                    o[e] = x[e];
                    if (c >= p.rot || !live) continue;
                    const int other = p.interleaved ? c ^ 1 : c >= half ? c - half : c + half;
                    float v;
                    if constexpr (kBF16) v = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(first)[other] << 16);
                    else v = reinterpret_cast<const float*>(first)[other];
                    o[e] = turned<kBF16>(x[e], v, whole(e));
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = o[e];
        }
        uint32_t scales;
        const uint32_t codes = quantise<kBF16, D / NG / 8>(x, scales);
        if (!live) return;
        *reinterpret_cast<uint32_t*>(page + code_at + (key ? 0 : v_codes)) = codes;
        if (ch % (PER / NG) == 0) *reinterpret_cast<uint32_t*>(page + scale_at + (key ? 0 : v_scales)) = scales;
    };
    const size_t row_step = HSTEP * D * ELT, page_step = (size_t)HSTEP * pp.page_bytes;
    if constexpr (kTok == 1) {  // keys and values side by side: a step of one token is one round of the block
        const char* row = h0 < p.Hkv ? k_row + (size_t)h0 * (D * ELT) : v_row + (size_t)(h0 - p.Hkv) * (D * ELT);
#pragma unroll 1
        for (int hb = 0; hb < heads; hb += HSTEP) {
            const int h = hb + h0, g = h < p.Hkv ? h : h - p.Hkv;
            const bool key = h < p.Hkv;
            if (hb > 0 && h < heads) {
                row = (key ? k_row : v_row) + (size_t)g * (D * ELT);
                load(key, row);
            }
            unit(key, row, dst + (size_t)g * pp.page_bytes, held && h < heads, [] {});
        }
    } else {
        auto half_of = [&](bool key, const char* base) {
            const char* row = base + (size_t)h0 * (D * ELT);
            unsigned char* page = dst + (size_t)h0 * pp.page_bytes;
#pragma unroll 1
            for (int h = h0; h < p.Hkv + h0; h += HSTEP) {  // as often for every thread
                unit(key, row, page, held && h < p.Hkv, [&] {
                    if (held && h + HSTEP < p.Hkv) load(key, row + row_step);
                    else if (key && held && h0 < p.Hkv && h + HSTEP >= p.Hkv && h < p.Hkv) load(false, v_row + (size_t)h0 * (D * ELT));
                });
                row += row_step;
                page += page_step;
            }
        };
        half_of(true, k_row);
        half_of(false, v_row);
    }
}

// Few tokens: a token's keys and values in one block, its queries in the next, so that a step waits for the longer of the
// two. Beyond: tiles of kKvTile tokens with their queries, which share places and angles (36,864 tokens apart, in tiles
// of 16 tokens and 8 of queries, 198 us against 183).
template <bool kBF16, int D, int NG, bool kVecQ, bool kVec>
__global__ void __launch_bounds__(kAppendThreads, kKvBlocks) art_append_kv4_few_kernel(const AppendKv4Params p) {
    if (blockIdx.x == 0) {
        append_check(p.a);
        return;
    }
    const int i = blockIdx.x - 1;
    if (i < p.a.T) append_kv4_tile<kBF16, D, NG, kVec, false, 1>(p, i);
    else if constexpr (kVecQ) rotate_token<kBF16, D>(p.a, i - p.a.T);
    else append_rows<kBF16, D, false, 1>(p.a, 0, i - p.a.T);
}
// kVecQ: queries turn in whole chunks; else they are taken two tokens at a time by the blocks behind the tiles'.
template <bool kBF16, int D, int NG, bool kVecQ, bool kVec>
__global__ void __launch_bounds__(kAppendThreads, kKvBlocks) art_append_kv4_kernel(const AppendKv4Params p) {
    if (blockIdx.x == 0) {
        append_check(p.a);
        return;
    }
    const int i = blockIdx.x - 1, tiles = (p.a.T + kKvTile - 1) / kKvTile;
    if (kVecQ || i < tiles) append_kv4_tile<kBF16, D, NG, kVec, kVecQ, kKvTile>(p, i);
    else if constexpr (!kVecQ) append_rows<kBF16, D, false, 2>(p.a, 0, i - tiles);
}

template <bool kBF16, int D, int NG>
static void launch_append_kv4(const AppendKv4Params& p, cudaStream_t st) {
    const int turn = p.a.interleaved ? p.a.rot : p.a.rot / 2;
    const bool vec = turn % 8 == 0, vec_q = turn % (kBF16 ? 8 : 4) == 0, q = p.a.q != nullptr;
    const bool few = p.a.T <= kFewTokensKv4;
    unsigned grid = 1u;
    if (few) grid += (unsigned)p.a.T * (q ? 2u : 1u);
    else grid += (unsigned)((p.a.T + kKvTile - 1) / kKvTile) + (q && !vec_q ? (unsigned)((p.a.T + 1) / 2) : 0u);
#define ART_APPEND4(VQ, V)                                                                              \
    (few ? art_append_kv4_few_kernel<kBF16, D, NG, VQ, V><<<grid, kAppendThreads, 0, st>>>(p)           \
         : art_append_kv4_kernel<kBF16, D, NG, VQ, V><<<grid, kAppendThreads, 0, st>>>(p))
    if (vec) ART_APPEND4(true, true);
    else if (vec_q) ART_APPEND4(true, false);
    else ART_APPEND4(false, false);
#undef ART_APPEND4
}

}  // namespace art

using namespace art;

extern "C" {

size_t art_kv4_page_bytes(const art_shape* shape, int32_t group) {
    if (check_cache_shape(shape) != ART_OK || !kv4_group_ok(shape->head_dim, group)) return 0;
    return (size_t)kv4_layout(shape->page_size, shape->head_dim, group).page_bytes;
}

size_t art_append_kv4_workspace_bytes(const art_shape* shape) { return shape ? sizeof(WsHeader) : 0; }

int art_append_kv4(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                   const int32_t* q_offsets, int32_t num_tokens, const int32_t* positions, const int32_t* block_table,
                   const int32_t* seq_lens, const float* inv_freq, const art_rope* rope, void* q_out, void* cache,
                   int32_t group, const art_shape* shape, void* workspace, size_t workspace_bytes, void* stream) {
    AppendKv4Params p;
    const int rc = append_setup(p.a, q, k, v, q_stride, k_stride, v_stride, q_offsets, num_tokens, positions, block_table,
                                seq_lens, inv_freq, rope, q_out, cache, cache, shape, workspace, workspace_bytes);
    if (rc == ART_OK || rc == ART_ERR_WORKSPACE)
        if (!kv4_group_ok(shape->head_dim, group)) return ART_ERR_UNSUPPORTED;
    if (rc != ART_OK) return rc;
    // blocks for queries and for keys and values
    if (num_tokens > 0x3fffffff) return ART_ERR_UNSUPPORTED;
    const art_shape& s = *shape;
    p.cache = static_cast<unsigned char*>(cache);
    const Kv4Layout l = kv4_layout(s.page_size, s.head_dim, group);
    p.slab = l.slab;
    p.slab_log2 = l.slab_log2;
    p.slab_bytes = l.slab_bytes;
    p.page_bytes = l.page_bytes;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int ng = s.head_dim / group;
    const bool bf = s.dtype == ART_DTYPE_BF16;
    if (s.head_dim == 128) {
        if (ng == 1) bf ? launch_append_kv4<true, 128, 1>(p, st) : launch_append_kv4<false, 128, 1>(p, st);
        else if (ng == 2) bf ? launch_append_kv4<true, 128, 2>(p, st) : launch_append_kv4<false, 128, 2>(p, st);
        else bf ? launch_append_kv4<true, 128, 4>(p, st) : launch_append_kv4<false, 128, 4>(p, st);
    } else {
        if (ng == 1) bf ? launch_append_kv4<true, 64, 1>(p, st) : launch_append_kv4<false, 64, 1>(p, st);
        else bf ? launch_append_kv4<true, 64, 2>(p, st) : launch_append_kv4<false, 64, 2>(p, st);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ART_OK : cuda_fail(e);
}

}  // extern "C"
