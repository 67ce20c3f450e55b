// art_attend.cuh -- attention of rows of queries over ranges of cached keys: the
// work that dense_extend and dense_decode_shared share.
//
// A row is one query head of one query token. The rows that see the same keys of
// one KV head form an item: for dense_extend the G heads of consecutive new tokens
// of a sequence; for dense_decode_shared the G heads of all sequences of a group,
// over the group's prefix, and the G heads of one sequence, over its own tokens.
// Rows are counted token by token, R = (token - tok0) * G + head in group, and cut
// into tiles of at most `rt` rows. Items are numbered entity by entity (a group, or
// a sequence), KV head by KV head, row tile by row tile.
//
// The items' costs (a part for the item and one for each key tile of 128 tokens (fp32: 64),
// on the absolute grid of the sequence) are laid end to end and cut into equal shares,
// one for each CTA of the main kernel; what a CTA gets of one item is a segment. An
// item inside one share is finished by its CTA; otherwise each segment leaves, per
// row, the unnormalised sum of p v, a reference m and the sum l of p, and the merge
// kernel joins them:
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i
// with m in units of log2 (scores times log2(e) / sqrt(d)).
//
// Every CTA lays out the whole work for itself (plan_share): the sequence lengths are
// on the device, and some microseconds of every CTA cost less than a kernel before
// the main one and the memset that its counters would need. A page id is checked where
// it is used; a bad one marks its segment, and the merge kernel zeroes the rows of the
// sequences that have such a segment. So a call is two kernels and nothing is zeroed
// beforehand. A row's query is read, by whatever CTAs, before its result is written (by the
// one CTA that had the whole item, after its last key, or by the merge kernel): out may be q.
#pragma once

#include "art_common.cuh"

namespace art {

constexpr int kKeyTile = 128;      // keys of a tile, bf16
constexpr int kKeyTileF32 = 64;    // ... and fp32
constexpr int kAttendCtas = 160;   // CTAs of the main kernel at most (one per SM)
constexpr int kRowsTc = 256;       // rows of an item's tile, bf16
constexpr int kItemRows = 64;      // ... and fp32
// Rows of an item that the warps take key by key, bf16: the rows of one mma. At 16 rows
// (16 sequences x 4 tokens x 4 heads behind 1k-8k) 64.5 us against 66.4 on tensor memory;
// with 64 such sequences 197 against 205.
constexpr int kSmallRows = 16;
constexpr int kSmallRowsF32 = 8;   // ... and fp32: as many as a lane's registers hold
// dense_extend: a share may grow by 1 / 32 at an end so that an item is not split. Chunks of
// 1-2k tokens: 1 / 64 364 us, 1 / 32 358, 1 / 16 364, 1 / 8 382. At head_dim 64 chunks 1 / 128 292,
// 1 / 32 297, 1 / 8 321; drafts 45.8, 45.8, 48.9. Where shares are small it moves little: an
// encoder's states (12 prompts, shares of about 108 units) 30.8, 30.8, 30.4, more of them (32) 120.4,
// 118.7, 115.3; fp32 chunks 36.8 with each.
constexpr int kSplitSlack = 32;
constexpr int kMaxGroups = 8192;   // groups of a dense_decode_shared call (their offsets are kept in shared memory)

// How far a row sees: all keys of the segment; up to its own token; up to the
// limit of its sequence (row_lim).
enum LimitKind : int { kLimAll = 0, kLimCausal = 1, kLimSeq = 2 };

struct alignas(16) Seg {
    int table_row;  // sequence whose block table holds the keys
    int tok0;       // query token of row 0 of the entity
    int r0, nrow;   // rows r0 .. r0 + nrow - 1 of the entity (nrow 0: nothing to do)
    int g;          // KV head
    int k0, k1;     // keys [k0, k1)
    int lim0, kind; // kLimCausal: row R sees keys below lim0 + R / G
    int prow;       // first row of its partial results, -1: writes the output
    int bad;        // set where a page id lies outside the pool
    int pad;
};
static_assert(sizeof(Seg) == 48, "three 16-byte words");

// A sequence's, or a group's, rows and keys.
struct Entity {
    int table_row, tok0, nrows;
    int k0, k1;  // keys of the last row
    int lim0, kind;
};
// ... and its place in the work, from which the merge kernel finds the pieces of its rows
struct alignas(16) EntityPlace {
    int nrows, k0, k1, start;  // start: its first cost unit
    int prow, hc, pad[2];      // its first partial row (dense_decode_shared), a KV head's cost
};
static_assert(sizeof(EntityPlace) == 32, "two 16-byte words");

// An item of dense_extend that starts in CTA c0's share and goes on in the next ones.
struct alignas(16) MergeItem {
    int tok0, r0, nrow, g;
    int c0, np;     // pieces: CTAs c0 .. c0 + np - 1 (np 0: none)
    int tiles, off; // its key tiles; cost units of its own before CTA c0 + 1's share
    int seq, pad[3];
};

struct PlanInfo {
    int quota;  // cost units of a share
    int ok;     // 0: bad offsets, nothing is computed
};

// Cost units of an item and of a key tile, by rows.
struct CostRule {
    int small_item, small_tile;  // up to small_rows rows
    int one_item, one_tile;      // up to 128 rows
    int two_item, two_tile;
};

struct AttendParams {
    const void *q, *k, *v;
    void* out;
    const int32_t *block_table, *seq_lens;
    const int32_t* offsets;  // dense_extend: q_offsets; dense_decode_shared: group_offsets
    const int32_t* prefix;   // dense_decode_shared: prefix_lens
    int shared, causal;
    int B, T, NG, NE;  // sequences, query tokens, groups, entities
    int Hq, Hkv, G, D, Ps, max_pages, num_pages;
    int rt, ctas;
    int kt_log2, small_rows;  // keys of a tile; rows of a small item
    CostRule cost;
    float scale_log2;  // log2(e) / sqrt(d)
    unsigned long long g_mul;  // ceil(2^34 / G): R / G = R * g_mul >> 34
    unsigned long long wait_ns;  // limit of the bounded waits
    int stall;         // test hook: the consumer warps first wait for what nothing completes
    // workspace
    WsHeader* hdr;
    PlanInfo* info;
    EntityPlace* place;  // per entity, then the end
    int* row_lim;        // per sequence: keys its rows see of its group's prefix, -1: a bad sequence
    int* group_of;       // per sequence: its group or -1
    int* cta_status;     // per CTA: status bits
    int2* cta_segs;      // per CTA: its segments [x, y)
    MergeItem* merge;    // per CTA: the item that its share starts inside of, by the first CTA it goes on in
    Seg* seg;            // segment of item i in CTA c: i + c
    float* part_o;       // partial results of a segment: [D / 4][nrow][4], D floats a row
    float2* part_ml;     // of each partial row: (m, l)
};

__device__ __forceinline__ int item_cost_tile(const AttendParams& p, int nrow) {
    return nrow <= p.small_rows ? p.cost.small_tile : nrow <= 128 ? p.cost.one_tile : p.cost.two_tile;
}
__device__ __forceinline__ int item_cost_base(const AttendParams& p, int nrow) {
    return nrow <= p.small_rows ? p.cost.small_item : nrow <= 128 ? p.cost.one_item : p.cost.two_item;
}
__device__ __forceinline__ int tiles_of(const AttendParams& p, int k0, int k1) {
    return ((k1 + (1 << p.kt_log2) - 1) >> p.kt_log2) - (k0 >> p.kt_log2);
}
// Key tiles of an item before cost unit x of it.
__device__ __forceinline__ int tiles_before(int x, int base, int per, int tiles) {
    if (x <= base) return 0;
    return min(tiles, (int)((unsigned)(x - base + per - 1) / (unsigned)per));
}

// First partial row of the piece of an item that CTA c holds. dense_extend keeps two
// slots per CTA (an item that starts in the share and goes on, one that came in);
// dense_decode_shared keeps every item's rows, shifted by one tile per CTA so that
// the pieces of an item lie apart.
__device__ __forceinline__ int piece_row_extend(int c, bool first, int rt) { return (2 * c + (first ? 1 : 0)) * rt; }

// Launches a kernel whose set-up may overlap the end of what runs before it on the
// stream (it waits by griddepcontrol.wait before it touches memory).
template <class... A>
inline cudaError_t launch_after(void (*kernel)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The shape checks of art_decode for the calls around the cache (max_visit and
// num_probe are not used).
int check_cache_shape(const art_shape* s);

// Sizes and costs of a call by its shape (bf16, fp32 caches).
void attend_shape(AttendParams& p, const art_shape& s);
// Sizes and workspace layout of a call; returns the bytes, or 0 where they pass the
// supported range. `base` null: only the bytes.
size_t attend_layout(AttendParams& p, unsigned char* base);
// The main kernel (`launch`, given `more`; null: the one of the shape's type) and the merge kernel.
using AttendLaunch = cudaError_t (*)(const AttendParams& p, const void* more, cudaStream_t st);
int attend_run(AttendParams& p, const art_shape& s, void* workspace, size_t workspace_bytes, cudaStream_t st,
               AttendLaunch launch = nullptr, const void* more = nullptr);

cudaError_t launch_attend_simt(const AttendParams& p, cudaStream_t st);  // fp32
cudaError_t launch_attend_tc(const AttendParams& p, cudaStream_t st);    // bf16

}  // namespace art
