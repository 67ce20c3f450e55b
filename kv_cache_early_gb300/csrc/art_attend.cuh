// art_attend.cuh -- attention of rows of queries over ranges of cached keys: the
// work list that dense_extend and dense_decode_shared share.
//
// A row is one query head of one query token. The rows that see the same keys of
// one KV head form an item: for dense_extend the G heads of consecutive new tokens
// of a sequence; for dense_decode_shared the G heads of all sequences of a group,
// over the group's prefix, and the G heads of one sequence, over its own tokens.
// Rows are counted token by token, R = (token - tok0) * G + head in group, and cut
// into tiles of at most `rt` rows.
//
// The items' key tiles (kKeyTile tokens on the absolute grid of the sequence) are
// laid end to end and cut into equal shares, one for each CTA of the main kernel;
// what a CTA gets of one item is a segment. An item inside one share is finished by
// its CTA; otherwise each segment leaves, per row, the unnormalised sum of p v, the
// maximum and the sum of p, and the merge kernel joins them:
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i
// with m in units of log2 (scores times log2(e) / sqrt(d)).
#pragma once

#include "art_common.cuh"

namespace art {

constexpr int kKeyTile = 128;      // keys of a tile
constexpr int kAttendCtas = 160;   // CTAs of the main kernel at most (one per SM)
constexpr int kRowsTc = 256;       // rows of an item's tile, bf16
constexpr int kItemRows = 64;      // ... and fp32

// How far a row sees: all keys of the segment; up to its own token; up to the
// limit of its sequence (row_lim).
enum LimitKind : int { kLimAll = 0, kLimCausal = 1, kLimSeq = 2 };

struct alignas(16) Seg {
    int table_row;  // sequence whose block table holds the keys
    int tok0;       // query token of row 0 of the entity
    int r0, nrow;   // rows r0 .. r0 + nrow - 1 of the entity
    int g;          // KV head
    int k0, k1;     // keys [k0, k1)
    int lim0, kind; // kLimCausal: row R sees keys below lim0 + R / G
    int prow;       // first row of its partial results, -1: writes the output
    int pad[2];
};
static_assert(sizeof(Seg) == 48, "three 16-byte words");

// A sequence's, or a group's, rows and keys.
struct alignas(16) Entity {
    int table_row, tok0, nrows;
    int k0, k1;  // keys of the last row
    int lim0, kind;
    int bad;
};
static_assert(sizeof(Entity) == 32, "two 16-byte words");

// An item that the merge kernel finishes (dense_extend).
struct alignas(16) MergeItem {
    int tok0, r0, nrow, g;
    int c0, np;  // pieces: CTAs c0 .. c0 + np - 1 (np 0: no keys)
    int pad[2];
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
    int rt, ctas, max_items, part_rows;
    float scale_log2;  // log2(e) / sqrt(d)
    unsigned long long g_mul;  // ceil(2^34 / G): R / G = R * g_mul >> 34
    unsigned long long wait_ns;  // limit of the bounded waits
    int stall;         // test hook: the consumer warps first wait for what nothing completes
    // workspace
    WsHeader* hdr;
    Entity* ent;
    int* row_lim;    // per sequence: keys its rows see of its group's prefix
    int* group_of;   // per sequence: its group or -1
    int* item0;      // per entity: its first item; [NE] all items
    int* prow0;      // per entity (dense_decode_shared): its first partial row
    int2* item_c;    // per item: first CTA, pieces
    int* cta_first;  // per CTA: its first segment; [ctas] the end
    Seg* seg;
    MergeItem* merge;
    int* merge_n;
    float* part_o;   // [part_rows][D]
    float2* part_ml; // [part_rows]: maximum (log2 units), sum
};

// First partial row of the piece of an item that CTA c holds. dense_extend keeps two
// slots per CTA (an item that starts in the share and goes on, one that came in);
// dense_decode_shared keeps every item's rows, shifted by one tile per CTA so that
// the pieces of an item lie apart.
__host__ __device__ inline int piece_row_extend(int c, bool first, int rt) { return (2 * c + (first ? 1 : 0)) * rt; }

cudaError_t launch_attend_simt(const AttendParams& p, cudaStream_t st);  // fp32
cudaError_t launch_attend_tc(const AttendParams& p, cudaStream_t st);    // bf16

}  // namespace art
