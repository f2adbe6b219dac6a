// q4k_prefix.cuh -- the plan of attention behind shared prefixes: made, and the shared part computed, in q4k_prefix.cu; the sequences'
// own parts, and the join of both, in q4k_own.cu.
//
// A group's shared part is the whole pages of its prefix that lie before every new token of its sequences. Its query rows
// (row r: new token r / rep of the group, query head r % rep of the kv head) are cut into row tiles; an item is a
// (group, row tile, kv head), and its units are the shared tokens, 128 at a time. Items are cut along the tokens into pieces for
// one CTA each; what a piece gives goes to a slot of the partial results of its own.
#pragma once

#include "q4k_paged.cuh"
#include "q4k_pieces.cuh"

namespace q4k {

struct PrefixGroup {
    int row0, n;        // its new tokens: rows row0 .. row0 + n - 1 of the inputs
    int lo, from;       // the shared tokens that some row sees: lo (a multiple of 16) .. from - 1
    int full_lo;        // from here on every row sees them
    int leader;         // the sequence whose row of the page table is read: the first with new tokens
    int tiles, rows;    // units of 128 tokens, row tiles (0: nothing is shared)
    int64_t unit0;      // its units' place on the line of all units
    int64_t item0;      // its first item
    int cta0;           // its first CTA, where pieces are not of two items
    int pad;
};
// What a CTA computes of an item.
struct alignas(16) PrefixPiece {
    int n;                    // units (0: none)
    int leader, head;         // whose pages, which kv head
    int row0;                 // the group's first row of the inputs
    int r0, rows;             // the row tile's first query row; the group's query rows
    int kv0, kv_hi, full_lo;  // tokens; from full_lo on every row sees them
    int slot;
    int next;                 // the CTA's next piece (an index above this one's), or -1
    int pad;
};
// Where an item's partial results are, and whose they are.
struct alignas(16) PrefixItem {
    int slot, slots;          // the first one, and how many
    int row0, r0, rows;       // as in PrefixPiece
    int head, pad[2];
};
// A row tile of a sequence (kOwnRows query rows of a kv head) and what it sees of the sequence's own tokens, in pieces for one warp each.
constexpr int kOwnRows = 8;
struct alignas(16) OwnTile {
    int seq, start, n, len;   // as SeqSpan
    int lo, hi;               // tokens lo (a multiple of 16) .. hi - 1 are seen by some row
    int tile;                 // the row tile
    int piece0, pieces;       // its first piece, and how many
    int first;                // its first query row among those of its group, or -1: it shares nothing
    int64_t item0;            // its group's first item
};
struct PrefixHead {
    int64_t units, items;
    int ctas;            // that compute the shared part
    int own_tiles;       // row tiles of the sequences
    int own_pieces;      // of all row tiles; a piece of each kv head
    int own_length;      // tokens of a piece, but for a tile's last
    unsigned next;       // the next (piece, kv head) to be taken
    int pad[3];
};
struct PrefixPlan {
    PrefixHead* head;
    PrefixGroup* group;   // [groups]
    int2* seq;            // [batch]: group (-1: none), tokens taken from its shared part
    PrefixPiece* piece;   // [kPrefixCtas + items]: a CTA's first piece, then the pieces that begin an item after another's in a CTA
    PrefixItem* item;     // [items]
    OwnTile* own;         // [owns]
    int2* own_piece;      // [own_slots / kv_heads]: row tile, first token
    int* pos;             // [m]: positions of the groups' rows, where there is a window
    float* sums;          // [slots][tile_rows][head_dim]
    float2* refs;         // [slots][tile_rows]: exponent that the sums and the denominator are relative to (-inf: nothing seen), denominator
    float* own_sums;      // [own_pieces * kv_heads][kOwnRows][head_dim]: the same of the sequences' own parts
    float2* own_refs;     // [own_pieces * kv_heads][kOwnRows]
    int tile_rows, groups;
    int64_t items, slots, owns, own_pieces;   // what the workspace has room for
};

// Query rows (of all heads) up to which prefixes are shared; beyond, every sequence reads its prefix itself. Partial results take most of the
// workspace: kOwnRows rows for each row tile of a sequence and kv head, however few it fills, and a row tile of the shared part for each group and kv
// head. At head_dim 128 that is 0.06 GB for 256 sequences of one token with 32/8 heads, 1.1 GB for 2^20 rows of 64 sequences, 2.5 GB for
// 4096 sequences in 2048 groups, 5.5 GB for 2^20 rows with a sequence and kv head each.
constexpr int64_t kPrefixMaxRows = 1 << 20;
constexpr int kPrefixCtas = 152;

struct OwnParams {
    PagedBatch B;
    PrefixPlan plan;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int kv_heads, group, window;
    float scale_log2;
    int* err_flag;
};
cudaError_t launch_own(const OwnParams& P, int dtype, int head_dim, cudaStream_t stream);   // after the shared part's launch
cudaError_t launch_join(const OwnParams& P, int dtype, int head_dim, cudaStream_t stream);

}  // namespace q4k
