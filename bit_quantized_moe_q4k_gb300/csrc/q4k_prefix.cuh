// q4k_prefix.cuh -- the plan of attention behind shared prefixes (q4k_prefix.cu makes it and computes the shared part; q4k_attn.cu
// computes each sequence's own part and joins both).
//
// A group's shared part is the whole pages of its prefix that lie before every new token of its sequences. Its query rows
// (row r: new token r / rep of the group, query head r % rep of the kv head) are cut into row tiles; an item is a
// (group, row tile, kv head), and the line of all items' 128-token units is cut into equal pieces, one a CTA. What a CTA
// computes of an item goes to slot (CTA + item) of the partial results, a place of its own: along the line one or the other grows.
#pragma once

#include "q4k_paged.cuh"

namespace q4k {

struct PrefixGroup {
    int row0, n;        // its new tokens: rows row0 .. row0 + n - 1 of the inputs
    int lo, from;       // the shared tokens that some row sees: lo (a multiple of 16) .. from - 1
    int full_lo;        // from here on every row sees them
    int leader;         // the sequence whose row of the page table is read
    int tiles, rows;    // units of 128 tokens, row tiles (0: nothing is shared)
    int64_t unit0;      // its place on the line of work
    int64_t item0;      // its first item
};
struct PrefixHead {
    int64_t units, items;
    int ctas, pad;
};
struct PrefixPlan {
    PrefixHead* head;
    PrefixGroup* group;   // [groups]
    int2* seq;            // [batch]: group (-1: none), tokens taken from its shared part
    int2* piece;          // [items]: first slot, slots
    int* pos;             // [m]: positions of the groups' rows, where there is a window
    float* sums;          // [slots][tile_rows][head_dim]
    float2* refs;         // [slots][tile_rows]: exponent that the sums and the denominator are relative to (-inf: nothing seen), denominator
    int tile_rows, groups;
    int64_t items, slots, units;  // what the workspace has room for, and the units there can be at most
};

// Rows up to here have partial results of at most half a gigabyte; beyond (hundreds of rows a kv head for each of thousands of
// sequences), every sequence reads its prefix itself.
constexpr int64_t kPrefixMaxRows = 1 << 20;
constexpr int kPrefixCtas = 152;

}  // namespace q4k
