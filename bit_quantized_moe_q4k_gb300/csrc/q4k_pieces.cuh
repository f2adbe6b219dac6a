// q4k_pieces.cuh -- into how many pieces the sequences' own parts behind shared prefixes are cut, and the room for them: what the plan
// (q4k_prefix.cu) and the workspace have to agree on. Plain arithmetic, for host and device.
#pragma once

#include <stdint.h>

namespace q4k {

// Warps that work on own parts at a time: twelve on each of 152 SMs.
constexpr int kOwnWarps = 4, kOwnCtas = 3 * 152;
// Pieces that the tokens of all row tiles and kv heads are cut into, beyond one for each tile's end: three for each two warps.
constexpr int kOwnPieces = kOwnCtas * kOwnWarps * 3 / 2;
// Tokens of a piece at least: less does not pay for its start.
constexpr int kOwnLeast = 128;

// Tokens of a piece, where the row tiles of one kv head see `tokens` in all. Rounded up at each step: never below tokens * kv_heads / kOwnPieces
// (nor, at its limit, below what a tile can see), so that tokens / own_length <= kOwnPieces / kv_heads.
constexpr int own_length(int64_t tokens, int kv_heads) {
    const int64_t share = (tokens * kv_heads + kOwnPieces - 1) / kOwnPieces, whole = (share + 31) & ~(int64_t)31;
    return (int)(whole < kOwnLeast ? kOwnLeast : whole > (int64_t)1 << 30 ? (int64_t)1 << 30 : whole);
}
// Pieces of a row tile that sees `tokens`; rows that see nothing are zeroed by one.
constexpr int pieces_of_tile(int tokens, int length) { return tokens <= length ? 1 : (tokens - 1) / length + 1; }
// Pieces of all `tiles` row tiles of a kv head at most: each tile's are below 1 + tokens / length.
constexpr int64_t most_own_pieces(int64_t tiles, int kv_heads) { return tiles + kOwnPieces / kv_heads; }

}  // namespace q4k
