// Plan table of cp_attn_shared: what the host lays out and the kernels read.
//
// Table (int32 words, see cp_shared_plan):
//   cta_first  [num_ctas + 1]     pieces of thread block c: cta_first[c] .. cta_first[c+1]-1
//   unit_first [num_units + 1]    pieces of unit u (consecutive)
//   row_first  [num_q_rows + 1]   entries of query row n
//   entries    [num_entries][2]   (unit of the row's segment's first tile and KV head 0,
//                                  row index within the segment)
//   (padded to 16 bytes)
//   pieces     [num_pieces]       SharedPiece
// Unit = (segment, tile of up to CPATTN_SHARED_ROWS packed rows, KV head), numbered
// tile-major within a segment: unit0 + tile * Hkv + head.
#pragma once
#include <cstdint>

#include "../../include/cpattn.h"

namespace cpattn {

// A run of keys of one unit, done by one thread block.
struct SharedPiece {
  int32_t q_row0, q_pos0, q_pos_step;  // of the segment
  int32_t r0;        // first packed row of the unit within the segment
  int32_t rows;      // packed rows of the unit, 1 .. CPATTN_SHARED_ROWS
  int32_t kv_head;
  int32_t kv_row;    // KV row of the piece's first key
  int32_t key0;      // its key number within the segment's run
  int32_t keys;      // keys of the piece, >= 1
  int32_t ws_row;    // first partial row in the workspace
  int32_t flags;     // kPieceSplit: two partials, the second at ws_row + rows
  int32_t unused;
};
static_assert(sizeof(SharedPiece) == 48, "three 16-byte words");
constexpr int kPieceSplit = 2;
constexpr int kSharedTileRows = 128;  // packed rows of one MMA tile
constexpr int kSharedTileKeys = 128;  // keys of one KV tile

// A unit of more than kSharedTileRows rows is two MMA tiles that use every KV
// tile (dual).  A smaller one is a single MMA tile whose KV tiles are dealt
// alternately to the two softmax warpgroups; each keeps its own sum, so a piece
// of two or more KV tiles leaves two partials (split).
__host__ __device__ __forceinline__ bool shared_dual(int rows) { return rows > kSharedTileRows; }

struct SharedTable {
  long long unit_first, row_first, entries, pieces, total;  // word offsets (cta_first at 0)
};
inline SharedTable shared_table(const cp_shared_plan_t& p) {
  SharedTable t;
  t.unit_first = (long long)p.num_ctas + 1;
  t.row_first = t.unit_first + p.num_units + 1;
  t.entries = t.row_first + p.num_q_rows + 1;
  t.pieces = (t.entries + 2LL * p.num_entries + 3) & ~3LL;
  t.total = t.pieces + (long long)p.num_pieces * (long long)(sizeof(SharedPiece) / 4);
  return t;
}

}  // namespace cpattn
