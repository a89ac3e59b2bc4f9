// Plan table of cp_attn_shared: what the host lays out and the kernels read.
//
// Table (int32 words, see cp_shared_plan):
//   ctas       [num_ctas]         SharedCta: the pieces of each thread block
//   pieces     [num_pieces]       SharedPiece, by the kind of their units
//   units      [num_units]        SharedUnit: the partial rows of a unit
//   row_first  [num_q_rows + 1]   entries of query row n (padded to an even word)
//   entries    [num_entries][2]   (unit of the row's segment's first tile and KV head 0,
//                                  row index within the segment)
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
  int32_t ws_row;    // first partial row in the workspace (`rows` of them)
  int32_t unused[2];
};
static_assert(sizeof(SharedPiece) == 48, "three 16-byte words");

// The pieces of one thread block.  Units come in three kinds, by their rows:
//   dual    more than kSharedTileRows: two MMA tiles that use every KV tile; both of the
//           block's softmax warpgroups (streams) work on it: [dual0, dual1);
//   single  one MMA tile; a piece goes to one stream: stream 0 has [single0, single1),
//           stream 1 [single1, single2), and stream 0 has as many KV tiles as stream 1
//           or one more;
//   small   at most kSharedSmallRows: [small0, small1), in blocks that have no others.
struct SharedCta {
  int32_t dual0, dual1, single0, single1, single2, small0, small1, unused;
};
static_assert(sizeof(SharedCta) == 32, "two 16-byte words");

constexpr int kSharedTileRows = 128;  // packed rows of one MMA tile
constexpr int kSharedTileKeys = 128;  // keys of one KV tile
constexpr int kSharedSmallRows = 8;   // packed rows of one warp-level MMA's columns
__host__ __device__ constexpr bool shared_dual(int rows) { return rows > kSharedTileRows; }
__host__ __device__ constexpr int shared_kind(int rows) {  // 0 dual, 1 single, 2 small
  return shared_dual(rows) ? 0 : rows > kSharedSmallRows ? 1 : 2;
}

// The partials of a unit: part j of its packed row r is workspace row ws_row + j * rows
// + r; the pieces in the order of their keys.
struct SharedUnit {
  int32_t ws_row, parts, rows, unused;
};
static_assert(sizeof(SharedUnit) == 16, "one 16-byte word");

struct SharedTable {
  long long pieces, units, row_first, entries, total;  // word offsets (ctas at 0)
};
inline SharedTable shared_table(const cp_shared_plan_t& p) {
  SharedTable t;
  t.pieces = p.num_ctas * (long long)(sizeof(SharedCta) / 4);
  t.units = t.pieces + p.num_pieces * (long long)(sizeof(SharedPiece) / 4);
  t.row_first = t.units + p.num_units * (long long)(sizeof(SharedUnit) / 4);
  t.entries = (t.row_first + p.num_q_rows + 2) & ~1LL;
  t.total = t.entries + 2LL * p.num_entries;
  return t;
}

}  // namespace cpattn
