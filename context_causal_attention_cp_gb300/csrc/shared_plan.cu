// Host plan of cp_attn_shared: units, their cut into pieces and the merge lists.
//
// The units (segment, packed-row tile, KV head) are walked in a fixed order and
// their keys dealt to the thread blocks one after the other: each block is
// filled up to a budget, so a unit is cut only where a block is full, and every
// block's cost is within a tile of the others'.  The smallest budget that needs
// no more than num_ctas blocks is found by bisection.  A piece costs its KV
// tiles plus a fixed part (its queries' load and its partial's store), so that
// short units are not shredded.  Nothing is allocated: each pass walks the
// segment table again.
#include <algorithm>
#include <cstdint>

#include "shared_plan.h"

namespace cpattn {
namespace {

constexpr int kKeys = kSharedTileKeys;
constexpr int kTileCost = 16;       // one KV tile for one MMA tile of rows
constexpr int kDualCost = 24;       // one KV tile for two
constexpr int kPieceCost = 16;      // a piece's fixed part
constexpr int tile_cost(int rows) { return shared_dual(rows) ? kDualCost : kTileCost; }
// partial rows that a piece leaves
constexpr bool split(int rows, long long keys) { return !shared_dual(rows) && keys > kKeys; }
constexpr int parts(int rows, long long keys) { return split(rows, keys) ? 2 * rows : rows; }
constexpr long long kMaxUnits = 1LL << 22;

long long last_pos(const cp_segment_t& s) {
  return (long long)s.q_pos0 + (long long)(s.q_len - 1) * s.q_pos_step;
}

// Calls f(segment, tile, rows, keys) for every packed-row tile: `keys` that its
// last row sees (its other rows see no more).
template <class F>
void for_each_tile(const cp_segment_t* segs, int num_segs, int g, F&& f) {
  for (int i = 0; i < num_segs; ++i) {
    const cp_segment_t& s = segs[i];
    const long long packed = (long long)s.q_len * g;
    for (long long r0 = 0; r0 < packed; r0 += CPATTN_SHARED_ROWS) {
      const int rows = (int)std::min<long long>(CPATTN_SHARED_ROWS, packed - r0);
      const long long pos = s.q_pos0 + ((r0 + rows - 1) / g) * s.q_pos_step;
      f(s, r0, rows, std::max<long long>(0, pos + 1));
    }
  }
}

// Deals every unit's keys; calls f(cta, segment, r0, rows, head, key0, keys) for
// each piece and u(segment, r0, rows, head) before a unit's first piece.
// Returns the number of blocks used, or max_ctas + 1 as soon as they do not do.
template <class U, class F>
int deal(const cp_segment_t* segs, int num_segs, int g, int Hkv, long long budget, int max_ctas,
         U&& u, F&& f) {
  int cta = 0;
  long long used = 0;
  bool full = false;
  for_each_tile(segs, num_segs, g, [&](const cp_segment_t& s, long long r0, int rows,
                                       long long keys) {
    for (int h = 0; h < Hkv && !full; ++h) {
      u(s, r0, rows, h);
      long long key0 = 0;
      while (key0 < keys) {
        const long long tiles = (keys - key0 + kKeys - 1) / kKeys;
        long long fit = (budget - used - kPieceCost) / tile_cost(rows);
        if (fit < 1) {
          if (++cta >= max_ctas) {
            full = true;
            return;
          }
          used = 0;
          continue;
        }
        fit = std::min(fit, tiles);
        const long long n = std::min(keys - key0, fit * kKeys);
        f(cta, s, r0, rows, h, key0, n);
        key0 += n;
        used += kPieceCost + fit * tile_cost(rows);
      }
    }
  });
  return full ? max_ctas + 1 : cta + 1;
}

bool plan_ok(const cp_shared_plan_t& p) {
  return p.num_q_rows >= 0 && p.Hq >= 1 && p.Hkv >= 1 && p.Hq % p.Hkv == 0 && p.num_ctas >= 1 &&
         p.num_ctas <= 4096 && p.num_units >= 0 && p.num_pieces >= 0 && p.num_entries >= 0 &&
         p.kv_rows >= 0 && p.ws_rows >= 0 && p.table_ints == shared_table(p).total;
}

int check_segments(const cp_segment_t* segs, int num_segs, int num_q_rows) {
  for (int i = 0; i < num_segs; ++i) {
    const cp_segment_t& s = segs[i];
    if (s.q_len < 0 || s.q_row0 < 0 || (long long)s.q_row0 + s.q_len > num_q_rows ||
        s.q_pos_step < 0 || s.kv_row0 < 0 || s.kv_len < 0 ||
        (s.q_len > 0 && last_pos(s) + 1 > s.kv_len))
      return CPATTN_ERR_INVALID_ARG;
    if ((long long)s.kv_row0 + s.kv_len > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  }
  return CPATTN_OK;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cp_shared_plan_size(const cp_segment_t* segs, int num_segs, int num_q_rows, int Hq,
                                   int Hkv, int num_ctas, cp_shared_plan_t* plan) {
  if (!plan || num_segs < 0 || (num_segs > 0 && !segs) || num_q_rows < 0 || Hq < 1 || Hkv < 1 ||
      Hq % Hkv != 0 || num_ctas < 1 || num_ctas > 4096)
    return CPATTN_ERR_INVALID_ARG;
  if (num_segs > kMaxUnits) return CPATTN_ERR_TOO_LARGE;
  const int rc = check_segments(segs, num_segs, num_q_rows);
  if (rc != CPATTN_OK) return rc;
  const int g = Hq / Hkv;
  long long tiles = 0, entries = 0, kv_rows = 0;
  for (int i = 0; i < num_segs; ++i) {
    const cp_segment_t& s = segs[i];
    tiles += ((long long)s.q_len * g + CPATTN_SHARED_ROWS - 1) / CPATTN_SHARED_ROWS;
    entries += s.q_len;
    if (s.q_len > 0)
      kv_rows = std::max(kv_rows, s.kv_row0 + std::max<long long>(0, last_pos(s) + 1));
  }
  if (tiles * Hkv > kMaxUnits || entries > 0x3fffffffLL) return CPATTN_ERR_TOO_LARGE;
  long long cost = 0;
  for_each_tile(segs, num_segs, g, [&](const cp_segment_t&, long long, int rows, long long keys) {
    if (keys > 0) cost += (kPieceCost + (keys + kKeys - 1) / kKeys * tile_cost(rows)) * Hkv;
  });
  // one block more than the average needs at most: the average, a whole piece
  // and a cut on either side
  long long lo = kPieceCost + kTileCost, hi = cost / num_ctas + 2 * (kPieceCost + kDualCost);
  auto none = [](auto&&...) {};
  while (deal(segs, num_segs, g, Hkv, hi, num_ctas, none, none) > num_ctas) hi *= 2;
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (deal(segs, num_segs, g, Hkv, mid, num_ctas, none, none) <= num_ctas) hi = mid;
    else lo = mid + 1;
  }
  if (hi > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  long long pieces = 0, ws_rows = 0;
  deal(segs, num_segs, g, Hkv, hi, num_ctas, none,
       [&](int, const cp_segment_t&, long long, int rows, int, long long, long long keys) {
         ++pieces;
         ws_rows += parts(rows, keys);
       });
  if (ws_rows > 0x7fffffffLL || pieces > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  plan->num_q_rows = num_q_rows;
  plan->Hq = Hq;
  plan->Hkv = Hkv;
  plan->num_ctas = num_ctas;
  plan->num_units = (int32_t)(tiles * Hkv);
  plan->num_pieces = (int32_t)pieces;
  plan->num_entries = (int32_t)entries;
  plan->kv_rows = (int32_t)kv_rows;
  plan->needs_merge = entries > 0;
  plan->budget = (int32_t)hi;
  plan->ws_rows = ws_rows;
  plan->table_ints = shared_table(*plan).total;
  return CPATTN_OK;
}

extern "C" int cp_shared_plan(const cp_segment_t* segs, int num_segs, const cp_shared_plan_t* plan,
                              int32_t* table) {
  if (!plan || !table || num_segs < 0 || (num_segs > 0 && !segs) || !plan_ok(*plan))
    return CPATTN_ERR_INVALID_ARG;
  const int rc = check_segments(segs, num_segs, plan->num_q_rows);
  if (rc != CPATTN_OK) return rc;
  const int g = plan->Hq / plan->Hkv, Hkv = plan->Hkv, N = plan->num_q_rows;
  const SharedTable T = shared_table(*plan);
  int32_t* cta_first = table;
  int32_t* unit_first = table + T.unit_first;
  int32_t* row_first = table + T.row_first;
  int32_t* entries = table + T.entries;
  auto* pieces = reinterpret_cast<SharedPiece*>(table + T.pieces);
  // the table must be the one that was sized: check the counts before writing
  long long tiles = 0, ents = 0, np = 0, ws = 0;
  for (int i = 0; i < num_segs; ++i) {
    tiles += ((long long)segs[i].q_len * g + CPATTN_SHARED_ROWS - 1) / CPATTN_SHARED_ROWS;
    ents += segs[i].q_len;
  }
  if (tiles * Hkv != plan->num_units || ents != plan->num_entries) return CPATTN_ERR_INVALID_ARG;
  auto none = [](auto&&...) {};
  const int used =
      deal(segs, num_segs, g, Hkv, plan->budget, plan->num_ctas, none,
           [&](int, const cp_segment_t&, long long, int rows, int, long long, long long keys) {
             ++np;
             ws += parts(rows, keys);
           });
  if (used > plan->num_ctas || np != plan->num_pieces || ws != plan->ws_rows)
    return CPATTN_ERR_INVALID_ARG;
  for (long long i = T.entries + 2 * ents; i < T.pieces; ++i) table[i] = 0;  // padding

  // entries of each query row, segment by segment
  for (int n = 0; n <= N; ++n) row_first[n] = 0;
  for (int i = 0; i < num_segs; ++i)
    for (int j = 0; j < segs[i].q_len; ++j) ++row_first[segs[i].q_row0 + j + 1];
  for (int n = 0; n < N; ++n) row_first[n + 1] += row_first[n];
  int32_t unit0 = 0;
  for (int i = 0; i < num_segs; ++i) {
    const cp_segment_t& s = segs[i];
    for (int j = 0; j < s.q_len; ++j) {
      const int32_t e = row_first[s.q_row0 + j]++;
      entries[2 * e] = unit0;
      entries[2 * e + 1] = j;
    }
    unit0 += (int32_t)(((long long)s.q_len * g + CPATTN_SHARED_ROWS - 1) / CPATTN_SHARED_ROWS) * Hkv;
  }
  for (int n = N; n > 0; --n) row_first[n] = row_first[n - 1];
  row_first[0] = 0;

  int32_t unit = 0, piece = 0, cta_now = -1, ws_row = 0;
  deal(segs, num_segs, g, Hkv, plan->budget, plan->num_ctas,
       [&](const cp_segment_t&, long long, int, int) { unit_first[unit++] = piece; },
       [&](int cta, const cp_segment_t& s, long long r0, int rows, int h, long long key0,
           long long keys) {
         while (cta_now < cta) cta_first[++cta_now] = piece;
         SharedPiece p{};
         p.q_row0 = s.q_row0;
         p.q_pos0 = s.q_pos0;
         p.q_pos_step = s.q_pos_step;
         p.r0 = (int32_t)r0;
         p.rows = rows;
         p.kv_head = h;
         p.kv_row = (int32_t)(s.kv_row0 + key0);
         p.key0 = (int32_t)key0;
         p.keys = (int32_t)keys;
         p.ws_row = ws_row;
         p.flags = split(rows, keys) ? kPieceSplit : 0;
         ws_row += parts(rows, keys);
         pieces[piece++] = p;
       });
  unit_first[unit] = piece;
  while (cta_now < plan->num_ctas) cta_first[++cta_now] = piece;
  return CPATTN_OK;
}

extern "C" int cp_shared_workspace_size(const cp_shared_plan_t* plan, int dv, int64_t* bytes) {
  if (!plan || !bytes || !plan_ok(*plan) || dv < 4 || dv % 4 || dv > 1024)
    return CPATTN_ERR_INVALID_ARG;
  *bytes = std::max<int64_t>(16, plan->ws_rows * (dv + 1) * 4);
  return CPATTN_OK;
}
