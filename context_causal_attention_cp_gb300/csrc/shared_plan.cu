// Host plan of cp_attn_shared: units, their cut into pieces and the merge lists.
//
// The units (segment, packed-row tile, KV head), kind by kind, are walked in a
// fixed order and their keys dealt to the thread blocks one after the other: each
// block is filled up to a budget, so a unit is cut only where a block is full (a block
// with small units has no others).  The smallest budget that needs no more than num_ctas
// blocks is found by bisection.  A piece costs its KV tiles plus a fixed part (its queries' load and its
// partial's store), so that short units are not shredded.  A block's run of single
// units is cut once more, at half its KV tiles, between the block's two streams.
// Nothing is allocated: each pass walks the segment table again.
#include <algorithm>
#include <cstdint>

#include "shared_plan.h"

namespace cpattn {
namespace {

constexpr int kKeys = kSharedTileKeys;
// Costs by the kind of unit (dual, single, small), of a KV tile and of a piece's fixed
// part, in about 80 ns.  Fitted to whole calls in bf16 at d = 128: a block's dual tile
// takes 1.9 us, a small tile 1.0, a small piece 1.1 besides.  The one table serves e4m3
// and d = 64, too: in e4m3 (2.6, 1.1 and 1.4 us) blocks with dual units end about a tenth
// later than an even deal would let them.
// The fixed part of a dual or single piece (its queries, 128 KB of partial rows, their
// merge) is 3 to 4 us, and its cost is above that, which keeps units in few pieces.
constexpr int kCosts[2][3] = {{24, 16, 12}, {90, 50, 20}};
long long tile_cost(int rows) { return kCosts[0][shared_kind(rows)]; }
long long piece_cost(int rows) { return kCosts[1][shared_kind(rows)]; }
constexpr int kMinCost = std::min({kCosts[0][0] + kCosts[1][0], kCosts[0][1] + kCosts[1][1],
                                   kCosts[0][2] + kCosts[1][2]});
constexpr int kMaxCost = std::max({kCosts[0][0] + kCosts[1][0], kCosts[0][1] + kCosts[1][1],
                                   kCosts[0][2] + kCosts[1][2]});
constexpr long long kMaxUnits = 1LL << 22;
constexpr int kMaxCtas = 4096;

long long last_pos(const cp_segment_t& s) {
  return (long long)s.q_pos0 + (long long)(s.q_len - 1) * s.q_pos_step;
}
// Whether some row of s sees a key (else its key run is not read and may lie anywhere).
bool sees_keys(const cp_segment_t& s) { return s.q_len > 0 && last_pos(s) >= 0; }
long long num_tiles(const cp_segment_t& s, int g) {
  return ((long long)s.q_len * g + CPATTN_SHARED_ROWS - 1) / CPATTN_SHARED_ROWS;
}
long long kv_tiles(long long keys) { return (keys + kKeys - 1) / kKeys; }

// The line of all units' keys.
struct Line {
  const cp_segment_t* segs;
  int num_segs, g, Hkv;
};
// A place in the line: the next key to deal is key0 of the unit (seg, tile, head).
struct Place {
  int kind = 0;          // units of this kind, then those of the next
  bool end = false;
  int seg = 0, head = 0;
  long long tile = 0, key0 = 0;
  long long unit0 = 0;   // unit of (seg, tile 0, head 0)
  int rows = 0;          // of the unit
  long long keys = 0;    // that the unit's last row sees (its other rows no more)
};
struct Cut {
  const cp_segment_t* seg;
  long long unit, r0, key0, keys;
  int rows, head;
};

void measure(const Line& L, Place& p) {
  const cp_segment_t& s = L.segs[p.seg];
  const long long packed = (long long)s.q_len * L.g, r0 = p.tile * CPATTN_SHARED_ROWS;
  p.rows = (int)std::min<long long>(CPATTN_SHARED_ROWS, packed - r0);
  const long long pos = s.q_pos0 + ((r0 + p.rows - 1) / L.g) * s.q_pos_step;
  p.keys = std::max<long long>(0, pos + 1);
}
// Moves p on to the next key, if it is past the last of its unit (or at a unit of
// the other kind or without keys).
void settle(const Line& L, Place& p) {
  while (!p.end) {
    if (p.seg >= L.num_segs) {
      const int kind = p.kind + 1;
      p = Place{};
      p.kind = kind;
      p.end = kind > 2;
      continue;
    }
    if (p.tile >= num_tiles(L.segs[p.seg], L.g)) {
      p.unit0 += p.tile * L.Hkv;
      ++p.seg;
      p.tile = p.key0 = 0;
      p.head = 0;
      continue;
    }
    measure(L, p);
    if (shared_kind(p.rows) != p.kind || p.keys == 0) {
      ++p.tile;
      p.head = 0;
      p.key0 = 0;
      continue;
    }
    if (p.key0 < p.keys) return;
    p.key0 = 0;
    if (++p.head >= L.Hkv) {
      p.head = 0;
      ++p.tile;
    }
  }
}
// The dual units of a segment's tiles read the same keys.  A tile whose units fill
// kAlignBlocks blocks begins with a block of its own, so that every tile is cut at the
// same keys and the blocks of all tiles meet a key while it is in L2 (a 64K prefix of
// 256 tokens with 1024 keys each, 8 KV heads: 315 us for the call instead of 315 to 365).
constexpr int kAlignBlocks = 8;
bool begins_block(const Line& L, const Place& p, long long budget) {
  return p.kind == 0 && p.tile > 0 && p.head == 0 && p.key0 == 0 &&
         L.Hkv * kv_tiles(p.keys) * tile_cost(p.rows) / kAlignBlocks >= budget;
}
// One thread block's share: calls f(cut) for each of its pieces.
template <class F>
void share(const Line& L, Place& p, long long budget, F&& f) {
  long long used = 0;
  settle(L, p);
  const bool small = p.kind == 2;
  for (; !p.end; settle(L, p)) {
    if ((p.kind == 2) != small || (used > 0 && begins_block(L, p, budget))) return;
    const long long cost = tile_cost(p.rows), fixed = piece_cost(p.rows);
    const long long fit = std::min((budget - used - fixed) / cost, kv_tiles(p.keys - p.key0));
    if (budget - used < fixed + cost) return;
    const long long n = std::min(p.keys - p.key0, fit * kKeys);
    f(Cut{L.segs + p.seg, p.unit0 + p.tile * L.Hkv + p.head, p.tile * CPATTN_SHARED_ROWS, p.key0, n,
          p.rows, p.head});
    p.key0 += n;
    used += fixed + fit * cost;
  }
}
bool fits(const Line& L, long long budget, int num_ctas) {
  Place p;
  for (int c = 0; c < num_ctas; ++c) share(L, p, budget, [](const Cut&) {});
  settle(L, p);
  return p.end;
}
// Calls f(cta, cut, stream) for every piece in the table's order of each kind (stream:
// that has a single piece).
template <class F>
void deal(const Line& L, long long budget, int num_ctas, F&& f) {
  Place p;
  for (int c = 0; c < num_ctas; ++c) {
    Place ahead = p;
    long long tiles = 0;
    share(L, ahead, budget, [&](const Cut& k) { if (shared_kind(k.rows) == 1) tiles += kv_tiles(k.keys); });
    long long left = (tiles + 1) / 2;  // KV tiles that stream 0 still takes
    share(L, p, budget, [&](const Cut& k) {
      if (shared_kind(k.rows) != 1) {
        f(c, k, 0);
        return;
      }
      Cut a = k, b = k;
      a.keys = std::min(k.keys, left * kKeys);
      b.key0 += a.keys;
      b.keys -= a.keys;
      left -= kv_tiles(a.keys);
      if (a.keys > 0) f(c, a, 0);
      if (b.keys > 0) f(c, b, 1);
    });
  }
}

bool plan_ok(const cp_shared_plan_t& p) {
  return p.num_q_rows >= 0 && p.Hq >= 1 && p.Hkv >= 1 && p.Hq % p.Hkv == 0 && p.num_ctas >= 2 &&
         p.num_ctas <= kMaxCtas && p.num_units >= 0 && p.num_pieces >= 0 && p.num_entries >= 0 &&
         p.kv_rows >= 0 && p.budget >= 0 && p.ws_rows >= 0 && p.table_ints == shared_table(p).total;
}

int check_segments(const cp_segment_t* segs, int num_segs, int num_q_rows) {
  for (int i = 0; i < num_segs; ++i) {
    const cp_segment_t& s = segs[i];
    if (s.q_len < 0 || s.q_row0 < 0 || (long long)s.q_row0 + s.q_len > num_q_rows ||
        s.q_pos_step < 0 || s.kv_len < 0)
      return CPATTN_ERR_INVALID_ARG;
    if (!sees_keys(s)) continue;
    if (s.kv_row0 < 0 || last_pos(s) + 1 > s.kv_len) return CPATTN_ERR_INVALID_ARG;
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
      Hq % Hkv != 0 || num_ctas < 2 || num_ctas > kMaxCtas)
    return CPATTN_ERR_INVALID_ARG;
  if (num_segs > kMaxUnits) return CPATTN_ERR_TOO_LARGE;
  const int rc = check_segments(segs, num_segs, num_q_rows);
  if (rc != CPATTN_OK) return rc;
  const Line L{segs, num_segs, Hq / Hkv, Hkv};
  long long tiles = 0, entries = 0, kv_rows = 0;
  for (int i = 0; i < num_segs; ++i) {
    const cp_segment_t& s = segs[i];
    tiles += num_tiles(s, L.g);
    entries += s.q_len;
    if (sees_keys(s)) kv_rows = std::max(kv_rows, s.kv_row0 + last_pos(s) + 1);
  }
  if (tiles * Hkv > kMaxUnits || entries > 0x3fffffffLL) return CPATTN_ERR_TOO_LARGE;
  long long cost = 0;
  {
    Place p;
    for (int part = 0; part < 2; ++part)  // the small units are a share of their own
      share(L, p, INT64_MAX / 4, [&](const Cut& k) {
        cost += piece_cost(k.rows) + kv_tiles(k.keys) * tile_cost(k.rows);
      });
  }
  long long lo = kMinCost, hi = std::max<long long>(lo, cost / num_ctas + 2 * kMaxCost);
  while (!fits(L, hi, num_ctas)) {
    // one block cannot hold small units and others: it takes two
    if (hi > (1LL << 40)) return CPATTN_ERR_INVALID_ARG;
    hi *= 2;
  }
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (fits(L, mid, num_ctas)) hi = mid;
    else lo = mid + 1;
  }
  if (hi > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  long long pieces = 0, ws_rows = 0;
  deal(L, hi, num_ctas, [&](int, const Cut& k, int) {
    ++pieces;
    ws_rows += k.rows;
  });
  if (ws_rows > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  plan->num_q_rows = num_q_rows;
  plan->Hq = Hq;
  plan->Hkv = Hkv;
  plan->num_ctas = num_ctas;
  plan->num_units = (int32_t)(tiles * Hkv);
  plan->num_pieces = (int32_t)pieces;
  plan->num_entries = (int32_t)entries;
  plan->kv_rows = (int32_t)kv_rows;
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
  const Line L{segs, num_segs, plan->Hq / plan->Hkv, plan->Hkv};
  const int N = plan->num_q_rows;
  // the table must be the one that was sized: check the counts before writing
  long long tiles = 0, ents = 0, np = 0, kinds[3] = {}, ws = 0;
  for (int i = 0; i < num_segs; ++i) {
    tiles += num_tiles(segs[i], L.g);
    ents += segs[i].q_len;
  }
  if (tiles * L.Hkv != plan->num_units || ents != plan->num_entries ||
      !fits(L, plan->budget, plan->num_ctas))
    return CPATTN_ERR_INVALID_ARG;
  deal(L, plan->budget, plan->num_ctas, [&](int, const Cut& k, int) {
    ++np;
    ++kinds[shared_kind(k.rows)];
    ws += k.rows;
  });
  if (np != plan->num_pieces || ws != plan->ws_rows) return CPATTN_ERR_INVALID_ARG;

  const SharedTable T = shared_table(*plan);
  auto* ctas = reinterpret_cast<SharedCta*>(table);
  auto* pieces = reinterpret_cast<SharedPiece*>(table + T.pieces);
  auto* units = reinterpret_cast<SharedUnit*>(table + T.units);
  int32_t* row_first = table + T.row_first;
  int32_t* entries = table + T.entries;

  // entries of each query row, segment by segment
  row_first[T.entries - T.row_first - 1] = 0;  // the padding
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
    unit0 += (int32_t)num_tiles(s, L.g) * L.Hkv;
  }
  for (int n = N; n > 0; --n) row_first[n] = row_first[n - 1];
  row_first[0] = 0;

  for (int u = 0; u < plan->num_units; ++u) units[u] = SharedUnit{};
  for (int c = 0; c < plan->num_ctas; ++c) ctas[c] = SharedCta{};
  // the next piece of each kind
  int32_t next[3] = {0, (int32_t)kinds[0], (int32_t)(kinds[0] + kinds[1])}, ws_row = 0;
  int cta = -1;
  auto open = [&](int c) {  // empty ranges from here on
    while (cta < c) {
      ++cta;
      ctas[cta].dual0 = ctas[cta].dual1 = next[0];
      ctas[cta].single0 = ctas[cta].single1 = ctas[cta].single2 = next[1];
      ctas[cta].small0 = ctas[cta].small1 = next[2];
    }
  };
  deal(L, plan->budget, plan->num_ctas, [&](int c, const Cut& k, int stream) {
    open(c);
    const int kind = shared_kind(k.rows);
    const int32_t at = next[kind]++;
    if (kind == 0) ctas[c].dual1 = at + 1;
    if (kind == 1 && stream == 0) ctas[c].single1 = at + 1;
    if (kind == 1) ctas[c].single2 = at + 1;
    if (kind == 2) ctas[c].small1 = at + 1;
    SharedPiece p{};
    p.q_row0 = k.seg->q_row0;
    p.q_pos0 = k.seg->q_pos0;
    p.q_pos_step = k.seg->q_pos_step;
    p.r0 = (int32_t)k.r0;
    p.rows = k.rows;
    p.kv_head = k.head;
    p.kv_row = (int32_t)(k.seg->kv_row0 + k.key0);
    p.key0 = (int32_t)k.key0;
    p.keys = (int32_t)k.keys;
    p.ws_row = ws_row;
    ws_row += k.rows;
    pieces[at] = p;
    SharedUnit& u = units[k.unit];  // (its pieces come one after the other)
    if (u.parts == 0) u.ws_row = p.ws_row;
    ++u.parts;
    u.rows = k.rows;
  });
  open(plan->num_ctas - 1);
  return CPATTN_OK;
}

extern "C" int cp_shared_workspace_size(const cp_shared_plan_t* plan, int dv, int64_t* bytes) {
  if (!plan || !bytes || !plan_ok(*plan) || dv < 4 || dv % 4 || dv > 1024)
    return CPATTN_ERR_INVALID_ARG;
  *bytes = std::max<int64_t>(16, plan->ws_rows * (dv + 1) * 4);
  return CPATTN_OK;
}
