// Threads, registers and shared memory of the two attention kernels over a paged cache, by
// themselves, so that a host program can look at their layouts.
#pragma once
#include "attn_tree.cuh"

namespace cpattn {
namespace {

constexpr int kPieces = 4;  // in the ring
using Pieces = PieceRing<kPieces>;

// ---- 128 and 256 rows (attn_tree_mma.cu) ----
constexpr int kKWarp = 8, kVWarp = 9, kMmaWarp = 10, kQWarp = 11, kConvertWarp = 12;
constexpr int kConvertWarps = 8, kConvertThreads = 32 * kConvertWarps;

template <int D, bool QUANT, bool DUAL>
struct MmaCfg {
  static constexpr int kThreads = QUANT ? 640 : 384;
  static constexpr int kRegsLaunch = QUANT ? 96 : 168;
  // (e4m3 dual: with 128 and 72 the other warps spill, trees of 64 464 against 440 us; single:
  // with 120 and 80 the softmax does, trees of 32 323 against 308 us)
  static constexpr int kRegsSoftmax = !QUANT ? 200 : DUAL ? 120 : 128, kRegsOther = !QUANT ? 104 : DUAL ? 80 : 72;
  static_assert(kRegsSoftmax * 256 + kRegsOther * (kThreads - 256) <= kRegsLaunch * kThreads,
                "register split exceeds the launch allocation");
  static constexpr int kQTile = BM * D * 2;
  static constexpr int kTile = BN * D * 2;  // a K or V tile of 16-bit elements
  static constexpr int kRawTile = BN * D;   // an e4m3 K or V tile
  static constexpr int kStages = QUANT ? (D == 128 ? 3 : 6) : D == 128 ? 5 : 10;
  static constexpr int kRawStages = !QUANT ? 0 : D == 64 ? 8 : 3;
  static constexpr int kRingOff = 2 * kQTile;
  static constexpr int kRawOff = kRingOff + kStages * kTile;
  static constexpr int kScaleOff = kRawOff + kRawStages * kRawTile;  // of each raw row, and (K) of V's
  static constexpr int kNoteOff = kScaleOff + kRawStages * BN * 8;   // RawNote of each raw tile
  static constexpr int kExpOff = kNoteOff + kRawStages * 16;         // (ek, ev) of tiles n mod 8
  static constexpr int kLiftOff = kExpOff + 64;                      // exponents of query rows, [kLifts][units][BM]
  // A place for each of the piece ring's: the softmax may look at a piece's exponents until it is
  // done with the piece, which its place in the ring waits for and the queries' buffer does not.
  static constexpr int kLifts = kPieces, kLiftRows = DUAL ? 2 * BM : BM;
  // Scales of tiles n mod kTails that hold new keys, [kTails][K, V][BN]: the softmax has them from the
  // conversion of a K tile to its P V, while the ring takes kStages more places, of which K has every
  // other one (and one ahead).
  static constexpr int kTails = !QUANT ? 0 : kStages + 3 < 2 * 4 ? 4 : 8;
  static_assert(!QUANT || 2 * kTails > kStages + 3, "scales of tiles in flight");
  static constexpr int kTailOff = kLiftOff + (QUANT ? kLifts * kLiftRows : 0);
  static constexpr int kMlOff = kTailOff + kTails * 2 * BN * 4;  // single: (m, l) of each stream's rows
  static constexpr int kEvOff = kMlOff + (DUAL ? 0 : 2 * BM * 8);    // and O's exponent
  static constexpr int kBadOff = kEvOff + (QUANT && !DUAL ? 2 * BM : 0);  // value rows that are not finite
  static constexpr int kPiecesOff = kBadOff + 2 * 2 * 16 + (QUANT ? kStages * 16 : 0);
  static constexpr int kBarOff = kPiecesOff + (int)sizeof(Pieces);
  static constexpr int kNumBars = 2 * kStages + 2 * kRawStages + 2 * 5 + 1;
  static constexpr int kWordOff = kBarOff + kNumBars * 8;
  static constexpr int kSumOff = (kWordOff + 64 + 7) & ~7;  // of tree_start, a word a warp
  static constexpr int kSmemBytes = kSumOff + kThreads / 32 * 8;
  static_assert(kBarOff % 8 == 0 && kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kTmemCols = 4 * 128;  // S of each stream, then O of each
};

// What a producer tells the converters about a raw tile.
struct alignas(16) RawNote {
  int live;   // rows up to the unit's end
  int fresh;  // first row that is a new key
  int first;  // of its piece and stream
};
static_assert(sizeof(RawNote) == 16, "kNoteOff's places");

// ---- 8 and 16 rows (attn_tree_small.cu) ----
constexpr int kSmallWarps = 8, kSmallThreads = 384;
constexpr int kMaxStages = 12;

template <int D, bool QUANT, int NQ>
struct TreeCfg {
  static constexpr int kRows = 8 * NQ;  // of a unit
  static constexpr int kTeams = QUANT ? 2 : 1;
  static constexpr int kKeys = BN * kTeams / kSmallWarps;  // of a warp in its team's tiles
  static constexpr int kTile = BN * D * (QUANT ? 1 : 2);
  static constexpr int kScales = QUANT ? BN * 4 : 0;  // the rows' scales, fp32
  static constexpr int kQ = kRows * D * 2;            // two of them
  static constexpr int kJoin = kSmallWarps * 8 * NQ * D * 4;
  static constexpr int kMl = kSmallWarps * 8 * NQ * 8;
  static constexpr int kFixed = 2 * kQ + kJoin + kMl + (int)sizeof(Pieces) + (2 * kMaxStages + 4) * 8 + 64 + 256 + 1024;
  static constexpr int kFit = (232448 - kFixed) / (kTile + kScales);
  // With two teams a multiple of 4: K and V of the tiles n, n + kStages / 2, ... share slots, and
  // then one team has them all, so that its warps see every phase of their barriers.
  static constexpr int kMost = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kStages = kTeams == 2 ? kMost / 4 * 4 : kMost;
  static constexpr int kScaleOff = kStages * kTile;
  static constexpr int kQOff = kScaleOff + kStages * kScales;
  static constexpr int kJoinOff = kQOff + 2 * kQ;
  static constexpr int kMlOff = kJoinOff + kJoin;  // (m, l) of each warp's rows
  static constexpr int kPiecesOff = kMlOff + kMl;
  static constexpr int kBarOff = kPiecesOff + (int)sizeof(Pieces);
  static constexpr int kWordOff = kBarOff + (2 * kStages + 4) * 8;
  static constexpr int kSumOff = kWordOff + 64;  // of tree_start
  static constexpr int kSmemBytes = kSumOff + 256 + 1024;  // + align slack
  static_assert(kStages >= 4 && kSmemBytes <= 232448, "shared memory budget");
};

}  // namespace
}  // namespace cpattn
