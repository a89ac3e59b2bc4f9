// Attention for a batch that shares keys (cp_attn_shared).
//
// A unit is up to CPATTN_SHARED_ROWS packed rows (query row i, head j of the KV
// head's group, at i*g + j) against one run of keys; the plan cuts the units
// into pieces and gives each thread block a list of them.  A piece's partial
// result per row is (O, L) over its keys,
//     L = ln sum_k exp(S_k),  O = sum_k exp(S_k - L) V_k,
// in fp32; the merge combines a row's partials by the log-sum-exp rule
//     m = max L_j, w_j = exp(L_j - m), O = sum w_j O_j / sum w_j, L = m + ln sum w_j.
//
// attn_shared_kernel: one resident block per SM walks its pieces; its loads, its
// MMAs and its queries run ahead across piece ends.
//   warps 0-7    two softmax warpgroups (streams), one row per thread: query rows
//                to shared memory (any group size, any stride), S from TMEM, online
//                softmax in base 2 with a lazily moved maximum, P back to TMEM in 16
//                bits, the partial to the workspace.
//   warp 8       producer: K and V tiles of 128 keys by TMA, in the order of use,
//                through one ring; of a run's last tile only the rows it has.
//   warps 9, 10  MMA issuers, one per stream: S = Q K^T and O += P V (tcgen05); one
//                stream's softmax runs under the other's MMAs.  Two, because one
//                thread's issue of both streams took 2300 cycles a step against 1270
//                of tensor work.
//   warps 12-15  (e4m3 cache) codes to f16 tiles.
// A unit of two MMA tiles (dual) gives both streams every KV tile; the pieces of
// units of one tile (single) belong to one stream each, and the streams' KV tiles
// alternate.  Blocks with units of up to 8 rows (small) run attn_shared_small.cuh.
//
// What bounds it: dual units the chain S -> softmax -> P -> P V of a stream, 3600 cycles
// a KV tile of which the two streams' MMAs hold 3000 (256 tokens of 32 heads on a 64K
// prefix, d = 128: 216 us a call in bf16, 1.27 PFLOP/s, 0.65 of cuBLAS; 272 us over
// codes, whose way through shared memory is half as long again).  Measured and not
// kept: P in two halves, turns before the last MMA, MMAs issued by whole warps, eight
// converter warps, a first tile over nothing that brings the code in.
//
// e4m3 cache: both products run in f16, which holds a code exactly and takes two
// instructions for two codes (bf16 takes 6.5, more than a step has issue slots
// for).  K row r enters as code * 2^(e_r - E), E the tile's largest e, and 2^E goes
// into the scores' factor.  An f16 ends at 2^-24: a row within 2^15 of the largest scale
// loses nothing, one down to 2^-24 of it less than 2^-32 of the tile's largest element
// (the rounding of code times factor; less than an fp32 score resolves), and one below
// that has a factor of 0 and counts as zeros, up to 2^-24 of that element.  V the same
// with E the largest e that the stream has met in the piece; O is rescaled when that
// grows, and a V row below 2^-24 adds nothing even where it has all of the weight.  A
// query row enters as f16 times the power of two that brings its largest element to
// [2^14, 2^15), so that elements down to 2^-30 of it keep bf16's 8 bits.  P in f16 is
// off by at most 2^-11 of a weight (bf16: 2^-8) down to 2^-21 of the largest weight, and
// by 2^-32 of the largest below that.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "shared_plan.h"
#include "trace.h"

namespace cpattn {
namespace {

constexpr int kRows = CPATTN_SHARED_ROWS;
constexpr int BN = kSharedTileKeys;
constexpr int kTailRows = 16;                   // box rows of the loads of a run's last tile
constexpr int kProducerWarp = 8, kMmaWarp = 9;  // MMA: 9 and 10
constexpr int kConvertWarp = 12;                // to 15
constexpr int kConvertThreads = 128;

struct SharedParams {
  const int32_t* table;
  long long pieces, units, row_first, entries;  // word offsets
  int num_units, num_pieces, num_entries, num_q_rows, Hq, Hkv, g;
  uint32_t g_mul, g_shift;  // n / g = umulhi(n, g_mul) >> g_shift, see group_div
  long long ws_rows;
  const __nv_bfloat16* q;
  long long q_row, q_head;
  const float* ks;
  const float* vs;
  long long s_head;
  int num_kv_rows;
  float scale_log2;
  void* o;
  int o_f32;
  float* lse;
  float* ws_o;
  float* ws_l;  // log2 units
  int32_t* status;
  unsigned long long timeout_ns;
  int withhold_q;  // test hook: queries are never published (see cp_attn_debug)
};

template <int D, bool QUANT>
struct SharedCfg {
  static constexpr int kThreads = QUANT ? 512 : 384;
  static constexpr int kRegsLaunch = QUANT ? 128 : 168;
  static constexpr int kRegsSoftmax = 200, kRegsOther = QUANT ? 56 : 104;
  static_assert(kRegsSoftmax * 256 + kRegsOther * (kThreads - 256) <= kRegsLaunch * kThreads,
                "register split exceeds the launch allocation");
  static constexpr int kQTile = BM * D * 2;
  static constexpr int kTile = BN * D * 2;  // a K or V tile of 16-bit elements
  static constexpr int kRawTile = BN * D;   // an e4m3 K or V tile
  // 227 KB hold five tiles of 32 KB beside the queries, or three and four of codes
  static constexpr int kStages = QUANT ? 3 : 5;
  static constexpr int kRawStages = QUANT ? 4 : 0;
  static constexpr int kRingOff = 2 * kQTile;
  static constexpr int kRawOff = kRingOff + kStages * kTile;
  static constexpr int kMulOff = kRawOff + kRawStages * kRawTile;  // f16 factor of each raw row
  static constexpr int kNoteOff = kMulOff + kRawStages * BN * 2;   // RawNote of each raw tile
  static constexpr int kExpOff = kNoteOff + kRawStages * 16;       // exponents, see RawNote::which
  static constexpr int kBarOff = kExpOff + 48;
  static constexpr int kNumBars = 4 * kStages + 2 * kRawStages + 8 + 4;
  static constexpr int kWordOff = kBarOff + kNumBars * 8;  // TMEM slot, abort, loads, phases, tiles[2]
  static constexpr int kSmemBytes = kWordOff + 32 + 1024;  // + align slack
  static_assert(kBarOff % 8 == 0 && kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kTmemCols = 512;  // S of each stream, then O of each
};

// Orders this thread's shared-memory accesses before later ones of the async proxy (TMA,
// tcgen05.mma reading shared memory).
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// What the producer tells the converters about a raw tile.
struct RawNote {
  static constexpr int kNoteV = 8;
  int live;     // rows up to the run's end
  int which;    // RingTile::which, | kNoteV of a V tile
  int ek, ev;   // of a K tile: E of it, and E of its V tile
};

// Bounded waits, of one thread and of a whole warp (uniform).  They read the timer
// only after a few hundred polls: it is far from the SM, and a read at every wait
// that does not succeed at once costs more than the wait.
constexpr uint32_t kPollsPerCheck = 256;
__device__ __forceinline__ bool give_up(uint64_t& t0, const volatile int* abort, uint64_t timeout) {
  const uint64_t now = global_timer_ns();
  if (t0 == 0) t0 = now;
  return (abort && *abort != 0) || now - t0 > timeout;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, const volatile int* abort,
                                         uint64_t timeout) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i)
    if (i % kPollsPerCheck == 0 && give_up(t0, abort, timeout)) return false;
  return true;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const volatile int* abort,
                                          uint64_t timeout) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i)
    if (i % kPollsPerCheck == 0 &&
        __shfl_sync(0xffffffffu, (int)give_up(t0, abort, timeout), 0))
      return false;
  return true;
}

// n / g for 0 <= n < 2^31: with 2^s the power of two from g on, g_mul = floor(2^(31+s)
// / g) + 1 and n g_mul 2^-(31+s) exceeds n / g by less than 1 / g.
__device__ __forceinline__ int group_div(const SharedParams& p, int n) {
  return p.g == 1 ? n : (int)(__umulhi((uint32_t)n, p.g_mul) >> p.g_shift);
}

__device__ __forceinline__ SharedPiece load_piece(const SharedParams& p, int i) {
  const int4* w = reinterpret_cast<const int4*>(p.table + p.pieces) + 3LL * i;
  const int4 a = __ldg(w), b = __ldg(w + 1), c = __ldg(w + 2);
  return SharedPiece{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, {c.z, c.w}};
}
__device__ __forceinline__ bool piece_ok(const SharedParams& p, const SharedPiece& pc, int kind) {
  return pc.rows >= 1 && pc.rows <= kRows && shared_kind(pc.rows) == kind && pc.r0 >= 0 &&
         pc.r0 <= 0x7fffffff - kRows && pc.q_row0 >= 0 &&
         (long long)pc.q_row0 + group_div(p, pc.r0 + pc.rows - 1) < p.num_q_rows &&
         pc.kv_head >= 0 && pc.kv_head < p.Hkv && pc.keys >= 1 && pc.key0 >= 0 && pc.kv_row >= 0 &&
         (long long)pc.kv_row + pc.keys <= p.num_kv_rows && pc.ws_row >= 0 &&
         (long long)pc.ws_row + pc.rows <= p.ws_rows;
}
__device__ __forceinline__ int num_tiles(int keys) { return (keys - 1) / BN + 1; }

__device__ __forceinline__ SharedCta load_cta(const SharedParams& p) {
  const int4* w = reinterpret_cast<const int4*>(p.table) + 2LL * blockIdx.x;
  const int4 a = __ldg(w);
  const int4 b = __ldg(w + 1);
  return SharedCta{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
// Checks every piece of this block's list against the buffers: the roles below walk
// the list on their own and rely on it.  tiles[s]: KV tiles of stream s's single units
// (zeroed by the caller before a barrier).  All threads call it; false (and
// CPATTN_ERR_RANGE) when the list cannot be run.
__device__ __forceinline__ bool check_list(const SharedParams& p, const SharedCta& c, int* tiles) {
  bool ok = c.dual0 >= 0 && c.dual0 <= c.dual1 && c.dual1 <= p.num_pieces && c.single0 >= 0 &&
            c.single0 <= c.single1 && c.single1 <= c.single2 && c.single2 <= p.num_pieces &&
            c.small0 >= 0 && c.small0 <= c.small1 && c.small1 <= p.num_pieces &&
            (c.small0 == c.small1 || (c.dual0 == c.dual1 && c.single0 == c.single2));
  if (ok) {
    for (int i = c.dual0 + threadIdx.x; i < c.dual1; i += blockDim.x)
      ok = ok && piece_ok(p, load_piece(p, i), 0);
    for (int i = c.small0 + threadIdx.x; i < c.small1; i += blockDim.x)
      ok = ok && piece_ok(p, load_piece(p, i), 2);
    for (int i = c.single0 + threadIdx.x; i < c.single2; i += blockDim.x) {
      const SharedPiece pc = load_piece(p, i);
      ok = ok && piece_ok(p, pc, 1);
      if (ok) atomicAdd(tiles + (i >= c.single1), num_tiles(pc.keys));
    }
  }
  ok = __syncthreads_and(ok);
  // (not for a list of small units: their path goes on to lay out this memory otherwise)
  if (ok && c.single0 < c.single2) ok = tiles[0] == tiles[1] || tiles[0] == tiles[1] + 1;
  if (!ok && threadIdx.x == 0) set_status(p.status, CPATTN_ERR_RANGE);
  return ok;
}

// Byte offset of 16-code chunk `chunk` of row `row` in a raw e4m3 tile: rows of D bytes,
// their chunks swizzled (128-byte swizzle at D = 128, 64-byte at D = 64).
template <int D>
__device__ __forceinline__ uint32_t code_at(int row, int chunk) {
  return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// Two barriers at once (their polls overlap).
__device__ __forceinline__ bool wait_warp2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           const volatile int* abort, uint64_t timeout) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
    if (__all_sync(0xffffffffu, x && y)) return true;
    if (i % kPollsPerCheck == 0 && __shfl_sync(0xffffffffu, (int)give_up(t0, abort, timeout), 0))
      return false;
  }
}

// One K or V tile of the ring.
struct RingTile {
  int kv_row, kv_head, live;  // its first row, head, and rows up to the run's end
  bool is_v, first;           // first: of its piece
  int which;  // 2 * stream + (step of the stream) % 2; of a dual unit: 4 + tile % 2
  __device__ __forceinline__ int user() const { return which >> 1; }  // stream, or 2: both
};
// Calls f(tile) for the K and V tiles of a list in the order in which the MMA warps
// use them, until it returns false: K0 V0 K1 V1 ... for dual units, then K0 K1 V0
// K2 V1 ... for the steps of the single units, step n being the next KV tile of
// stream n & 1.
template <class F>
__device__ __forceinline__ bool for_each_ring_tile(const SharedParams& p, const SharedCta& c,
                                                   int steps, F&& f) {
  int tile = 0;
  for (int i = c.dual0; i < c.dual1; ++i) {
    const SharedPiece pc = load_piece(p, i);
    RingTile r{pc.kv_row, pc.kv_head, pc.keys, false, true, 0};
    for (const int end = 2 * (tile + num_tiles(pc.keys)); 2 * tile < end;) {
      r.which = 4 + (tile & 1);
      if (!f(r)) return false;
      if (r.is_v) {
        ++tile;
        r.kv_row += BN;
        r.live -= BN;
        r.first = false;
      }
      r.is_v = !r.is_v;
    }
  }
  int next0 = c.single0, next1 = c.single1;
  RingTile t0{0, 0, 0, false, true, 0}, t1 = t0;  // the streams' last K tiles
  for (int j = 0; j < 2 * steps; ++j) {
    const bool is_v = j == 2 * steps - 1 || (j > 0 && !(j & 1));
    const int n = j == 2 * steps - 1 ? steps - 1 : is_v ? (j - 2) >> 1 : (j + 1) >> 1;
    RingTile r = n & 1 ? t1 : t0;
    r.is_v = is_v;
    if (!is_v) {
      r.kv_row += BN;
      r.live -= BN;
      r.first = r.live <= 0;
      if (r.first) {
        const SharedPiece pc = load_piece(p, n & 1 ? next1++ : next0++);
        r.kv_row = pc.kv_row;
        r.kv_head = pc.kv_head;
        r.live = pc.keys;
      }
      r.which = 2 * (n & 1) + ((n >> 1) & 1);
      if (n & 1) t1 = r;
      else t0 = r;
    }
    if (!f(r)) return false;
  }
  return true;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four e4m3 codes as f16, times m (f16 in both halves).
__device__ __forceinline__ uint2 codes_to_f16(uint32_t c, uint32_t m) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)c));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(c >> 16)));
  return make_uint2(mul_f16x2(h0, m), mul_f16x2(h1, m));
}
__device__ __forceinline__ float exp2_int(int e) {  // e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// Exponent of a scale s >= 0, such that exp2_int takes it and its negative.
__device__ __forceinline__ int exponent_of(float s) {
  return min(max((int)(__float_as_uint(s) >> 23) - 127, -126), 126);
}
// Factor f s of a raw e4m3 score, f > 0 of its query row and s of its key (or key tile).
// Not below a normal number: a zero row over zero keys would come to 0, and a masked -inf
// times 0 is NaN.  Not infinite: a score of 0 between orthogonal large rows stays 0.  A
// raw score is below 2^31 (2^15 448 d), so that with a raised factor it is still nothing.
__device__ __forceinline__ float score_factor(float f, float s) {
  return fminf(fmaxf(f * s, 0x1p-126f), 0x1.fffffep127f);
}
constexpr uint32_t idesc_16bit_f32(bool f16, int M, int N, int b_mn) {
  return idesc_bf16_f32(M, N, 0, b_mn) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}

// f16 weights are taken by a maximum that is kF16Lift too small: an f16 below 2^-14 loses
// bits, which now begins at 2^-21 of the largest weight (and ends the weight at 2^-32),
// and the largest stays below 2^16.
constexpr float kF16Lift = 7.f;
static_assert(kF16Lift + kMaxSlack < 16.f, "f16 range");

// One KV tile for the rows of a warp (one per lane).  S from TMEM, masked to the `here`
// visible keys of the tile, online softmax in base 2, P (16 bits) back over S, and where
// there is an O (`has_o`), O rescaled when the maximum moves or o_scale != 1.
template <int D, bool QUANT>
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint32_t o_addr, int here, bool has_o,
                                             float o_scale, float sl2, float& m_run,
                                             float& m_use, float& l_run) {
  float x[BN];
  {
    uint32_t v[BN];
#pragma unroll
    for (int q = 0; q < BN / 32; ++q) tmem_ld32p(s_addr + q * 32, v + q * 32);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < BN; ++c) x[c] = __uint_as_float(v[c]);
  }
  if (here < BN) {
#pragma unroll
    for (int c = 0; c < BN; ++c)
      if (c >= here) x[c] = -INFINITY;
  }
  float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
  for (int c = 4; c + 8 <= BN; c += 8) {
    mx0 = fmax3(mx0, x[c], x[c + 1]);
    mx1 = fmax3(mx1, x[c + 2], x[c + 3]);
    mx2 = fmax3(mx2, x[c + 4], x[c + 5]);
    mx3 = fmax3(mx3, x[c + 6], x[c + 7]);
  }
  mx0 = fmax3(mx0, x[BN - 4], x[BN - 3]);
  mx1 = fmax3(mx1, x[BN - 2], x[BN - 1]);
  const float mx = fmaf(fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)), sl2, QUANT ? -kF16Lift : 0.f);
  // The maximum moves only when a tile raises it by more than kMaxSlack (log2
  // units): exponentials stay below 2^kMaxSlack, l uses the same maximum, and O in
  // TMEM is rescaled only then.
  const bool move = mx > m_run + kMaxSlack;
  const float m_new = move ? mx : m_run;
  const float m_new_use = (m_new == -INFINITY) ? 0.f : m_new;
  const float alpha = move ? ex2_approx(m_run - m_new_use) : 1.f;
  float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
  for (int q = 0; q < BN / 32; ++q) {
    uint32_t pk[16];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float a, b;
      ffma2(a, b, x[q * 32 + c], x[q * 32 + c + 1], sl2, sl2, -m_new_use, -m_new_use);
      a = ex2_approx(a);
      b = ex2_approx(b);
      fadd2(sum0, sum1, sum0, sum1, a, b);
      // P in 16 bits, the second product's operand type: off by at most 2^-8 (bf16) or
      // 2^-11 (f16) of each weight; l sums the unrounded values
      pk[c >> 1] = QUANT ? pack_f16x2(a, b) : pack_bf16x2(a, b);
    }
    tmem_st16(s_addr + q * 16, pk);
  }
  l_run = l_run * alpha + (sum0 + sum1);
  const bool need = has_o && (move || o_scale != 1.f);
  if (__any_sync(0xffffffffu, need)) {
    const float a = need ? alpha * o_scale : 1.f;
    uint32_t v[32];
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      tmem_ld32(o_addr + q * 32, v);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * a);
      tmem_st32(o_addr + q * 32, v);
    }
  }
  tmem_wait_st();
  m_run = m_new;
  m_use = m_new_use;
}

// Partial rows in the workspace: those of one piece by chunks of 8 columns, so
// that the lanes of a warp, a row each, store to one place.  Offset of column 8 c of row
// r of `rows`, from the first row's place at D floats a row.
__device__ __forceinline__ int partial_at(int c, int r, int rows) { return (c * rows + r) * 8; }

// 32 bytes, a whole sector.
__device__ __forceinline__ void store8(float* at, const float (&f)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "f"(f[0]), "f"(f[1]),
               "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

}  // namespace
}  // namespace cpattn

#include "attn_shared_small.cuh"  // run_small, on the pieces above

namespace cpattn {
namespace {

template <int D, bool QUANT>
__global__ void __launch_bounds__(SharedCfg<D, QUANT>::kThreads, 1)
attn_shared_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_k_tail,
                   const __grid_constant__ CUtensorMap tm_v_tail, const SharedParams p) {
  using C = SharedCfg<D, QUANT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + 3 * C::kStages;
  uint64_t* raw_full = empty + C::kStages;
  uint64_t* raw_empty = raw_full + C::kRawStages;
  uint64_t* q_full = raw_empty + C::kRawStages;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* turn = o_full + 2;
  uint64_t* bar_drain = turn + 2;
  uint16_t* raw_mul = reinterpret_cast<uint16_t*>(smem + C::kMulOff);
  RawNote* raw_note = reinterpret_cast<RawNote*>(smem + C::kNoteOff);
  int2* tile_exp = reinterpret_cast<int2*>(smem + C::kExpOff);  // (ek, ev) by RingTile::which
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kWordOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued_loads = reinterpret_cast<volatile int*>(tmem_slot + 2);  // for the abort drain
  volatile int* issued_phases = issued_loads + 1;
  int* stream_tiles = reinterpret_cast<int*>(tmem_slot + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_trigger();  // the merge may be scheduled as blocks of this grid end
  // the block's list and the tensor maps travel while the barriers are set up
  SharedCta list = load_cta(p);
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_k_tail);
    prefetch_tmap(&tm_v_tail);
  }
  if (threadIdx.x < 2) stream_tiles[threadIdx.x] = 0;
  __syncthreads();
  if (list.dual0 == list.dual1 && list.single0 == list.single2 && list.small0 == list.small1) return;  // no work
  if (!check_list(p, list, stream_tiles)) return;
  if (list.small0 < list.small1) {
    run_small<D, QUANT>(p, list, smem, &tm_k, &tm_v, &tm_k_tail, &tm_v_tail);
    return;
  }
  const int steps = stream_tiles[0] + stream_tiles[1];  // of the single units
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      for (int u = 0; u < 3; ++u) mbar_init(full + u * C::kStages + i, QUANT ? kConvertThreads : 1);
      mbar_init(empty + i, 2);  // a commit of each stream
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(raw_full + i, 2);  // the TMA copy and the factors
      mbar_init(raw_empty + i, kConvertThreads);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 128);
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 128);
      mbar_init(o_full + s, 1);
      mbar_init(turn + s, 1);
      mbar_init(bar_drain + s, 1);
    }
    *abort_flag = 0;
    *issued_loads = *issued_phases = 0;
    fence_barrier_init();
  }
  if (warp == kProducerWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t q_base = smem_u32(smem);
  const uint32_t ring_base = smem_u32(smem + C::kRingOff);
  // A ring slot has a full barrier for each user (stream 0, stream 1, both), so that
  // every waiter sees all phases of the barriers it waits on; their parities are kept
  // as bits of a word, `user * kStages + slot`.
  auto full_bit = [](int user, int slot) { return user * C::kStages + slot; };
  // Ring places of step n of the single units, behind dual_seq places of dual units.
  auto k_place = [](int n) { return n == 0 ? 0 : 2 * n - 1; };
  auto v_place = [&](int n) { return n == steps - 1 ? 2 * n + 1 : 2 * n + 2; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kProducerWarp) {
      // ---------------------------------------------------------- producer --
      // bf16: one lane.  e4m3: the whole warp, which also turns the scales of the
      // tile's rows into f16 factors, one tile behind the copies it starts.
      constexpr int kSt = QUANT ? C::kRawStages : C::kStages;
      constexpr int kBytes = QUANT ? C::kRawTile : C::kTile;
      constexpr int kChunks = QUANT ? 1 : D / 64;   // boxes across a row
      constexpr int kLine = kBytes / BN / kChunks;  // bytes of a box row
      uint64_t* const emptyb = QUANT ? raw_empty : empty;
      uint8_t* const ring = smem + (QUANT ? C::kRawOff : C::kRingOff);
      auto copy = [&](const RingTile& r, int slot, uint64_t* bar) {
        uint8_t* dst = ring + slot * kBytes;
        if (r.live > BN - kTailRows) {
          mbar_arrive_expect_tx(bar, kBytes);
          const CUtensorMap* tm = r.is_v ? &tm_v : &tm_k;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d(dst + c * BN * kLine, tm, bar, c * 64, r.kv_head, r.kv_row);
        } else {
          const int boxes = (r.live + kTailRows - 1) / kTailRows;
          mbar_arrive_expect_tx(bar, boxes * kTailRows * kLine * kChunks);
          const CUtensorMap* tm = r.is_v ? &tm_v_tail : &tm_k_tail;
          for (int x = 0; x < boxes; ++x)
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_3d(dst + (c * BN + x * kTailRows) * kLine, tm, bar, c * 64, r.kv_head,
                          r.kv_row + x * kTailRows);
        }
      };
      int seq = 0;
      uint32_t phases = 0;  // (bf16) loads of each full barrier, mod 2
      bool ok = true;
      if constexpr (!QUANT) {
        if (lane == 0)
          ok = for_each_ring_tile(p, list, steps, [&](const RingTile& r) {
            const int slot = seq % kSt;
            if (!wait_one(emptyb + slot, ((seq / kSt) & 1) ^ 1, abort_flag, p.timeout_ns))
              return false;
            copy(r, slot, full + full_bit(r.user(), slot));
            phases ^= 1u << full_bit(r.user(), slot);
            ++seq;
            return true;
          });
      } else {
        // The scales' lines are fetched to L1 when a tile's copy starts, and read a tile
        // later (held in registers instead, the loop waited for them: 2000 cycles a tile).
        RingTile last{};        // the tile whose factors are still to be made
        int ev0 = 0, ev1 = 0;   // E of each stream's V rows
        auto scale_at = [&](const float* scales, const RingTile& r) {
          return scales + (long long)r.kv_head * p.s_head + r.kv_row;
        };
        auto factors = [&]() {
          const int slot = (seq - 1) % kSt;
          const bool second = last.user() == 1;
          const float* at = scale_at(last.is_v ? p.vs : p.ks, last) + lane;
          const float* at_v = scale_at(p.vs, last) + lane;
          float sc[4], mv = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool live = i * 32 + lane < last.live;
            sc[i] = live ? __ldg(at + i * 32) : 0.f;
            if (!last.is_v && live) mv = fmaxf(mv, __ldg(at_v + i * 32));
          }
          int ev = second ? ev1 : ev0, e = ev;
          if (!last.is_v) {
            float mk = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
            // (scales are not negative: their bits order as integers)
            mk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mk)));
            mv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mv)));
            e = exponent_of(mk);
            ev = last.first ? exponent_of(mv) : max(ev, exponent_of(mv));
            if (second) ev1 = ev;
            else ev0 = ev;
          }
          const float inv = exp2_int(-e);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            raw_mul[slot * BN + i * 32 + lane] = (uint16_t)pack_f16x2(sc[i] * inv, 0.f);
          if (lane == 0) raw_note[slot] = RawNote{last.live, last.which | (last.is_v ? RawNote::kNoteV : 0), e, ev};
          __syncwarp();
          if (lane == 0) mbar_arrive(raw_full + slot);
        };
        ok = for_each_ring_tile(p, list, steps, [&](const RingTile& r) {
          const int slot = seq % kSt;
          if (!wait_warp(emptyb + slot, ((seq / kSt) & 1) ^ 1, abort_flag, p.timeout_ns)) return false;
          if (lane == 0) copy(r, slot, raw_full + slot);
          __syncwarp();
          // lanes 0-15 the lines of this tile's scales, 16-31 those of a K tile's V
          // (32-byte steps: a tile's 512 bytes start anywhere)
          const int row = (lane & 15) * 8 + (lane & 1 ? 7 : 0);
          if (row < r.live && (lane < 16 || !r.is_v))
            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                scale_at(lane >= 16 || r.is_v ? p.vs : p.ks, r) + row));
          if (seq > 0) factors();
          last = r;
          ++seq;
          return true;
        });
        if (ok && seq > 0) factors();
        // given up: the last copy's barrier still wants its second arrival
        if (!ok && seq > 0 && lane == 0) mbar_arrive(raw_full + (seq - 1) % kSt);
      }
      if (lane == 0) {
        *issued_loads = seq;
        *issued_phases = (int)phases;
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ------------------------------------------- MMA issuer of one stream --
      // Its steps in order: P V of a step, then Q K^T of its next, whose S overwrites
      // the P that the former reads (the tensor core keeps their order).
      const int s = warp - kMmaWarp;
      if (lane == 0) {
        constexpr uint32_t kIdescQK = idesc_16bit_f32(QUANT, BM, BN, 0);
        constexpr uint32_t kIdescPV = idesc_16bit_f32(QUANT, BM, D, 1);
        const uint64_t qd = smem_desc_sw128(q_base, 16, 1024) + (uint64_t)((s * C::kQTile) >> 4);
        const uint64_t dk0 = smem_desc_sw128(ring_base, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(ring_base, BN * 128, 1024);
        const uint32_t s_tmem = tmem_base + s * BN, o_tmem = tmem_base + 2 * BN + s * D;
        auto issue_qk = [&](int slot) {
          const uint64_t kd = dk0 + (uint64_t)((slot * C::kTile) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            constexpr int kChunk = (BM * 128) >> 4;
            const uint64_t off = (uint64_t)((kk >> 2) * kChunk + (kk & 3) * 2);
            mma_ss(s_tmem, qd + off, kd + off, kIdescQK, kk > 0 ? 1u : 0u);
          }
        };
        auto issue_pv = [&](int slot, bool first) {
          const uint64_t vd = dv0 + (uint64_t)((slot * C::kTile) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(o_tmem, s_tmem + kk * 8, vd + (uint64_t)(kk * ((16 * 128) >> 4)), kIdescPV,
                   (!first || kk > 0) ? 1u : 0u);
        };
        const int single_end = s ? list.single2 : list.single1;
        int i = list.dual0;  // piece whose keys come next
        bool dual = i < list.dual1;
        if (!dual) i = s ? list.single1 : list.single0;
        int dual_seq = 0;    // ring places of the dual tiles so far
        int n = s;           // step of the single units
        int step = 0, pieces = 0;
        bool ok = true;
        int left = 0;        // KV tiles of the current piece behind the one in S
        uint32_t phases = 0;
        auto wait_tile = [&](int user, int slot) {
          const int b = full_bit(user, slot);
          const uint32_t parity = (phases >> b) & 1;
          phases ^= 1u << b;
          return wait_one(full + b, parity, abort_flag, p.timeout_ns);
        };
        int k_slot = 0, v_slot = 0;                // of the stream's next step
        bool next_dual = false, next_head = false;
        // Finds the stream's next step; waits for its queries, at a piece's head, and
        // its K tile.  False when there is none or a wait ran out.
        auto prepare = [&]() {
          next_head = left == 0;
          if (next_head) {
            if (dual && i == list.dual1) {
              dual = false;
              i = s ? list.single1 : list.single0;
            }
            if (!dual && i >= single_end) return false;
            left = num_tiles(load_piece(p, i++).keys);
            ok = wait_one(q_full + s, pieces++ & 1, abort_flag, p.timeout_ns);
          }
          --left;
          next_dual = dual;
          if (dual) {
            k_slot = dual_seq % C::kStages;
            v_slot = (dual_seq + 1) % C::kStages;
            dual_seq += 2;
          } else {
            k_slot = (dual_seq + k_place(n)) % C::kStages;
            v_slot = (dual_seq + v_place(n)) % C::kStages;
            n += 2;
          }
          ok = ok && wait_tile(dual ? 2 : s, k_slot);
          return ok;
        };
        auto begin_step = [&]() {
          tc_fence_after();
          issue_qk(k_slot);
          mma_commit(s_full + s);
          mma_commit(empty + k_slot);
          if (!next_dual) mbar_arrive(empty + k_slot);  // the other stream does not use the tile
        };
        // Bursts by turns: for dual units, and for single ones when each stream has one
        // piece (they have as many KV tiles, or stream 0 one more; 8 tokens on a 128K
        // prefix 112 -> 108 us).  With several, a stream would wait for the other's ends.
        const bool one_each = list.single1 - list.single0 == 1 && list.single2 - list.single1 == 1;
        bool more = prepare();
        if (more) begin_step();
        while (more) {
          const int slot = v_slot;
          const bool first = next_head, last = left == 0, both = next_dual, turns = both || one_each;
          ok = wait_tile(both ? 2 : s, slot);
          if (ok && turns && !last) more = prepare();
          ok = ok && wait_one(p_full + s, step & 1, abort_flag, p.timeout_ns);
          // The streams' bursts of MMAs alternate, so that each stream's softmax runs under
          // the other's MMAs; without the turns the two fall into step and the tensor
          // core idles during both softmaxes.
          if (ok && turns && (s == 1 || step > 0))
            ok = wait_one(turn + s, (s == 1 ? step : step - 1) & 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          tc_fence_after();
          issue_pv(slot, first);
          if (last) mma_commit(o_full + s);
          mma_commit(empty + slot);
          if (!both) mbar_arrive(empty + slot);
          if (turns && !last) begin_step();
          if (turns) mbar_arrive(turn + (s ^ 1));
          if (!turns || last) {
            more = prepare();
            if (more) begin_step();
          }
          ++step;
        }
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        // every MMA and commit issued by this thread has completed
        mma_commit(bar_drain + s);
        wait_one(bar_drain + s, 0, nullptr, p.timeout_ns);
      }
    }
    if constexpr (QUANT) if (warp >= kConvertWarp) {
      // --------------------------------------------------- codes to f16 tiles --
      // Warp w has rows 32w .. 32w+31 of every tile; of a row, lane l has 8 codes of
      // each 64 (so that 8 lanes store 8 different banks' chunks).  Rows behind the
      // last key become zeros (0 * NaN is NaN, so masking P alone would not keep stale
      // rows out).
      const int w = warp - kConvertWarp;
      const int rl = lane >> 3, cl = lane & 7;  // row of four, 8-code chunk
      int tiles = 2 * steps;
      for (int i = list.dual0; i < list.dual1; ++i) tiles += 2 * num_tiles(load_piece(p, i).keys);
      // chunk places of rows r and r + 4 of a row's 128-byte line
      const uint32_t swz[2] = {(uint32_t)((cl ^ rl) << 4), (uint32_t)((cl ^ (rl + 4)) << 4)};
      // and of the codes of rows r and r + 4 (every eighth row is swizzled alike)
      constexpr int kBatch = 4, kHalves = D / 64;
      uint32_t from[2][kHalves];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          from[x][h] = code_at<D>(w * 32 + rl + 4 * x, h * 4 + (cl >> 1)) + (cl & 1) * 8;
      bool ok = true;
      for (int seq = 0; seq < tiles; ++seq) {
        const int raw = seq % C::kRawStages, slot = seq % C::kStages;
        ok = wait_warp2(empty + slot, ((seq / C::kStages) & 1) ^ 1, raw_full + raw,
                        (seq / C::kRawStages) & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        const RawNote note = raw_note[raw];
        if (w == 0 && lane == 0 && note.which < RawNote::kNoteV)
          tile_exp[note.which] = make_int2(note.ek, note.ev);
        const uint8_t* src = smem + C::kRawOff + raw * C::kRawTile;
        const uint16_t* mul = raw_mul + raw * BN + w * 32 + rl;
        uint8_t* dst = smem + C::kRingOff + slot * C::kTile + (w * 32 + rl) * 128;
        const int live = note.live - w * 32 - rl;
        // loads of a batch before its stores: the compiler cannot tell them apart
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 4 * kBatch) {
          uint2 v[kBatch][kHalves];
          uint32_t m[kBatch];
#pragma unroll
          for (int x = 0; x < kBatch; ++x) {
            m[x] = mul[r0 + 4 * x];
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              v[x][h] = *reinterpret_cast<const uint2*>(src + from[x & 1][h] + (r0 + 4 * (x & ~1)) * D);
          }
          if (live < 32) {
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                if (r0 + 4 * x >= live) v[x][h] = make_uint2(0, 0);
          }
#pragma unroll
          for (int x = 0; x < kBatch; ++x)
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              const uint32_t m2 = m[x] * 0x10001u;
              const uint2 a = codes_to_f16(v[x][h].x, m2), b = codes_to_f16(v[x][h].y, m2);
              *reinterpret_cast<uint4*>(dst + h * (BN * 128) + (r0 + 4 * x) * 128 + swz[x & 1]) =
                  make_uint4(a.x, a.y, b.x, b.y);
            }
        }
        fence_async_shared();
        mbar_arrive(full + full_bit((note.which & (RawNote::kNoteV - 1)) >> 1, slot));
        mbar_arrive(raw_empty + raw);
      }
      if (!ok && lane == 0) {
        set_status(p.status, CPATTN_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // ----------------------------------------------------------- softmax --
    const int s = warp >> 2;          // stream
    const int wq = warp & 3;          // TMEM lane quarter
    const int trow = wq * 32 + lane;  // row within the MMA tile
    const uint32_t s_addr = tmem_base + ((uint32_t)(wq * 32) << 16) + s * BN;
    const uint32_t o_addr = tmem_base + ((uint32_t)(wq * 32) << 16) + 2 * BN + s * D;
    uint8_t* const q_line = smem + s * C::kQTile + trow * 128;
    auto q_chunk = [&](int c) {  // 16-byte chunk c of this thread's query row (128-byte swizzle)
      return q_line + (c >> 3) * (BM * 128) + (((c & 7) ^ (trow & 7)) << 4);
    };
    auto row_of = [&](const SharedPiece& pc) {
      // (a single unit's rows in the other half for stream 1: other schedulers' warps)
      return shared_dual(pc.rows) ? s * BM + trow : trow ^ (s * (BM / 2));
    };
    // The warp's query rows of a piece to shared memory, asynchronously (D / 8 lanes to a
    // row: a thread for each row would touch 32 lines with every instruction, 4000 cycles
    // a piece); q_ready() publishes them, and returns the factor of this row's scores.
    auto load_q = [&](const SharedPiece& pc) {
      constexpr int kLanes = D / 8;  // of a row
      const int r = row_of(pc);
      const __nv_bfloat16* row = nullptr;
      if (r < pc.rows) {
        const int packed = pc.r0 + r, qi = group_div(p, packed);
        row = p.q + (long long)(pc.q_row0 + qi) * p.q_row +
              (long long)(pc.kv_head * p.g + packed - qi * p.g) * p.q_head;
      }
      const int c = lane % kLanes;
      uint32_t dst = q_base + s * C::kQTile + (c >> 3) * (BM * 128) + wq * 32 * 128;
#pragma unroll 4
      for (int i = lane / kLanes; i < 32; i += 32 / kLanes) {
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), i));
        if (src)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           dst + i * 128 + (((c & 7) ^ (i & 7)) << 4)),
                       "l"(src + c * 8)
                       : "memory");
      }
    };
    auto q_ready = [&](const SharedPiece& pc) {
      float factor = p.scale_log2;
      asm volatile("cp.async.wait_all;" ::: "memory");
      if constexpr (QUANT) {
        __syncwarp();  // (the row came by other lanes' copies)
        if (row_of(pc) < pc.rows) {
          // bf16 to f16 in place, times 2^f with 2^f max|q| in [2^14, 2^15)
          uint32_t mx = 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(q_chunk(c));
            mx = __vmaxu2(__vmaxu2(mx, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                          __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
          }
          const int e = (int)(max(mx & 0xFFFFu, mx >> 16) >> 7) - 127;  // of max|q|
          const int f = min(max(14 - e, -126), 126);
          const float up = exp2_int(f);
          factor *= exp2_int(-f);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            uint4* const at = reinterpret_cast<uint4*>(q_chunk(c));
            uint4 v = *at;
            uint32_t* const x = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = pack_f16x2(__uint_as_float(x[i] << 16) * up,
                                __uint_as_float(x[i] & 0xFFFF0000u) * up);
            *at = v;
          }
        }
      }
      fence_async_shared();
      if (!p.withhold_q) mbar_arrive(q_full + s);
      return factor;
    };
    // the stream's pieces: the dual ones, then its own
    const int single0 = s ? list.single1 : list.single0, single1 = s ? list.single2 : list.single1;
    const int duals = list.dual1 - list.dual0, pieces = duals + single1 - single0;
    auto piece = [&](int i) {
      return load_piece(p, i < duals ? list.dual0 + i : single0 + i - duals);
    };
    SharedPiece np{};
    float factor = p.scale_log2;
    if (pieces > 0) {
      np = piece(0);
      load_q(np);
      factor = q_ready(np);
    }
    int step = 0;      // of the stream
    int dual_seq = 0;  // ring places of the dual tiles before this piece
    uint32_t phases = 0;
    bool ok = true;
    for (int i = 0; i < pieces; ++i) {
      const SharedPiece pc = np;
      const bool more = i + 1 < pieces;
      if (more) np = piece(i + 1);
      const bool dual = i < duals;
      const int T = num_tiles(pc.keys);
      const int r = row_of(pc);
      const bool warp_live = (r & ~31) < pc.rows;
      int seen = 0;  // keys of the piece that this row sees
      if (r < pc.rows) {
        const long long pos = (long long)pc.q_pos0 + (long long)group_div(p, pc.r0 + r) * pc.q_pos_step;
        seen = (int)max(0LL, min((long long)pc.keys, pos + 1 - pc.key0));
      }
      float m_run = -INFINITY, l_run = 0.f, m_use = 0.f;
      int ev = 0;  // exponent of O
      for (int t = 0; t < T; ++t) {
        ok = wait_warp(s_full + s, step & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        tc_fence_after();
        // the piece's last S is done: its query tile is free for the next piece
        if (t == T - 1 && more) load_q(np);
        float sl2 = factor, o_scale = 1.f;
        if constexpr (QUANT) {
          // written before the K tile of this step went to the tensor core, and not
          // again before this step's P has been used
          const volatile int2* e =
              tile_exp + (dual ? 4 + ((dual_seq / 2 + t) & 1) : 2 * s + ((step - dual_seq / 2) & 1));
          const int ek = e->x, ev_now = e->y;
          sl2 = score_factor(sl2, exp2_int(ek));
          if (t > 0 && ev_now != ev) o_scale = exp2_int(max(ev - ev_now, -126));
          ev = ev_now;
        }
        if (warp_live) {
          const int here = seen - t * BN;  // visible keys of this tile
          softmax_tile<D, QUANT>(s_addr, o_addr, here, t > 0, o_scale, sl2, m_run, m_use, l_run);
        }
        if constexpr (!QUANT) {
          // V rows behind the last key become zeros (0 * NaN is NaN, so masking P
          // alone would not keep stale rows out); both streams do it to a shared tile
          const int user = dual ? 2 : s, n = 2 * (step - dual_seq / 2) + s;
          const int k_bit = full_bit(user, (dual_seq + (dual ? 2 * t : k_place(n))) % C::kStages);
          const int v_slot = (dual_seq + (dual ? 2 * t + 1 : v_place(n))) % C::kStages;
          const int v_bit = full_bit(user, v_slot), live = pc.keys - t * BN;
          phases ^= 1u << k_bit;
          if (live < BN) {
            ok = wait_warp(full + v_bit, (phases >> v_bit) & 1, abort_flag, p.timeout_ns);
            if (!ok) break;
            uint8_t* tile = smem + C::kRingOff + v_slot * C::kTile;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              for (int at = live * 8 + trow; at < BN * 8; at += 128)
                *reinterpret_cast<uint4*>(tile + c * BN * 128 + at * 16) = make_uint4(0, 0, 0, 0);
            fence_async_shared();
          }
          phases ^= 1u << v_bit;
        }
        tc_fence_before();
        mbar_arrive(p_full + s);
        ++step;
      }
      if (!ok) break;
      if (more) factor = q_ready(np);
      if (dual) dual_seq += 2 * T;
      ok = wait_warp(o_full + s, i & 1, abort_flag, p.timeout_ns);
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        const bool none = l_run == 0.f;  // (a NaN sum is not none)
        const float inv = none ? 0.f : exp2_int(ev) / l_run;
        float* dst = p.ws_o + (long long)pc.ws_row * D;
        constexpr int kCols = QUANT ? 64 : D;  // (register budget)
#pragma unroll
        for (int q = 0; q < D / kCols; ++q) {
          uint32_t v[kCols];
#pragma unroll
          for (int c = 0; c < kCols; c += 32) tmem_ld32p(o_addr + q * kCols + c, v + c);
          tmem_wait_ld();
          if (r < pc.rows) {
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
              float f[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) f[x] = none ? 0.f : __uint_as_float(v[c + x]) * inv;
              store8(dst + partial_at((q * kCols + c) / 8, r, pc.rows), f);
            }
          }
        }
        if (r < pc.rows) p.ws_l[(long long)pc.ws_row + r] = none ? -INFINITY : m_use + lg2_approx(l_run);
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) {
      set_status(p.status, CPATTN_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (warp == kProducerWarp) {
    if (lane == 0 && *abort_flag) {
      // let the copies in flight land before the shared memory goes: the last load of
      // each barrier that had one (a barrier without loads passes: its phase before
      // the first counts as done)
      if constexpr (QUANT) {
        const int n = *issued_loads;
        for (int j = max(0, n - C::kRawStages); j < n; ++j)
          wait_one(raw_full + j % C::kRawStages, (j / C::kRawStages) & 1, nullptr, p.timeout_ns);
      } else {
        const uint32_t phases = (uint32_t)*issued_phases;
        for (int b = 0; b < 3 * C::kStages; ++b)
          wait_one(full + b, ((phases >> b) & 1) ^ 1, nullptr, p.timeout_ns);
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// Merge of the partials of J heads of a query row (J = 1, 2, 4 dividing g, so that they
// are J rows side by side of the same unit), `ways` warps for them, each an interleaved
// share of the partials.  Bound by latency or, with many rows, by the partials' bytes:
// the plan's words are read before the wait for the attention kernel, so that two
// dependent loads are left after it, the L of up to 32 / J partials and their O.  A lane
// has 4 columns of each of its chunks, all of one row (see partial_at: a chunk's J rows
// are contiguous).
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
template <int D, int J>
struct MergeCfg {
  static constexpr int kLanes = 2 * J;                                 // of a chunk's J rows
  static constexpr int kVec = D * J / 128 > 0 ? D * J / 128 : 1;       // 16-byte loads of a partial
  // partials of a warp whose O loads are in flight together (12 or 16 vectors cost J = 4
  // more in registers than they gain)
  static constexpr int kLoads = (J == 1 ? 16 : 8) / kVec;
};

template <int V>
struct MergeSum {  // sum_j 2^(L_j - m) (1, O_j), this lane's row and columns
  float m, w, o[V][4];
};

// The share `way` of `ways` of the partials of heads h0 .. h0 + J - 1; false (and
// CPATTN_ERR_RANGE) when the plan's words lead out of the buffers.
template <int D, int J>
__device__ __forceinline__ bool merge_share(const SharedParams& p, int h0, int e0, int e1, int way, int ways,
                                            int lane, MergeSum<MergeCfg<D, J>::kVec>& sum) {
  using C = MergeCfg<D, J>;
  const unsigned all = 0xffffffffu;
  const int kvh = h0 / p.g, j0 = h0 - kvh * p.g;
  const int mine = (lane >> 1) % J, chunk = lane / C::kLanes;  // the lane's row, first chunk
  float m_l = -INFINITY;  // sum.m of row lane % J
  bool waited = false;
  for (int eb = e0; eb < e1; eb += 32) {
    // lane e: the partials of entry eb + e
    SharedUnit un{0, 0, 1, 0};
    int at = 0;
    bool ok = true;
    if (eb + lane < e1) {
      const int2 en = __ldg(reinterpret_cast<const int2*>(p.table + p.entries) + eb + lane);
      const long long packed = (long long)en.y * p.g + j0;
      const long long unit = en.x + packed / kRows * p.Hkv + kvh;
      ok = en.x >= 0 && en.y >= 0 && unit < p.num_units;
      if (ok) {
        const int4 w = __ldg(reinterpret_cast<const int4*>(p.table + p.units) + unit);
        un = SharedUnit{w.x, w.y, w.z, w.w};
        at = (int)(packed % kRows);
        ok = un.ws_row >= 0 && un.parts >= 0 &&
             (un.parts == 0 || (at + J <= un.rows && un.rows <= kRows &&
                                un.ws_row + (long long)un.parts * un.rows <= p.ws_rows));
      }
    }
    if (!__all_sync(all, ok)) return false;
    int upto = un.parts;  // partials of this entry and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(all, upto, o);
      if (lane >= o) upto += x;
    }
    const int total = __shfl_sync(all, upto, 31), entries = min(32, e1 - eb);
    for (int b = way; b < total; b += 32 / J * ways) {
      // lane l: row l % J of partial b + (l / J) * ways
      const int part = b + lane / J * ways;
      long long first = 0;  // workspace row of the partial's first
      int rows = 1, row = 0;
      for (int e = 0; e < entries; ++e) {
        const int end = __shfl_sync(all, upto, e), cnt = __shfl_sync(all, un.parts, e);
        const int ws_row = __shfl_sync(all, un.ws_row, e), r = __shfl_sync(all, un.rows, e);
        const int a = __shfl_sync(all, at, e);
        if (part >= end - cnt && part < end) {
          first = ws_row + (long long)(part - (end - cnt)) * r;
          rows = r;
          row = a;
        }
      }
      if (!waited) grid_dep_wait();  // the attention kernel before this one wrote the partials
      waited = true;
      const int cnt = min(32 / J, (total - b + ways - 1) / ways);
      const float l = part < total ? __ldcg(p.ws_l + first + row + lane % J) : -INFINITY;
      float4 x[C::kLoads][C::kVec];
      auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
          const int from = (i0 + i) * J & 31;
          const float* src = p.ws_o + __shfl_sync(all, first, from) * D;
          const int r = __shfl_sync(all, rows, from), r0 = __shfl_sync(all, row, from);
#pragma unroll
          for (int v = 0; v < C::kVec; ++v) {
            const int c = v * (32 / C::kLanes) + chunk;
            x[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + i < cnt && c < D / 8)
              x[i][v] = __ldcg(reinterpret_cast<const float4*>(src + partial_at(c, r0 + mine, r)) + (lane & 1));
          }
        }
      };
      load(0);
      float mx = l;
#pragma unroll
      for (int o = 16; o >= J; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(all, mx, o));
      const float mn = fmaxf(m_l, mx), use = mn == -INFINITY ? 0.f : mn;
      const float w = exp2f(l - use);  // (a NaN partial stays one)
      float ws = w;
#pragma unroll
      for (int o = 16; o >= J; o >>= 1) ws += __shfl_xor_sync(all, ws, o);
      const float old = __shfl_sync(all, exp2f(m_l - use), mine);
      m_l = mn;
      sum.w = sum.w * old + __shfl_sync(all, ws, mine);
#pragma unroll
      for (int v = 0; v < C::kVec; ++v)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum.o[v][c] *= old;
      sum.m = __shfl_sync(all, mn, mine);
      for (int i0 = 0; i0 < cnt; i0 += C::kLoads) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
          const float wi = __shfl_sync(all, w, ((i0 + i) * J & 31) + mine);
          if (i0 + i < cnt)
#pragma unroll
            for (int v = 0; v < C::kVec; ++v) {
              sum.o[v][0] = fmaf(wi, x[i][v].x, sum.o[v][0]);
              sum.o[v][1] = fmaf(wi, x[i][v].y, sum.o[v][1]);
              sum.o[v][2] = fmaf(wi, x[i][v].z, sum.o[v][2]);
              sum.o[v][3] = fmaf(wi, x[i][v].w, sum.o[v][3]);
            }
        }
      }
    }
  }
  return true;
}

template <int D, int J>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const SharedParams p, int ways) {
  using C = MergeCfg<D, J>;
  constexpr int V = C::kVec;
  __shared__ MergeSum<V> parts[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, way = warp % ways;
  const long long u = (long long)blockIdx.x * (kMergeWarps / ways) + warp / ways;
  const int groups = p.Hq / J;  // of heads
  int n = 0, h0 = 0;
  MergeSum<V> sum;
  sum.m = -INFINITY;
  sum.w = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int c = 0; c < 4; ++c) sum.o[v][c] = 0.f;
  bool write = false;
  if (u < (long long)p.num_q_rows * groups) {
    n = (int)(u / groups);
    h0 = (int)(u - (long long)n * groups) * J;
    const int e0 = __ldg(p.table + p.row_first + n), e1 = __ldg(p.table + p.row_first + n + 1);
    if (e0 != e1) {  // (a row of no segment is left as it is)
      write = e0 >= 0 && e1 > e0 && e1 <= p.num_entries &&
              merge_share<D, J>(p, h0, e0, e1, way, ways, lane, sum);
      if (!write && lane == 0) set_status(p.status, CPATTN_ERR_RANGE);
    }
  }
  grid_dep_wait();  // no block ends before the kernel that this launch may overlap
  if (ways > 1) {
    parts[warp][lane] = sum;
    __syncthreads();
    if (way > 0) return;
    for (int x = 1; x < ways; ++x) {
      const MergeSum<V>& other = parts[warp + x][lane];
      const float mn = fmaxf(sum.m, other.m), use = mn == -INFINITY ? 0.f : mn;
      const float a = exp2f(sum.m - use), b = exp2f(other.m - use);
      sum.w = sum.w * a + other.w * b;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum.o[v][c] = sum.o[v][c] * a + other.o[v][c] * b;
      sum.m = mn;
    }
  }
  if (!write) return;
  const float inv = sum.w == 0.f ? 0.f : 1.f / sum.w;
  const long long row = (long long)n * p.Hq + h0 + (lane >> 1) % J;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * (32 / C::kLanes) + lane / C::kLanes;
    if (c >= D / 8) break;
    const long long out = row * D + c * 8 + (lane & 1) * 4;
    const float4 f = make_float4(sum.o[v][0] * inv, sum.o[v][1] * inv, sum.o[v][2] * inv, sum.o[v][3] * inv);
    if (p.o_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.o) + out) = f;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + out) =
          make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
  }
  if (lane < 2 * J && (lane & 1) == 0)
    p.lse[row] = sum.w == 0.f ? -INFINITY : (sum.m + log2f(sum.w)) * kLn2;
}

// Warps for a row's J heads: enough that a warp loads its partials in two goes (their
// average is ws_rows / rows), e.g. 152 partials a row at one token on a 256K prefix, but
// no more than let all blocks reside at once (two to an SM): a block takes 5 us, mostly
// for its chain of loads, and a second wave of them as much again.
constexpr int kMergeResident = 2 * 152;
template <int D, int J>
int launch_merge(const SharedParams& p, bool behind, cudaStream_t stream) {
  const long long rows = (long long)p.num_q_rows * p.Hq;
  int ways = 1;
  while (ways < kMergeWarps && p.ws_rows > rows * ways * 2 * MergeCfg<D, J>::kLoads) ways *= 2;
  while (ways > 1 && rows / J * ways > (long long)kMergeResident * kMergeWarps) ways /= 2;
  const long long blocks = (rows / J * ways + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  const cudaError_t e = launch_kernel(shared_merge_kernel<D, J>, (unsigned)blocks, kMergeThreads, 0, stream,
                                      behind, p, ways);
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}
// behind: the kernel before it on the stream is this call's, not one that may still
// write the plan's table.
template <int D>
int launch_merge(const SharedParams& p, bool behind, cudaStream_t stream) {
  return p.g % 4 == 0   ? launch_merge<D, 4>(p, behind, stream)
         : p.g % 2 == 0 ? launch_merge<D, 2>(p, behind, stream)
                        : launch_merge<D, 1>(p, behind, stream);
}

// 3-D map of a code buffer (cols, heads, rows) with a D-column x 1-head box, rows
// packed in shared memory and swizzled over their length (see code_at); out-of-range
// rows read as zero.
bool make_code_map(CUtensorMap* m, const void* base, int cols, int heads, long long rows,
                   long long head_stride, long long row_stride, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride, (cuuint64_t)row_stride};
  cuuint32_t box[3] = {(cuuint32_t)cols, 1, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct SharedMaps {  // full tiles, then the tail boxes
  CUtensorMap k, v, k_tail, v_tail;
};

template <int D, bool QUANT>
int launch_shared(const SharedMaps& m, const SharedParams& p, int num_ctas, cudaStream_t stream) {
  using C = SharedCfg<D, QUANT>;
  constexpr int kSmem = std::max(C::kSmemBytes, SmallCfg<D, QUANT>::kSmemBytes);
  auto kern = attn_shared_kernel<D, QUANT>;
  if (!allow_smem(kern, kSmem)) return CPATTN_ERR_CUDA;
  // setmaxnreg.inc waits until the block's launch allocation covers the split;
  // refuse a build whose register count could not (a property of this binary).
  static int regs_ok = 0;  // 0 not checked yet, 1 ok, -1 refused
  if (regs_ok == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return CPATTN_ERR_CUDA;
    regs_ok = fa.numRegs * C::kThreads >=
                      C::kRegsSoftmax * 256 + C::kRegsOther * (C::kThreads - 256)
                  ? 1
                  : -1;
  }
  if (regs_ok < 0) return CPATTN_ERR_UNSUPPORTED;
  return launch_kernel(kern, (unsigned)num_ctas, C::kThreads, kSmem, stream, false, m.k, m.v,
                       m.k_tail, m.v_tail, p) == cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cp_attn_shared(const cp_shared_plan_t* plan, const int32_t* table_dev,
                              const void* q, int64_t q_row_stride, int64_t q_head_stride,
                              const void* k, int64_t k_row_stride, int64_t k_head_stride,
                              const float* k_scales, const void* v, int64_t v_row_stride,
                              int64_t v_head_stride, const float* v_scales, int64_t scale_stride,
                              int num_kv_rows, int d, int dv, float scale, void* o, int o_is_fp32,
                              float* lse, void* workspace, int64_t workspace_bytes,
                              int32_t* status_dev, cudaStream_t stream) {
  CPATTN_TRACE("cp_attn_shared");
  int64_t need = 0;
  const int rc = cp_shared_workspace_size(plan, dv, &need);
  if (rc != CPATTN_OK) return rc;
  if (!((d == 64 && dv == 64) || (d == 128 && dv == 128))) return CPATTN_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || num_kv_rows < 0 || (k_scales != nullptr) != (v_scales != nullptr))
    return CPATTN_ERR_INVALID_ARG;
  if (plan->num_entries == 0) return CPATTN_OK;  // no rows: nothing to write
  if (!table_dev || !q || !o || !lse || !workspace || workspace_bytes < need ||
      num_kv_rows < plan->kv_rows || (plan->num_pieces > 0 && (!k || !v)))
    return CPATTN_ERR_INVALID_ARG;
  const bool quant = k_scales != nullptr;
  const int64_t per16 = quant ? 16 : 8;  // elements in 16 bytes
  if (!a16(table_dev) || !a16(q) || !a16(k) || !a16(v) || !a16(o) ||
      (reinterpret_cast<uintptr_t>(workspace) & 31u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(k_scales) & 3u) ||
      (reinterpret_cast<uintptr_t>(v_scales) & 3u) || q_row_stride % 8 || q_head_stride % 8 ||
      k_row_stride % per16 || k_head_stride % per16 || v_row_stride % per16 ||
      v_head_stride % per16)
    return CPATTN_ERR_ALIGNMENT;
  if (q_row_stride < 0 || q_head_stride < 0 || k_head_stride < d || v_head_stride < dv ||
      k_row_stride < (int64_t)(plan->Hkv - 1) * k_head_stride + d ||
      v_row_stride < (int64_t)(plan->Hkv - 1) * v_head_stride + dv ||
      (quant && scale_stride < num_kv_rows))
    return CPATTN_ERR_INVALID_ARG;

  const SharedTable T = shared_table(*plan);
  SharedParams p{};
  p.table = table_dev;
  p.pieces = T.pieces;
  p.units = T.units;
  p.row_first = T.row_first;
  p.entries = T.entries;
  p.num_units = plan->num_units;
  p.num_pieces = plan->num_pieces;
  p.num_entries = plan->num_entries;
  p.num_q_rows = plan->num_q_rows;
  p.Hq = plan->Hq;
  p.Hkv = plan->Hkv;
  p.g = plan->Hq / plan->Hkv;
  for (p.g_shift = 0; (1LL << (p.g_shift + 1)) < p.g; ++p.g_shift) {}  // s - 1
  p.g_mul = (uint32_t)((1ULL << (32 + p.g_shift)) / p.g + 1);
  p.ws_rows = plan->ws_rows;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.ks = k_scales;
  p.vs = v_scales;
  p.s_head = scale_stride;
  p.num_kv_rows = num_kv_rows;
  p.scale_log2 = scale * kLog2e;
  p.o = o;
  p.o_f32 = o_is_fp32 ? 1 : 0;
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_l = p.ws_o + plan->ws_rows * dv;
  p.status = status_dev;
  p.timeout_ns = attn_debug().timeout_ns;
  p.withhold_q = attn_debug().withhold_q;
  if (plan->num_pieces > 0) {
    SharedMaps m;
    auto map = [&](CUtensorMap* t, const void* base, int dim, int64_t hs, int64_t rs, int box_rows) {
      return quant ? make_code_map(t, base, dim, plan->Hkv, num_kv_rows, hs, rs, box_rows)
                   : make_map(t, base, dim, plan->Hkv, num_kv_rows, hs, rs, box_rows);
    };
    if (!map(&m.k, k, d, k_head_stride, k_row_stride, BN) ||
        !map(&m.v, v, dv, v_head_stride, v_row_stride, BN) ||
        !map(&m.k_tail, k, d, k_head_stride, k_row_stride, kTailRows) ||
        !map(&m.v_tail, v, dv, v_head_stride, v_row_stride, kTailRows))
      return CPATTN_ERR_CUDA;
    const int n = plan->num_ctas;
    const int r = d == 128 ? (quant ? launch_shared<128, true>(m, p, n, stream)
                                    : launch_shared<128, false>(m, p, n, stream))
                           : (quant ? launch_shared<64, true>(m, p, n, stream)
                                    : launch_shared<64, false>(m, p, n, stream));
    if (r != CPATTN_OK) return r;
  }
  const bool behind = plan->num_pieces > 0;
  return d == 128 ? launch_merge<128>(p, behind, stream) : launch_merge<64>(p, behind, stream);
}
