// cp_attn_tree for few rows a request and KV head (a decode step, a short draft): warp-level
// MMAs in registers.
//
// A 128-row MMA tile would be nearly empty, and HBM gives a block a KV tile of 128 keys every
// 1.4 us (bf16, d = 128): so eight warps work on registers, with 16x8x16 MMAs that have keys
// (and then the columns of V) as their 16 rows and queries as their 8 columns:
//     S^T = K Q^T,   O^T += V^T P^T.
// A unit has NQ columns of 8 rows, and the warps share its KV tiles' keys: 16 each, or (e4m3,
// where the decoding's latency counts) in two teams that take turns at the tiles, 32 each.
// Each warp keeps its own maximum, sum and output; at a piece's end the eight are joined in
// shared memory.  Three more warps feed them: K and V pages by TMA, one lane a page, (e4m3)
// with their scales by asynchronous copies; and the query rows, by the warp that walks the
// block's share.  A warp's step issues the products of its next keys between the softmax and
// the second product of these.
//
// Fragments are loaded as they lie in memory.  K Q^T sums over d in any order, so lane
// (g = lane / 4, c = lane % 4) takes whole 16-byte chunks of key rows g and g + 8 and of
// query row g the same ones: a chunk's elements 4x .. 4x+3 are its share of one k-step.
// V of a bf16 tile goes through the transposing matrix load.  V codes: the lane reads the
// g-th eighth of the columns of its keys 2c, 2c+1, 2c+8, 2c+9 and joins two rows' bytes into
// a pair for each column, so rows g and g + 8 of product x are columns g D/8 + 2x and + 1.
// Codes enter as f16, exact; K's scale multiplies the score, V's is taken relative to the
// largest that the warp has met (O is rescaled when that grows); among new keys, of which a row
// may not see all, V's scale multiplies the weight, relative to the largest that the row has seen.
//
// Measured, 32/8 heads, d = 128: 64 tokens on up to 8K keys each, bf16 175 us (6.7 TB/s, the copy
// bandwidth), e4m3 111 us (5.5 TB/s: codes to f16 and the copies of the scales); one token on 1K
// 11 us, of which tree_start takes 2, the first piece's walk 1.5, its tiles 3 and the merge 4.
#include <algorithm>
#include <atomic>

#include "attn_tree_smem.cuh"

namespace cpattn {
namespace {

constexpr int kWarps = kSmallWarps;
constexpr int kThreads = kSmallThreads;  // a third warpgroup: K's loader, V's, the walker, and one that idles
constexpr int kRegsLaunch = 168, kRegsWork = 208, kRegsOther = 88;
static_assert(kRegsWork * 256 + kRegsOther * 128 <= kRegsLaunch * kThreads, "register split exceeds the launch's");

// The 256 threads of the eight warps; true when any of them says so.
__device__ __forceinline__ bool bar_warps(bool any) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)any)
      : "memory");
  return r != 0;
}

// First element of the lane's 16-byte query chunk x: bf16, chunks 2c and 2c + 1 of each
// 128 bytes; e4m3, the two halves of its code chunks (2c, 2c + 1 of a row of 128, c of 64).
template <int D, bool QUANT>
__device__ __forceinline__ int q_chunk(int c, int x) {
  if (QUANT) return (D == 128 ? 2 * c + (x >> 1) : c) * 16 + (x & 1) * 8;
  return (x >> 1) * 64 + (2 * c + (x & 1)) * 8;
}
// Place of column d of row r of a warp's part of the join buffer (bank swizzle: a store's
// lanes have 8 columns, or 8 groups of four, of the rows 2 c + e).
template <bool QUANT>
__device__ __forceinline__ int join_at(int d, int r) {
  return d ^ (((r >> 1) & 3) << (QUANT ? 2 : 3));
}

template <int D, bool QUANT, int NQ>
struct Warp {
  using C = TreeCfg<D, QUANT, NQ>;
  static constexpr int kOut = D / 16, kLoads = QUANT ? D / 64 : D / 32;
  static constexpr int kTeams = C::kTeams, kKeys = C::kKeys, kBlocks = kKeys / 16;
  uint32_t base;  // shared memory
  uint8_t* mem;
  uint64_t *full, *empty, *q_full, *q_empty;
  const volatile int* abort;
  int warp, lane, g, c, team, key0;  // key0: the warp's first key of its team's tiles

  __device__ __forceinline__ void release(uint64_t* bar) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  __device__ __forceinline__ uint32_t scale_at(int slot, int row) const {
    return base + C::kScaleOff + slot * C::kScales + row * 4;
  }

  // K of 16 keys from `key` on: chunks of rows g and g + 8, as they lie.
  struct Keys {
    uint4 v[2][kLoads];
    float scale[2];
  };
  __device__ __forceinline__ void load_k(Keys& k, int slot, int key) const {
    const uint32_t tile = base + slot * C::kTile;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = key + 8 * j + g;
#pragma unroll
      for (int x = 0; x < kLoads; ++x)
        k.v[j][x] = QUANT ? lds128(tile + code_at<D>(row, D == 128 ? 2 * c + x : c))
                          : lds128(tile + (x >> 1) * (BN * 128) + row * 128 +
                                   (((2 * c + (x & 1)) ^ (row & 7)) << 4));
      k.scale[j] = QUANT ? lds_f32(scale_at(slot, row)) : 1.f;
    }
  }
  // s[n]: keys g (0, 1) and g + 8 (2, 3), rows 8n + 2c and 8n + 2c + 1; for one column of
  // rows two chains, for their latency
  __device__ __forceinline__ void product(const Keys& k, const uint32_t (&q)[NQ][kOut][2],
                                          const float (&factor)[NQ][2], float (&s)[NQ][4]) const {
    float s2[NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int y = 0; y < 4; ++y) s[n][y] = s2[n][y] = 0.f;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const uint32_t u0[4] = {k.v[0][x].x, k.v[0][x].y, k.v[0][x].z, k.v[0][x].w};
      const uint32_t u1[4] = {k.v[1][x].x, k.v[1][x].y, k.v[1][x].z, k.v[1][x].w};
      if constexpr (!QUANT) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          mma_16816<false>(s[n], u0[0], u1[0], u0[1], u1[1], q[n][2 * x][0], q[n][2 * x][1]);
          mma_16816<false>(s2[n], u0[2], u1[2], u0[3], u1[3], q[n][2 * x + 1][0], q[n][2 * x + 1][1]);
        }
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t a0 = e4m3x2_to_f16x2(u0[y]), a1 = e4m3x2_to_f16x2(u1[y]);
          const uint32_t a2 = e4m3x2_to_f16x2(u0[y] >> 16), a3 = e4m3x2_to_f16x2(u1[y] >> 16);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            mma_16816<true>(y & 1 ? s2[n] : s[n], a0, a1, a2, a3, q[n][4 * x + y][0], q[n][4 * x + y][1]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int y = 0; y < 4; ++y)
        s[n][y] = (s[n][y] + s2[n][y]) *
                  (QUANT ? score_factor(factor[n][y & 1], k.scale[y >> 1]) : factor[n][y & 1]);
  }

  // Which of the warp's value rows of a tile hold an infinity or NaN, in their scale or a code.
  __device__ __forceinline__ uint32_t bad_rows(int slot) const {
    constexpr int kParts = 32 / kKeys;                          // lanes of a row
    constexpr int kN = D * (QUANT ? 1 : 2) / 16 / kParts;       // chunks of a lane
    const uint32_t tile = base + slot * C::kTile;
    const int row = key0 + lane / kParts;
    bool bad = QUANT && !(lds_f32(scale_at(slot, row)) < INFINITY);
#pragma unroll
    for (int x = 0; x < kN; ++x) {
      const int ch = lane % kParts * kN + x;
      const uint4 v = lds128(QUANT ? tile + code_at<D>(row, ch)
                                   : tile + (ch >> 3) * (BN * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if constexpr (QUANT)
          bad = bad || __vcmpeq4(u[y] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
        else
          bad = bad || __vcmpgeu2(u[y] & 0x7FFF7FFFu, 0x7F807F80u) != 0;
    }
    return __reduce_or_sync(0xffffffffu, bad ? 1u << (lane / kParts) : 0u);
  }

  __device__ bool piece(const TreeParams& p, const TreePiece& pc, int n_piece, int n0) const;
};

template <int D, bool QUANT, int NQ>
__device__ __forceinline__ bool Warp<D, QUANT, NQ>::piece(const TreeParams& p, const TreePiece& pc, int n_piece,
                                                          int n0) const {
  constexpr int NS = C::kStages;
  const unsigned all = 0xffffffffu;
  const int qb = n_piece & 1;
  const int tile0 = pc.t0 * BN;  // first key
  // ---- queries: row g of each column ----
  uint32_t q[NQ][kOut][2];
  float factor[NQ][2];
  bool ok = wait_warp(q_full + qb, (n_piece >> 1) & 1, abort, p.timeout_ns);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    uint4 v[D / 32];
    const int row = 8 * n + g;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      v[x] = lds128(base + C::kQOff + qb * C::kQ + row * (D * 2) +
                    (((q_chunk<D, QUANT>(c, x) >> 3) ^ (row & 7)) << 4));
      if (row >= pc.rows) v[x] = make_uint4(0, 0, 0, 0);
    }
    float f_row = p.scale_log2;
    if constexpr (QUANT) {
      // bf16 to f16 times 2^f with 2^f max|q| in [2^14, 2^15)
      uint32_t mx = 0;
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
        mx = __vmaxu2(__vmaxu2(mx, __vmaxu2(v[x].x & 0x7FFF7FFFu, v[x].y & 0x7FFF7FFFu)),
                      __vmaxu2(v[x].z & 0x7FFF7FFFu, v[x].w & 0x7FFF7FFFu));
      mx = max(mx & 0xFFFFu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(all, mx, 1));
      mx = max(mx, __shfl_xor_sync(all, mx, 2));
      const int f = min(max(14 - ((int)(mx >> 7) - 127), -126), 126);
      const float up = exp2_int(f);
      f_row *= exp2_int(-f);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        uint32_t* const u = &v[x].x;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          u[y] = pack_f16x2(__uint_as_float(u[y] << 16) * up, __uint_as_float(u[y] & 0xFFFF0000u) * up);
      }
    }
    factor[n][0] = __shfl_sync(all, f_row, 8 * c);      // of row 2c
    factor[n][1] = __shfl_sync(all, f_row, 8 * c + 4);  // and the next
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      q[n][2 * x][0] = v[x].x;
      q[n][2 * x][1] = v[x].y;
      q[n][2 * x + 1][0] = v[x].z;
      q[n][2 * x + 1][1] = v[x].w;
    }
  }
  release(q_empty + qb);
  float o[NQ][kOut][4], m_run[NQ][2], m_use[NQ][2], l_run[NQ][2];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
#pragma unroll
    for (int x = 0; x < kOut; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[n][x][y] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m_run[n][e] = -INFINITY;
      m_use[n][e] = l_run[n][e] = 0.f;
    }
  }
  // (e4m3) exponent of O: ev while the rows see the same keys, and from there on (`parted`) a row's own,
  // which lies where the join will have the row's (m, l): the loop has no register for it
  int ev = -126;
  bool parted = false;
  int2* const own = reinterpret_cast<int2*>(mem + C::kMlOff) + warp * (8 * NQ);
  auto wait_k = [&](int n) {
    const int place = k_place<false>(n);
    return wait_warp(full + place % NS, (place / NS) & 1, abort, p.timeout_ns);
  };
  auto wait_v = [&](int n) {
    const int place = v_place<false>(n);
    return wait_warp(full + place % NS, (place / NS) & 1, abort, p.timeout_ns);
  };
  float s[kBlocks][NQ][4];
  auto scores = [&](int n) {  // of the block's n-th tile
    const int slot = k_place<false>(n) % NS;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      Keys k;
      load_k(k, slot, key0 + 16 * b);
      product(k, q, factor, s[b]);
    }
  };
  // Where rows see different keys V's codes enter the product as they are, and a value's scale its
  // weight: it must reach no row that does not see the key, as a factor for all rows would.  It is
  // taken relative to a power of two above all scales that the row has seen, so that a weight of up to
  // 2^15 stays one of f16.  (A key that a row does not see has a weight of 0.)  A row at a time, a key a
  // lane, through the warp's part of the join: on the registers that hold the weights it is so much
  // code that tiles that do not come here take longer, too (decode of 64 113.2 against 111.2 us).
  auto weigh = [&](int slot, uint32_t spoilt, float (&alpha)[NQ][2], bool& any) {
    constexpr int kPitch = 33;  // floats
    static_assert(!QUANT || (kKeys == 32 && kPitch <= D), "a key a lane, and rows of the join");
    float* const w = reinterpret_cast<float*>(mem + C::kJoinOff) + warp * (8 * NQ) * D;
    auto each = [&](auto&& f) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) f(s[b][x][y], w[(8 * x + 2 * c + (y & 1)) * kPitch + 16 * b + g + 8 * (y >> 1)]);
    };
    each([](float& weight, float& at) { at = weight; });
    const float f = (spoilt >> lane) & 1u ? 0.f : lds_f32(scale_at(slot, key0 + lane));
    __syncwarp();
    const int before = parted && lane < 8 * NQ ? own[lane].x : ev;  // of row `lane`
    int after = ev;
#pragma unroll 4
    for (int r = 0; r < 8 * NQ; ++r) {
      const float weight = w[r * kPitch + lane];
      const int now = max(__shfl_sync(all, before, r), exponent_of(__uint_as_float(__reduce_max_sync(
                                                           all, weight != 0.f ? __float_as_uint(f) : 0u))) + 1);
      w[r * kPitch + lane] = weight != 0.f ? weight * (f * exp2_int(1 - now) * 0.5f) : 0.f;
      if (lane == r) after = now;
    }
    if (lane < 8 * NQ) own[lane] = make_int2(after, before - after);
    parted = true;
    __syncwarp();
    each([](float& weight, float& at) { weight = at; });
#pragma unroll
    for (int x = 0; x < NQ; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int down = own[8 * x + 2 * c + e].y;
        alpha[x][e] *= exp2_int(max(down, -126));
        any = any || down != 0;
      }
  };
  int t = kTeams == 1 ? 0 : (n0 ^ team) & 1;  // the team's first tile
  if (t < pc.tiles) {
    ok = ok && wait_k(n0 + t);
    if (ok) {
      if (tile0 + t * BN + key0 < pc.keys) scores(n0 + t);
      release(empty + k_place<false>(n0 + t) % NS);
    }
  }
  for (; t < pc.tiles && ok; t += kTeams) {
    const int n = n0 + t, v_slot = v_place<false>(n) % NS, at = tile0 + t * BN + key0;
    const bool more = t + kTeams < pc.tiles;
    ok = wait_v(n);
    if (more) ok = ok && wait_k(n + kTeams);
    if (!ok) break;
    const bool work = at < pc.keys, next_work = more && at + kTeams * BN < pc.keys;
    const uint32_t tile = base + v_slot * C::kTile;
    uint32_t alive = ~0u;  // value rows that count: up to the last key, and (new keys) finite
    uint32_t pb[kBlocks][NQ][2];
    bool apart = false;  // (e4m3) rows may see different keys of the warp's
    if (work) {
      const bool masked = at + kKeys > pc.L;  // new keys among them, or keys behind the last
      apart = QUANT && masked && (p.mask || pc.T > 1);
      uint32_t spoilt = 0;  // new keys whose value rows are not finite
      if (masked) {
        if (pc.keys - at < kKeys) alive = (1u << (pc.keys - at)) - 1u;
        const uint32_t fresh = at >= pc.L ? ~0u : ~0u << min(31, pc.L - at);
        const uint32_t bad = bad_rows(v_slot) & alive & fresh;
        alive &= ~bad;
        spoilt = bad;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int kk = 16 * b + g + (y >> 1) * 8, node = at + kk - pc.L;
              const int r = 8 * x + 2 * c + (y & 1);
              if (at + kk >= pc.keys) s[b][x][y] = -INFINITY;
              else if (node < 0 || r >= pc.rows) continue;
              else if (!sees(p, pc, group_div(p, pc.r0 + r), node)) s[b][x][y] = -INFINITY;
              else if ((bad >> kk) & 1u) s[b][x][y] = __uint_as_float(0x7FC00000u);  // the row becomes NaN
            }
      }
      // ---- softmax, base 2; the maximum moves only when a step raises it by more than
      // kMaxSlack, so that O is seldom rescaled ----
      bool any = false;
      float alpha[NQ][2];
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) mx = fmaxf(mx, fmaxf(s[b][x][e], s[b][x][e + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(all, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(all, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(all, mx, 16));
          if (QUANT) mx -= kF16Lift;
          const bool move = mx > m_run[x][e] + kMaxSlack;
          const float m_new = move ? mx : m_run[x][e];
          const float use = m_new == -INFINITY ? 0.f : m_new;
          alpha[x][e] = move ? ex2_approx(m_run[x][e] - use) : 1.f;
          any = any || move;
          m_run[x][e] = m_new;
          m_use[x][e] = use;
          float sum = 0.f;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const float a = ex2_approx(s[b][x][e] - use), z = ex2_approx(s[b][x][e + 2] - use);
            sum += a + z;
            s[b][x][e] = a;
            s[b][x][e + 2] = z;
          }
          l_run[x][e] = l_run[x][e] * alpha[x][e] + sum;
        }
      }
      if (apart) weigh(v_slot, spoilt, alpha, any);
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        // P in 16 bits, the second product's operand type: off by at most 2^-8 (bf16) or
        // 2^-11 (f16) of each weight; l sums the unrounded values.  Queries by rows, keys
        // by columns now
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            pb[b][x][hh] = transpose_8x8(QUANT ? pack_f16x2(s[b][x][2 * hh], s[b][x][2 * hh + 1])
                                               : pack_bf16x2(s[b][x][2 * hh], s[b][x][2 * hh + 1]));
      }
      if (__any_sync(all, any)) {
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
          for (int y = 0; y < kOut; ++y)
#pragma unroll
            for (int z = 0; z < 4; ++z) o[x][y][z] *= alpha[x][z & 1];
      }
    }
    // ---- the next tile's S, then O += P V ----
    if (more) {
      if (next_work) scores(n + kTeams);
      release(empty + k_place<false>(n + kTeams) % NS);
    }
    if (work) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const uint32_t live = alive >> (16 * b);
        if constexpr (!QUANT) {
          // keys 2c, 2c + 1 (and + 8) of a column
          uint32_t mask[2] = {~0u, ~0u};
          if (alive != ~0u)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t two = live >> (2 * c + 8 * x);
              mask[x] = (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u);
            }
          // matrix x of the load: columns 8 (x & 1) of 16, keys 8 (x >> 1)
          const int row = key0 + 16 * b + (lane & 7) + 8 * (lane >> 4), col = (lane >> 3) & 1;
#pragma unroll
          for (int x = 0; x < kOut; ++x) {
            const int chunk = 2 * x + col;
            const uint32_t from = tile + (chunk >> 3) * (BN * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
            uint32_t v[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(from));
#pragma unroll
            for (int y = 0; y < NQ; ++y)
              mma_16816<false>(o[y][x], v[0] & mask[0], v[1] & mask[0], v[2] & mask[1], v[3] & mask[1], pb[b][y][0],
                               pb[b][y][1]);
          }
        } else {
          // the lane's codes of the keys 2c, 2c + 1, 2c + 8, 2c + 9, and their scales
          uint32_t u[4][D / 32];
          float f[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = key0 + 16 * b + 2 * c + (x >> 1) * 8 + (x & 1);
            f[x] = lds_f32(scale_at(v_slot, row));
            if constexpr (D == 128) {
              const uint4 v = lds128(tile + code_at<D>(row, g));
              u[x][0] = v.x; u[x][1] = v.y; u[x][2] = v.z; u[x][3] = v.w;
            } else {
              const uint2 v = lds64(tile + code_at<D>(row, g >> 1) + (g & 1) * 8);
              u[x][0] = v.x; u[x][1] = v.y;
            }
          }
          if (apart || alive != ~0u) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (apart) f[x] = exp2_int(ev);  // (the weights have them: a factor of 1)
              if (!((live >> (2 * c + (x >> 1) * 8 + (x & 1))) & 1u)) {
                f[x] = 0.f;
#pragma unroll
                for (int y = 0; y < D / 32; ++y) u[x][y] = 0u;
              }
            }
          }
          // factors of the lane's keys, relative to 2^ev
          const int e = exponent_of(__uint_as_float(
              __reduce_max_sync(all, __float_as_uint(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]))))));
          if (e > ev) {  // (the same for the warp)
            const float down = exp2_int(max(ev - e, -126));
#pragma unroll
            for (int y = 0; y < NQ; ++y)
#pragma unroll
              for (int x = 0; x < kOut; ++x)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[y][x][z] *= down;
            ev = e;
          }
          const float inv = exp2_int(-ev);
          const uint32_t f0 = pack_f16x2(f[0] * inv, f[1] * inv), f1 = pack_f16x2(f[2] * inv, f[3] * inv);
#pragma unroll
          for (int x = 0; x < kOut; ++x) {  // columns 2x, 2x + 1 of the lane's
            const uint32_t a = __byte_perm(u[0][x >> 1], u[1][x >> 1], x & 1 ? 0x7362 : 0x5140);
            const uint32_t z = __byte_perm(u[2][x >> 1], u[3][x >> 1], x & 1 ? 0x7362 : 0x5140);
            const uint32_t a0 = mul_f16x2(e4m3x2_to_f16x2(a), f0), a1 = mul_f16x2(e4m3x2_to_f16x2(a >> 16), f0);
            const uint32_t a2 = mul_f16x2(e4m3x2_to_f16x2(z), f1), a3 = mul_f16x2(e4m3x2_to_f16x2(z >> 16), f1);
#pragma unroll
            for (int y = 0; y < NQ; ++y) mma_16816<true>(o[y][x], a0, a1, a2, a3, pb[b][y][0], pb[b][y][1]);
          }
        }
      }
    }
    release(empty + v_slot);
  }
  // ---- join the warps of a row: O = sum_w f_w O_w / L, f_w = 2^(m_w - M), L = sum f_w l_w ----
  float* const join = reinterpret_cast<float*>(mem + C::kJoinOff);
  float2* const ml = reinterpret_cast<float2*>(mem + C::kMlOff);
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = l_run[n][e];
      l += __shfl_xor_sync(all, l, 4);
      l += __shfl_xor_sync(all, l, 8);
      l += __shfl_xor_sync(all, l, 16);
      const int r = 8 * n + 2 * c + e;  // of the warp's
      const float down = QUANT ? exp2_int(parted ? own[r].x : ev) : 1.f;
      if (QUANT) __syncwarp();
      if (g == 0) ml[warp * (8 * NQ) + r] = make_float2(m_use[n][e], l);
      float* const dst = join + (warp * (8 * NQ) + r) * D;
      if constexpr (!QUANT) {
#pragma unroll
        for (int x = 0; x < kOut; ++x) {
          dst[join_at<QUANT>(16 * x + g, r)] = o[n][x][e];
          dst[join_at<QUANT>(16 * x + 8 + g, r)] = o[n][x][e + 2];
        }
      } else {
#pragma unroll
        for (int x = 0; x < kOut; x += 2)
          *reinterpret_cast<float4*>(dst + join_at<QUANT>(g * (D / 8) + 2 * x, r)) =
              make_float4(o[n][x][e] * down, o[n][x][e + 2] * down, o[n][x + 1][e] * down, o[n][x + 1][e + 2] * down);
      }
    }
  // (a warp that gave up still comes here, so that none waits for it)
  ok = !bar_warps(!ok);
  if (!ok) return false;
  for (int i = warp * 32 + lane; i < pc.rows * (D / 4); i += 32 * kWarps) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;  // row, column
    float M = -INFINITY, Lsum = 0.f;
    float2 v[kWarps];
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
      v[y] = ml[y * (8 * NQ) + r];
      if (v[y].y != 0.f) M = fmaxf(M, v[y].x);  // (m of a warp without keys means nothing)
    }
    if (M == -INFINITY) M = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
      const float4 part = *reinterpret_cast<const float4*>(join + (y * (8 * NQ) + r) * D + join_at<QUANT>(d, r));
      if (v[y].y == 0.f) continue;
      const float fw = ex2_approx(v[y].x - M);
      Lsum += fw * v[y].y;
      sum.x = fmaf(fw, part.x, sum.x);
      sum.y = fmaf(fw, part.y, sum.y);
      sum.z = fmaf(fw, part.z, sum.z);
      sum.w = fmaf(fw, part.w, sum.w);
    }
    const float inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
    const float4 out = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    const float lse2 = Lsum == 0.f ? -INFINITY : M + lg2_approx(Lsum);
    if (pc.slot >= 0) {
      const long long slot = (long long)pc.slot * C::kRows;
      *reinterpret_cast<float4*>(p.ws_o + slot * D + partial_at(d >> 3, r, C::kRows) + (d & 4)) = out;
      if (d == 0) p.ws_l[slot + r] = lse2;
    } else {
      const int packed = pc.r0 + r, node = group_div(p, packed);
      const long long at = (long long)(pc.row0 + node) * p.Hq + pc.kv_head * p.g + packed - node * p.g;
      if (p.o_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * D + d) = out;
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + d) =
            make_uint2(pack_bf16x2(out.x, out.y), pack_bf16x2(out.z, out.w));
      if (d == 0) p.lse[at] = lse2 * kLn2;
    }
  }
  return true;
}

template <int D, bool QUANT, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
attn_tree_small_kernel(const __grid_constant__ TreeMaps maps, const TreeParams p) {
  using C = TreeCfg<D, QUANT, NQ>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;
  uint64_t* q_empty = q_full + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kWordOff);
  volatile int* issued = abort_flag + 1;  // K and V tiles, for the abort drain
  Pieces& pieces = *reinterpret_cast<Pieces*>(smem + C::kPiecesOff);
  long long* found = reinterpret_cast<long long*>(smem + C::kWordOff + 16);
  auto& sums = *reinterpret_cast<long long (*)[kThreads / 32]>(smem + C::kSumOff);
  static_assert(C::kSumOff + sizeof(sums) + 1024 <= C::kSmemBytes, "shared memory of the launch");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_trigger();  // the merge may be scheduled as blocks of this grid end
  if (threadIdx.x == 0) {
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.k_tail);
    prefetch_tmap(&maps.v_tail);
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, QUANT ? 33 : 1);  // the TMA copies and each lane's scales
      mbar_init(empty + i, kWarps / C::kTeams);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 32);  // each lane's copies
      mbar_init(q_empty + i, kWarps);
    }
    pieces.init(kWarps);
    *abort_flag = 0;
    issued[0] = issued[1] = 0;
    fence_barrier_init();
  }
  const TreeStart start = tree_start(p, sums, found);  // (its barriers publish those above)
  TreePiece pc;
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWarps || warp == kWarps + 1) {  // K, V
      constexpr int kChunks = QUANT ? 1 : D / 64;     // boxes across a row
      constexpr int kLine = C::kTile / BN / kChunks;  // bytes of a box row
      const bool is_v = warp > kWarps;
      const int whole_log = min(7, p.log_page);
      TileLoader<kPieces> w(pieces);
      int n = 0;
      bool ok = true;
      // (e4m3: a tile two ahead; bf16, where a tile takes longer: one)
      LoadTile cur = w.next(p, abort_flag), next{}, later{};
      if (QUANT) next = w.next(p, abort_flag);
      for (; cur.live; ++n) {
        if (QUANT) later = w.next(p, abort_flag);
        const int place = is_v ? v_place<false>(n) : k_place<false>(n), slot = place % NS, row = cur.row(p);
        ok = wait_warp(empty + slot, ((place / NS) & 1) ^ 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        copy_tile<kChunks, kLine>(p, is_v ? &maps.v : &maps.k, is_v ? &maps.v_tail : &maps.k_tail,
                                  smem + slot * C::kTile, full + slot, cur, row, whole_log);
        if constexpr (QUANT) {
          copy_scales(p, is_v ? p.vs : p.ks, cur, row, smem_u32(smem + C::kScaleOff + slot * C::kScales));
          arrive_copies(full + slot);
        }
        cur = QUANT ? next : w.next(p, abort_flag);
        next = later;
      }
      ok = ok && w.ok;
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        issued[is_v ? 1 : 0] = n;
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
    } else if (warp == kWarps + 2) {  // walks the share, two pieces ahead of the queries that it loads
      // (the first piece's queries are on their way before the second is walked)
      TreeWalker<kPieces> walker(p, start, pieces);
      TreePiece pc;
      bool ok = true;
      for (int i = 0;; ++i) {
        walker.upto(p, i == 0 ? 0 : i + 2, abort_flag);
        ok = walker.ok && pieces.get(i, pc, abort_flag, p.timeout_ns);
        if (!ok || pc.tiles == 0) break;
        const int qb = i & 1;
        ok = wait_warp(q_empty + qb, ((i >> 1) & 1) ^ 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        // the query rows, 16-byte chunks swizzled over a row's length
        for (int x = lane; x < pc.rows * (D / 8); x += 32) {
          const int r = x / (D / 8), ch = x % (D / 8), packed = pc.r0 + r, node = group_div(p, packed);
          const __nv_bfloat16* src = p.q + (long long)(pc.row0 + node) * p.q_row +
                                     (long long)(pc.kv_head * p.g + packed - node * p.g) * p.q_head + ch * 8;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           smem_u32(smem + C::kQOff + qb * C::kQ) + r * (D * 2) + ((ch ^ (r & 7)) << 4)),
                       "l"(src)
                       : "memory");
        }
        if (!p.withhold_q) arrive_copies(q_full + qb);
        fetch_masks(p, pc);
        if (i == 0) walker.upto(p, 2, abort_flag);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        walker.end(p);
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWork));
    Warp<D, QUANT, NQ> w;
    w.base = smem_u32(smem);
    w.mem = smem;
    w.full = full;
    w.empty = empty;
    w.q_full = q_full;
    w.q_empty = q_empty;
    w.abort = abort_flag;
    w.warp = warp;
    w.lane = lane;
    w.g = lane >> 2;
    w.c = lane & 3;
    w.team = warp * C::kTeams / kWarps;
    w.key0 = warp % (kWarps / C::kTeams) * C::kKeys;
    int n0 = 0;  // KV tiles before the piece
    bool ok = true;
    for (int n = 0;; ++n) {
      ok = pieces.get(n, pc, abort_flag, p.timeout_ns);
      // (all eight warps go on, or none)
      if (bar_warps(!ok || pc.tiles == 0)) break;
      ok = w.piece(p, pc, n, n0);
      if (!ok) break;
      n0 += pc.tiles;
      if (lane == 0) pieces.done(n);
    }
    if (!ok && lane == 0) {
      set_status(p.status, CPATTN_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  __syncthreads();
  // (after an abort) let the copies in flight land before the shared memory goes
  if (warp == kWarps && lane == 0 && *abort_flag) drain_tiles<false>(full, NS, issued[0], issued[1], p.timeout_ns);
}

template <int D, bool QUANT, int NQ>
int launch(const TreeMaps& m, const TreeParams& p, int num_ctas, cudaStream_t stream) {
  using C = TreeCfg<D, QUANT, NQ>;
  auto kern = attn_tree_small_kernel<D, QUANT, NQ>;
  if (!allow_smem(kern, C::kSmemBytes)) return CPATTN_ERR_CUDA;
  static std::atomic<int> covered{0};
  if (!split_covered(kern, kThreads, kRegsWork * 256 + kRegsOther * 128, covered)) return CPATTN_ERR_UNSUPPORTED;
  return launch_kernel(kern, (unsigned)num_ctas, kThreads, C::kSmemBytes, stream, false, m, p) == cudaSuccess
             ? CPATTN_OK
             : CPATTN_ERR_CUDA;
}
template <int NQ>
int launch(const TreeMaps& m, const TreeParams& p, int d, bool quant, int num_ctas, cudaStream_t stream) {
  return d == 128 ? (quant ? launch<128, true, NQ>(m, p, num_ctas, stream)
                           : launch<128, false, NQ>(m, p, num_ctas, stream))
                  : (quant ? launch<64, true, NQ>(m, p, num_ctas, stream)
                           : launch<64, false, NQ>(m, p, num_ctas, stream));
}

}  // namespace

int launch_tree_small(const TreeMaps& m, const TreeParams& p, int d, bool quant, int num_ctas, cudaStream_t stream) {
  return p.unit_rows == 8 ? launch<1>(m, p, d, quant, num_ctas, stream) : launch<2>(m, p, d, quant, num_ctas, stream);
}

}  // namespace cpattn
