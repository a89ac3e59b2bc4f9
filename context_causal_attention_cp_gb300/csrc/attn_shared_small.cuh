// Small units of cp_attn_shared: at most kSharedSmallRows packed rows, e.g. one token's
// heads of a KV group against the request's own keys.
//
// A 128-row MMA tile would be nearly empty, and the trips through tensor memory (S out,
// P in, O out) take longer than a KV tile's way from HBM.  So a block that has small
// units works on registers, with warp-level 16x8x16 MMAs that have the keys (and then
// the columns of V) as their 16 rows and the queries as their 8 columns:
//     S^T = K Q^T,   O^T += V^T P^T.
// Eight warps share each KV tile, 16 keys each, and each keeps its own maximum, sum and
// output; at a piece's end the eight are joined in shared memory.  The ninth warp loads:
// K and V tiles by TMA, the query rows and (e4m3) the scales by asynchronous copies, all
// of them ahead across piece ends.  A warp's step issues the products of the next tile's
// keys between the softmax and the second product of this one.
//
// What bounds it: HBM in bf16 (256 tokens with 1024 keys each: 166 us, 6.5 TB/s, 0.96 of a
// copy), the instructions that decode in e4m3 (133 us, 4.5 TB/s).  A piece costs 1.1 us
// (e4m3 1.4) besides its tiles.  Queries as the MMAs' 16 rows take twice the MMAs and
// registers: 1.0 -> 1.2 us a KV tile where HBM does not bind (e4m3 1.1 -> 1.4).  Two teams
// of four warps on pieces of their own leave each half the ring (slower by a third), and
// a next piece's queries and first product before the last step of this one help short
// pieces (140 us for 1024 of 128 keys instead of 152) and cost long ones more.
//
// Fragments are loaded as they lie in memory.  K Q^T sums over d in any order, so lane
// (g = lane / 4, c = lane % 4) takes whole 16-byte chunks of key rows g and g + 8 and of
// query row g the same ones: a chunk's elements 4x .. 4x+3 are its share of one k-step.
// The chunks 2c and 2c + 1 of each 128 bytes meet no bank conflict under the 128-byte
// swizzle.  V of a bf16 tile goes through the transposing matrix load.  V codes: the lane
// reads the g-th eighth of the columns of its keys 2c, 2c+1, 2c+8, 2c+9 and joins two
// rows' bytes into a pair for each column, so rows g and g + 8 of product x are columns
// g D/8 + 2x and + 1.
#pragma once
#include <cstdint>

#include "attn_tiles.cuh"

namespace cpattn {
namespace {

constexpr int kSmallWarps = 8, kSmallKeys = BN / kSmallWarps;  // keys of a warp in a KV tile
static_assert(kSmallKeys == 16 && kSharedSmallRows == 8, "an MMA's rows (and one k-step), and its columns");
constexpr int kMaxSmallStages = 12;

template <int D, bool QUANT>
struct SmallCfg {
  static constexpr int kTile = BN * D * (QUANT ? 1 : 2);
  static constexpr int kScales = QUANT ? BN * 4 : 0;   // the rows' scales, fp32
  static constexpr int kQ = kSharedSmallRows * D * 2;  // two of them
  static constexpr int kJoin = kSmallWarps * kSharedSmallRows * D * 4;
  static constexpr int kMl = 2 * kSmallWarps * kSharedSmallRows * 8;
  static constexpr int kFixed = 2 * kQ + kJoin + kMl + (2 * kMaxSmallStages + 4) * 8 + 16 + 1024;
  static constexpr int kFit = (232448 - kFixed) / (kTile + kScales);
  static constexpr int kStages = kFit < kMaxSmallStages ? kFit : kMaxSmallStages;
  static constexpr int kScaleOff = kStages * kTile;
  static constexpr int kQOff = kScaleOff + kStages * kScales;
  static constexpr int kJoinOff = kQOff + 2 * kQ;
  static constexpr int kMlOff = kJoinOff + kJoin;  // (m, l) of each warp's rows, two of them
  static constexpr int kBarOff = kMlOff + kMl;
  static constexpr int kWordOff = kBarOff + (2 * kStages + 4) * 8;
  static constexpr int kSmemBytes = kWordOff + 16 + 1024;  // + align slack
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// The 256 threads of the eight warps; true when any of them says so.
__device__ __forceinline__ bool bar_small(bool any) {
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

// What a warp needs to work on the pieces.
template <int D, bool QUANT>
struct SmallWarp {
  uint32_t base;  // shared memory
  uint8_t* mem;
  uint64_t *full, *empty, *q_full, *q_empty;
  const volatile int* abort;
  int warp, g, c, lane;
  __device__ __forceinline__ void release(uint64_t* bar) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  __device__ __forceinline__ uint32_t scale_at(int slot, int row) const {
    using C = SmallCfg<D, QUANT>;
    return base + C::kScaleOff + slot * C::kScales + row * 4;
  }
};

// K of a warp's 16 keys: chunks of rows g and g + 8, as they lie.
template <int D, bool QUANT>
struct SmallK {
  static constexpr int kLoads = QUANT ? D / 64 : D / 32;
  uint4 v[2][kLoads];
  float scale[2];
  __device__ __forceinline__ void load(const SmallWarp<D, QUANT>& w, int slot) {
    const uint32_t tile = w.base + slot * SmallCfg<D, QUANT>::kTile;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = w.warp * kSmallKeys + 8 * j + w.g;
#pragma unroll
      for (int x = 0; x < kLoads; ++x)
        v[j][x] = QUANT ? lds128(tile + code_at<D>(row, D == 128 ? 2 * w.c + x : w.c))
                        : lds128(tile + (x >> 1) * (BN * 128) + row * 128 +
                                 (((2 * w.c + (x & 1)) ^ (row & 7)) << 4));
      scale[j] = QUANT ? lds_f32(w.scale_at(slot, row)) : 1.f;
    }
  }
  // s: keys g (0, 1) and g + 8 (2, 3), queries 2c, 2c + 1; two chains, for their latency
  __device__ __forceinline__ void product(const uint32_t (&q)[D / 16][2], const float (&factor)[2],
                                          float (&s)[4]) const {
    float s2[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) s[y] = s2[y] = 0.f;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const uint32_t u0[4] = {v[0][x].x, v[0][x].y, v[0][x].z, v[0][x].w};
      const uint32_t u1[4] = {v[1][x].x, v[1][x].y, v[1][x].z, v[1][x].w};
      if constexpr (!QUANT) {
        mma_16816<false>(s, u0[0], u1[0], u0[1], u1[1], q[2 * x][0], q[2 * x][1]);
        mma_16816<false>(s2, u0[2], u1[2], u0[3], u1[3], q[2 * x + 1][0], q[2 * x + 1][1]);
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y)
          mma_16816<true>(y & 1 ? s2 : s, e4m3x2_to_f16x2(u0[y]), e4m3x2_to_f16x2(u1[y]),
                          e4m3x2_to_f16x2(u0[y] >> 16), e4m3x2_to_f16x2(u1[y] >> 16), q[4 * x + y][0],
                          q[4 * x + y][1]);
      }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
      s[y] = (s[y] + s2[y]) * (QUANT ? score_factor(factor[y & 1], scale[y >> 1]) : factor[y & 1]);
  }
};

// One piece; n its number in the list, seq the ring place of its first
// tile; turns: the last piece used a half of the join buffer.
template <int D, bool QUANT>
__device__ __forceinline__ bool small_piece(const SharedParams& p, const SmallWarp<D, QUANT>& w,
                                            const SharedPiece& pc, int n, int& seq, bool& turns) {
  using C = SmallCfg<D, QUANT>;
  constexpr int NS = C::kStages, kOut = D / 16;
  const unsigned all = 0xffffffffu;
  const int g = w.g, c = w.c, key0 = w.warp * kSmallKeys, T = num_tiles(pc.keys), qb = n & 1;
  // keys of the piece that the rows 2c, 2c + 1 see, that any and that all rows see
  int seen[2], last_seen = 0, full_seen = pc.keys;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * c + e;
    seen[e] = 0;
    if (r < pc.rows) {
      const long long pos = (long long)pc.q_pos0 + (long long)group_div(p, pc.r0 + r) * pc.q_pos_step;
      seen[e] = (int)max(0LL, min((long long)pc.keys, pos + 1 - pc.key0));
      last_seen = max(last_seen, seen[e]);
      full_seen = min(full_seen, seen[e]);
    }
  }
  last_seen = __reduce_max_sync(all, last_seen);
  full_seen = __reduce_min_sync(all, full_seen);
  // ---- queries: row g ----
  uint32_t q[D / 16][2];
  float factor[2];
  bool ok = wait_warp(w.q_full + qb, (n >> 1) & 1, w.abort, p.timeout_ns);
  uint4 v[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    v[x] = lds128(w.base + C::kQOff + qb * C::kQ + g * (D * 2) +
                  (((q_chunk<D, QUANT>(c, x) >> 3) ^ g) << 4));
    if (g >= pc.rows) v[x] = make_uint4(0, 0, 0, 0);
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
  factor[0] = __shfl_sync(all, f_row, 8 * c);      // of row 2c
  factor[1] = __shfl_sync(all, f_row, 8 * c + 4);  // and the next
#pragma unroll
  for (int x = 0; x < D / 32; ++x) {
    q[2 * x][0] = v[x].x;
    q[2 * x][1] = v[x].y;
    q[2 * x + 1][0] = v[x].z;
    q[2 * x + 1][1] = v[x].w;
  }
  w.release(w.q_empty + qb);
  float o[kOut][4];
#pragma unroll
  for (int x = 0; x < kOut; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
  float m_run[2], m_use[2], l_run[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    m_run[e] = -INFINITY;
    m_use[e] = l_run[e] = 0.f;
  }
  int ev = -126;  // (e4m3) exponent of O
  SmallK<D, QUANT> k;
  float s[4];
  ok = ok && wait_warp(w.full + seq % NS, (seq / NS) & 1, w.abort, p.timeout_ns);
  if (ok) {
    if (key0 < last_seen) {  // (some row sees some of the warp's keys)
      k.load(w, seq % NS);
      k.product(q, factor, s);
    }
    w.release(w.empty + seq % NS);
  }
  for (int t = 0; t < T && ok; ++t, seq += 2) {
    const int at0 = t * BN + key0, v_slot = (seq + 1) % NS, k_slot = (seq + 2) % NS;
    const bool work = at0 < last_seen, next = t + 1 < T, next_work = next && at0 + BN < last_seen;
    ok = wait_warp(w.full + v_slot, ((seq + 1) / NS) & 1, w.abort, p.timeout_ns) &&
         (!next || wait_warp(w.full + k_slot, ((seq + 2) / NS) & 1, w.abort, p.timeout_ns));
    if (!ok) break;
    if (next_work) k.load(w, k_slot);
    const uint32_t tile = w.base + v_slot * C::kTile;
    const int live = pc.keys - at0;  // of the warp's keys
    // (e4m3) the lane's codes of the keys 2c, 2c + 1, 2c + 8, 2c + 9, and their scales
    uint32_t u[4][D / 32];
    float f[4];
    if constexpr (QUANT) {
      if (work) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = key0 + 2 * c + (x >> 1) * 8 + (x & 1);
          f[x] = lds_f32(w.scale_at(v_slot, row));
          if constexpr (D == 128) {
            const uint4 v = lds128(tile + code_at<D>(row, g));
            u[x][0] = v.x; u[x][1] = v.y; u[x][2] = v.z; u[x][3] = v.w;
          } else {
            const uint2 v = lds64(tile + code_at<D>(row, g >> 1) + (g & 1) * 8);
            u[x][0] = v.x; u[x][1] = v.y;
          }
        }
        if (live < kSmallKeys) {  // rows behind the last key are zeros
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (2 * c + (x >> 1) * 8 + (x & 1) >= live) {
              f[x] = 0.f;
#pragma unroll
              for (int y = 0; y < D / 32; ++y) u[x][y] = 0u;
            }
        }
      }
    }
    // ---- softmax, base 2; the maximum moves as in softmax_tile ----
    uint32_t pb[2];
    if (work) {
      if (at0 + kSmallKeys > full_seen) {
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (at0 + g + (y >> 1) * 8 >= seen[y & 1]) s[y] = -INFINITY;
      }
      float alpha[2];
      bool any = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[e], s[e + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(all, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(all, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(all, mx, 16));
        if (QUANT) mx -= kF16Lift;
        const bool move = mx > m_run[e] + kMaxSlack;
        const float m_new = move ? mx : m_run[e];
        const float use = m_new == -INFINITY ? 0.f : m_new;
        alpha[e] = move ? ex2_approx(m_run[e] - use) : 1.f;
        any = any || move;
        m_run[e] = m_new;
        m_use[e] = use;
        const float a = ex2_approx(s[e] - use), z = ex2_approx(s[e + 2] - use);
        l_run[e] = l_run[e] * alpha[e] + (a + z);
        s[e] = a;
        s[e + 2] = z;
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)  // keys g, g + 8
        // P in 16 bits, as in softmax_tile; queries by rows, keys by columns now
        pb[hh] = transpose_8x8(QUANT ? pack_f16x2(s[2 * hh], s[2 * hh + 1])
                                     : pack_bf16x2(s[2 * hh], s[2 * hh + 1]));
      if (__any_sync(all, any)) {
#pragma unroll
        for (int x = 0; x < kOut; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[x][y] *= alpha[y & 1];
      }
    }
    // ---- the next tile's S, then O += P V ----
    if (next_work) k.product(q, factor, s);
    if (next) w.release(w.empty + k_slot);
    if (work) {
      if constexpr (!QUANT) {
        // keys 2c, 2c + 1 (and + 8) of a column: rows behind the last key are zeros
        uint32_t mask[2] = {~0u, ~0u};
        if (live < kSmallKeys)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            mask[x] = (2 * c + 8 * x < live ? 0xFFFFu : 0u) | (2 * c + 8 * x + 1 < live ? 0xFFFF0000u : 0u);
        // matrix x of the load: columns 8 (x & 1) of 16, keys 8 (x >> 1)
        const int row = key0 + (w.lane & 7) + 8 * (w.lane >> 4), col = (w.lane >> 3) & 1;
#pragma unroll
        for (int x = 0; x < kOut; ++x) {
          const int chunk = 2 * x + col;
          const uint32_t at =
              tile + (chunk >> 3) * (BN * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
          uint32_t v[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(at));
          mma_16816<false>(o[x], v[0] & mask[0], v[1] & mask[0], v[2] & mask[1], v[3] & mask[1], pb[0],
                           pb[1]);
        }
      } else {
        // factors of the lane's keys, relative to 2^ev
        const int e = exponent_of(__uint_as_float(__reduce_max_sync(
            all, __float_as_uint(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]))))));
        if (e > ev) {  // (the same for the warp)
          const float down = exp2_int(max(ev - e, -126));
#pragma unroll
          for (int x = 0; x < kOut; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[x][y] *= down;
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
          mma_16816<true>(o[x], a0, a1, a2, a3, pb[0], pb[1]);
        }
      }
    }
    w.release(w.empty + v_slot);
  }
  // ---- join the warps: O = sum_w f_w O_w / L, f_w = 2^(m_w - M), L = sum f_w l_w; up to 4
  // rows in the halves of the buffer in turn, so that the next piece need not wait for
  // this one's readers ----
  const float down = exp2_int(ev);
  const bool halves = pc.rows <= kSharedSmallRows / 2;
  float* const join = reinterpret_cast<float*>(w.mem + C::kJoinOff + (halves && (n & 1) ? C::kJoin / 2 : 0));
  const int stride = halves ? kSharedSmallRows / 2 : kSharedSmallRows;  // rows of a warp's part
  float2* const ml = reinterpret_cast<float2*>(w.mem + C::kMlOff) + (n & 1) * (kSmallWarps * kSharedSmallRows);
  float l[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] = l_run[e];
    l[e] += __shfl_xor_sync(all, l[e], 4);
    l[e] += __shfl_xor_sync(all, l[e], 8);
    l[e] += __shfl_xor_sync(all, l[e], 16);
  }
  // the buffer's last readers: only between pieces that take turns none are left
  if (!halves || !turns) bar_small(false);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * c + e;
    if (r >= pc.rows) break;
    if (g == 0) ml[w.warp * kSharedSmallRows + r] = make_float2(m_use[e], l[e]);
    float* const dst = join + (w.warp * stride + r) * D;
    if constexpr (!QUANT) {
#pragma unroll
      for (int x = 0; x < kOut; ++x) {
        dst[join_at<QUANT>(16 * x + g, r)] = o[x][e];
        dst[join_at<QUANT>(16 * x + 8 + g, r)] = o[x][e + 2];
      }
    } else {
#pragma unroll
      for (int x = 0; x < kOut; x += 2)
        *reinterpret_cast<float4*>(dst + join_at<QUANT>(g * (D / 8) + 2 * x, r)) =
            make_float4(o[x][e] * down, o[x][e + 2] * down, o[x + 1][e] * down,
                        o[x + 1][e + 2] * down);
    }
  }
  // (a warp that gave up still comes here, so that none waits for it)
  ok = !bar_small(!ok);
  if (!ok) return false;
  for (int i = w.warp * 32 + w.lane; i < pc.rows * (D / 4); i += 32 * kSmallWarps) {
    const int x = i / (D / 4), d = i % (D / 4) * 4;  // row, column
    float m[kSmallWarps], lw[kSmallWarps], M = -INFINITY, L = 0.f;
    float4 part[kSmallWarps];
#pragma unroll
    for (int y = 0; y < kSmallWarps; ++y) {
      const float2 v = ml[y * kSharedSmallRows + x];
      part[y] = *reinterpret_cast<const float4*>(join + (y * stride + x) * D + join_at<QUANT>(d, x));
      m[y] = v.x;
      lw[y] = v.y;
      if (lw[y] != 0.f) M = fmaxf(M, m[y]);  // (m of a warp without keys means nothing)
    }
    if (M == -INFINITY) M = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kSmallWarps; ++y) {
      if (lw[y] == 0.f) continue;
      const float fw = ex2_approx(m[y] - M);
      L += fw * lw[y];
      sum.x = fmaf(fw, part[y].x, sum.x);
      sum.y = fmaf(fw, part[y].y, sum.y);
      sum.z = fmaf(fw, part[y].z, sum.z);
      sum.w = fmaf(fw, part[y].w, sum.w);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<float4*>(p.ws_o + (long long)pc.ws_row * D + partial_at(d >> 3, x, pc.rows) + (d & 4)) =
        make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    if (d == 0) p.ws_l[(long long)pc.ws_row + x] = L == 0.f ? -INFINITY : M + lg2_approx(L);
  }
  turns = halves;
  return true;
}

template <int D, bool QUANT>
__device__ __forceinline__ void run_small(const SharedParams& p, const SharedCta& list, uint8_t* smem,
                                          const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                          const CUtensorMap* tm_k_tail, const CUtensorMap* tm_v_tail) {
  using C = SmallCfg<D, QUANT>;
  constexpr int NS = C::kStages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;
  uint64_t* q_empty = q_full + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kWordOff);
  volatile int* issued_loads = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, QUANT ? 33 : 1);  // the TMA copy and each lane's scales
      mbar_init(empty + i, kSmallWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 32);  // each lane's copies
      mbar_init(q_empty + i, kSmallWarps);
    }
    *abort_flag = 0;
    *issued_loads = 0;
    fence_barrier_init();
  }
  __syncthreads();
  auto arrive_copies = [&](uint64_t* bar) {  // when this lane's copies so far have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
  };

  if (warp >= kSmallWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SharedCfg<D, QUANT>::kRegsOther));
    if (warp == kProducerWarp) {
      constexpr int kChunks = QUANT ? 1 : D / 64;      // boxes across a row
      constexpr int kLine = C::kTile / BN / kChunks;   // bytes of a box row
      int seq = 0;
      bool ok = true;
      for (int i = list.small0; i < list.small1 && ok; ++i) {
        const SharedPiece pc = load_piece(p, i);
        const int n = i - list.small0, qb = n & 1;
        ok = wait_warp(q_empty + qb, ((n >> 1) & 1) ^ 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        // the query rows, 16-byte chunks swizzled over a row's length
        for (int x = lane; x < pc.rows * (D / 8); x += 32) {
          const int r = x / (D / 8), ch = x % (D / 8), packed = pc.r0 + r, qi = group_div(p, packed);
          const __nv_bfloat16* src = p.q + (long long)(pc.q_row0 + qi) * p.q_row +
                                     (long long)(pc.kv_head * p.g + packed - qi * p.g) * p.q_head + ch * 8;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           smem_u32(smem + C::kQOff + qb * C::kQ) + r * (D * 2) + ((ch ^ (r & 7)) << 4)),
                       "l"(src)
                       : "memory");
        }
        if (!p.withhold_q) arrive_copies(q_full + qb);
        for (int u = 0; u < 2 * num_tiles(pc.keys); ++u, ++seq) {  // K0 V0 K1 V1 ...
          const int slot = seq % NS, t = u >> 1, row = pc.kv_row + t * BN, live = pc.keys - t * BN;
          const bool is_v = u & 1;
          ok = wait_warp(empty + slot, ((seq / NS) & 1) ^ 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          uint8_t* dst = smem + slot * C::kTile;
          if (lane == 0) {
            const bool whole = live > BN - kTailRows;
            const int boxes = whole ? 1 : (live + kTailRows - 1) / kTailRows;
            const int rows = whole ? BN : kTailRows;  // of a box
            const CUtensorMap* tm = whole ? (is_v ? tm_v : tm_k) : (is_v ? tm_v_tail : tm_k_tail);
            mbar_arrive_expect_tx(full + slot, boxes * rows * kLine * kChunks);
            for (int x = 0; x < boxes; ++x)
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                tma_load_3d(dst + (c * BN + x * rows) * kLine, tm, full + slot, c * 64, pc.kv_head,
                            row + x * rows);
          }
          __syncwarp();
          if constexpr (QUANT) {
            const float* src = (is_v ? p.vs : p.ks) + (long long)pc.kv_head * p.s_head + row + lane;
            const uint32_t at = smem_u32(smem + C::kScaleOff + slot * C::kScales) + lane * 4;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x * 32 + lane < live)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + x * 128),
                             "l"(src + x * 32)
                             : "memory");
            arrive_copies(full + slot);
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        *issued_loads = seq;
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SharedCfg<D, QUANT>::kRegsSoftmax));
    const SmallWarp<D, QUANT> w{smem_u32(smem), smem, full, empty, q_full, q_empty, abort_flag,
                                warp, lane >> 2, lane & 3, lane};
    int seq = 0;
    bool ok = true, turns = true;
    SharedPiece np = load_piece(p, list.small0);
    for (int i = list.small0; i < list.small1 && ok; ++i) {
      const SharedPiece pc = np;
      if (i + 1 < list.small1) np = load_piece(p, i + 1);
      ok = small_piece<D, QUANT>(p, w, pc, i - list.small0, seq, turns);
    }
    if (!ok && lane == 0) {
      set_status(p.status, CPATTN_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  }
  __syncthreads();
  if (warp == kProducerWarp && lane == 0 && *abort_flag) {
    // let the copies in flight land before the shared memory goes
    const int n = *issued_loads;
    for (int j = max(0, n - NS); j < n; ++j)
      wait_one(full + j % NS, (j / NS) & 1, nullptr, p.timeout_ns);
  }
}

}  // namespace
}  // namespace cpattn
