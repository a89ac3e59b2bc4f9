// Small units of cp_attn_shared: at most kSharedSmallRows packed rows, e.g. one token's
// heads of a KV group against the request's own keys.
//
// A 128-row MMA tile would be nearly empty, and the trips through tensor memory (S out,
// P in, O out) take longer than a KV tile's way from HBM.  So a block that has small
// units works on registers: eight warps share each KV tile, 16 keys each, with warp-level
// 16x8x16 MMAs, and each keeps its own maximum, sum and 16 x D output; at a piece's end
// the eight are joined in shared memory.  What bounds it is HBM: a KV tile costs a warp
// about 100 instructions (250 with codes) and the block 64 KB (33 KB).  The ninth warp
// loads: K and V tiles by TMA, the query rows and (e4m3) the scales by asynchronous
// copies, all of them ahead across piece ends.  A warp's step issues the products of the
// next tile's keys between the softmax and the second product of this one, so that their
// latencies overlap.
//
// Fragments are loaded as they lie in memory.  Q K^T sums over d in any order, so lane
// (key g = lane / 4, c = lane % 4) takes whole 16-byte chunks of a key row, and of a
// query row the same ones: a chunk's elements 4x .. 4x+3 are its share of one k-step.
// The chunks 2c and 2c + 1 of each 128 bytes meet no bank conflict under the 128-byte
// swizzle.  V of a bf16 tile goes through the transposing matrix load.  V codes: lane
// (d group g, c) reads 16 codes of each of its keys 2c, 2c+1, 2c+8, 2c+9, and joins two
// rows' bytes into a pair for each d, so column 8j + g of the MMAs' output is d = 16g + j.
#pragma once
#include <cstdint>

#include "attn_common.cuh"
#include "shared_plan.h"

namespace cpattn {
namespace {

constexpr int kSmallWarps = 8, kSmallKeys = BN / kSmallWarps;  // keys of a warp in a KV tile
static_assert(kSmallKeys == 16, "one MMA k-step");
constexpr int kMaxSmallStages = 12;

template <int D, bool QUANT>
struct SmallCfg {
  static constexpr int kTile = BN * D * (QUANT ? 1 : 2);
  static constexpr int kScales = QUANT ? BN * 4 : 0;  // the rows' scales, fp32
  static constexpr int kQ = kSharedSmallRows * D * 2;  // two of them
  static constexpr int kJoinRows = 8;                  // rows that are joined in one round
  static constexpr int kJoin = kSmallWarps * kJoinRows * D * 4;
  static constexpr int kMl = 2 * kSmallWarps * kJoinRows * 8;
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

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {  // the low half
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}

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
// Place of column d of row r in a warp's part of the join buffer (bank swizzle).
template <int D>
__device__ __forceinline__ int join_at(int d, int r) {
  return d ^ (((d >> 5) & 3) << 2) ^ ((r & (D / 16 - 1)) << 4);
}

// One KV tile's K for a warp: the chunks of its keys (row = key0 + 8j + g), as they lie.
template <int D, bool QUANT>
struct SmallK {
  static constexpr int kLoads = QUANT ? D / 64 : D / 32;
  uint4 v[2][kLoads];
  float2 scale[2];  // (e4m3) of the keys 8j + 2c, + 1
  __device__ __forceinline__ void load(uint32_t tile, const float* scales, int key0, int g, int c) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = key0 + 8 * j + g;
#pragma unroll
      for (int x = 0; x < kLoads; ++x)
        v[j][x] = QUANT ? lds128(tile + code_at<D>(row, D == 128 ? 2 * c + x : c))
                        : lds128(tile + (x >> 1) * (BN * 128) + row * 128 +
                                 (((2 * c + (x & 1)) ^ (row & 7)) << 4));
      if (QUANT) scale[j] = *reinterpret_cast<const float2*>(scales + key0 + 8 * j + 2 * c);
    }
  }
  // s[j]: keys 8j + 2c, + 1 of rows g, g + 8; two chains a product, for their latency
  __device__ __forceinline__ void product(const uint32_t (&q)[D / 16][4], const float (&factor)[2],
                                          float (&s)[2][4]) const {
    float s2[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int y = 0; y < 4; ++y) s[j][y] = s2[j][y] = 0.f;
#pragma unroll
    for (int x = 0; x < kLoads; ++x)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (!QUANT) {
          mma_16816<false>(s[j], q[2 * x], v[j][x].x, v[j][x].y);
          mma_16816<false>(s2[j], q[2 * x + 1], v[j][x].z, v[j][x].w);
        } else {
          const uint32_t w[4] = {v[j][x].x, v[j][x].y, v[j][x].z, v[j][x].w};
#pragma unroll
          for (int y = 0; y < 4; ++y)
            mma_16816<true>(y & 1 ? s2[j] : s[j], q[4 * x + y], e4m3x2_to_f16x2(w[y]),
                            e4m3x2_to_f16x2(w[y] >> 16));
        }
      }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        s[j][2 * hh] = (s[j][2 * hh] + s2[j][2 * hh]) * (QUANT ? factor[hh] * scale[j].x : factor[hh]);
        s[j][2 * hh + 1] =
            (s[j][2 * hh + 1] + s2[j][2 * hh + 1]) * (QUANT ? factor[hh] * scale[j].y : factor[hh]);
      }
  }
};

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
        arrive_copies(q_full + qb);
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
    const int g = lane >> 2, c = lane & 3;
    const int key0 = warp * kSmallKeys;   // the warp's keys of a tile
    const uint32_t smem_base = smem_u32(smem);
    constexpr int kSteps = D / 16;        // k-steps of Q K^T
    constexpr int kOut = D / 8;           // column blocks of O
    auto scales_of = [&](int slot) {
      return reinterpret_cast<const float*>(smem + C::kScaleOff + slot * C::kScales);
    };
    int seq = 0;
    bool ok = true, turns = true;  // turns: the last piece used a half of the join buffer
    SharedPiece np = load_piece(p, list.small0);
    for (int i = list.small0; i < list.small1; ++i) {
      const SharedPiece pc = np;
      if (i + 1 < list.small1) np = load_piece(p, i + 1);
      const int T = num_tiles(pc.keys), n = i - list.small0, qb = n & 1;
      int seen[2], last_seen = 0, full_seen = pc.keys;  // keys that any, that all rows see
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = g + 8 * hh;
        seen[hh] = 0;
        if (r < pc.rows) {
          const long long pos = (long long)pc.q_pos0 + (long long)group_div(p, pc.r0 + r) * pc.q_pos_step;
          seen[hh] = (int)max(0LL, min((long long)pc.keys, pos + 1 - pc.key0));
          last_seen = max(last_seen, seen[hh]);
          full_seen = min(full_seen, seen[hh]);
        }
      }
      last_seen = __reduce_max_sync(0xffffffffu, last_seen);
      full_seen = __reduce_min_sync(0xffffffffu, full_seen);
      // ---- queries: rows g and g + 8 ----
      uint32_t q[kSteps][4];
      float factor[2] = {p.scale_log2, p.scale_log2};
      ok = wait_warp(q_full + qb, (n >> 1) & 1, abort_flag, p.timeout_ns);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = g + 8 * hh;
        uint4 v[D / 32];
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          v[x] = lds128(smem_base + C::kQOff + qb * C::kQ + r * (D * 2) +
                        (((q_chunk<D, QUANT>(c, x) >> 3) ^ (r & 7)) << 4));
          if (r >= pc.rows) v[x] = make_uint4(0, 0, 0, 0);
        }
        if constexpr (QUANT) {
          // bf16 to f16 times 2^f with 2^f max|q| in [2^14, 2^15)
          uint32_t mx = 0;
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            mx = __vmaxu2(__vmaxu2(mx, __vmaxu2(v[x].x & 0x7FFF7FFFu, v[x].y & 0x7FFF7FFFu)),
                          __vmaxu2(v[x].z & 0x7FFF7FFFu, v[x].w & 0x7FFF7FFFu));
          mx = max(mx & 0xFFFFu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int f = min(max(14 - ((int)(mx >> 7) - 127), -126), 126);
          const float up = exp2_int(f);
          factor[hh] *= exp2_int(-f);
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t* const w = &v[x].x;
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = pack_f16x2(__uint_as_float(w[y] << 16) * up, __uint_as_float(w[y] & 0xFFFF0000u) * up);
          }
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          q[2 * x][hh] = v[x].x;
          q[2 * x][hh + 2] = v[x].y;
          q[2 * x + 1][hh] = v[x].z;
          q[2 * x + 1][hh + 2] = v[x].w;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty + qb);
      float o[kOut][4];
#pragma unroll
      for (int x = 0; x < kOut; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
      float m_run[2] = {-INFINITY, -INFINITY}, m_use[2] = {0.f, 0.f}, l_run[2] = {0.f, 0.f};
      int ev = -126;  // (e4m3) exponent of O
      // S of a tile; t the tile, seq_t its K tile's place
      auto begin_s = [&](SmallK<D, QUANT>& k, int t, int seq_t) {
        const int slot = seq_t % NS;
        if (!wait_warp(full + slot, (seq_t / NS) & 1, abort_flag, p.timeout_ns)) return false;
        if (t * BN + key0 < last_seen)  // (some row sees some of the warp's keys)
          k.load(smem_base + slot * C::kTile, scales_of(slot), key0, g, c);
        return true;
      };
      auto release = [&](int slot) {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + slot);
      };
      SmallK<D, QUANT> k;
      float s[2][4];
      ok = ok && begin_s(k, 0, seq);
      if (ok) {
        if (key0 < last_seen) k.product(q, factor, s);
        release(seq % NS);
      }
      for (int t = 0; t < T && ok; ++t, seq += 2) {
        const int v_slot = (seq + 1) % NS, at0 = t * BN + key0;
        const bool work = at0 < last_seen, next = t + 1 < T, next_work = next && at0 + BN < last_seen;
        ok = wait_warp(full + v_slot, ((seq + 1) / NS) & 1, abort_flag, p.timeout_ns);
        if (ok && next) ok = begin_s(k, t + 1, seq + 2);
        if (!ok) break;
        const uint32_t tile = smem_base + v_slot * C::kTile;
        const int live = pc.keys - at0;  // of the warp's keys
        // (e4m3) the lane's codes of the keys 2c, 2c + 1, 2c + 8, 2c + 9 and their scales
        uint32_t w[4][D / 32];
        float f[4];
        if constexpr (QUANT) {
          if (work) {
            const float* sc = scales_of(v_slot) + key0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = 2 * c + (x >> 1) * 8 + (x & 1), row = key0 + key;
              f[x] = sc[key];
              if constexpr (D == 128) {
                const uint4 v = lds128(tile + code_at<D>(row, g));
                w[x][0] = v.x; w[x][1] = v.y; w[x][2] = v.z; w[x][3] = v.w;
              } else {
                const uint2 v = lds64(tile + code_at<D>(row, g >> 1) + (g & 1) * 8);
                w[x][0] = v.x; w[x][1] = v.y;
              }
              if (key >= live) {  // rows behind the last key are zeros
                f[x] = 0.f;
#pragma unroll
                for (int y = 0; y < D / 32; ++y) w[x][y] = 0u;
              }
            }
          }
        }
        // ---- softmax, base 2; the maximum moves as in softmax_tile ----
        uint32_t pa[4];
        if (work) {
          if (at0 + kSmallKeys > full_seen) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                if (at0 + 8 * j + 2 * c + (y & 1) >= seen[y >> 1]) s[j][y] = -INFINITY;
          }
          float alpha[2];
          bool any = false;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float mx = fmaxf(fmaxf(s[0][2 * hh], s[0][2 * hh + 1]), fmaxf(s[1][2 * hh], s[1][2 * hh + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const bool move = mx > m_run[hh] + kMaxSlack;
            const float m_new = move ? mx : m_run[hh];
            const float use = m_new == -INFINITY ? 0.f : m_new;
            alpha[hh] = move ? ex2_approx(m_run[hh] - use) : 1.f;
            any = any || move;
            m_run[hh] = m_new;
            m_use[hh] = use;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float a = ex2_approx(s[j][2 * hh] - use), b = ex2_approx(s[j][2 * hh + 1] - use);
              sum += a + b;
              // P in 16 bits, as in softmax_tile
              pa[2 * j + hh] = QUANT ? pack_f16x2(a, b) : pack_bf16x2(a, b);
            }
            l_run[hh] = l_run[hh] * alpha[hh] + sum;
          }
          if (__any_sync(0xffffffffu, any)) {
#pragma unroll
            for (int x = 0; x < kOut; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) o[x][y] *= alpha[y >> 1];
          }
        }
        // ---- the next tile's S, then O += P V ----
        if (next_work) k.product(q, factor, s);
        if (next) release((seq + 2) % NS);
        if (work) {
          if constexpr (!QUANT) {
            // keys 2c, 2c + 1 (and + 8) of a column: rows behind the last key are zeros
            uint32_t mask[2] = {~0u, ~0u};
            if (live < kSmallKeys)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                mask[x] = (2 * c + 8 * x < live ? 0xFFFFu : 0u) | (2 * c + 8 * x + 1 < live ? 0xFFFF0000u : 0u);
            // matrix x of the load: keys 8 (x & 1), columns 8 (x >> 1) of 16
            const int row = key0 + (lane & 15);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const int chunk = 2 * x + (lane >> 4);
              const uint32_t at = tile + (chunk >> 3) * (BN * 128) + row * 128 +
                                  (((chunk & 7) ^ (row & 7)) << 4);
              uint32_t v[4];
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                           : "r"(at));
              mma_16816<false>(o[2 * x], pa, v[0] & mask[0], v[1] & mask[1]);
              mma_16816<false>(o[2 * x + 1], pa, v[2] & mask[0], v[3] & mask[1]);
            }
          } else {
            // factors of the lane's keys, relative to 2^ev
            const uint32_t mx = __reduce_max_sync(
                0xffffffffu, __float_as_uint(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]))));
            const int e = exponent_of(__uint_as_float(mx));
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
            for (int y = 0; y < D / 32; ++y) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {  // two columns at a time
                const uint32_t a = __byte_perm(w[0][y], w[1][y], z ? 0x7362 : 0x5140);
                const uint32_t b = __byte_perm(w[2][y], w[3][y], z ? 0x7362 : 0x5140);
                mma_16816<true>(o[4 * y + 2 * z], pa, mul_f16x2(e4m3x2_to_f16x2(a), f0),
                                mul_f16x2(e4m3x2_to_f16x2(b), f1));
                mma_16816<true>(o[4 * y + 2 * z + 1], pa, mul_f16x2(e4m3x2_to_f16x2(a >> 16), f0),
                                mul_f16x2(e4m3x2_to_f16x2(b >> 16), f1));
              }
            }
          }
        }
        release(v_slot);
      }
      // ---- join the warps: O = sum_w f_w O_w / L, f_w = 2^(m_w - M), L = sum f_w l_w,
      // rows 0-7 and then 8-15; up to 4 rows in the halves of the buffer in turn, so that
      // the next piece need not wait for this one's readers ----
      const float down = exp2_int(ev);
      const bool halves = pc.rows <= C::kJoinRows / 2;
      float* const join = reinterpret_cast<float*>(smem + C::kJoinOff + (halves && (n & 1) ? C::kJoin / 2 : 0));
      const int stride = halves ? C::kJoinRows / 2 : C::kJoinRows;  // rows of a warp's part
      float2* const ml = reinterpret_cast<float2*>(smem + C::kMlOff) + (n & 1) * (kSmallWarps * C::kJoinRows);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        if (hh * C::kJoinRows >= pc.rows && hh > 0) break;
        const int r = g + 8 * hh;
        float l = l_run[hh];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        // the buffer's last readers: only between pieces that take turns none are left
        if (!halves || !turns || hh > 0) bar_small(false);
        if (r < pc.rows) {
          if (c == 0) ml[warp * C::kJoinRows + g] = make_float2(m_use[hh], l);
          float* const dst = join + (warp * stride + g) * D;
#pragma unroll
          for (int x = 0; x < kOut; ++x) {
            if constexpr (!QUANT) {  // columns 8x + 2c, + 1
              *reinterpret_cast<float2*>(dst + join_at<D>(8 * x + 2 * c, g)) =
                  make_float2(o[x][2 * hh], o[x][2 * hh + 1]);
            } else if (x % 4 == 0) {  // column 8x + y of the MMAs is d = y (D / 8) + x, y = 2c, 2c + 1
#pragma unroll
              for (int y = 0; y < 2; ++y)
                *reinterpret_cast<float4*>(dst + join_at<D>((2 * c + y) * (D / 8) + x, g)) =
                    make_float4(o[x][2 * hh + y] * down, o[x + 1][2 * hh + y] * down,
                                o[x + 2][2 * hh + y] * down, o[x + 3][2 * hh + y] * down);
            }
          }
        }
        // (a warp that gave up still comes here, so that none waits for it)
        ok = !bar_small(!ok);
        if (!ok) break;
        const int rows = min(C::kJoinRows, pc.rows - hh * C::kJoinRows);
        for (int u = threadIdx.x; u < rows * (D / 4); u += 32 * kSmallWarps) {
          const int x = u / (D / 4), d = u % (D / 4) * 4;  // row of the round
          float m[kSmallWarps], lw[kSmallWarps], M = -INFINITY, L = 0.f;
          float4 part[kSmallWarps];
#pragma unroll
          for (int y = 0; y < kSmallWarps; ++y) {
            const float2 v = ml[y * C::kJoinRows + x];
            part[y] = *reinterpret_cast<const float4*>(join + (y * stride + x) * D + join_at<D>(d, x));
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
          const int row = hh * C::kJoinRows + x;
          *reinterpret_cast<float4*>(p.ws_o + (long long)pc.ws_row * D + partial_at(d >> 3, row, pc.rows) +
                                     (d & 4)) =
              make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
          if (d == 0) p.ws_l[(long long)pc.ws_row + row] = L == 0.f ? -INFINITY : M + lg2_approx(L);
        }
      }
      if (!ok) break;
      turns = halves;
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
