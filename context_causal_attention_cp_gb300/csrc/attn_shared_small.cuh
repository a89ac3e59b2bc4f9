// Small units of cp_attn_shared: at most kSharedSmallRows packed rows, e.g. one token's
// heads of a KV group against the request's own keys.
//
// A 128-row MMA tile would be nearly empty, and the trips through tensor memory (S out,
// P in, O out) take longer than a KV tile's way from HBM.  So a block that has small
// units works on registers: eight warps share each KV tile, 16 keys each, with warp-level
// 16x8x16 MMAs, and each keeps its own maximum, sum and 16 x D output; at a piece's end
// the eight are joined in shared memory.  What bounds it is HBM: a KV tile costs a warp
// about 100 instructions (250 with codes) and the block 64 KB (33 KB).
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
  static constexpr int kJoin = kSmallWarps * kSharedSmallRows * D * 4;
  static constexpr int kFixed = kJoin + kSmallWarps * kSharedSmallRows * 8 + 2 * kMaxSmallStages * 8 + 64 + 1024;
  static constexpr int kFit = (232448 - kFixed) / (kTile + kScales);
  static constexpr int kStages = kFit < kMaxSmallStages ? kFit : kMaxSmallStages;
  static constexpr int kScaleOff = kStages * kTile;
  static constexpr int kJoinOff = kScaleOff + kStages * kScales;
  static constexpr int kMlOff = kJoinOff + kJoin;  // (m, l) of each warp's rows
  static constexpr int kBarOff = kMlOff + kSmallWarps * kSharedSmallRows * 8;
  static constexpr int kWordOff = kBarOff + 2 * kStages * 8;
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

template <int D, bool QUANT>
__device__ __forceinline__ void run_small(const SharedParams& p, const SharedCta& list, uint8_t* smem,
                                          const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                          const CUtensorMap* tm_k_tail, const CUtensorMap* tm_v_tail) {
  using C = SmallCfg<D, QUANT>;
  constexpr int NS = C::kStages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + NS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kWordOff);
  volatile int* issued_loads = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, QUANT ? 33 : 1);  // the TMA copy and each lane's scales
      mbar_init(empty + i, kSmallWarps);
    }
    *abort_flag = 0;
    *issued_loads = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp >= kSmallWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SharedCfg<D, QUANT>::kRegsOther));
    if (warp == kProducerWarp && (QUANT || lane == 0)) {
      constexpr int kChunks = QUANT ? 1 : D / 64;      // boxes across a row
      constexpr int kLine = C::kTile / BN / kChunks;   // bytes of a box row
      int seq = 0;
      bool ok = true;
      for (int i = list.small0; i < list.small1 && ok; ++i) {
        const SharedPiece pc = load_piece(p, i);
        for (int u = 0; u < 2 * num_tiles(pc.keys); ++u, ++seq) {  // K0 V0 K1 V1 ...
          const int slot = seq % NS, t = u >> 1, row = pc.kv_row + t * BN, live = pc.keys - t * BN;
          const bool is_v = u & 1;
          const uint32_t parity = ((seq / NS) & 1) ^ 1;
          ok = QUANT ? wait_warp(empty + slot, parity, abort_flag, p.timeout_ns)
                     : wait_one(empty + slot, parity, abort_flag, p.timeout_ns);
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
          if constexpr (QUANT) {
            __syncwarp();
            const float* src = (is_v ? p.vs : p.ks) + (long long)pc.kv_head * p.s_head + row + lane;
            const uint32_t at = smem_u32(smem + C::kScaleOff + slot * C::kScales) + lane * 4;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x * 32 + lane < live)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + x * 128),
                             "l"(src + x * 32)
                             : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                             smem_u32(full + slot))
                         : "memory");
          }
        }
      }
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
    float* const join = reinterpret_cast<float*>(smem + C::kJoinOff);
    float2* const ml = reinterpret_cast<float2*>(smem + C::kMlOff);
    int seq = 0;
    bool ok = true;
    for (int i = list.small0; i < list.small1; ++i) {
      const SharedPiece pc = load_piece(p, i);
      // ---- queries: rows g and g + 8 ----
      uint32_t q[kSteps][4];
      float factor[2];
      int seen[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = g + 8 * hh;
        seen[hh] = 0;
        factor[hh] = p.scale_log2;
        uint4 v[D / 32];
        if (r < pc.rows) {
          const int packed = pc.r0 + r, qi = group_div(p, packed);
          const __nv_bfloat16* src = p.q + (long long)(pc.q_row0 + qi) * p.q_row +
                                     (long long)(pc.kv_head * p.g + packed - qi * p.g) * p.q_head;
          const long long pos = (long long)pc.q_pos0 + (long long)qi * pc.q_pos_step;
          seen[hh] = (int)max(0LL, min((long long)pc.keys, pos + 1 - pc.key0));
          // bf16: chunks 2c, 2c + 1 of each 128 bytes; e4m3: the 16-element chunks that
          // the lane's code chunks stand for
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            v[x] = __ldg(reinterpret_cast<const uint4*>(src + q_chunk<D, QUANT>(c, x)));
        } else {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) v[x] = make_uint4(0, 0, 0, 0);
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
      const int seen_all = max(seen[0], seen[1]);
      const int last_seen = __reduce_max_sync(0xffffffffu, seen_all);
      const int first_seen = min(pc.rows > g ? seen[0] : pc.keys, pc.rows > g + 8 ? seen[1] : pc.keys);
      const int full_seen = __reduce_min_sync(0xffffffffu, first_seen);  // keys that all rows see
      float o[kOut][4];
#pragma unroll
      for (int x = 0; x < kOut; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
      float m_run[2] = {-INFINITY, -INFINITY}, m_use[2] = {0.f, 0.f}, l_run[2] = {0.f, 0.f};
      int ev = -126;  // (e4m3) exponent of O
      const int T = num_tiles(pc.keys);
      for (int t = 0; t < T; ++t, seq += 2) {
        const int ks = seq % NS, vs = (seq + 1) % NS;
        const int at0 = t * BN + key0;           // the warp's first key
        const bool work = at0 < last_seen;       // some row sees some of its keys
        ok = wait_warp(full + ks, (seq / NS) & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        // ---- S = Q K^T: keys 8j + 2c, + 1 of rows g, g + 8 ----
        float s[2][4];
        if (work) {
          float s2[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[j][y] = s2[j][y] = 0.f;
          const uint32_t tile = smem_base + ks * C::kTile;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int row = key0 + 8 * j + g;
            if constexpr (!QUANT) {
#pragma unroll
              for (int x = 0; x < D / 32; ++x) {
                const uint4 k = lds128(tile + (x >> 1) * (BN * 128) + row * 128 +
                                       (((2 * c + (x & 1)) ^ (row & 7)) << 4));
                mma_16816<false>(s[j], q[2 * x], k.x, k.y);
                mma_16816<false>(s2[j], q[2 * x + 1], k.z, k.w);
              }
            } else {
#pragma unroll
              for (int x = 0; x < D / 64; ++x) {
                const uint4 k = lds128(tile + code_at<D>(row, D == 128 ? 2 * c + x : c));
                const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const uint32_t b0 = e4m3x2_to_f16x2(w[y]), b1 = e4m3x2_to_f16x2(w[y] >> 16);
                  if (y & 1) mma_16816<true>(s2[j], q[4 * x + y], b0, b1);
                  else mma_16816<true>(s[j], q[4 * x + y], b0, b1);
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float k0 = 1.f, k1 = 1.f;
            if constexpr (QUANT) {
              const float2 x = *reinterpret_cast<const float2*>(smem + C::kScaleOff + ks * C::kScales +
                                                                (key0 + 8 * j + 2 * c) * 4);
              k0 = x.x;
              k1 = x.y;
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              s[j][2 * hh] = (s[j][2 * hh] + s2[j][2 * hh]) * (factor[hh] * k0);
              s[j][2 * hh + 1] = (s[j][2 * hh + 1] + s2[j][2 * hh + 1]) * (factor[hh] * k1);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + ks);
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
        ok = wait_warp(full + vs, ((seq + 1) / NS) & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        if (work) {
          const uint32_t tile = smem_base + vs * C::kTile;
          const int live = pc.keys - at0;  // of the warp's keys
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
            // factors of the keys 2c, 2c + 1, 2c + 8, 2c + 9, relative to 2^ev
            float f[4];
            const float* sc = reinterpret_cast<const float*>(smem + C::kScaleOff + vs * C::kScales) + key0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = 2 * c + (x >> 1) * 8 + (x & 1);
              f[x] = key < live ? sc[key] : 0.f;
            }
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
            uint32_t w[4][D / 32];  // the lane's codes of its four keys
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = 2 * c + (x >> 1) * 8 + (x & 1), row = key0 + key;
              if constexpr (D == 128) {
                const uint4 v = lds128(tile + code_at<D>(row, g));
                w[x][0] = v.x; w[x][1] = v.y; w[x][2] = v.z; w[x][3] = v.w;
              } else {
                const uint2 v = lds64(tile + code_at<D>(row, g >> 1) + (g & 1) * 8);
                w[x][0] = v.x; w[x][1] = v.y;
              }
              if (key >= live)
#pragma unroll
                for (int y = 0; y < D / 32; ++y) w[x][y] = 0u;
            }
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
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + vs);
      }
      // ---- join the warps: O = sum_w f_w O_w / L, f_w = 2^(m_w - M), L = sum f_w l_w ----
      const float down = exp2_int(ev);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = g + 8 * hh;
        float l = l_run[hh];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (r < pc.rows) {
          if (c == 0) ml[warp * kSharedSmallRows + r] = make_float2(m_use[hh], l);
          float* const dst = join + (warp * kSharedSmallRows + r) * D;
#pragma unroll
          for (int x = 0; x < kOut; ++x) {
            if constexpr (!QUANT) {  // columns 8x + 2c, + 1
              *reinterpret_cast<float2*>(dst + join_at<D>(8 * x + 2 * c, r)) =
                  make_float2(o[x][2 * hh], o[x][2 * hh + 1]);
            } else if (x % 4 == 0) {  // column 8x + n of the MMAs is d = n (D / 8) + x, n = 2c, 2c + 1
#pragma unroll
              for (int n = 0; n < 2; ++n)
                *reinterpret_cast<float4*>(dst + join_at<D>((2 * c + n) * (D / 8) + x, r)) =
                    make_float4(o[x][2 * hh + n] * down, o[x + 1][2 * hh + n] * down,
                                o[x + 2][2 * hh + n] * down, o[x + 3][2 * hh + n] * down);
            }
          }
        }
      }
      // (a warp that gave up still comes here, so that none waits for it)
      if (bar_small(!ok)) {
        ok = false;
        break;
      }
      for (int u = threadIdx.x; u < pc.rows * (D / 4); u += 32 * kSmallWarps) {
        const int r = u / (D / 4), d = u % (D / 4) * 4;
        float m[kSmallWarps], l[kSmallWarps], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) {
          const float2 x = ml[w * kSharedSmallRows + r];
          m[w] = x.x;
          l[w] = x.y;
          if (l[w] != 0.f) M = fmaxf(M, m[w]);  // (m of a warp without keys means nothing)
        }
        if (M == -INFINITY) M = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) {
          const float f = l[w] == 0.f ? 0.f : ex2_approx(m[w] - M);
          L += f * l[w];
          const float4 x = *reinterpret_cast<const float4*>(join + (w * kSharedSmallRows + r) * D +
                                                           join_at<D>(d, r));
          if (l[w] != 0.f) {
            sum.x = fmaf(f, x.x, sum.x);
            sum.y = fmaf(f, x.y, sum.y);
            sum.z = fmaf(f, x.z, sum.z);
            sum.w = fmaf(f, x.w, sum.w);
          }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<float4*>(p.ws_o + ((long long)pc.ws_row + r) * D + d) =
            make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        if (d == 0) p.ws_l[(long long)pc.ws_row + r] = L == 0.f ? -INFINITY : M + lg2_approx(L);
      }
      bar_small(false);
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
