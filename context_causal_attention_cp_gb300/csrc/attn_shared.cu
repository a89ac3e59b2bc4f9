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
// attn_shared_kernel: one resident block per SM walks its pieces; its loads run
// ahead across piece ends.
//   warps 0-7    two softmax warpgroups (streams), one row per thread: query rows
//                to shared memory (any group size, any stride), S from TMEM, online
//                softmax in base 2 with a lazily moved maximum, P back to TMEM as
//                bf16, the partial to the workspace.
//   warp 8       TMA producer: K and V tiles of 128 keys, in the order of use,
//                through one ring.
//   warp 9       MMA issuer: S = Q K^T and O += P V (tcgen05), the two streams in
//                turn, so that one stream's softmax runs under the other's MMAs.
//   warp 10      zeroes the V rows behind a piece's last key (0 * NaN is NaN, so
//                masking P alone would not keep stale rows out).
//   warps 12-15  (e4m3 cache) codes to bf16 tiles, exactly: code * 2^e has 4
//                significant bits.  Rows behind the last key become zeros there.
// A unit of two MMA tiles (dual) gives both streams every KV tile; a smaller
// unit deals its KV tiles alternately to the streams, each with its own sums.
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
constexpr int kConvertWarp = 12;  // first of the four that decode e4m3 tiles

struct SharedParams {
  const int32_t* table;
  long long unit_first, row_first, entries, pieces;  // word offsets
  int num_units, num_pieces, num_entries, num_q_rows, Hq, Hkv, g;
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
};

template <int D, bool QUANT>
struct SharedCfg {
  static constexpr int kThreads = QUANT ? 512 : 384;
  static constexpr int kRegsLaunch = QUANT ? 128 : 168;
  static constexpr int kRegsSoftmax = 200, kRegsOther = QUANT ? 56 : 104;
  static_assert(kRegsSoftmax * 256 + kRegsOther * (kThreads - 256) <= kRegsLaunch * kThreads,
                "register split exceeds the launch allocation");
  static constexpr int kProducerWarp = 8, kMmaWarp = 9, kFixWarp = 10;
  static constexpr int kQTile = BM * D * 2;
  static constexpr int kTile = BN * D * 2;     // a bf16 K or V tile
  static constexpr int kRawTile = BN * D;      // an e4m3 K or V tile
  // 227 KB hold five tiles of 32 KB beside the queries, or three and four of codes
  static constexpr int kStages = QUANT ? 3 : 5;
  static constexpr int kRawStages = QUANT ? 4 : 0;
  static constexpr int kRingOff = 2 * kQTile;
  static constexpr int kRawOff = kRingOff + kStages * kTile;
  static constexpr int kBarOff = kRawOff + kRawStages * kRawTile;
  static constexpr int kNumBars = 2 * kStages + 2 * kRawStages + 8 + 3;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16 + 1024;  // + align slack
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kTmemCols = 512;  // S of each stream, then O of each
};

// A piece of the table, checked against the buffers; false (and
// CPATTN_ERR_RANGE) when it does not fit them.  Every warp of the block reads
// the same words and decides the same.
__device__ __forceinline__ bool load_piece(const SharedParams& p, int i, SharedPiece& pc) {
  const int4* w = reinterpret_cast<const int4*>(p.table + p.pieces) + 3LL * i;
  const int4 a = __ldg(w), b = __ldg(w + 1), c = __ldg(w + 2);
  pc = SharedPiece{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
  const int parts = pc.flags & kPieceSplit ? 2 : 1;
  const bool ok = pc.rows >= 1 && pc.rows <= kRows && pc.r0 >= 0 && pc.q_row0 >= 0 &&
                  (long long)pc.q_row0 + ((long long)pc.r0 + pc.rows - 1) / p.g < p.num_q_rows &&
                  pc.kv_head >= 0 && pc.kv_head < p.Hkv && pc.keys >= 1 && pc.key0 >= 0 &&
                  pc.kv_row >= 0 && (long long)pc.kv_row + pc.keys <= p.num_kv_rows &&
                  pc.ws_row >= 0 && (long long)pc.ws_row + (long long)parts * pc.rows <= p.ws_rows &&
                  (parts == 2) == (!shared_dual(pc.rows) && pc.keys > BN);
  if (!ok) set_status(p.status, CPATTN_ERR_RANGE);
  return ok;
}

// Order of a piece's K and V tiles in the ring, T KV tiles in all: the order in
// which the MMA warp first uses them (see its loop).  dual: K0 V0 K1 V1 ...;
// otherwise K0 K1 V0 K2 V1 ... K(T-1) V(T-2) V(T-1).
__device__ __forceinline__ int k_place(bool dual, int t) { return dual ? 2 * t : (t == 0 ? 0 : 2 * t - 1); }
__device__ __forceinline__ int v_place(bool dual, int t, int T) {
  return dual ? 2 * t + 1 : (t == T - 1 ? 2 * T - 1 : 2 * t + 2);
}
__device__ __forceinline__ void tile_at(bool dual, int j, int T, bool& is_v, int& t) {
  if (dual) {
    is_v = j & 1;
    t = j >> 1;
  } else if (j == 2 * T - 1) {
    is_v = true;
    t = T - 1;
  } else if (j == 0 || (j & 1)) {
    is_v = false;
    t = (j + 1) >> 1;
  } else {
    is_v = true;
    t = (j - 2) >> 1;
  }
}

// Four e4m3 codes times a power of two, as bf16 (exact: the low halves of the
// fp32 products are zero, so the upper halves are the bf16 values).
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t c, float scale) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)c));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(c >> 16)));
  float x[4];
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(x[0]), "=f"(x[1]) : "r"(h0));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(x[2]), "=f"(x[3]) : "r"(h1));
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= scale;
  return make_uint2(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x7632),
                    __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x7632));
}

template <int D, bool QUANT>
__global__ void __launch_bounds__(SharedCfg<D, QUANT>::kThreads, 1)
attn_shared_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const SharedParams p) {
  using C = SharedCfg<D, QUANT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint64_t* raw_full = empty + C::kStages;
  uint64_t* raw_empty = raw_full + C::kRawStages;
  uint64_t* q_full = raw_empty + C::kRawStages;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* fix_req = o_full + 2;
  uint64_t* fix_done = fix_req + 1;
  uint64_t* bar_drain = fix_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_trigger();  // the merge may be scheduled as blocks of this grid end

  const int first = __ldg(p.table + blockIdx.x), last = __ldg(p.table + blockIdx.x + 1);
  if (first < 0 || last > p.num_pieces) {
    if (threadIdx.x == 0) set_status(p.status, CPATTN_ERR_RANGE);
    return;
  }
  if (first >= last) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + i, QUANT ? 128 : 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < C::kRawStages; ++i) {
      mbar_init(raw_full + i, 1);
      mbar_init(raw_empty + i, 128);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 128);
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 128);
      mbar_init(o_full + s, 1);
    }
    mbar_init(fix_req, 1);
    mbar_init(fix_done, 32);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    tmem_slot[2] = 0;
    fence_barrier_init();
  }
  if (warp == C::kProducerWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  volatile int* issued_loads = reinterpret_cast<volatile int*>(tmem_slot + 2);  // for the abort drain
  const uint32_t q_base = smem_u32(smem);
  const uint32_t ring_base = smem_u32(smem + C::kRingOff);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == C::kProducerWarp) {
      // ---------------------------------------------------------- producer --
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        constexpr int kSt = QUANT ? C::kRawStages : C::kStages;
        constexpr int kBytes = QUANT ? C::kRawTile : C::kTile;
        uint64_t* const fullb = QUANT ? raw_full : full;
        uint64_t* const emptyb = QUANT ? raw_empty : empty;
        uint8_t* const ring = smem + (QUANT ? C::kRawOff : C::kRingOff);
        int seq = 0;
        bool ok = true;
        for (int i = first; i < last && ok; ++i) {
          SharedPiece pc;
          if (!load_piece(p, i, pc)) continue;
          const bool dual = shared_dual(pc.rows);
          const int T = (pc.keys + BN - 1) / BN;
          for (int j = 0; j < 2 * T; ++j, ++seq) {
            bool is_v;
            int t;
            tile_at(dual, j, T, is_v, t);
            const int slot = seq % kSt;
            ok = mbar_wait(emptyb + slot, ((seq / kSt) & 1) ^ 1, abort_flag, p.timeout_ns);
            if (!ok) break;
            mbar_arrive_expect_tx(fullb + slot, kBytes);
            const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
            const int row = pc.kv_row + t * BN;
            if (QUANT) {
              tma_load_3d(ring + slot * kBytes, tm, fullb + slot, 0, pc.kv_head, row);
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(ring + slot * kBytes + c * BN * 128, tm, fullb + slot, c * 64,
                            pc.kv_head, row);
            }
          }
        }
        *issued_loads = seq;
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
      }
    } else if (warp == C::kMmaWarp) {
      // -------------------------------------------------------- MMA issuer --
      // Step n of a piece is a (KV tile, stream) pair, the streams in turn; while
      // stream s works on P of step n the tensor core has step n + 1.  S of step
      // n + 2 overwrites P of step n, whose PV was issued before it.
      if (lane == 0) {
        constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, 0, 0);
        constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, 0, 1);
        const uint64_t dq0 = smem_desc_sw128(q_base, 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(ring_base, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(ring_base, BN * 128, 1024);
        int seq0 = 0;                  // ring place of the piece's first tile
        int steps[2] = {0, 0}, pieces[2] = {0, 0}, fixes = 0;
        bool ok = true;
        for (int i = first; i < last && ok; ++i) {
          SharedPiece pc;
          if (!load_piece(p, i, pc)) continue;
          const bool dual = shared_dual(pc.rows);
          const int T = (pc.keys + BN - 1) / BN;
          const int N = dual ? 2 * T : T;
          const bool ragged = !QUANT && pc.keys % BN != 0;
          auto wait_tile = [&](int seq) {
            const bool r = mbar_wait(full + seq % C::kStages, (seq / C::kStages) & 1, abort_flag,
                                     p.timeout_ns);
            tc_fence_after();
            return r;
          };
          auto issue_qk = [&](int n) {
            const int s = n & 1, t = dual ? n >> 1 : n;
            const int seq = seq0 + k_place(dual, t), slot = seq % C::kStages;
            if (n < 2) {
              if (!mbar_wait(q_full + s, pieces[s] & 1, abort_flag, p.timeout_ns)) return false;
              tc_fence_after();
            }
            if (!(dual && s == 1) && !wait_tile(seq)) return false;
            const uint64_t qd = dq0 + (uint64_t)((s * C::kQTile) >> 4);
            const uint64_t kd = dk0 + (uint64_t)((slot * C::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              constexpr int kChunk = (BM * 128) >> 4;
              const uint64_t off = (uint64_t)((kk >> 2) * kChunk + (kk & 3) * 2);
              mma_ss(tmem_base + s * BN, qd + off, kd + off, kIdescQK, kk > 0 ? 1u : 0u);
            }
            mma_commit(s_full + s);
            if (!(dual && s == 0)) mma_commit(empty + slot);
            return true;
          };
          ok = issue_qk(0);
          if (ok && N > 1) ok = issue_qk(1);
          for (int n = 0; n < N && ok; ++n) {
            const int s = n & 1, t = dual ? n >> 1 : n;
            const int seq = seq0 + v_place(dual, t, T), slot = seq % C::kStages;
            const bool first_use = !(dual && s == 1);
            const bool fix = ragged && t == T - 1 && first_use;
            if (first_use) {
              ok = wait_tile(seq);
              if (ok && fix) mbar_arrive(fix_req);
            }
            if (ok) ok = mbar_wait(p_full + s, steps[s] & 1, abort_flag, p.timeout_ns);
            if (ok && fix) ok = mbar_wait(fix_done, fixes++ & 1, abort_flag, p.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            ++steps[s];
            const uint64_t vd = dv0 + (uint64_t)((slot * C::kTile) >> 4);
            const uint32_t dt = tmem_base + 2 * BN + s * D, pt = tmem_base + s * BN;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              mma_ts(dt, pt + kk * 8, vd + (uint64_t)(kk * ((16 * 128) >> 4)), kIdescPV,
                     (n >= 2 || kk > 0) ? 1u : 0u);
            if (n + 2 >= N) mma_commit(o_full + s);
            if (!(dual && s == 0)) mma_commit(empty + slot);
            if (n + 2 < N) ok = issue_qk(n + 2);
          }
          ++pieces[0];
          if (N > 1) ++pieces[1];
          seq0 += 2 * T;
        }
        if (!ok) {
          set_status(p.status, CPATTN_ERR_TIMEOUT);
          *abort_flag = 1;
        }
        // every MMA and commit issued by this thread has completed
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0, nullptr, p.timeout_ns);
      }
    } else if (!QUANT && warp == C::kFixWarp) {
      // ------------------------------------------ V rows behind the last key --
      int seq0 = 0, fixes = 0;
      for (int i = first; i < last; ++i) {
        SharedPiece pc;
        if (!load_piece(p, i, pc)) continue;
        const int T = (pc.keys + BN - 1) / BN, live = pc.keys - (T - 1) * BN;
        if (live < BN) {
          const int seq = seq0 + 2 * T - 1, slot = seq % C::kStages;
          if (!mbar_wait_warp(fix_req, fixes & 1, abort_flag, p.timeout_ns) ||
              !mbar_wait_warp(full + slot, (seq / C::kStages) & 1, abort_flag, p.timeout_ns))
            break;  // the MMA warp's own wait runs out as well and reports
          ++fixes;
          for (int c = 0; c < D / 64; ++c) {
            uint4* tile = reinterpret_cast<uint4*>(smem + C::kRingOff + slot * C::kTile + c * BN * 128);
            for (int at = live * 8 + lane; at < BN * 8; at += 32) tile[at] = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
          mbar_arrive(fix_done);
        }
        seq0 += 2 * T;
      }
    }
    if constexpr (QUANT) if (warp >= kConvertWarp) {
      // ------------------------------------------------- codes to bf16 tiles --
      // Warp w has rows 32w .. 32w+31 of every tile, D / 16 lanes to a row.
      const int w = warp - kConvertWarp;
      constexpr int kLanes = D / 16, kRowsPer = 32 / kLanes;
      const int rl = lane / kLanes, cl = lane % kLanes;  // row in the group, 16-code chunk
      int seq = 0;
      bool ok = true;
      for (int i = first; i < last && ok; ++i) {
        SharedPiece pc;
        if (!load_piece(p, i, pc)) continue;
        const bool dual = shared_dual(pc.rows);
        const int T = (pc.keys + BN - 1) / BN;
        const long long srow = (long long)pc.kv_head * p.s_head + pc.kv_row + w * 32 + lane;
        auto load_scale = [&](int j) {
          bool is_v;
          int t;
          tile_at(dual, j, T, is_v, t);
          const bool live = t * BN + w * 32 + lane < pc.keys;
          return live ? __ldg((is_v ? p.vs : p.ks) + srow + t * BN) : 0.f;
        };
        float next = load_scale(0);
        for (int j = 0; j < 2 * T; ++j, ++seq) {
          const float scale = next;
          if (j + 1 < 2 * T) next = load_scale(j + 1);
          bool is_v;
          int t;
          tile_at(dual, j, T, is_v, t);
          const int live = pc.keys - t * BN;
          const int raw = seq % C::kRawStages, slot = seq % C::kStages;
          ok = mbar_wait_warp(raw_full + raw, (seq / C::kRawStages) & 1, abort_flag, p.timeout_ns) &&
               mbar_wait_warp(empty + slot, ((seq / C::kStages) & 1) ^ 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          const uint8_t* src = smem + C::kRawOff + raw * C::kRawTile;
          uint8_t* dst = smem + C::kRingOff + slot * C::kTile;
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += kRowsPer) {
            const int row = w * 32 + r0 + rl;
            const float sc = __shfl_sync(0xffffffffu, scale, r0 + rl);
            uint4 a = *reinterpret_cast<const uint4*>(src + row * D + cl * 16);
            if (row >= live) a = make_uint4(0, 0, 0, 0);
            const uint2 x0 = codes_to_bf16(a.x, sc), x1 = codes_to_bf16(a.y, sc);
            const uint2 x2 = codes_to_bf16(a.z, sc), x3 = codes_to_bf16(a.w, sc);
            uint8_t* line = dst + (cl >> 2) * (BN * 128) + row * 128;
            const int c0 = (cl & 3) * 2;  // 16-byte chunk of the row's 128 bytes
            *reinterpret_cast<uint4*>(line + ((c0 ^ (row & 7)) << 4)) = make_uint4(x0.x, x0.y, x1.x, x1.y);
            *reinterpret_cast<uint4*>(line + (((c0 + 1) ^ (row & 7)) << 4)) =
                make_uint4(x2.x, x2.y, x3.x, x3.y);
          }
          fence_async_shared();
          mbar_arrive(full + slot);
          mbar_arrive(raw_empty + raw);
        }
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
    const float sl2 = p.scale_log2;
    // The stream's next piece with KV tiles for it, from index i on; last if none.
    SharedPiece np;
    auto find = [&](int i) {
      for (; i < last; ++i)
        if (load_piece(p, i, np) && (s == 0 || shared_dual(np.rows) || np.keys > BN)) break;
      return i;
    };
    // This thread's query row of piece np to shared memory (128-byte swizzle).
    auto load_q = [&]() {
      const int r = shared_dual(np.rows) ? s * BM + trow : trow;
      if (r < np.rows) {
        const int packed = np.r0 + r, qi = packed / p.g;
        const __nv_bfloat16* src = p.q + (long long)(np.q_row0 + qi) * p.q_row +
                                   (long long)(np.kv_head * p.g + packed - qi * p.g) * p.q_head;
        uint8_t* dst = smem + s * C::kQTile + trow * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (BM * 128) + (((c & 7) ^ (trow & 7)) << 4)) =
              __ldg(reinterpret_cast<const uint4*>(src) + c);
      }
      fence_async_shared();
      mbar_arrive(q_full + s);
    };
    int step = 0, done = 0;
    bool ok = true;
    int i = find(first);
    if (i < last) load_q();
    while (i < last) {
      const SharedPiece pc = np;
      const bool dual = shared_dual(pc.rows);
      const int T = (pc.keys + BN - 1) / BN;
      const int r = dual ? s * BM + trow : trow;
      const bool warp_live = (dual ? s * BM : 0) + wq * 32 < pc.rows;
      int seen = 0;  // keys of the piece that this row sees
      if (r < pc.rows) {
        const long long pos = (long long)pc.q_pos0 + (long long)((pc.r0 + r) / p.g) * pc.q_pos_step;
        seen = (int)max(0LL, min((long long)pc.keys, pos + 1 - pc.key0));
      }
      float m_run = -INFINITY, l_run = 0.f, m_use = 0.f;
      for (int t = dual ? 0 : s; t < T; t += dual ? 1 : 2, ++step) {
        ok = mbar_wait_warp(s_full + s, step & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          float x[BN];
          {
            uint32_t v[BN];
#pragma unroll
            for (int q = 0; q < BN / 32; ++q) tmem_ld32p(s_addr + q * 32, v + q * 32);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < BN; ++c) x[c] = __uint_as_float(v[c]);
          }
          const int here = seen - t * BN;  // visible keys of this tile
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
          const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
          // The maximum moves only when a tile raises it by more than kMaxSlack
          // (log2 units): exponentials stay below 2^kMaxSlack, l uses the same
          // maximum, and O in TMEM is rescaled only then.
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
              // P in bf16 (half a step, 2^-8 of each weight; l sums the unrounded
              // values): the second product's operand type
              pk[c >> 1] = pack_bf16x2(a, b);
            }
            tmem_st16(s_addr + q * 16, pk);
          }
          l_run = l_run * alpha + (sum0 + sum1);
          const bool need = t > (dual ? 0 : s) && move;
          if (__any_sync(0xffffffffu, need)) {
            const float a = need ? alpha : 1.f;
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
        tc_fence_before();
        mbar_arrive(p_full + s);
      }
      if (ok) ok = mbar_wait_warp(o_full + s, done & 1, abort_flag, p.timeout_ns);
      if (!ok) break;
      ++done;
      tc_fence_after();
      // the query tile is free (its last product is done): the next piece's rows
      // go in before this one's store, so that its first S overlaps the store
      i = find(i + 1);
      if (i < last) load_q();
      if (warp_live) {
        const bool none = l_run == 0.f;  // (a NaN sum is not none)
        const float inv = none ? 0.f : 1.f / l_run;
        const long long row = (long long)pc.ws_row + r +
                              ((pc.flags & kPieceSplit) && s == 1 ? pc.rows : 0);
        float* dst = p.ws_o + row * D;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t v[32];
          tmem_ld32(o_addr + q * 32, v);
          tmem_wait_ld();
          if (r < pc.rows) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float4 f = make_float4(__uint_as_float(v[c]) * inv, __uint_as_float(v[c + 1]) * inv,
                                     __uint_as_float(v[c + 2]) * inv, __uint_as_float(v[c + 3]) * inv);
              if (none) f = make_float4(0.f, 0.f, 0.f, 0.f);
              *reinterpret_cast<float4*>(dst + q * 32 + c) = f;
            }
          }
        }
        if (r < pc.rows) p.ws_l[row] = none ? -INFINITY : m_use + lg2_approx(l_run);
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
  if (warp == C::kProducerWarp) {
    if (lane == 0 && *abort_flag) {
      // let the copies in flight land before the shared memory goes
      constexpr int kSt = QUANT ? C::kRawStages : C::kStages;
      uint64_t* const fullb = QUANT ? raw_full : full;
      const int n = *issued_loads;
      for (int j = max(0, n - kSt); j < n; ++j)
        mbar_wait(fullb + j % kSt, (j / kSt) & 1, nullptr, p.timeout_ns);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// One warp per (query row, head): its partials, in the order of its segments.
template <int D>
__global__ void __launch_bounds__(256) shared_merge_kernel(const SharedParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  grid_dep_wait();  // the attention kernel before this one wrote the partials
  const long long u = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (u >= (long long)p.num_q_rows * p.Hq) return;
  const int n = (int)(u / p.Hq), h = (int)(u % p.Hq), kvh = h / p.g, j = h % p.g;
  const int e0 = p.table[p.row_first + n], e1 = p.table[p.row_first + n + 1];
  if (e0 == e1) return;
  if (e0 < 0 || e1 > p.num_entries) {
    if (lane == 0) set_status(p.status, CPATTN_ERR_RANGE);
    return;
  }
  float m = -INFINITY, sw = 0.f, acc[E];
#pragma unroll
  for (int c = 0; c < E; ++c) acc[c] = 0.f;
  for (int e = e0; e < e1; ++e) {
    const long long packed = (long long)p.table[p.entries + 2 * e + 1] * p.g + j;
    const long long unit = p.table[p.entries + 2 * e] + packed / kRows * p.Hkv + kvh;
    if (packed < 0 || unit < 0 || unit >= p.num_units) {
      if (lane == 0) set_status(p.status, CPATTN_ERR_RANGE);
      return;
    }
    const int p0 = p.table[p.unit_first + unit], p1 = p.table[p.unit_first + unit + 1];
    if (p0 < 0 || p1 > p.num_pieces) {
      if (lane == 0) set_status(p.status, CPATTN_ERR_RANGE);
      return;
    }
    for (int i = p0; i < p1; ++i) {
      const SharedPiece& pc = reinterpret_cast<const SharedPiece*>(p.table + p.pieces)[i];
      for (int part = 0; part <= (pc.flags & kPieceSplit ? 1 : 0); ++part) {
        const long long row = (long long)pc.ws_row + packed % kRows + part * pc.rows;
        if (row < 0 || row >= p.ws_rows) {
          if (lane == 0) set_status(p.status, CPATTN_ERR_RANGE);
          return;
        }
        const float lj = p.ws_l[row];
        const float mn = fmaxf(m, lj);
        const float use = mn == -INFINITY ? 0.f : mn;  // a NaN partial stays one
        const float a = exp2f(m - use), w = exp2f(lj - use);
        sw = sw * a + w;
#pragma unroll
        for (int c = 0; c < E; ++c) acc[c] = fmaf(acc[c], a, w * p.ws_o[row * D + lane * E + c]);
        m = mn;
      }
    }
  }
  const float inv = sw == 0.f ? 0.f : 1.f / sw;
  const long long out = ((long long)n * p.Hq + h) * D + lane * E;
#pragma unroll
  for (int c = 0; c < E; ++c) {
    if (p.o_f32) static_cast<float*>(p.o)[out + c] = acc[c] * inv;
    else static_cast<__nv_bfloat16*>(p.o)[out + c] = __float2bfloat16_rn(acc[c] * inv);
  }
  if (lane == 0) p.lse[(long long)n * p.Hq + h] = sw == 0.f ? -INFINITY : (m + log2f(sw)) * kLn2;
}

// 3-D map of a code buffer (cols, heads, rows) with a D-column x 1-head x 128-row
// box, rows packed in shared memory; out-of-range rows read as zero.
bool make_code_map(CUtensorMap* m, const void* base, int cols, int heads, long long rows,
                   long long head_stride, long long row_stride) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)head_stride, (cuuint64_t)row_stride};
  cuuint32_t box[3] = {(cuuint32_t)cols, 1, BN};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool QUANT>
int launch_shared(const CUtensorMap& mk, const CUtensorMap& mv, const SharedParams& p, int num_ctas,
                  cudaStream_t stream) {
  using C = SharedCfg<D, QUANT>;
  auto kern = attn_shared_kernel<D, QUANT>;
  if (!allow_smem(kern, C::kSmemBytes)) return CPATTN_ERR_CUDA;
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
  return launch_kernel(kern, (unsigned)num_ctas, C::kThreads, C::kSmemBytes, stream, false, mk, mv,
                       p) == cudaSuccess
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
  if (!a16(table_dev) || !a16(q) || !a16(k) || !a16(v) || !a16(o) || !a16(workspace) ||
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
  p.unit_first = T.unit_first;
  p.row_first = T.row_first;
  p.entries = T.entries;
  p.pieces = T.pieces;
  p.num_units = plan->num_units;
  p.num_pieces = plan->num_pieces;
  p.num_entries = plan->num_entries;
  p.num_q_rows = plan->num_q_rows;
  p.Hq = plan->Hq;
  p.Hkv = plan->Hkv;
  p.g = plan->Hq / plan->Hkv;
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
  if (plan->num_pieces > 0) {
    CUtensorMap mk, mv;
    if (quant ? !make_code_map(&mk, k, d, plan->Hkv, num_kv_rows, k_head_stride, k_row_stride) ||
                    !make_code_map(&mv, v, dv, plan->Hkv, num_kv_rows, v_head_stride, v_row_stride)
              : !make_map(&mk, k, d, plan->Hkv, num_kv_rows, k_head_stride, k_row_stride) ||
                    !make_map(&mv, v, dv, plan->Hkv, num_kv_rows, v_head_stride, v_row_stride))
      return CPATTN_ERR_CUDA;
    const int r = d == 128 ? (quant ? launch_shared<128, true>(mk, mv, p, plan->num_ctas, stream)
                                    : launch_shared<128, false>(mk, mv, p, plan->num_ctas, stream))
                           : (quant ? launch_shared<64, true>(mk, mv, p, plan->num_ctas, stream)
                                    : launch_shared<64, false>(mk, mv, p, plan->num_ctas, stream));
    if (r != CPATTN_OK) return r;
  }
  const long long blocks = ((long long)plan->num_q_rows * plan->Hq + 7) / 8;
  if (blocks > 0x7fffffffLL) return CPATTN_ERR_TOO_LARGE;
  const cudaError_t e = launch_kernel(d == 128 ? shared_merge_kernel<128> : shared_merge_kernel<64>,
                                      (unsigned)blocks, 256, 0, stream, true, p);
  return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA;
}
